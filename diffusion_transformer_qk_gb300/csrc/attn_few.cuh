// Attention of a few queries (a pooling token, a step of decoding) over many
// keys for sm_103a (formulas: qknr_attn.h).
//
// Bound by HBM: every key and value is read once, for the ROWS = group *
// seq_q <= 4 queries of a key head together.  A 128-row tile of the tensor
// cores would be almost empty and the one CTA that owns it waits for its own
// softmax between two loads, so the products are plain FMAs here and the warps
// run independently.  A team of D/8 lanes takes 8 keys at a time, 8 columns a
// lane, K and V in flight together (8 KB a warp, 128 KB an SM).  The 8 partial
// dot products are summed across the team by swapping halves, so that each
// lane ends with one key's score (8 shuffles instead of 32) and takes one
// exponential.  Each team keeps a running maximum, sum and accumulator per
// query; a CTA's teams join in order through shared memory, and CTAs share a
// key head's keys like the tiles' contraction in attn_kernel.cuh.
#pragma once

#include "attn_kernel.cuh"

namespace qknr {

// One query: two CTAs of 8 warps per SM with 128 registers a thread; several:
// one CTA of 12 warps with 168.
__host__ __device__ constexpr int few_threads(int rows) { return rows == 1 ? 256 : 384; }
__host__ __device__ constexpr int few_ctas(int rows) { return rows == 1 ? 2 : 1; }       // per SM
constexpr int kFewRows = 4;   // queries of a key head at most
constexpr int kFewKeys = 8;   // keys of a team's step

// The query and head of row r of a key head's rows.
struct FewRow {
  int i, h;
  __device__ __forceinline__ FewRow(const AttnParams& p, int hk, int r)
      : i(r % p.seq_q), h(hk * p.group + r / p.seq_q) {}
};

// Sums s[0..7] over a team's lanes; the lane keeps key `few_key`'s.
template <int L>
__device__ __forceinline__ float few_sum(float (&s)[kFewKeys], int lane) {
#pragma unroll
  for (int off = L / 2, n = kFewKeys / 2; n >= 1; off >>= 1, n >>= 1) {
    const bool upper = lane & off;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float give = upper ? s[j] : s[j + n];
      const float keep = upper ? s[j + n] : s[j];
      s[j] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, off));
    }
  }
  // 16 lanes: the last two hold halves of the same key
  return L == 16 ? __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], 1)) : s[0];
}
// The lane's key: its upper three bits in the team choose the halves.
template <int L>
__device__ __forceinline__ int few_key(int lane) {
  return L == 16 ? (lane >> 1) & 7 : lane & 7;
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(few_threads(R), few_ctas(R)) attn_few_kernel(const __grid_constant__ AttnParams p) {
  constexpr int L = D / 8, TPW = 32 / L, WARPS = few_threads(R) / 32, TEAMS = WARPS * TPW;
  __shared__ __align__(16) float sums[WARPS][R][D];
  __shared__ float2 stats[WARPS][R];              // (maximum, sum)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane % L;
  const int rows = p.group * p.seq_q;
  grid_dependency_wait();
  grid_dependents_launch();
  AttnWork w;
  for (int s = 0; attn_work(p, s, w); ++s) {
    const int b = w.tile / p.heads_k, hk = w.tile - b * p.heads_k;
    const int q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
    const int k_len = clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
    float2 q[R][4], acc[R][4];
    float m[R], l[R];
    int limit[R], n = 0;                          // keys [0, limit) are seen
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
      limit[r] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[r][e] = acc[r][e] = make_float2(0.0f, 0.0f);
      const FewRow at(p, hk, r);
      if (r >= rows || at.i >= q_len) continue;
      limit[r] = p.causal ? min(max(at.i + k_len - q_len + 1, 0), k_len) : k_len;
      n = max(n, limit[r]);
      const char* src = p.q_in + (static_cast<long long>(b) * p.seq_q + at.i) * p.q_stride + at.h * (D * 2) + col * 16;
      if (in_span(src, 16, p.sp_q, p.status)) Elem<T>::unpack(*reinterpret_cast<const uint4*>(src), q[r]);
    }
    int begin, end;
    attn_cut(w, n, begin, end);
    const long long first = static_cast<long long>(b) * p.seq_k;
    const char* kp = p.k_in + first * p.k_stride + hk * (D * 2) + col * 16;
    const char* vp = p.v_in + first * p.v_stride + hk * (D * 2) + col * 16;
    for (int k0 = begin + warp * TPW * kFewKeys; k0 < end; k0 += TEAMS * kFewKeys) {   // the same for a whole warp
      const int mine = k0 + lane / L * kFewKeys;
      uint4 kr[kFewKeys], vr[kFewKeys];
#pragma unroll
      for (int j = 0; j < kFewKeys; ++j) {
        const char* src = kp + (mine + j) * p.k_stride;
        kr[j] = make_uint4(0, 0, 0, 0);
        if (mine + j < end && in_span(src, 16, p.sp_k, p.status)) kr[j] = __ldcs(reinterpret_cast<const uint4*>(src));
      }
#pragma unroll
      for (int j = 0; j < kFewKeys; ++j) {
        const char* src = vp + (mine + j) * p.v_stride;
        vr[j] = make_uint4(0, 0, 0, 0);
        if (mine + j < end && in_span(src, 16, p.sp_v, p.status)) vr[j] = __ldcs(reinterpret_cast<const uint4*>(src));
      }
      float prob[R];
      {
        float dot[R][kFewKeys];
#pragma unroll
        for (int j = 0; j < kFewKeys; ++j) {
          float2 x[4];
          Elem<T>::unpack(kr[j], x);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float2 d = __fmul2_rn(q[r][0], x[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) d = __ffma2_rn(q[r][e], x[e], d);
            dot[r][j] = __fadd_rn(d.x, d.y);
          }
        }
        const int key = mine + few_key<L>(lane);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float sum = few_sum<L>(dot[r], lane);
          const float score = key < end && key < limit[r] ? sum : -INFINITY;
          float top = score;
#pragma unroll
          for (int off = L / 2; off >= L / 8; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          top = fmaxf(top, m[r]);
          const float base = top == -INFINITY ? 0.0f : top;   // no key so far: every p is zero
          const float old = exp2_approx(__fmul_rn(__fsub_rn(m[r], base), p.scale_log2));
          prob[r] = exp2_approx(__fmul_rn(__fsub_rn(score, base), p.scale_log2));
          m[r] = top;
          l[r] = __fmaf_rn(l[r], old, prob[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] = __fmul2_rn(acc[r][e], make_float2(old, old));
        }
      }
#pragma unroll
      for (int j = 0; j < kFewKeys; ++j) {
        float2 x[4];
        Elem<T>::unpack(vr[j], x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float pj = __shfl_sync(0xffffffffu, prob[r], L == 16 ? 2 * j : j, L);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] = __ffma2_rn(make_float2(pj, pj), x[e], acc[r][e]);
        }
      }
    }
    // the warp's teams
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int off = L / 2; off >= L / 8; off >>= 1) l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xffffffffu, l[r], off));
#pragma unroll
      for (int off = L; off < 32; off <<= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, m[r], off);
        const float top = fmaxf(m[r], other), base = top == -INFINITY ? 0.0f : top;
        const float f = exp2_approx(__fmul_rn(__fsub_rn(m[r], base), p.scale_log2));
        m[r] = top;
        l[r] = __fmul_rn(l[r], f);
        l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xffffffffu, l[r], off));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[r][e] = __fmul2_rn(acc[r][e], make_float2(f, f));
          acc[r][e].x = __fadd_rn(acc[r][e].x, __shfl_xor_sync(0xffffffffu, acc[r][e].x, off));
          acc[r][e].y = __fadd_rn(acc[r][e].y, __shfl_xor_sync(0xffffffffu, acc[r][e].y, off));
        }
      }
      if (lane < L) {
        float4* dst = reinterpret_cast<float4*>(&sums[warp][r][col * 8]);
        dst[0] = make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y);
        dst[1] = make_float4(acc[r][2].x, acc[r][2].y, acc[r][3].x, acc[r][3].y);
      }
      if (lane == 0) stats[warp][r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    // the CTA's warps: a thread per two columns of a row
    const int r = threadIdx.x / (D / 2), c = threadIdx.x % (D / 2) * 2;
    if (r < R && r < rows) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) top = fmaxf(top, stats[i][r].x);
      const float base = top == -INFINITY ? 0.0f : top;
      float total = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        const float f = exp2_approx(__fmul_rn(__fsub_rn(stats[i][r].x, base), p.scale_log2));
        total = __fmaf_rn(f, stats[i][r].y, total);
        o = __ffma2_rn(make_float2(f, f), *reinterpret_cast<const float2*>(&sums[i][r][c]), o);
      }
      const FewRow at(p, hk, r);
      if (w.slot >= 0) {
        const long long k = static_cast<long long>(w.slot) * rows + r;
        if (in_span(p.part + k * D + c, 8, p.sp_part, p.status)) *reinterpret_cast<float2*>(p.part + k * D + c) = o;
        if (c == 0 && in_span(p.stats + 2 * k, 8, p.sp_stats, p.status))
          *reinterpret_cast<float2*>(p.stats + 2 * k) = make_float2(top, total);
      } else {
        const bool some = total != 0.0f;
        const float inv = some ? __frcp_rn(total) : 0.0f;
        const long long row = static_cast<long long>(b) * p.seq_q + at.i;
        char* dst = p.o + row * p.o_stride + at.h * (D * 2) + c * 2;
        if (in_span(dst, 4, p.sp_o, p.status))
          *reinterpret_cast<uint32_t*>(dst) = some ? pack2<T>(__fmul_rn(o.x, inv), __fmul_rn(o.y, inv)) : 0u;
        float* lse = p.lse + (static_cast<long long>(b) * p.heads_q + at.h) * p.seq_q + at.i;
        if (c == 0 && in_span(lse, 4, p.sp_lse, p.status)) *lse = some ? __fmaf_rn(top, p.scale, logf(total)) : -INFINITY;
      }
    }
    __syncthreads();
  }
}

}  // namespace qknr
