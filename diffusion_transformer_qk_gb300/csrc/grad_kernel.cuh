// Backward pass of the fused QK-RMSNorm + RoPE for sm_103a (formulas:
// qknr_grad.h).
//
// Bound by HBM: x and the incoming gradient are read once, the gradient of x
// is written once.  A team of D/8 lanes takes one head of one token, 8 values
// a lane, so the two sums over the head are shuffles inside the team.  A lane
// holds 4 rotation pairs: the two members of a pair meet in one thread (16
// contiguous bytes when interleaved, two 8-byte pieces D/2 apart when
// rotated by halves) and neither is read twice or shuffled.  A CTA takes a
// run of (token, head) items of Q, then of K, its teams side by side, so that
// a token's table row comes from HBM once and then from L1; every lane copies
// its share of the next kGradDepth items into shared-memory slots of its own
// (cp.async, 48 KB a CTA in flight and no barrier: a lane reads only what it
// copied).  At 2 x 4608 tokens of 48 heads x 128, with a copy of V's gradient,
// it takes 155 us, 5.9 TB/s.  Each lane's columns never change, so its share of
// dgamma stays in registers; a CTA's teams add theirs in order through shared
// memory and write one partial row.
#pragma once

#include "qknr_ptx.cuh"

namespace qknr {

struct GradSide {             // Q or K
  const char* x;
  const char* dy;
  char* dx;
  long long x_stride, dy_stride, dx_stride;       // bytes per row
  const float* gamma;
  int heads;
  MemSpan sp_x, sp_dy, sp_dx, sp_gamma;
};

struct GradParams {
  GradSide side[2];
  const char* dv;
  char* dv_out;
  long long dv_stride, dv_out_stride;
  int v_chunks;               // 16-byte chunks per row to copy (0: none)
  long long tokens;
  long long cos_rows;
  const char* cos;
  const char* sin;
  long long table_stride;     // bytes between table rows
  int head_stride;            // bytes between heads of a table row (0: shared)
  float* parts;               // [grid][2][D]
  float eps, inv_d;
  int* status;
  MemSpan sp_dv, sp_dv_out, sp_cos, sp_sin, sp_ws;
};

constexpr int kGradThreads = 256;
constexpr int kGradDepth = 6;                     // items in flight per team
constexpr int kGradSlots = kGradThreads * 32;     // bytes of one item of every team: x and dy
constexpr int kGradSmem = kGradSlots * kGradDepth;

// The 4 pairs of a lane, two to a register pair: `f` the first members, `s`
// the second.
struct GradPairs {
  float2 f[2], s[2];
};

template <typename T, bool RH>
__device__ __forceinline__ GradPairs grad_unpack(const uint4& r) {
  float2 X[4];
  Elem<T>::unpack(r, X);
  if (RH) return GradPairs{{X[0], X[1]}, {X[2], X[3]}};
  return GradPairs{{make_float2(X[0].x, X[1].x), make_float2(X[2].x, X[3].x)},
                   {make_float2(X[0].y, X[1].y), make_float2(X[2].y, X[3].y)}};
}

template <typename T, bool RH>
__device__ __forceinline__ uint4 grad_pack(const GradPairs& v) {
  if (RH) {
    const float2 O[4] = {v.f[0], v.f[1], v.s[0], v.s[1]};
    return Elem<T>::pack(O);
  }
  const float2 O[4] = {make_float2(v.f[0].x, v.s[0].x), make_float2(v.f[0].y, v.s[0].y),
                       make_float2(v.f[1].x, v.s[1].x), make_float2(v.f[1].y, v.s[1].y)};
  return Elem<T>::pack(O);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const char* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// A lane's 16 bytes of a head into its slot (`head`: the lane's first byte).
template <int D, bool RH>
__device__ __forceinline__ void grad_copy(uint32_t slot, const char* head) {
  if (RH) {
    copy_async<8>(slot, head);
    copy_async<8>(slot + 8, head + D);
  } else {
    copy_async<16>(slot, head);
  }
}

// the same 8 values of a table row (`row`: the lane's first value)
template <typename CT, int D, bool RH>
__device__ __forceinline__ GradPairs grad_table(const char* row) {
  const unsigned char* at = reinterpret_cast<const unsigned char*>(row);
  GradPairs v;
  if (RH) {
    load_table4<CT>(at, v.f);
    load_table4<CT>(at + D / 2 * sizeof(CT), v.s);
    return v;
  }
  float2 a[4];
  load_table8<CT>(at, a);
  return GradPairs{{make_float2(a[0].x, a[1].x), make_float2(a[2].x, a[3].x)},
                   {make_float2(a[0].y, a[1].y), make_float2(a[2].y, a[3].y)}};
}

// The place of an item (token, head) and of the team's next one.
struct GradWalk {
  long long left;             // the team's items from here on
  int h, step_h, heads;
  // byte offsets advance by `by`, and by `wrap` more when the head wraps into the next token
  __device__ __forceinline__ bool next() {
    --left;
    h += step_h;
    if (h < heads) return false;
    h -= heads;
    return true;
  }
};

template <typename T, typename CT, int D, bool RH>
__global__ void __launch_bounds__(kGradThreads, 3) qk_grad_kernel(const __grid_constant__ GradParams p) {
  constexpr int L = D / 8;                        // lanes per team
  constexpr int TEAMS = kGradThreads / L;
  extern __shared__ __align__(16) unsigned char smem[];   // [kGradDepth][x, dy][thread][16]
  float(*acc)[D] = reinterpret_cast<float(*)[D]>(smem);   // when the items are done: the teams' sums
  static_assert(TEAMS * D * 4 <= kGradSmem, "shared memory");
  const uint32_t slots = smem_addr(smem) + threadIdx.x * 16;
  const int team = threadIdx.x / L, lane = threadIdx.x % L;
  const int first = RH ? lane * 8 : lane * 16;    // the lane's first byte of a head
  constexpr long long step = TEAMS;
  grid_dependency_wait();
  grid_dependents_launch();

#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const GradSide& sd = p.side[w];
    const int H = sd.heads;
    GradPairs gamma, acc_w;
#pragma unroll
    for (int i = 0; i < 2; ++i) gamma.f[i] = gamma.s[i] = acc_w.f[i] = acc_w.s[i] = make_float2(0.0f, 0.0f);
    if (H > 0 && in_span(sd.gamma, D * 4, sd.sp_gamma, p.status)) {
      // 4-byte aligned only
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* f = sd.gamma + (RH ? lane * 4 + 2 * i : lane * 8 + 4 * i);
        gamma.f[i] = make_float2(f[0], f[RH ? 1 : 2]);
        const float* s = RH ? f + D / 2 : f + 1;
        gamma.s[i] = make_float2(s[0], s[RH ? 1 : 2]);
      }
    }
    // the CTA's run of items
    const long long all = p.tokens * H, run = (all + gridDim.x - 1) / gridDim.x;
    const long long it0 = blockIdx.x * run + team, items = (blockIdx.x + 1) * run < all ? (blockIdx.x + 1) * run : all;
    const long long t0 = H ? it0 / H : 0, step_t = H ? step / H : 0;
    GradWalk at{it0 < items ? (items - it0 + step - 1) / step : 0, H ? static_cast<int>(it0 - t0 * H) : 0,
                H ? static_cast<int>(step - step_t * H) : 0, H};
    GradWalk ahead = at;
    const long long h0 = at.h * (D * 2) + first, hb = at.step_h * (D * 2), wrap = -static_cast<long long>(H) * (D * 2);
    const char* fx = sd.x + t0 * sd.x_stride + h0;
    const char* fd = sd.dy + t0 * sd.dy_stride + h0;
    char* dst = sd.dx + t0 * sd.dx_stride + h0;
    const long long x_by = step_t * sd.x_stride + hb, d_by = step_t * sd.dy_stride + hb,
                    o_by = step_t * sd.dx_stride + hb;
    // table row of the item, t % cos_rows, kept by addition
    const long long step_row = step_t % p.cos_rows;
    long long row = t0 % p.cos_rows;
    int f_slot = 0, slot = 0;
    GradPairs c{}, n{};
    bool fresh = true;
    auto fetch = [&]() {
      if (ahead.left > 0) {
        if (in_span(fx - first, D * 2, sd.sp_x, p.status) && in_span(fd - first, D * 2, sd.sp_dy, p.status)) {
          grad_copy<D, RH>(slots + f_slot, fx);
          grad_copy<D, RH>(slots + f_slot + kGradSlots / 2, fd);
        }
        fx += x_by;
        fd += d_by;
        if (ahead.next()) {
          fx += sd.x_stride + wrap;
          fd += sd.dy_stride + wrap;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      f_slot = f_slot == kGradSmem - kGradSlots ? 0 : f_slot + kGradSlots;
    };
    for (int i = 0; i < kGradDepth; ++i) fetch();
    // the whole warp goes round together (the shuffles below), so a team
    // past the end walks along and stores nothing
    while (__any_sync(0xffffffffu, at.left > 0)) {
      const bool live = at.left > 0;
      asm volatile("cp.async.wait_group %0;" ::"n"(kGradDepth - 1) : "memory");
      const unsigned char* mine = smem + slot + threadIdx.x * 16;
      const GradPairs x = grad_unpack<T, RH>(*reinterpret_cast<const uint4*>(mine));
      const GradPairs d = grad_unpack<T, RH>(*reinterpret_cast<const uint4*>(mine + kGradSlots / 2));
      slot = slot == kGradSmem - kGradSlots ? 0 : slot + kGradSlots;
      // a team's heads of one token share its table row
      if (live && fresh) {
        const long long off = row * p.table_stride + at.h * p.head_stride;
        if (in_span(p.cos + off, D * sizeof(CT), p.sp_cos, p.status) &&
            in_span(p.sin + off, D * sizeof(CT), p.sp_sin, p.status)) {
          const int mine_at = (RH ? lane * 4 : lane * 8) * static_cast<int>(sizeof(CT));
          c = grad_table<CT, D, RH>(p.cos + off + mine_at);
          n = grad_table<CT, D, RH>(p.sin + off + mine_at);
        }
      }
      fetch();
      GradPairs y, g;
      float2 sq = make_float2(0.0f, 0.0f), gx = sq;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // o1 = y1 cos1 - y2 sin1, o2 = y2 cos2 + y1 sin2
        y.f[i] = __ffma2_rn(d.f[i], c.f[i], __fmul2_rn(d.s[i], n.s[i]));
        y.s[i] = __ffma2_rn(d.s[i], c.s[i], __fmul2_rn(make_float2(-d.f[i].x, -d.f[i].y), n.f[i]));
        g.f[i] = __fmul2_rn(y.f[i], gamma.f[i]);
        g.s[i] = __fmul2_rn(y.s[i], gamma.s[i]);
        sq = __ffma2_rn(x.f[i], x.f[i], __ffma2_rn(x.s[i], x.s[i], sq));
        gx = __ffma2_rn(g.f[i], x.f[i], __ffma2_rn(g.s[i], x.s[i], gx));
      }
      // the two sums over the team share one tree: its upper lanes take gx
      const bool upper = lane & (L / 2);
      const float a = __fadd_rn(sq.x, sq.y), b = __fadd_rn(gx.x, gx.y);
      float t = __fadd_rn(upper ? b : a, __shfl_xor_sync(0xffffffffu, upper ? a : b, L / 2));
#pragma unroll
      for (int off = L / 4; off >= 1; off >>= 1) t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, off));
      const float other = __shfl_xor_sync(0xffffffffu, t, L / 2);
      const float r = rsqrtf(__fmaf_rn(upper ? other : t, p.inv_d, p.eps));
      const float m = __fmul_rn(__fmul_rn(__fmul_rn(r, r), r), __fmul_rn(upper ? t : other, -p.inv_d));
      if (live) {
        const float2 R = make_float2(r, r), M = make_float2(m, m);
        GradPairs o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc_w.f[i] = __ffma2_rn(y.f[i], __fmul2_rn(x.f[i], R), acc_w.f[i]);
          acc_w.s[i] = __ffma2_rn(y.s[i], __fmul2_rn(x.s[i], R), acc_w.s[i]);
          o.f[i] = __ffma2_rn(x.f[i], M, __fmul2_rn(g.f[i], R));
          o.s[i] = __ffma2_rn(x.s[i], M, __fmul2_rn(g.s[i], R));
        }
        if (in_span(dst - first, D * 2, sd.sp_dx, p.status)) {
          const uint4 v = grad_pack<T, RH>(o);
          if (RH) {
            store8(dst, make_uint2(v.x, v.y));
            store8(dst + D, make_uint2(v.z, v.w));
          } else {
            store16(dst, v);
          }
        }
      }
      dst += o_by;
      row += step_row;
      fresh = step_t > 0 || p.head_stride > 0;
      if (at.next()) {
        dst += sd.dx_stride + wrap;
        ++row;
        fresh = true;
      }
      if (row >= p.cos_rows) row -= p.cos_rows;
    }
    // this side's partial row
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* f = &acc[team][RH ? lane * 4 + 2 * i : lane * 8 + 4 * i];
      float* s = RH ? f + D / 2 : f + 1;
      f[0] = acc_w.f[i].x;
      f[RH ? 1 : 2] = acc_w.f[i].y;
      s[0] = acc_w.s[i].x;
      s[RH ? 1 : 2] = acc_w.s[i].y;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.0f;
      for (int g = 0; g < TEAMS; ++g) s = __fadd_rn(s, acc[g][threadIdx.x]);
      float* out = p.parts + (static_cast<long long>(blockIdx.x) * 2 + w) * D + threadIdx.x;
      if (in_span(out, 4, p.sp_ws, p.status)) *out = s;
    }
    __syncthreads();                              // the slots are free again
  }

  // V's gradient, copied, eight pieces a thread in flight
  if (p.v_chunks > 0) {
    const long long items = p.tokens * p.v_chunks, vstep = static_cast<long long>(gridDim.x) * kGradThreads;
    constexpr int kPieces = 8;
    const long long vt = vstep / p.v_chunks;
    const int vc = static_cast<int>(vstep - vt * p.v_chunks);
    long long it = static_cast<long long>(blockIdx.x) * kGradThreads + threadIdx.x;
    long long t = it / p.v_chunks;
    int c = static_cast<int>(it - t * p.v_chunks);
    while (it < items) {
      uint4 v[kPieces];
      char* dst[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        dst[i] = nullptr;
        if (it < items) {
          const char* src = p.dv + t * p.dv_stride + c * 16;
          char* to = p.dv_out + t * p.dv_out_stride + c * 16;
          if (in_span(src, 16, p.sp_dv, p.status) && in_span(to, 16, p.sp_dv_out, p.status)) {
            v[i] = __ldcs(reinterpret_cast<const uint4*>(src));
            dst[i] = to;
          }
        }
        it += vstep;
        t += vt;
        c += vc;
        if (c >= p.v_chunks) {
          c -= p.v_chunks;
          ++t;
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (dst[i]) store16(dst[i], v[i]);
    }
  }
}

}  // namespace qknr
