// Attention forward and backward for sm_103a (formulas: qknr_attn.h).
//
// All four kernels' products run on tcgen05 with operands that TMA leaves in
// shared memory and accumulators in tensor memory; the probabilities (and the
// score gradients) go back to tensor memory as 16-bit left operands of the
// second product, in the columns whose scores they replace.  One thread
// issues every MMA; MMAs of one thread run in order, so a product that
// overwrites an operand of an earlier one needs no wait in between.
//
// Roles of a CTA's 12 warps: 0-7 are two groups of four that each cover the
// 128 lanes of tensor memory (a thread owns one row of a score tile), warp 8
// issues the MMAs, warp 9 the TMA loads, warps 10 and 11 fill up the third
// group, whose registers go to the first two (and hand round the queries'
// statistics in the dk, dv kernel).  Every wait is bounded; a role that
// gives up sets the CTA's abort flag, drains what it started and leaves.
#pragma once

#include "tc.cuh"

namespace qknr {

struct AttnParams {
  CUtensorMap map_q, map_k, map_v, map_do;
  const char* o_in;           // backward: the forward's output
  const char* dout;
  char* o;
  char* dq;
  char* dk;
  char* dv;
  float* lse;
  float* delta;               // [batch][heads_q][seq_q]
  long long o_stride, dout_stride, dq_stride, dk_stride, dv_stride;   // bytes per row
  const int* q_lens;
  const int* k_lens;
  int batch, seq_q, seq_k, heads_q, heads_k, group;
  int causal;
  float scale, scale_log2;
  int tiles;                  // row tiles of a head
  unsigned flags;
  int* status;
  unsigned long long wait_limit_ns;
  MemSpan sp_o, sp_dout, sp_dq, sp_dk, sp_dv, sp_lse, sp_delta, sp_q_lens, sp_k_lens;
};

constexpr int kAttnThreads = 384;
constexpr int kAttnMmaWarp = 8, kAttnLoadWarp = 9;
constexpr int kTile = 128;                        // rows of a tile, both ways
// Registers: 384 threads start with 168 each; 2 x 128 x 208 + 128 x 80 fit in
// the 384 x 168 that the block was launched with.
constexpr int kAttnWorkRegs = 208, kAttnIssueRegs = 80;
static_assert(2 * kAttnWorkRegs + kAttnIssueRegs <= 3 * 168, "register split above the launch's total");
constexpr float kLog2e = 1.4426950408889634f;

template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int D>
constexpr int kTileBytes = kTile * D * 2;

__device__ __forceinline__ int clamp_len(const int* lens, int b, int most, const MemSpan& sp, int* status) {
  if (lens == nullptr || !in_span(lens + b, 4, sp, status)) return most;
  const int n = lens[b];
  return n < 0 ? 0 : (n > most ? most : n);
}

// Rows [first, 128) of a tile become zero, so that whatever lies past a
// sample's length meets the zero probabilities of masked places as zero.  A
// whole warp; the swizzle moves chunks inside a row only.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int first, int lane) {
  const int chunks = (kTile - first) * 8;
#pragma unroll
  for (int half = 0; half < D / 64; ++half)
    for (int c = lane; c < chunks; c += 32)
      reinterpret_cast<uint4*>(tile + half * (kTile * 128) + first * 128)[c] = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  __syncwarp();
}

// D[128 x N] (+)= A[128 x D] B[N x D]^T, both tiles contracted over their columns
template <typename T, int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = mma_desc<T>(kTile, kTile, false);
  const uint32_t da = desc_k_major(a), db = desc_k_major(b);
  mma_ss<false>(d, da, db, idesc);
#pragma unroll
  for (int k = 1; k < D / 16; ++k) {
    const uint32_t off = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
    mma_ss<true>(d, da + off, db + off, idesc);
  }
}

// D[128 x D] (+)= A[128 x 128] B[128 x D]: A 16-bit in tensor memory (SPLIT:
// its second 64 columns start 64 columns on), B contracted over its rows
template <typename T, int D, bool SPLIT>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  constexpr uint32_t idesc = mma_desc<T>(kTile, D, true);
  const uint32_t db = desc_mn_major(b, kTile * 128);
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    mma_ts(d, a + (SPLIT ? (k / 4) * 64 + (k % 4) * 8 : k * 8), db + k * (2048 >> 4), idesc, accumulate || k > 0);
}

// A place in a ring of N stages, stepped without divisions: the issuing warp's
// instructions between two products are time the tensor cores may stand still.
template <int N>
struct RingPos {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      phase ^= 1u;
    }
  }
};

// The common part of the kernels: barriers, tensor memory, bounded waits.
struct AttnCta {
  unsigned char* smem;
  uint32_t base;              // shared address of the tiles
  uint32_t bars;              // first barrier
  volatile int* abort_flag;
  int* status;
  unsigned long long limit;
  int warp, lane;

  // One thread.  Bounded like bounded_wait(), but inline: a kernel that moves
  // registers between its warps makes no calls.
  __device__ __forceinline__ bool wait1(int i, uint32_t phase) const {
    const uint32_t b = bar(i);
    if (mbar_try_wait(b, phase & 1u)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait_sleep(b, phase & 1u, 20000u)) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > limit) {
        *abort_flag = 1;
        if (status) atomicCAS(status, 0, kStatusTimeout);
        return false;
      }
    }
    return true;
  }
  // Whole warp; the same answer in every lane.
  __device__ __forceinline__ bool wait(int i, uint32_t phase) const {
    return __all_sync(0xffffffffu, wait1(i, phase));
  }
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // a warp's arrival after its tensor memory accesses
  __device__ __forceinline__ void arrive(int i) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  }
};

// 16 bytes of a row at a time: 32 accumulator values from tensor memory to
// their place in a row of the output, times f (zero where the row has no value)
template <typename T>
__device__ __forceinline__ void store_cols(char* dst, const float (&v)[32], float f, bool some) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 w;
    uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ww[i] = some ? pack2<T>(__fmul_rn(v[c * 8 + 2 * i], f), __fmul_rn(v[c * 8 + 2 * i + 1], f)) : 0u;
    reinterpret_cast<uint4*>(dst)[c] = w;
  }
}

// ---------------------------------------------------------------------------
// forward: a CTA takes 256 queries of one head as two tiles whose softmaxes
// alternate with each other's products.

namespace fwd {
constexpr int kStages = 4;                        // K and V tiles in flight, in turn
enum { Q_FULL = 0, KV_FULL = 2, KV_EMPTY = KV_FULL + kStages, S_FULL = KV_EMPTY + kStages, P_FULL = S_FULL + 2,
       O_DONE = P_FULL + 2, DRAIN = O_DONE + 2, BARS = DRAIN + 1 };
template <int D>
constexpr int kSmem = (2 + kStages) * kTileBytes<D> + 256;
// The running maximum is only raised, and the accumulator rescaled, when the
// new one is more than 2^8 above: p stays below 2^8, which 16-bit floats and
// the fp32 sums hold as exactly as values below one.
constexpr float kSlack = 8.0f;
}  // namespace fwd

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_forward_kernel(const __grid_constant__ AttnParams p) {
  using namespace fwd;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + (2 + kStages) * kTileBytes<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
            __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), i >= P_FULL && i < O_DONE ? 4 : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();

  const int tile = p.causal ? p.tiles - 1 - static_cast<int>(blockIdx.x % p.tiles) : static_cast<int>(blockIdx.x % p.tiles);
  const int h = static_cast<int>(blockIdx.x / p.tiles % p.heads_q), b = static_cast<int>(blockIdx.x / p.tiles / p.heads_q);
  const int q0 = tile * 2 * kTile;
  const int q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
  const int k_len = clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
  const int diag = k_len - q_len;                 // causal: query i sees keys up to i + diag
  int nb[2];                                      // key blocks of each query tile
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = q0 + t * kTile;
    int last = first + kTile < q_len ? first + kTile : q_len;
    int keys = first >= q_len ? 0 : (p.causal ? last + diag : k_len);
    keys = keys < 0 ? 0 : (keys > k_len ? k_len : keys);
    nb[t] = (keys + kTile - 1) / kTile;
  }
  const int blocks = nb[0] > nb[1] ? nb[0] : nb[1];
  const uint32_t ring = c.base + 2 * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && blocks > 0) {
      const int hk = h / p.group;
      int issued = 0;
      bool ok = !(p.flags & 1u);                  // test only: issue nothing
      if (ok) {
        for (int t = 0; t < 2; ++t) {
          if (nb[t] == 0) continue;
          mbar_arrive_expect_tx(c.bar(Q_FULL + t), kTileBytes<D>);
          tma_load_tile(c.base + t * kTileBytes<D>, &p.map_q, q0 + t * kTile, h, b, c.bar(Q_FULL + t));
        }
        for (int i = 0; i < 2 * blocks; ++i) {
          const int s = i % kStages;
          if (!c.wait1(KV_EMPTY + s, (i / kStages + 1) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(c.bar(KV_FULL + s), kTileBytes<D>);
          tma_load_tile(ring + s * kTileBytes<D>, i & 1 ? &p.map_v : &p.map_k, (i / 2) * kTile, hk, b, c.bar(KV_FULL + s));
          ++issued;
        }
      }
      if (!ok || *abort_flag) {
        // copies in flight end before the CTA leaves its shared memory
        const unsigned long long t0 = global_timer_ns();
        for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          while (!mbar_try_wait(c.bar(KV_FULL + i % kStages), (i / kStages) & 1) && global_timer_ns() - t0 < c.limit) {
          }
        for (int t = 0; t < 2; ++t)
          while (!(p.flags & 1u) && nb[t] && !mbar_try_wait(c.bar(Q_FULL + t), 0) && global_timer_ns() - t0 < c.limit) {
          }
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp) {
    // S_t(0), then per block: O_t += P_t V, S_t(next)
    bool ok = blocks > 0;
    for (int t = 0; t < 2 && ok; ++t)
      if (nb[t]) ok = c.wait(Q_FULL + t, 0);
    ok = ok && c.wait(KV_FULL, 0);
    tc_fence_after();
    if (ok && elect_one()) {
      for (int t = 0; t < 2; ++t)
        if (nb[t]) {
          mma_rows<T, D>(tmem + t * kTile, c.base + t * kTileBytes<D>, ring);
          mma_commit(c.bar(S_FULL + t));
        }
      mma_commit(c.bar(KV_EMPTY));
    }
    for (int j = 0; ok && j < blocks; ++j) {
      const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % kStages, sk = ik % kStages;
      ok = c.wait(KV_FULL + sv, iv / kStages);
      if (!ok) break;
      if (k_len < p.seq_k && (j + 1) * kTile > k_len)
        zero_rows<D>(smem + (2 + sv) * kTileBytes<D>, k_len - j * kTile, c.lane);
      if (j + 1 < blocks) ok = c.wait(KV_FULL + sk, ik / kStages);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && j < nb[t]) {
          ok = c.wait(P_FULL + t, j);
          tc_fence_after();
          if (ok && elect_one()) {
            mma_cols<T, D, false>(tmem + 2 * kTile + t * kTile, tmem + t * kTile, ring + sv * kTileBytes<D>, j > 0);
            mma_commit(c.bar(O_DONE + t));
          }
        }
        if (t == 1 && ok && elect_one()) mma_commit(c.bar(KV_EMPTY + sv));
        if (ok && elect_one() && j + 1 < nb[t]) {
          mma_rows<T, D>(tmem + t * kTile, c.base + t * kTileBytes<D>, ring + sk * kTileBytes<D>);
          mma_commit(c.bar(S_FULL + t));
        }
      }
      if (ok && elect_one() && j + 1 < blocks) mma_commit(c.bar(KV_EMPTY + sk));
    }
    if (!ok && blocks > 0) {
      // MMAs in flight end before tensor memory is given back
      if (elect_one()) mma_commit(c.bar(DRAIN));
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(c.bar(DRAIN), 0) && global_timer_ns() - t0 < c.limit) {
      }
    }
    __syncwarp();
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // softmax: a thread per query
    const int t = c.warp >> 2, n = nb[t];
    const int row = q0 + t * kTile + (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const uint32_t ts = tmem + t * kTile + lanes, to = tmem + 2 * kTile + t * kTile + lanes;
    int limit = row < q_len ? (p.causal ? row + diag + 1 : k_len) : 0;   // keys this query sees
    limit = limit < 0 ? 0 : (limit > k_len ? k_len : limit);
    const float sl = p.scale_log2, slack = kSlack / sl;
    float m = -INFINITY;
    float2 sum = make_float2(0.0f, 0.0f);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = c.wait(S_FULL + t, j);
      if (!ok) break;
      tc_fence_after();
      float s[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_load32(ts + 32 * i, s[i]);
      tmem_wait_load(s[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) tmem_loaded(s[i]);
      const int seen = limit - j * kTile;
      if (__any_sync(0xffffffffu, seen < kTile)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) s[i][e] = 32 * i + e < seen ? s[i][e] : -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mx[i] = fmaxf(s[i][0], s[i][1]);
#pragma unroll
        for (int e = 2; e < 32; e += 2) mx[i] = fmaxf(mx[i], fmaxf(s[i][e], s[i][e + 1]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = top;
      } else if (__any_sync(0xffffffffu, top > m + slack)) {
        const float raised = fmaxf(m, top);
        const float f = raised == m ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(m, raised), sl));
        m = raised;
        sum = __fmul2_rn(sum, make_float2(f, f));
        ok = c.wait(O_DONE + t, j - 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_load32(to + 32 * i, o);
          tmem_wait_load(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __fmul_rn(o[e], f);
          tmem_store32(to + 32 * i, o);
        }
      }
      // a row that has seen nothing yet: exp2(-inf - 0) = 0
      const float shift = m == -INFINITY ? 0.0f : __fmul_rn(-m, sl);
      const float2 SL = make_float2(sl, sl), SH = make_float2(shift, shift);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __ffma2_rn(make_float2(s[i][2 * e], s[i][2 * e + 1]), SL, SH);
          const float2 y = make_float2(exp2_approx(x.x), exp2_approx(x.y));
          sum = __fadd2_rn(sum, y);
          w[e] = pack2<T>(y.x, y.y);
        }
        tmem_store16(ts + 16 * i, w);
      }
      tmem_wait_store();
      c.arrive(P_FULL + t);
    }
    if (ok && n > 0) ok = c.wait(O_DONE + t, n - 1);
    tc_fence_after();
    const float total = __fadd_rn(sum.x, sum.y);
    const bool some = total != 0.0f;
    const float inv = some ? __frcp_rn(total) : 0.0f;
    const bool mine = row < p.seq_q;
    if (ok) {
      const long long at = (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + row;
      if (mine && in_span(p.lse + at, 4, p.sp_lse, p.status))
        p.lse[at] = some ? __fmaf_rn(m, p.scale, logf(total)) : -INFINITY;
      char* dst = p.o + (static_cast<long long>(b) * p.seq_q + row) * p.o_stride + h * (D * 2);
      const bool fits = mine && in_span(dst, D * 2, p.sp_o, p.status);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
        if (n > 0) {
          tmem_load32(to + 32 * i, o);
          tmem_wait_load(o);
        }
        if (fits) store_cols<T>(dst + 64 * i, o, inv, some);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// backward
//
// Powers of two that the 16-bit operands carry through their products and
// the epilogues take out again.  P gets 2^kP, in the exponent: fp16 keeps the
// small probabilities of long rows out of its subnormals (P <= 1, so 2^14 is
// in range), bf16 those that ex2.approx would flush to zero.  dS gets 2^kS.
template <typename T>
struct GradScale;
template <>
struct GradScale<__half> {
  static constexpr float kP = 14.0f, kS = 0.0f;
};
template <>
struct GradScale<__nv_bfloat16> {
  static constexpr float kP = 24.0f, kS = 24.0f;
};
__device__ __forceinline__ constexpr float grad_scale_down(float k) {   // 2^-k
  return k == 0.0f ? 1.0f : (k == 14.0f ? 1.0f / 16384.0f : 1.0f / 16777216.0f);
}
// ds = (2^kP p) * (dp * kC - delta * kC)
template <typename T>
constexpr float kGradC = GradScale<T>::kP == GradScale<T>::kS ? 1.0f : 1.0f / 16384.0f;

// delta = rowsum(do * o), one team of D/8 lanes per row

template <typename T, int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnParams p) {
  constexpr int L = D / 8, TEAMS = 256 / L;
  const int team = threadIdx.x / L, lane = threadIdx.x % L;
  const long long items = static_cast<long long>(p.batch) * p.seq_q * p.heads_q;
  grid_dependency_wait();
  // (row, head) with the heads of a row next to each other
  for (long long first = static_cast<long long>(blockIdx.x) * TEAMS; first < items;
       first += static_cast<long long>(gridDim.x) * TEAMS) {
    const long long it = first + team;
    float s = 0.0f;
    const long long row = it / p.heads_q;
    const int h = static_cast<int>(it - row * p.heads_q);
    if (it < items) {
      const char* a = p.o_in + row * p.o_stride + h * (D * 2) + lane * 16;
      const char* d = p.dout + row * p.dout_stride + h * (D * 2) + lane * 16;
      if (in_span(a, 16, p.sp_o, p.status) && in_span(d, 16, p.sp_dout, p.status)) {
        float2 x[4], y[4];
        Elem<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(a)), x);
        Elem<T>::unpack(*reinterpret_cast<const uint4*>(d), y);
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __ffma2_rn(x[i], y[i], acc);
        s = __fadd_rn(acc.x, acc.y);
      }
    }
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    if (it < items && lane == 0) {
      const long long b = row / p.seq_q;
      float* out = p.delta + (b * p.heads_q + h) * p.seq_q + (row - b * p.seq_q);
      if (in_span(out, 4, p.sp_delta, p.status)) *out = s;
    }
  }
  grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// backward, dq: a CTA takes 128 queries of one head and walks their keys.
// Per block S = Q K^T, dP = dO V^T, dQ += dS K.  The scores have two buffers,
// so the next block's S is there when this block's dS is done.

namespace dq {
constexpr int kK = 3, kV = 2;                     // K and V tiles in flight
enum { Q_FULL = 0, K_FULL = 1, K_EMPTY = K_FULL + kK, V_FULL = K_EMPTY + kK, V_EMPTY = V_FULL + kV,
       S_FULL = V_EMPTY + kV, DP_FULL = S_FULL + 2, DP_FREE, DS_FULL, DONE, DRAIN, BARS };
template <int D>
constexpr int kSmem = (2 + kK + kV) * kTileBytes<D> + 256;
}  // namespace dq

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_dq_kernel(const __grid_constant__ AttnParams p) {
  using namespace dq;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + (2 + kK + kV) * kTileBytes<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
            __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), i == DP_FREE || i == DS_FULL ? 8 : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();

  const int tile = p.causal ? p.tiles - 1 - static_cast<int>(blockIdx.x % p.tiles) : static_cast<int>(blockIdx.x % p.tiles);
  const int h = static_cast<int>(blockIdx.x / p.tiles % p.heads_q), b = static_cast<int>(blockIdx.x / p.tiles / p.heads_q);
  const int q0 = tile * kTile;
  const int q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
  const int k_len = clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
  const int diag = k_len - q_len;
  const int last = q0 + kTile < q_len ? q0 + kTile : q_len;
  int keys = q0 >= q_len ? 0 : (p.causal ? last + diag : k_len);
  keys = keys < 0 ? 0 : (keys > k_len ? k_len : keys);
  const int n = (keys + kTile - 1) / kTile;
  const uint32_t sq = c.base, sdo = c.base + kTileBytes<D>, sk = c.base + 2 * kTileBytes<D>,
                 sv = c.base + (2 + kK) * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && n > 0) {
      const int hk = h / p.group;
      int ik = 0, iv = 0;
      bool ok = !(p.flags & 1u);
      if (ok) {
        mbar_arrive_expect_tx(c.bar(Q_FULL), 2 * kTileBytes<D>);
        tma_load_tile(sq, &p.map_q, q0, h, b, c.bar(Q_FULL));
        tma_load_tile(sdo, &p.map_do, q0, h, b, c.bar(Q_FULL));
        RingPos<kK> k;
        RingPos<kV> v;
        for (int j = 0; j < n; ++j, k.step(), v.step()) {
          ok = c.wait1(K_EMPTY + k.s, k.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(K_FULL + k.s), kTileBytes<D>);
          tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_k, j * kTile, hk, b, c.bar(K_FULL + k.s));
          ++ik;
          ok = c.wait1(V_EMPTY + v.s, v.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(V_FULL + v.s), kTileBytes<D>);
          tma_load_tile(sv + v.s * kTileBytes<D>, &p.map_v, j * kTile, hk, b, c.bar(V_FULL + v.s));
          ++iv;
        }
      }
      if (!ok || *abort_flag) {
        const unsigned long long t0 = global_timer_ns();
        for (int i = ik > kK ? ik - kK : 0; i < ik; ++i)
          while (!mbar_try_wait(c.bar(K_FULL + i % kK), (i / kK) & 1) && global_timer_ns() - t0 < c.limit) {
          }
        for (int i = iv > kV ? iv - kV : 0; i < iv; ++i)
          while (!mbar_try_wait(c.bar(V_FULL + i % kV), (i / kV) & 1) && global_timer_ns() - t0 < c.limit) {
          }
        while (!(p.flags & 1u) && !mbar_try_wait(c.bar(Q_FULL), 0) && global_timer_ns() - t0 < c.limit) {
        }
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp) {
    bool ok = n > 0;
    const bool ragged = k_len < p.seq_k;
    // Blocks whose scores, dP and dQ products come next, and their stages.
    RingPos<kK> ks, kd;
    RingPos<kV> vs;
    int js = 0, jv = 0;
    // the block's K (V) has landed, with nothing past the sample's keys
    auto have = [&](int full, int tile_at, uint32_t phase, int j) {
      const bool got = c.wait(full, phase);
      if (got && ragged && (j + 1) * kTile > k_len)
        zero_rows<D>(smem + tile_at * kTileBytes<D>, k_len - j * kTile, c.lane);
      return got;
    };
    auto scores = [&]() {
      if (!have(K_FULL + ks.s, 2 + ks.s, ks.phase, js)) return false;
      if (elect_one()) {
        mma_rows<T, D>(tmem + (js & 1) * kTile, sq, sk + ks.s * kTileBytes<D>);
        mma_commit(c.bar(S_FULL + (js & 1)));
      }
      ks.step();
      ++js;
      return true;
    };
    auto grads = [&]() {
      if (!have(V_FULL + vs.s, 2 + kK + vs.s, vs.phase, jv)) return false;
      if (elect_one()) {
        mma_rows<T, D>(tmem + 2 * kTile, sdo, sv + vs.s * kTileBytes<D>);
        mma_commit(c.bar(DP_FULL));
        mma_commit(c.bar(V_EMPTY + vs.s));
      }
      vs.step();
      ++jv;
      return true;
    };
    ok = ok && c.wait(Q_FULL, 0) && scores() && grads() && (n == 1 || scores());
    for (int j = 0; ok && j < n; ++j) {
      if (j + 1 < n) {
        ok = c.wait(DP_FREE, j);
        tc_fence_after();
        if (!ok) break;
        ok = grads();
        if (!ok) break;
      }
      ok = c.wait(DS_FULL, j);
      tc_fence_after();
      if (!ok) break;
      if (elect_one()) {
        mma_cols<T, D, true>(tmem + 3 * kTile, tmem + (j & 1) * kTile, sk + kd.s * kTileBytes<D>, j > 0);
        mma_commit(c.bar(K_EMPTY + kd.s));
      }
      kd.step();
      if (j + 2 < n) ok = scores();
    }
    if (ok && elect_one()) mma_commit(c.bar(DONE));
    if (!ok && n > 0) {
      if (elect_one()) mma_commit(c.bar(DRAIN));
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(c.bar(DRAIN), 0) && global_timer_ns() - t0 < c.limit) {
      }
    }
    __syncwarp();
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // a thread per query and half of the block's keys
    const int half = c.warp >> 2;
    const int row = q0 + (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const bool valid = row < q_len;
    int limit = valid ? (p.causal ? row + diag + 1 : k_len) : 0;
    limit = limit < 0 ? 0 : (limit > k_len ? k_len : limit);
    float lse2 = INFINITY, delta = 0.0f;          // p = 0 for a row that sees nothing
    const long long at = (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + row;
    if (limit > 0 && in_span(p.lse + at, 4, p.sp_lse, p.status) && in_span(p.delta + at, 4, p.sp_delta, p.status)) {
      const float v = p.lse[at];
      lse2 = v == -INFINITY ? INFINITY : __fmul_rn(v, kLog2e);
      delta = p.delta[at];
    }
    const float nl = GradScale<T>::kP - lse2, nd = -delta * kGradC<T>;
    const float2 SL = make_float2(p.scale_log2, p.scale_log2), NL = make_float2(nl, nl), ND = make_float2(nd, nd),
                 C = make_float2(kGradC<T>, kGradC<T>);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t ts = tmem + (j & 1) * kTile + half * 64 + lanes, tdp = tmem + 2 * kTile + half * 64 + lanes;
      ok = c.wait(S_FULL + (j & 1), j >> 1);
      if (!ok) break;
      tc_fence_after();
      float s[2][32];
      tmem_load32(ts, s[0]);
      tmem_load32(ts + 32, s[1]);
      tmem_wait_load(s[0]);
      tmem_loaded(s[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = __ffma2_rn(make_float2(s[i][e], s[i][e + 1]), SL, NL);
          s[i][e] = exp2_approx(x.x);
          s[i][e + 1] = exp2_approx(x.y);
        }
      ok = c.wait(DP_FULL, j);
      if (!ok) break;
      tc_fence_after();
      float d[2][32];
      tmem_load32(tdp, d[0]);
      tmem_load32(tdp + 32, d[1]);
      tmem_wait_load(d[0]);
      tmem_loaded(d[1]);
      c.arrive(DP_FREE);
      const int seen = limit - j * kTile - half * 64;
      if (__any_sync(0xffffffffu, seen < 64)) {
        // p = 0 and a finite dp - delta where the row does not see the key
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            s[i][e] = 32 * i + e < seen ? s[i][e] : 0.0f;
            d[i][e] = 32 * i + e < seen ? d[i][e] : 0.0f;
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __fmul2_rn(make_float2(s[i][2 * e], s[i][2 * e + 1]),
                                      __ffma2_rn(make_float2(d[i][2 * e], d[i][2 * e + 1]), C, ND));
          w[e] = pack2<T>(x.x, x.y);
        }
        tmem_store16(ts + 16 * i, w);
      }
      tmem_wait_store();
      c.arrive(DS_FULL);
    }
    if (ok && n > 0) ok = c.wait(DONE, 0);
    tc_fence_after();
    char* dst = p.dq + (static_cast<long long>(b) * p.seq_q + row) * p.dq_stride + h * (D * 2) + half * D;
    const bool fits = ok && row < p.seq_q && in_span(dst, D, p.sp_dq, p.status);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      float v[32];
      if (ok && n > 0) {
        tmem_load32(tmem + 3 * kTile + half * (D / 2) + 32 * i + lanes, v);
        tmem_wait_load(v);
      }
      if (fits) store_cols<T>(dst + 64 * i, v, p.scale * grad_scale_down(GradScale<T>::kS), n > 0 && limit > 0);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// backward, dk and dv: a CTA takes 128 keys of one key head and walks the
// queries of every head that shares it.  Per block, transposed so that P and
// dS come out as left operands: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO,
// dK += dS^T Q.

namespace dkv {
constexpr int kQ = 3, kO = 2;                     // Q and dO tiles in flight
enum { KV_FULL = 0, Q_FULL = 1, Q_EMPTY = Q_FULL + kQ, O_FULL = Q_EMPTY + kQ, O_EMPTY = O_FULL + kO,
       S_FULL = O_EMPTY + kO, P_FULL, DP_FULL, DS_FULL, ROWS, ROWS_FREE = ROWS + 2,
       DONE = ROWS_FREE + 2, DRAIN, BARS };
constexpr int kRowBytes = 2 * 2 * kTile * 4;      // two buffers of (lse, delta) of a tile's queries
template <int D>
constexpr int kSmem = (2 + kQ + kO) * kTileBytes<D> + kRowBytes + 256;
}  // namespace dkv

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_dkv_kernel(const __grid_constant__ AttnParams p) {
  using namespace dkv;
  extern __shared__ __align__(1024) unsigned char smem[];
  float* rows = reinterpret_cast<float*>(smem + (2 + kQ + kO) * kTileBytes<D>);   // [2][2][128]
  unsigned char* ctl = smem + (2 + kQ + kO) * kTileBytes<D> + kRowBytes;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
            __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), i == P_FULL || i == DS_FULL || (i >= ROWS_FREE && i < DONE) ? 8 : (i >= ROWS && i < ROWS_FREE ? 2 : 1));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();

  const int hk = static_cast<int>(blockIdx.x / p.tiles % p.heads_k), b = static_cast<int>(blockIdx.x / p.tiles / p.heads_k);
  const int k0 = static_cast<int>(blockIdx.x % p.tiles) * kTile;
  const int q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
  const int k_len = clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
  const int diag = k_len - q_len;
  // query tiles [first, end) see one of these keys
  int first = 0, end = (q_len + kTile - 1) / kTile;
  if (p.causal && k0 - diag > 0) first = (k0 - diag) / kTile;
  if (k0 >= k_len || first > end) first = end;
  const int per_head = end - first, n = per_head * p.group;
  const uint32_t sk = c.base, sv = c.base + kTileBytes<D>, sq = c.base + 2 * kTileBytes<D>,
                 sdo = c.base + (2 + kQ) * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && n > 0) {
      int iq = 0, io = 0;
      bool ok = !(p.flags & 1u);
      if (ok) {
        mbar_arrive_expect_tx(c.bar(KV_FULL), 2 * kTileBytes<D>);
        tma_load_tile(sk, &p.map_k, k0, hk, b, c.bar(KV_FULL));
        tma_load_tile(sv, &p.map_v, k0, hk, b, c.bar(KV_FULL));
        RingPos<kQ> q;
        RingPos<kO> o;
        int h = hk * p.group, t = first;
        for (int i = 0; i < n; ++i, q.step(), o.step()) {
          ok = c.wait1(Q_EMPTY + q.s, q.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(Q_FULL + q.s), kTileBytes<D>);
          tma_load_tile(sq + q.s * kTileBytes<D>, &p.map_q, t * kTile, h, b, c.bar(Q_FULL + q.s));
          ++iq;
          ok = c.wait1(O_EMPTY + o.s, o.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(O_FULL + o.s), kTileBytes<D>);
          tma_load_tile(sdo + o.s * kTileBytes<D>, &p.map_do, t * kTile, h, b, c.bar(O_FULL + o.s));
          ++io;
          if (++t == end) {
            t = first;
            ++h;
          }
        }
      }
      if (!ok || *abort_flag) {
        const unsigned long long t0 = global_timer_ns();
        for (int i = iq > kQ ? iq - kQ : 0; i < iq; ++i)
          while (!mbar_try_wait(c.bar(Q_FULL + i % kQ), (i / kQ) & 1) && global_timer_ns() - t0 < c.limit) {
          }
        for (int i = io > kO ? io - kO : 0; i < io; ++i)
          while (!mbar_try_wait(c.bar(O_FULL + i % kO), (i / kO) & 1) && global_timer_ns() - t0 < c.limit) {
          }
        while (!(p.flags & 1u) && !mbar_try_wait(c.bar(KV_FULL), 0) && global_timer_ns() - t0 < c.limit) {
        }
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp) {
    bool ok = n > 0;
    const bool ragged = q_len < p.seq_q;
    // Blocks whose scores, dP, dV and dK products come next.
    RingPos<kQ> qs, qd;
    RingPos<kO> os, od;
    int ts = first, to = first;                   // their query tiles
    // the tile has landed, with nothing past the sample's queries
    auto have = [&](int full, int tile_at, uint32_t phase, int& t) {
      const bool got = c.wait(full, phase);
      if (got && ragged && (t + 1) * kTile > q_len) zero_rows<D>(smem + tile_at * kTileBytes<D>, q_len - t * kTile, c.lane);
      if (++t == end) t = first;
      return got;
    };
    auto scores = [&]() {
      if (!have(Q_FULL + qs.s, 2 + qs.s, qs.phase, ts)) return false;
      if (elect_one()) {
        mma_rows<T, D>(tmem, sk, sq + qs.s * kTileBytes<D>);
        mma_commit(c.bar(S_FULL));
      }
      qs.step();
      return true;
    };
    auto grads = [&]() {
      if (!have(O_FULL + os.s, 2 + kQ + os.s, os.phase, to)) return false;
      if (elect_one()) {
        mma_rows<T, D>(tmem + kTile, sv, sdo + os.s * kTileBytes<D>);
        mma_commit(c.bar(DP_FULL));
      }
      os.step();
      return true;
    };
    ok = ok && c.wait(KV_FULL, 0) && scores() && grads();
    for (int i = 0; ok && i < n; ++i) {
      ok = c.wait(P_FULL, i);
      tc_fence_after();
      if (!ok) break;
      if (elect_one()) {
        mma_cols<T, D, true>(tmem + 2 * kTile, tmem, sdo + od.s * kTileBytes<D>, i > 0);
        mma_commit(c.bar(O_EMPTY + od.s));
      }
      od.step();
      if (i + 1 < n) {
        ok = scores();
        if (!ok) break;
      }
      ok = c.wait(DS_FULL, i);
      tc_fence_after();
      if (!ok) break;
      if (elect_one()) {
        mma_cols<T, D, true>(tmem + 3 * kTile, tmem + kTile, sq + qd.s * kTileBytes<D>, i > 0);
        mma_commit(c.bar(Q_EMPTY + qd.s));
      }
      qd.step();
      if (i + 1 < n) ok = grads();
    }
    if (ok && elect_one()) mma_commit(c.bar(DONE));
    if (!ok && n > 0) {
      if (elect_one()) mma_commit(c.bar(DRAIN));
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(c.bar(DRAIN), 0) && global_timer_ns() - t0 < c.limit) {
      }
    }
    __syncwarp();
  } else if (c.warp >= kAttnMmaWarp) {
    // Warps 10 and 11 hand round kP - lse (log2) and -delta kC of the blocks'
    // queries, up to two blocks ahead.  A query past the length or with no
    // key gets -inf: p = 0.
    const bool second = c.warp == kAttnMmaWarp + 3;
    const float* source = second ? p.delta : p.lse;
    const MemSpan& sp_source = second ? p.sp_delta : p.sp_lse;
    int h = hk * p.group, t = first;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const float* at = source + (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + t * kTile + c.lane;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = t * kTile + 32 * e + c.lane;
        v[e] = second ? 0.0f : -INFINITY;
        if (q < q_len && in_span(at + 32 * e, 4, sp_source, p.status)) v[e] = at[32 * e];
      }
      // the block before last has been read
      ok = i < 2 || c.wait(ROWS_FREE + (i & 1), (i >> 1) - 1);
      if (!ok) break;
      float* out = rows + (i & 1) * 2 * kTile + (second ? kTile : 0) + c.lane;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[32 * e] = second ? -v[e] * kGradC<T> : (v[e] == -INFINITY ? -INFINITY : __fmaf_rn(v[e], -kLog2e, GradScale<T>::kP));
      __syncwarp();
      if (c.lane == 0) mbar_arrive(c.bar(ROWS + (i & 1)));
      if (++t == end) {
        t = first;
        ++h;
      }
    }
  } else {
    more_registers<kAttnWorkRegs>();
    // a thread per key and half of the block's queries
    const int half = c.warp >> 2;
    const int key = k0 + (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const uint32_t ts = tmem + half * 64 + lanes, tdp = tmem + kTile + half * 64 + lanes;
    const float2 SL = make_float2(p.scale_log2, p.scale_log2), C = make_float2(kGradC<T>, kGradC<T>);
    bool ok = true;
    int t = first;                                // the block's query tile
    for (int i = 0; i < n; ++i) {
      const float* mine = rows + (i & 1) * 2 * kTile;
      const float4* nl = reinterpret_cast<const float4*>(mine + half * 64);
      const float4* nd = reinterpret_cast<const float4*>(mine + kTile + half * 64);
      ok = c.wait(ROWS + (i & 1), i >> 1) && c.wait(S_FULL, i);
      if (!ok) break;
      tc_fence_after();
      float s[2][32];
      tmem_load32(ts, s[0]);
      tmem_load32(ts + 32, s[1]);
      tmem_wait_load(s[0]);
      tmem_loaded(s[1]);
      // query q0 + c sees this key when c >= from
      const int from = p.causal ? key - diag - t * kTile - half * 64 : 0;
      if (++t == end) t = first;
      const bool masked = __any_sync(0xffffffffu, from > 0);
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 l4 = nl[a * 8 + e];
          float* x = &s[a][4 * e];
          const float2 u = __ffma2_rn(make_float2(x[0], x[1]), SL, make_float2(l4.x, l4.y));
          const float2 v = __ffma2_rn(make_float2(x[2], x[3]), SL, make_float2(l4.z, l4.w));
          x[0] = exp2_approx(u.x);
          x[1] = exp2_approx(u.y);
          x[2] = exp2_approx(v.x);
          x[3] = exp2_approx(v.y);
        }
      if (masked) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 32; ++e) s[a][e] = 32 * a + e >= from ? s[a][e] : 0.0f;
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack2<T>(s[a][2 * e], s[a][2 * e + 1]);
        tmem_store16(ts + 16 * a, w);
      }
      tmem_wait_store();
      c.arrive(P_FULL);
      ok = c.wait(DP_FULL, i);
      if (!ok) break;
      tc_fence_after();
      float d[2][32];
      tmem_load32(tdp, d[0]);
      tmem_load32(tdp + 32, d[1]);
      tmem_wait_load(d[0]);
      tmem_loaded(d[1]);
      if (masked) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 32; ++e) d[a][e] = 32 * a + e >= from ? d[a][e] : 0.0f;
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 d4 = nd[a * 8 + e];
          const float* x = &s[a][4 * e];
          const float2 u = __fmul2_rn(make_float2(x[0], x[1]),
                                      __ffma2_rn(make_float2(d[a][4 * e], d[a][4 * e + 1]), C, make_float2(d4.x, d4.y)));
          const float2 v = __fmul2_rn(make_float2(x[2], x[3]),
                                      __ffma2_rn(make_float2(d[a][4 * e + 2], d[a][4 * e + 3]), C, make_float2(d4.z, d4.w)));
          w[2 * e] = pack2<T>(u.x, u.y);
          w[2 * e + 1] = pack2<T>(v.x, v.y);
        }
        tmem_store16(tdp + 16 * a, w);
      }
      tmem_wait_store();
      c.arrive(DS_FULL);
      if (c.lane == 0) mbar_arrive(c.bar(ROWS_FREE + (i & 1)));
    }
    if (ok && n > 0) ok = c.wait(DONE, 0);
    tc_fence_after();
    // the first group writes dv, the second dk
    const float f = half ? p.scale * grad_scale_down(GradScale<T>::kS) : grad_scale_down(GradScale<T>::kP);
    char* dst = half ? p.dk + (static_cast<long long>(b) * p.seq_k + key) * p.dk_stride + hk * (D * 2)
                     : p.dv + (static_cast<long long>(b) * p.seq_k + key) * p.dv_stride + hk * (D * 2);
    const bool fits = ok && key < p.seq_k && in_span(dst, D * 2, half ? p.sp_dk : p.sp_dv, p.status);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float v[32];
      if (ok && n > 0) {
        tmem_load32(tmem + (2 + half) * kTile + 32 * i + lanes, v);
        tmem_wait_load(v);
      }
      if (fits) store_cols<T>(dst + 64 * i, v, f, n > 0 && key < k_len);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  grid_dependents_launch();
}

}  // namespace qknr
