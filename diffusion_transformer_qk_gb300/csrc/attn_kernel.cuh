// Attention forward and backward for sm_103a (formulas: qknr_attn.h).
//
// The products of the three kernels here that have some (forward, dq, and dk
// with dv) run on tcgen05 with operands that TMA leaves in shared memory and
// accumulators in tensor memory; the probabilities (and the score gradients) go
// back to tensor memory as 16-bit left operands of the second product, in the
// columns whose scores they replace.  Operands of one product have one type, so
// that rounding is what 16-bit queries, keys and values cost: h of each
// probability, where the formula in 32 bits rounds the output alone.  MMAs of
// one thread run in order, so a product that overwrites an operand of an
// earlier one needs no wait in between.
//
// Roles of a CTA's 12 warps: 0-7 are two groups of four that each cover the
// 128 lanes of tensor memory (a thread owns one row of a score tile), warp 8
// issues the MMAs, warp 9 the TMA loads.  In the backward kernels warp 10
// issues a second chain of products that does not depend on the first one's
// order, so that what one warp spends on waits the other's products fill; in
// the dk, dv kernel warp 11 hands round the queries' statistics.  The third
// group's registers go to the first two.
//
// Persistent CTAs, one per SM.  Tile w of CTA c is tile w * CTAs + c, so that
// CTAs next to each other read the same keys; the tiles left over after the
// last full wave are cut along their contraction into as many equal parts as
// there are CTAs, whose fp32 partial results attn_join_*_kernel adds in a
// fixed order.  A causal mask's tiles go out whole, or all of them as two
// halves, costly ones first.
// A tile's loads, its first products and the previous tile's epilogue overlap.
// Every wait is bounded; a role that gives up sets the CTA's abort flag,
// drains what it started and leaves.
#pragma once

#include "tc.cuh"

namespace qknr {

struct AttnParams {
  CUtensorMap map_q, map_k, map_v, map_do;
  CUtensorMap map_out;        // o or dq: boxes of kOutRows rows of a warp
  const char* q_in;           // few queries: read without a map
  long long q_stride;
  const char* o_in;           // backward: the forward's output
  const char* dout;
  char* o;
  char* dq;
  char* dk;
  char* dv;
  float* lse;
  float* delta;               // [batch][heads_q][seq_q]
  // fp16 backward: what dS's powers of two come from
  const char* v_in;
  long long v_stride;
  float* dout_norm;           // |do| of each row, like delta
  float* v_top;               // [delta kernel's CTAs] none of its rows of v is longer
  int v_tops;
  float* ds_top;              // [batch][heads_q][q_tiles][4] the largest bound on |ds| among 32 rows
  int q_tiles;                // 128-row tiles of the queries
  long long o_stride, dout_stride, dq_stride, dk_stride, dv_stride;   // bytes per row
  const int* q_lens;
  const int* k_lens;
  int batch, seq_q, seq_k, heads_q, heads_k, group;
  int causal;
  float scale, scale_log2;
  int tiles;                  // row tiles of a head
  int total;                  // tiles in all
  int halves;                 // every tile goes out as two halves of its contraction
  int waves;                  // whole tiles (or halves) per CTA
  int rem;                    // tiles after those, shared out among all CTAs
  float* part;                // their partial results, two slots per CTA
  float* stats;               // forward: (maximum, sum) of the slots' rows
  unsigned flags;
  int* status;
  unsigned long long wait_limit_ns;
  MemSpan sp_q, sp_o, sp_dout, sp_dq, sp_dk, sp_dv, sp_lse, sp_delta, sp_q_lens, sp_k_lens, sp_part, sp_stats,
      sp_v, sp_dout_norm, sp_v_top, sp_ds_top;
};

constexpr int kAttnThreads = 384;
constexpr int kAttnMmaWarp = 8, kAttnLoadWarp = 9, kAttnMma2Warp = 10, kAttnRowWarp = 11;
constexpr int kTile = 128;                        // rows of a tile, both ways
constexpr int kFewRows = 16;                      // rows of a tile of a few queries (attn_few.cuh)
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

// the same with A 16-bit in tensor memory
template <typename T, int D>
__device__ __forceinline__ void mma_rows_ts(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = mma_desc<T>(kTile, kTile, false);
  const uint32_t db = desc_k_major(b);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    mma_ts(d, a + k * 8, db + (((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4), idesc, k > 0);
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
  __device__ __forceinline__ void skip(int n) {
    s += n;
    phase ^= static_cast<uint32_t>(s / N) & 1u;
    s %= N;
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
  // Whole warp, three barriers that are likely to be complete: lane 0 looks at
  // the first, lane 1 at the second, the others at the third.  Shared memory
  // answers slowly while the tensor cores read it: one look after the other
  // costs 100 to 150 cycles each.
  __device__ __forceinline__ bool wait(int i, uint32_t pi, int j, uint32_t pj, int k, uint32_t pk) const {
    const int mine = lane == 0 ? i : (lane == 1 ? j : k);
    const uint32_t phase = lane == 0 ? pi : (lane == 1 ? pj : pk);
    if (__all_sync(0xffffffffu, mbar_test(bar(mine), phase & 1u))) return true;
    return wait(i, pi) && wait(j, pj) && wait(k, pk);
  }
  // One thread, giving up: the last `n` of `issued` copies into a ring of n
  // stages end before the CTA leaves its shared memory.
  __device__ __forceinline__ void drain(int full, int n, int issued) const {
    const unsigned long long t0 = global_timer_ns();
    for (int i = issued > n ? issued - n : 0; i < issued; ++i)
      while (!mbar_try_wait(bar(full + i % n), static_cast<uint32_t>(i / n) & 1u) && global_timer_ns() - t0 < limit) {
      }
  }
  // Whole warp, giving up: the MMAs in flight end before tensor memory is given back.
  __device__ __forceinline__ void drain_mma(int i) const {
    if (elect_one()) mma_commit(bar(i));
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar(i), 0) && global_timer_ns() - t0 < limit) {
    }
    __syncwarp();
  }
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // a warp's arrival after its tensor memory accesses
  __device__ __forceinline__ void arrive(int i) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  }
};

// One piece of a CTA's work: a tile and which part of its contraction, in
// 1024ths; `slot` is where a partial result goes (-1: the tile is whole).
constexpr int kUnits = 1024;
struct AttnWork {
  int tile, u0, u1, slot;
};

// first unit of CTA c's share of the tiles left over
__device__ __forceinline__ long long attn_share(const AttnParams& p, long long c, int ctas) {
  return c * p.rem * kUnits / ctas;
}

__device__ __forceinline__ bool attn_work(const AttnParams& p, int s, AttnWork& w) {
  const int n = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  if (s < p.waves) {
    // with a causal mask a wave's tiles cost less and less: every other wave
    // goes round the other way
    const int item = s * n + (p.causal && (s & 1) ? n - 1 - c : c), second = item & 1;
    w = p.halves ? AttnWork{item >> 1, second * (kUnits / 2), (second + 1) * (kUnits / 2), item} : AttnWork{item, 0, kUnits, -1};
    return w.tile < p.total;
  }
  const int k = s - p.waves;
  if (p.rem == 0 || k > 1) return false;
  const long long v0 = attn_share(p, c, n), v1 = attn_share(p, c + 1, n);
  const int r = static_cast<int>(v0 / kUnits) + k;
  const long long lo = v0 > static_cast<long long>(r) * kUnits ? v0 : static_cast<long long>(r) * kUnits;
  const long long hi = v1 < static_cast<long long>(r + 1) * kUnits ? v1 : static_cast<long long>(r + 1) * kUnits;
  if (lo >= hi) return false;
  w = AttnWork{p.waves * n + r, static_cast<int>(lo - static_cast<long long>(r) * kUnits),
               static_cast<int>(hi - static_cast<long long>(r) * kUnits), 2 * c + k};
  return true;
}

// The tile's place.  Without a causal mask the tiles of a head follow each
// other; with one, tiles of the same cost do (`heavy_last`: the later rows
// cost more), the costly ones first.
struct AttnPlace {
  int t, h, b;
};
__device__ __forceinline__ AttnPlace attn_place(const AttnParams& p, int tile, int heads, bool heavy_last) {
  if (p.causal) {
    const int per = heads * p.batch, t = tile / per, r = tile - t * per;
    return AttnPlace{heavy_last ? p.tiles - 1 - t : t, r % heads, r / heads};
  }
  const int r = tile / p.tiles;
  return AttnPlace{tile - r * p.tiles, r % heads, r / heads};
}

// iterations [begin, end) of n that a piece takes
__device__ __forceinline__ void attn_cut(const AttnWork& w, int n, int& begin, int& end) {
  begin = static_cast<int>(static_cast<long long>(n) * w.u0 / kUnits);
  end = static_cast<int>(static_cast<long long>(n) * w.u1 / kUnits);
}

// Epilogue stores.  A thread holds pieces of its own row; stored as they are,
// every store instruction touches 32 rows, a cache line each (6000 cycles for
// a 128 x 128 tile).  Where shared memory is left, a warp stages its rows
// there and one TMA store writes them.
constexpr int kOutRows = 32;

// 32 accumulator values of each row of a warp, times f (zero where the row has
// no value), in the output's type: chunks [first, first + 4) of the staged
// rows, COLS values each, where the map's swizzle expects them.
template <typename T, int COLS>
__device__ __forceinline__ void stage_cols(unsigned char* stage, int first, const float (&v)[32], float f, bool some, int lane) {
  const int flip = COLS == 64 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 w;
    uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ww[i] = some ? pack2<T>(__fmul_rn(v[c * 8 + 2 * i], f), __fmul_rn(v[c * 8 + 2 * i + 1], f)) : 0u;
    *reinterpret_cast<uint4*>(stage + lane * (COLS * 2) + (((first + c) ^ flip) << 4)) = w;
  }
}

// Elsewhere the four lanes of a quad first swap 16-byte chunks: afterwards
// v[k] is chunk (lane & 3) of the quad's k-th row, and an instruction writes 64
// bytes of each of eight rows (3700 cycles).
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step <<= 1) {
    const bool upper = lane & step;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & step) continue;
      uint4& lo = v[k];
      uint4& hi = v[k + step];
      uint4 give = upper ? lo : hi;
      give.x = __shfl_xor_sync(0xffffffffu, give.x, step);
      give.y = __shfl_xor_sync(0xffffffffu, give.y, step);
      give.z = __shfl_xor_sync(0xffffffffu, give.z, step);
      give.w = __shfl_xor_sync(0xffffffffu, give.w, step);
      if (upper) lo = give;
      else hi = give;
    }
  }
}

// 32 accumulator values of each row of a warp, times f (zero where the row has
// no value), in the output's type.  `dst`: this thread's place in its own row;
// rows are `stride` bytes apart, the warp's first `rows` of them are there.
template <typename T>
__device__ __forceinline__ void store_cols(char* dst, long long stride, int rows, const float (&v)[32], float f, bool some,
                                           int lane) {
  uint4 w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t* ww = reinterpret_cast<uint32_t*>(&w[c]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ww[i] = some ? pack2<T>(__fmul_rn(v[c * 8 + 2 * i], f), __fmul_rn(v[c * 8 + 2 * i + 1], f)) : 0u;
  }
  quad_transpose(w, lane);
  char* at = dst - (lane & 3) * stride + (lane & 3) * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if ((lane & ~3) + k < rows) *reinterpret_cast<uint4*>(at + k * stride) = w[k];
}

// the same values as a partial result: fp32 rows of D values, times f
template <int D>
__device__ __forceinline__ void store_part(float* dst, const float (&v)[32], float f, bool some, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float* x = &v[16 * h + 4 * c];
      w[c] = some ? make_uint4(__float_as_uint(x[0] * f), __float_as_uint(x[1] * f), __float_as_uint(x[2] * f), __float_as_uint(x[3] * f))
                  : make_uint4(0, 0, 0, 0);
    }
    quad_transpose(w, lane);
    float* at = dst - (lane & 3) * D + (lane & 3) * 4 + 16 * h;
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(at + k * D) = w[k];
  }
}

// ---------------------------------------------------------------------------
// The forward kernels' P carries 2^kPLift into its product and into the sum,
// which takes it out again.  In fp16 a probability below 2^-25 of the row's
// largest would round to zero: of N keys up to N 2^-25 of the sum, more than
// half a step of the output from 16384 on.  With 2^7 that is N 2^-32.
template <typename T>
constexpr float kPLift = 0.0f;
template <>
constexpr float kPLift<__half> = 7.0f;
// the log of a sum of such values
template <typename T>
__device__ __forceinline__ float log_sum(float total) {
  return logf(kPLift<T> == 0.0f ? total : __fmul_rn(total, 1.0f / 128.0f));
}

// ---------------------------------------------------------------------------
// forward: a tile is 256 queries of one head, two halves whose softmaxes
// alternate with each other's products, so that the tensor cores work on one
// while the other's row maxima, exponentials and conversions run.  One thread
// issues all products: with two the kernel is no faster.  At 2 x 4608 x 48 x
// 128 it takes 685 us, 1.52 PFLOP/s, near what the power limit leaves of a
// plain matrix product (1.71 sustained).

namespace fwd {
constexpr int kRows = 2 * kTile;
constexpr int kK = 2, kV = 2;                     // K and V tiles in flight
enum { Q_FULL = 0, Q_EMPTY = 2, K_FULL = 4, K_EMPTY = K_FULL + kK, V_FULL = K_EMPTY + kK, V_EMPTY = V_FULL + kV,
       S_FULL = V_EMPTY + kV, P_FULL = S_FULL + 2, O_DONE = P_FULL + 2, O_FREE = O_DONE + 2, DRAIN = O_FREE + 2, BARS };
__device__ __forceinline__ int arrivals(int i) {
  return (i >= P_FULL && i < O_DONE) || (i >= O_FREE && i < DRAIN) ? 4 : 1;
}
constexpr int kStage = kOutRows * 128;            // a warp's staged rows: 64 columns
template <int D>
constexpr int kCtl = (2 + kK + kV) * kTileBytes<D> + 8 * kStage;
template <int D>
constexpr int kSmem = kCtl<D> + 256;
// The running maximum is only raised, and the accumulator rescaled, when the
// new one is more than 2^8 above: p stays below 2^8 (2^15 with kPLift), which
// 16-bit floats and the fp32 sums hold as exactly as values below one.
constexpr float kSlack = 8.0f;

struct Seg {
  int b, h, q0, slot;
  int q_len, k_len, diag;     // causal: query i sees keys up to i + diag
  int begin;                  // first key block
  int nb[2];                  // key blocks of each half
  int blocks;
};
}  // namespace fwd

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_forward_kernel(const __grid_constant__ AttnParams p) {
  using namespace fwd;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + kCtl<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  const AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
                  __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), arrivals(i));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();
  grid_dependents_launch();

  auto segment = [&](int s, Seg& g) {
    AttnWork w;
    if (!attn_work(p, s, w)) return false;
    const AttnPlace at = attn_place(p, w.tile, p.heads_q, true);
    g.b = at.b;
    g.h = at.h;
    g.q0 = at.t * kRows;
    g.slot = w.slot;
    g.q_len = clamp_len(p.q_lens, at.b, p.seq_q, p.sp_q_lens, p.status);
    g.k_len = clamp_len(p.k_lens, at.b, p.seq_k, p.sp_k_lens, p.status);
    g.diag = g.k_len - g.q_len;
    int nb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = g.q0 + t * kTile, last = first + kTile < g.q_len ? first + kTile : g.q_len;
      int keys = first >= g.q_len ? 0 : (p.causal ? last + g.diag : g.k_len);
      keys = keys < 0 ? 0 : (keys > g.k_len ? g.k_len : keys);
      nb[t] = (keys + kTile - 1) / kTile;
    }
    int end;
    attn_cut(w, nb[0] > nb[1] ? nb[0] : nb[1], g.begin, end);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int last = nb[t] < end ? nb[t] : end;
      g.nb[t] = last > g.begin ? last - g.begin : 0;
    }
    g.blocks = g.nb[0] > g.nb[1] ? g.nb[0] : g.nb[1];
    return true;
  };
  const uint32_t sk = c.base + 2 * kTileBytes<D>, sv = c.base + (2 + kK) * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && !(p.flags & 1u)) {         // test only: issue nothing
      RingPos<kK> k;
      RingPos<kV> v;
      int uses[2] = {0, 0}, ik = 0, iv = 0;
      bool ok = true;
      Seg g;
      for (int s = 0; ok && segment(s, g); ++s) {
        {
          // the next tile's queries come from HBM: on their way while this one's keys come from L2
          Seg next;
          if (segment(s + 1, next))
            for (int t = 0; t < 2; ++t)
              if (next.nb[t]) tma_prefetch_tile(&p.map_q, next.q0 + t * kTile, next.h, next.b);
        }
        for (int t = 0; t < 2 && ok; ++t) {
          if (g.nb[t] == 0) continue;
          ok = c.wait1(Q_EMPTY + t, uses[t] + 1);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(Q_FULL + t), kTileBytes<D>);
          tma_load_tile(c.base + t * kTileBytes<D>, &p.map_q, g.q0 + t * kTile, g.h, g.b, c.bar(Q_FULL + t));
          ++uses[t];
        }
        const int hk = g.h / p.group;
        for (int j = 0; ok && j < g.blocks; ++j, k.step(), v.step()) {
          ok = c.wait1(K_EMPTY + k.s, k.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(K_FULL + k.s), kTileBytes<D>);
          tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_k, (g.begin + j) * kTile, hk, g.b, c.bar(K_FULL + k.s));
          ++ik;
          ok = c.wait1(V_EMPTY + v.s, v.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(V_FULL + v.s), kTileBytes<D>);
          tma_load_tile(sv + v.s * kTileBytes<D>, &p.map_v, (g.begin + j) * kTile, hk, g.b, c.bar(V_FULL + v.s));
          ++iv;
        }
      }
      if (!ok || *abort_flag) {
        c.drain(K_FULL, kK, ik);
        c.drain(V_FULL, kV, iv);
        c.drain(Q_FULL, 1, uses[0]);
        c.drain(Q_FULL + 1, 1, uses[1]);
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp) {
    // S_t(0), then per block and half in turn: O_t += P_t V, S_t(next)
    RingPos<kK> k;
    RingPos<kV> v;
    int uses[2] = {0, 0}, done[2] = {0, 0};       // tiles, blocks of each half so far
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      if (g.blocks == 0) continue;
      const int n0 = g.nb[0], n1 = g.nb[1], blocks = g.blocks;
      // the block whose V has rows past the sample's keys
      const int ragged = g.k_len < p.seq_k ? g.k_len / kTile - g.begin : blocks;
      ok = (n0 == 0 || c.wait(Q_FULL, uses[0])) && (n1 == 0 || c.wait(Q_FULL + 1, uses[1])) && c.wait(K_FULL + k.s, k.phase);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = t ? n1 : n0;
          if (n == 0) continue;
          mma_rows<T, D>(tmem + t * kTile, c.base + t * kTileBytes<D>, sk + k.s * kTileBytes<D>);
          mma_commit(c.bar(S_FULL + t));
          if (n == 1) mma_commit(c.bar(Q_EMPTY + t));
        }
        mma_commit(c.bar(K_EMPTY + k.s));
      }
      k.step();
      for (int j = 0; ok && j < blocks; ++j) {
        const bool more = j + 1 < blocks;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = t ? n1 : n0;
          const uint32_t ts = tmem + t * kTile, to = tmem + 2 * kTile + t * kTile;
          // this block's V, the next one's K, the half's P
          const int bv = V_FULL + v.s, bk = more ? K_FULL + k.s : bv, bp = j < n ? P_FULL + t : bv;
          const uint32_t pv = v.phase, pk = more ? k.phase : pv, pp = j < n ? done[t] : pv;
          if (t == 0) {
            ok = c.wait(bv, pv, bk, pk, bp, pp);
            if (!ok) break;
            if (j >= ragged) zero_rows<D>(smem + (2 + kK + v.s) * kTileBytes<D>, g.k_len - (g.begin + j) * kTile, c.lane);
          } else if (j < n) {
            ok = c.wait(bp, pp);
            if (!ok) break;
          }
          if (j < n) {
            ++done[t];
            // the accumulator has been read for the tile before
            ok = j > 0 || uses[t] == 0 || c.wait(O_FREE + t, uses[t] - 1);
            if (!ok) break;
          }
          tc_fence_after();
          if (elect_one()) {
            if (j < n) {
              mma_cols<T, D, false>(to, ts, sv + v.s * kTileBytes<D>, j > 0);
              mma_commit(c.bar(O_DONE + t));
            }
            if (t == 1) mma_commit(c.bar(V_EMPTY + v.s));
            if (j + 1 < n) {
              mma_rows<T, D>(ts, c.base + t * kTileBytes<D>, sk + k.s * kTileBytes<D>);
              mma_commit(c.bar(S_FULL + t));
              if (j + 2 == n) mma_commit(c.bar(Q_EMPTY + t));
            }
            if (t == 1 && more) mma_commit(c.bar(K_EMPTY + k.s));
          }
        }
        v.step();
        if (more) k.step();
      }
      uses[0] += n0 > 0;
      uses[1] += n1 > 0;
    }
    if (!ok) c.drain_mma(DRAIN);
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // softmax: a thread per query
    const int t = c.warp >> 2, r = (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const uint32_t ts = tmem + t * kTile + lanes, to = tmem + 2 * kTile + t * kTile + lanes;
    unsigned char* stage = smem + (2 + kK + kV) * kTileBytes<D> + c.warp * kStage;
    const float sl = p.scale_log2, slack = kSlack / sl;
    int done = 0;                                 // blocks so far
    bool ok = true;
    Seg g;
    for (int sg = 0; ok && segment(sg, g); ++sg) {
      const int n = t ? g.nb[1] : g.nb[0];
      int limit;                                  // keys from the first block on that this query sees
      {
        const int row = g.q0 + t * kTile + r;
        limit = row < g.q_len ? (p.causal ? row + g.diag + 1 : g.k_len) : 0;
        limit = (limit < 0 ? 0 : (limit > g.k_len ? g.k_len : limit)) - g.begin * kTile;
      }
      float m = -INFINITY;
      float2 sum = make_float2(0.0f, 0.0f);
      for (int j = 0; j < n; ++j, ++done) {
        ok = c.wait(S_FULL + t, done);
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
          for (int e = 2; e < 32; e += 2) mx[i] = max3(mx[i], s[i][e], s[i][e + 1]);
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + slack)) {
          const float raised = fmaxf(m, top);
          const float f = raised == m ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(m, raised), sl));
          m = raised;
          sum = __fmul2_rn(sum, make_float2(f, f));
          ok = c.wait(O_DONE + t, done - 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            tmem_fetch16(to + 16 * i, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), f));
            tmem_store16(to + 16 * i, o);
          }
        }
        // a row that has seen nothing yet: exp2(-inf - 0) = 0
        const float shift = m == -INFINITY ? 0.0f : (kPLift<T> == 0.0f ? __fmul_rn(-m, sl) : __fmaf_rn(-m, sl, kPLift<T>));
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
      if (!ok) break;
      if (n > 0) {
        ok = c.wait(O_DONE + t, done - 1);
        if (!ok) break;
        tc_fence_after();
      }
      const float total = __fadd_rn(sum.x, sum.y);
      const bool some = total != 0.0f;
      const float inv = some ? __frcp_rn(total) : 0.0f;
      segment(sg, g);                             // again: the loop above has no registers to keep it in
      const int row = g.q0 + t * kTile + r;
      const long long at = static_cast<long long>(g.slot) * kRows + t * kTile + r;   // a part's row
      if (g.slot >= 0) {
        // a part of the keys: unnormalised, with its maximum and sum
        if (in_span(p.stats + 2 * at, 8, p.sp_stats, p.status))
          *reinterpret_cast<float2*>(p.stats + 2 * at) = make_float2(m, total);
      } else {
        const long long l = (static_cast<long long>(g.b) * p.heads_q + g.h) * p.seq_q + row;
        if (row < p.seq_q && in_span(p.lse + l, 4, p.sp_lse, p.status))
          p.lse[l] = some ? __fmaf_rn(m, p.scale, log_sum<T>(total)) : -INFINITY;
      }
      // checked builds: the rows of a part that this warp writes (a store by TMA stays inside its map)
      const bool fits = __all_sync(0xffffffffu, g.slot < 0 || in_span(p.part + at * D, 4 * D, p.sp_part, p.status));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
        if (n > 0) {
          tmem_load32(to + 32 * i, o);
          tmem_wait_load(o);
          if (i == D / 32 - 1) c.arrive(O_FREE + t);
        }
        if (!fits) continue;
        if (g.slot >= 0) {
          store_part<D>(p.part + at * D + 32 * i, o, 1.0f, n > 0, c.lane);
          continue;
        }
        if (i % 2 == 0) {
          // the store before has read the stage
          if (c.lane == 0) tma_store_wait_read();
          __syncwarp();
        }
        stage_cols<T, 64>(stage, 4 * (i % 2), o, inv, some, c.lane);
        if (i % 2 == 1) {
          fence_async_shared();
          __syncwarp();
          if (c.lane == 0 && row < p.seq_q) tma_store_box(&p.map_out, smem_addr(stage), 0, row, i / 2, g.h, g.b);
        }
      }
    }
    if (c.lane == 0) tma_store_wait();
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// The parts of the r-th tile that was cut, `tile`: count of them; where it was
// shared out they belong to CTAs first, first + 1, ...  Part i's slot is slot(i).
struct AttnParts {
  int tile, first, count, late;
  bool halves;
  __device__ __forceinline__ AttnParts(const AttnParams& p, int r, int ctas) : halves(p.halves) {
    if (halves) {
      tile = first = r;
      count = 2;
      late = 0;
      return;
    }
    tile = p.waves * ctas + r;
    const long long unit0 = static_cast<long long>(r) * kUnits;
    int c = static_cast<int>(static_cast<long long>(r) * ctas / p.rem);
    while (c > 0 && attn_share(p, c, ctas) > unit0) --c;
    while (attn_share(p, c + 1, ctas) <= unit0) ++c;
    first = c;
    late = attn_share(p, c, ctas) < unit0;        // its share began in the tile before
    while (c < ctas && attn_share(p, c, ctas) < unit0 + kUnits) ++c;
    count = c - first;
  }
  __device__ __forceinline__ int slot(int i) const { return halves ? 2 * first + i : 2 * (first + i) + (i == 0 ? late : 0); }
};

// tiles that were cut
__device__ __forceinline__ int attn_cut_tiles(const AttnParams& p) { return p.halves ? p.total : p.rem; }

// Joins the parts of the tiles that were shared out: a warp per query row.
// FEW: the parts are those of a few queries (attn_few.cuh), a tile up to
// kFewRows of a key head's group * seq_q rows.
//   o = sum_i w_i o_i / sum_i w_i l_i,  w_i = exp2((m_i - max m) scale)
template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(256) attn_join_forward_kernel(const __grid_constant__ AttnParams p, int ctas) {
  const int kRows = FEW ? min(p.group * p.seq_q, kFewRows) : fwd::kRows;
  const int item = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (item >= attn_cut_tiles(p) * kRows) return;
  const int r = item / kRows, q = item % kRows;
  const AttnParts parts(p, r, ctas);
  int b, h, row;
  if (FEW) {
    const int key_head = parts.tile / p.tiles, x = (parts.tile - key_head * p.tiles) * kFewRows + q;
    if (x >= p.group * p.seq_q) return;
    b = key_head / p.heads_k;
    h = (key_head - b * p.heads_k) * p.group + x / p.seq_q;
    row = x % p.seq_q;
  } else {
    const AttnPlace at = attn_place(p, parts.tile, p.heads_q, true);
    b = at.b;
    h = at.h;
    row = at.t * kRows + q;
    if (row >= p.seq_q) return;
  }
  float m = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < parts.count; ++i) {
    const float* st = p.stats + (static_cast<long long>(parts.slot(i)) * kRows + q) * 2;
    if (in_span(st, 8, p.sp_stats, p.status)) m = fmaxf(m, *st);
  }
  float total = 0.0f;
  float2 acc[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) acc[e] = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int i = 0; i < parts.count; ++i) {
    const long long k = static_cast<long long>(parts.slot(i)) * kRows + q;
    if (!in_span(p.stats + 2 * k, 8, p.sp_stats, p.status) || !in_span(p.part + k * D, 4 * D, p.sp_part, p.status)) continue;
    const float2 st = *reinterpret_cast<const float2*>(p.stats + 2 * k);
    // a part that saw no key has sum 0, maximum -inf and zeros
    const float w = st.x == m ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(st.x, m), p.scale_log2));
    total = __fmaf_rn(w, st.y, total);
    const float2* src = reinterpret_cast<const float2*>(p.part + k * D) + lane;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = __ffma2_rn(make_float2(w, w), src[32 * e], acc[e]);
  }
  const bool some = total != 0.0f;
  const float inv = some ? __frcp_rn(total) : 0.0f;
  const long long l = (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + row;
  if (lane == 0 && in_span(p.lse + l, 4, p.sp_lse, p.status))
    p.lse[l] = some ? __fmaf_rn(m, p.scale, log_sum<T>(total)) : -INFINITY;
  char* dst = p.o + (static_cast<long long>(b) * p.seq_q + row) * p.o_stride + h * (D * 2);
  if (!in_span(dst, D * 2, p.sp_o, p.status)) return;
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    reinterpret_cast<uint32_t*>(dst)[lane + 32 * e] =
        some ? pack2<T>(__fmul_rn(acc[e].x, inv), __fmul_rn(acc[e].y, inv)) : 0u;
}

// ---------------------------------------------------------------------------
// backward
//
// Powers of two that the 16-bit operands carry through their products and
// the epilogues take out again.  P gets 2^kP, in the exponent: fp16 keeps the
// small probabilities of long rows out of its subnormals (P <= 1, so 2^14 is
// in range), bf16 those that ex2.approx would flush to zero.
//
// dS gets 2^kS.  bf16 has the exponents of fp32, so a constant does.  fp16 has
// not: dS = P (dP - delta) is as small as the incoming gradient over the number
// of keys and as large as |do| |v|, and with no factor gradients of 1e-5 over
// 4096 keys lose four of five dS to zero.  Its factor comes from the bound
// |dP - delta| <= b = 2 |do| V, where no row of v is longer than V (o is a mean
// of v's rows): with 2^e <= b < 2^(e+1), 2^14 P (dP - delta) 2^-e stays below
// 2^15, and half a subnormal step is 2^-39 b.  In dq a row is a query and has a
// factor of its own; in dk all queries of a sample's key head go into one sum
// and share the largest b.  At 4096 x 24 x 128 the bounds cost 20 us (4 %), at
// 8 x 1 x 4096 x 24 x 128, where v's 200 MB are read once more for them, 34 of
// 390.
template <typename T>
struct GradScale;
template <>
struct GradScale<__half> {
  static constexpr float kP = 14.0f;
  static constexpr bool kFromData = true;
};
template <>
struct GradScale<__nv_bfloat16> {
  static constexpr float kP = 24.0f;              // kS too
  static constexpr bool kFromData = false;
};
__device__ __forceinline__ constexpr float grad_scale_down(float k) {   // 2^-k
  return k == 14.0f ? 1.0f / 16384.0f : 1.0f / 16777216.0f;
}
// ds = (2^kP p) * (dp * lift - delta * lift), lift = 2^(kS - kP): 2^-e for the
// bound b, 1 where it says nothing (no gradient, infinities)
template <typename T>
__device__ __forceinline__ float grad_lift(float b) {
  if (!GradScale<T>::kFromData) return 1.0f;
  const bool use = b >= 0x1p-100f && b < INFINITY;
  return use ? __uint_as_float((254u << 23) - (__float_as_uint(b) & 0x7f800000u)) : 1.0f;
}
// 2^-kS, exact
template <typename T>
__device__ __forceinline__ float grad_unlift(float lift) {
  const float down = grad_scale_down(GradScale<T>::kP);
  return GradScale<T>::kFromData ? __uint_as_float((254u << 23) - __float_as_uint(lift)) * down : down;
}

__device__ __forceinline__ float square_sum(const float2 (&v)[4]) {
  float2 acc = __fmul2_rn(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) acc = __ffma2_rn(v[i], v[i], acc);
  return __fadd_rn(acc.x, acc.y);
}

// the largest of a warp's values, in every lane (a NaN does not count)
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// delta = rowsum(do * o), one team of D/8 lanes per row.  Bound by HBM (50 us
// for 2 x 8190 x 40 x 128, 6.7 TB/s).  Worked out inside the dq kernel instead,
// whose tiles load do anyway, each tile waits for its rows of o: the same time
// there, 150 against 145 us at 3 x 1999 x 16 on 4 heads x 64, causal.
// fp16: also |do| of each row and a bound on the rows of v (GradScale).
template <typename T, int D>
__global__ void __launch_bounds__(256, 8) attn_delta_kernel(const __grid_constant__ AttnParams p) {
  constexpr int L = D / 8, TEAMS = 256 / L;
  const int team = threadIdx.x / L, lane = threadIdx.x % L;
  const long long items = static_cast<long long>(p.batch) * p.seq_q * p.heads_q;
  grid_dependency_wait();
  // (row, head) with the heads of a row next to each other
  for (long long first = static_cast<long long>(blockIdx.x) * TEAMS; first < items;
       first += static_cast<long long>(gridDim.x) * TEAMS) {
    const long long it = first + team;
    float s = 0.0f, n = 0.0f;
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
        if (GradScale<T>::kFromData) n = square_sum(y);
      }
    }
    if (GradScale<T>::kFromData) {
      // two sums share one tree: the upper lanes take the second
      const bool upper = lane & (L / 2);
      s = __fadd_rn(upper ? n : s, __shfl_xor_sync(0xffffffffu, upper ? s : n, L / 2));
    } else {
      s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, L / 2));
    }
#pragma unroll
    for (int off = L / 4; off >= 1; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    if (it < items && lane % (L / 2) == 0) {
      const long long b = row / p.seq_q, at = (b * p.heads_q + h) * p.seq_q + (row - b * p.seq_q);
      if (lane == 0) {
        if (in_span(p.delta + at, 4, p.sp_delta, p.status)) p.delta[at] = s;
      } else if (GradScale<T>::kFromData && in_span(p.dout_norm + at, 4, p.sp_dout_norm, p.status)) {
        p.dout_norm[at] = __fsqrt_rn(s);
      }
    }
  }
  if (GradScale<T>::kFromData) {
    // No row of v that counts is longer than this: a lane keeps the largest sum
    // of its 8 columns, and a team's rows all stay below the sum over its lanes
    // (about sqrt(2) times the longest row; no shuffles until the end).
    constexpr int N = 2;                          // rows in flight
    const long long rows_v = static_cast<long long>(p.batch) * p.seq_k * p.heads_k, step = static_cast<long long>(gridDim.x) * TEAMS;
    const int h_step = static_cast<int>(step % p.heads_k), row_step = static_cast<int>(step / p.heads_k);
    long long it = static_cast<long long>(blockIdx.x) * TEAMS + team;
    int row = static_cast<int>(it / p.heads_k), h = static_cast<int>(it - static_cast<long long>(row) * p.heads_k);
    float top = 0.0f;
    while (it < rows_v) {
      uint4 x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (it < rows_v) {
          const char* src = p.v_in + row * p.v_stride + h * (D * 2) + lane * 16;
          bool counts = in_span(src, 16, p.sp_v, p.status);
          if (p.k_lens) {
            const int b = row / p.seq_k;
            counts = counts && row - b * p.seq_k < clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
          }
          if (counts) x[i] = *reinterpret_cast<const uint4*>(src);
          it += step;
          row += row_step;
          h += h_step;
          if (h >= p.heads_k) {
            h -= p.heads_k;
            ++row;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float2 y[4];
        Elem<T>::unpack(x[i], y);
        top = fmaxf(top, square_sum(y));
      }
    }
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) top = __fadd_rn(top, __shfl_xor_sync(0xffffffffu, top, off));
    __shared__ float tops[8];
    top = warp_max(top);
    if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, tops[i]);
      if (in_span(p.v_top + blockIdx.x, 4, p.sp_v_top, p.status)) p.v_top[blockIdx.x] = __fsqrt_rn(top);
    }
  }
  grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// backward, dq: a tile is 128 queries of one head, its iterations blocks of
// 128 keys.  Per block S = Q K^T, dP = dO V^T, dQ += dS K.
//
// Tensor memory holds S, dP, dQ, dS and Q (columns 0, 128, 256, 384, 448).  Q
// as a left operand in tensor memory takes 32 KB off the shared memory that a
// block's products read (160 KB, a quarter more than the tensor cores' time
// for it) and leaves room for a third V tile in flight; it comes through the
// K ring as the tile's first item, and the threads that own its rows copy it.
// S is free for the next block as soon as it has been read into registers.

namespace dq {
constexpr int kK = 3, kV = 2;                     // K (and Q) and V tiles in flight
constexpr int kColS = 0, kColDp = kTile, kColDq = 2 * kTile, kColDs = 3 * kTile, kColQ = 3 * kTile + 64;
enum { O_FULL = 0, O_EMPTY, K_FULL, K_EMPTY = K_FULL + kK, V_FULL = K_EMPTY + kK, V_EMPTY = V_FULL + kV,
       Q_READY = V_EMPTY + kV, S_FULL, S_FREE, DP_FULL, DP_FREE, DS_FULL, DS_FREE, DONE, ACC_FREE, DRAIN,
       BARS = DRAIN + 2 };
__device__ __forceinline__ int arrivals(int i) {
  return i == Q_READY || i == S_FREE || i == DP_FREE || i == DS_FULL || i == ACC_FREE ? 8 : 1;
}
template <int D>
constexpr int kStage = kOutRows * D;              // a warp's staged rows: D / 2 columns
template <int D>
constexpr int kCtl = (1 + kK + kV) * kTileBytes<D> + 8 * kStage<D>;
template <int D>
constexpr int kSmem = kCtl<D> + 256;

struct Seg {
  int b, h, q0, slot;
  int q_len, k_len, diag;
  int begin, n;               // key blocks [begin, begin + n)
  bool opens;                 // the tile's first piece
};
}  // namespace dq

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_dq_kernel(const __grid_constant__ AttnParams p) {
  using namespace dq;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + kCtl<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  const AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
                  __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), arrivals(i));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();
  grid_dependents_launch();

  auto segment = [&](int s, Seg& g) {
    AttnWork w;
    if (!attn_work(p, s, w)) return false;
    const AttnPlace at = attn_place(p, w.tile, p.heads_q, true);
    g.b = at.b;
    g.h = at.h;
    g.q0 = at.t * kTile;
    g.slot = w.slot;
    g.opens = w.u0 == 0;
    g.q_len = clamp_len(p.q_lens, at.b, p.seq_q, p.sp_q_lens, p.status);
    g.k_len = clamp_len(p.k_lens, at.b, p.seq_k, p.sp_k_lens, p.status);
    g.diag = g.k_len - g.q_len;
    const int last = g.q0 + kTile < g.q_len ? g.q0 + kTile : g.q_len;
    int keys = g.q0 >= g.q_len ? 0 : (p.causal ? last + g.diag : g.k_len);
    keys = keys < 0 ? 0 : (keys > g.k_len ? g.k_len : keys);
    int end;
    attn_cut(w, (keys + kTile - 1) / kTile, g.begin, end);
    g.n = end - g.begin;
    return true;
  };
  const uint32_t sdo = c.base, sk = c.base + kTileBytes<D>, sv = c.base + (1 + kK) * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && !(p.flags & 1u)) {         // test only: issue nothing
      RingPos<kK> k;
      RingPos<kV> v;
      int ik = 0, iv = 0, io = 0;
      bool ok = true;
      Seg g;
      for (int s = 0; ok && segment(s, g); ++s) {
        {
          // the next tile's queries come from HBM: on their way while this one's keys come from L2
          Seg next;
          if (segment(s + 1, next) && next.n > 0) {
            tma_prefetch_tile(&p.map_q, next.q0, next.h, next.b);
            tma_prefetch_tile(&p.map_do, next.q0, next.h, next.b);
          }
        }
        if (g.n == 0) continue;
        const int hk = g.h / p.group;
        for (int j = -1; j < g.n; ++j) {
          // Q, then K blocks
          ok = c.wait1(K_EMPTY + k.s, k.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(K_FULL + k.s), kTileBytes<D>);
          if (j < 0)
            tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_q, g.q0, g.h, g.b, c.bar(K_FULL + k.s));
          else
            tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_k, (g.begin + j) * kTile, hk, g.b, c.bar(K_FULL + k.s));
          ++ik;
          k.step();
          if (j < 0) continue;
          if (j == 0) {
            ok = c.wait1(O_EMPTY, io + 1);
            if (!ok) break;
            mbar_arrive_expect_tx(c.bar(O_FULL), kTileBytes<D>);
            tma_load_tile(sdo, &p.map_do, g.q0, g.h, g.b, c.bar(O_FULL));
            ++io;
          }
          ok = c.wait1(V_EMPTY + v.s, v.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(V_FULL + v.s), kTileBytes<D>);
          tma_load_tile(sv + v.s * kTileBytes<D>, &p.map_v, (g.begin + j) * kTile, hk, g.b, c.bar(V_FULL + v.s));
          ++iv;
          v.step();
        }
      }
      if (!ok || *abort_flag) {
        c.drain(K_FULL, kK, ik);
        c.drain(V_FULL, kV, iv);
        c.drain(O_FULL, 1, io);
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp) {
    // S(0), then per block S(next), when S has been read, and dQ
    RingPos<kK> ks, kd;                           // stages of the next S and dQ
    int done = 0, live = 0;                       // blocks of the tiles before, tiles
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      if (g.n == 0) continue;
      const int n = g.n, ragged = g.k_len < p.seq_k ? g.k_len / kTile - g.begin : n;
      // block j's S: its K has landed, with nothing past the sample's keys
      auto scores = [&](int j) {
        if (!c.wait(K_FULL + ks.s, ks.phase)) return false;
        if (j >= ragged) zero_rows<D>(smem + (1 + ks.s) * kTileBytes<D>, g.k_len - (g.begin + j) * kTile, c.lane);
        if (j > 0 && !c.wait(S_FREE, done + j - 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          mma_rows_ts<T, D>(tmem + kColS, tmem + kColQ, sk + ks.s * kTileBytes<D>);
          mma_commit(c.bar(S_FULL));
        }
        ks.step();
        return true;
      };
      // Q has been copied: its place in the ring is free
      ok = c.wait(Q_READY, live);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) mbar_arrive(c.bar(K_EMPTY + ks.s));
      __syncwarp();
      ks.step();
      kd.step();
      ok = scores(0);
      for (int j = 0; ok && j < n; ++j) {
        if (j + 1 < n) ok = scores(j + 1);
        // the accumulator has been read for the tile before
        ok = ok && (j > 0 || live == 0 || c.wait(ACC_FREE, live - 1)) && c.wait(DS_FULL, done + j);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_cols<T, D, false>(tmem + kColDq, tmem + kColDs, sk + kd.s * kTileBytes<D>, j > 0);
          mma_commit(c.bar(K_EMPTY + kd.s));
          mma_commit(c.bar(DS_FREE));
          if (j + 1 == n) mma_commit(c.bar(DONE));
        }
        kd.step();
      }
      done += n;
      ++live;
    }
    if (!ok) c.drain_mma(DRAIN);
  } else if (c.warp == kAttnMma2Warp) {
    // dP of each block, when the block's before has been read
    RingPos<kV> v;
    int done = 0, live = 0;
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      if (g.n == 0) continue;
      const int n = g.n, ragged = g.k_len < p.seq_k ? g.k_len / kTile - g.begin : n;
      ok = c.wait(O_FULL, live);
      for (int j = 0; ok && j < n; ++j, ++done) {
        ok = c.wait(V_FULL + v.s, v.phase);
        if (!ok) break;
        if (j >= ragged) zero_rows<D>(smem + (1 + kK + v.s) * kTileBytes<D>, g.k_len - (g.begin + j) * kTile, c.lane);
        ok = done == 0 || c.wait(DP_FREE, done - 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_rows<T, D>(tmem + kColDp, sdo, sv + v.s * kTileBytes<D>);
          mma_commit(c.bar(DP_FULL));
          mma_commit(c.bar(V_EMPTY + v.s));
          if (j + 1 == n) mma_commit(c.bar(O_EMPTY));
        }
        v.step();
      }
      ++live;
    }
    if (!ok) c.drain_mma(DRAIN + 1);
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // a thread per query and half of the block's keys
    const int half = c.warp >> 2, r = (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    RingPos<kK> k;                                // the K ring's place of the next tile's Q
    bool ready = false;                           // it has been copied
    // the next tile's Q: this thread's half of its row, to tensor memory
    auto copy_q = [&]() {
      if (!c.wait(K_FULL + k.s, k.phase)) return false;
      const unsigned char* row_q = smem + (1 + k.s) * kTileBytes<D> + r * 128;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        // 32 values: four chunks of the row, where the swizzle has put them
        const int first = half * (D / 16) + 4 * i;
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int chunk = first + e;
          const uint4 x =
              *reinterpret_cast<const uint4*>(row_q + (chunk >> 3) * (kTile * 128) + (((chunk & 7) ^ (r & 7)) << 4));
          w[4 * e] = x.x;
          w[4 * e + 1] = x.y;
          w[4 * e + 2] = x.z;
          w[4 * e + 3] = x.w;
        }
        tmem_store16(tmem + kColQ + first * 4 + lanes, w);
      }
      tmem_wait_store();
      c.arrive(Q_READY);
      return true;
    };
    float v_top = 0.0f;                           // no row of v is longer
    if (GradScale<T>::kFromData) {
#pragma unroll 4
      for (int i = c.lane; i < p.v_tops; i += 32)
        if (in_span(p.v_top + i, 4, p.sp_v_top, p.status)) v_top = fmaxf(v_top, p.v_top[i]);
      v_top = warp_max(v_top);
    }
    // a tile's row: log-sum, delta and the bound on |dP - delta|
    auto row_stats = [&](const Seg& g, float& lse, float& delta, float& bound) {
      const long long at = (static_cast<long long>(g.b) * p.heads_q + g.h) * p.seq_q + g.q0 + r;
      lse = delta = bound = 0.0f;
      if (g.q0 + r < p.seq_q && in_span(p.lse + at, 4, p.sp_lse, p.status) && in_span(p.delta + at, 4, p.sp_delta, p.status)) {
        lse = p.lse[at];
        delta = p.delta[at];
        if (GradScale<T>::kFromData && in_span(p.dout_norm + at, 4, p.sp_dout_norm, p.status))
          bound = __fmul_rn(2.0f * v_top, p.dout_norm[at]);
      }
    };
    unsigned char* stage = smem + (1 + kK + kV) * kTileBytes<D> + c.warp * kStage<D>;
    float lse = 0.0f, delta = 0.0f, bound = 0.0f;
    int done = 0, live = 0;                       // blocks and tiles so far
    bool ok = true;
    Seg g;
    for (int sg = 0; ok && segment(sg, g); ++sg) {
      const int row = g.q0 + r;
      int limit = row < g.q_len ? (p.causal ? row + g.diag + 1 : g.k_len) : 0;
      limit = limit < 0 ? 0 : (limit > g.k_len ? g.k_len : limit);
      if (!ready) row_stats(g, lse, delta, bound);
      if (GradScale<T>::kFromData && half == 0 && g.opens) {
        // for dk, dv: the largest bound of these 32 queries
        const float top = warp_max(limit > 0 ? bound : 0.0f);
        float* at = p.ds_top + ((static_cast<long long>(g.b) * p.heads_q + g.h) * p.q_tiles + g.q0 / kTile) * 4 + c.warp;
        if (c.lane == 0 && in_span(at, 4, p.sp_ds_top, p.status)) *at = top;
      }
      const float lift = grad_lift<T>(bound);
      // p = 0 for a row that sees nothing
      const float lse2 = limit == 0 || lse == -INFINITY ? INFINITY : __fmul_rn(lse, kLog2e);
      const float nl = GradScale<T>::kP - lse2, nd = -delta * lift;
      const float2 SL = make_float2(p.scale_log2, p.scale_log2), NL = make_float2(nl, nl), ND = make_float2(nd, nd),
                   C = make_float2(lift, lift);
      if (g.n > 0) {
        if (!ready) ok = copy_q();
        if (!ok) break;
        k.skip(g.n + 1);
        ready = false;
      }
      for (int j = 0; j < g.n; ++j, ++done) {
        const uint32_t ts = tmem + kColS + half * 64 + lanes, tdp = tmem + kColDp + half * 64 + lanes;
        ok = c.wait(S_FULL, done);
        if (!ok) break;
        tc_fence_after();
        float s[2][32];
        tmem_load32(ts, s[0]);
        tmem_load32(ts + 32, s[1]);
        tmem_wait_load(s[0]);
        tmem_loaded(s[1]);
        c.arrive(S_FREE);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = __ffma2_rn(make_float2(s[i][e], s[i][e + 1]), SL, NL);
            s[i][e] = exp2_approx(x.x);
            s[i][e + 1] = exp2_approx(x.y);
          }
        ok = c.wait(DP_FULL, done);
        if (!ok) break;
        tc_fence_after();
        float d[2][32];
        tmem_load32(tdp, d[0]);
        tmem_load32(tdp + 32, d[1]);
        tmem_wait_load(d[0]);
        tmem_loaded(d[1]);
        c.arrive(DP_FREE);
        const int seen = limit - (g.begin + j) * kTile - half * 64;
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
        if (done > 0) {
          // dQ has read the dS of the block before
          ok = c.wait(DS_FREE, done - 1);
          if (!ok) break;
          tc_fence_after();
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
          tmem_store16(tmem + kColDs + half * 32 + 16 * i + lanes, w);
        }
        tmem_wait_store();
        c.arrive(DS_FULL);
      }
      if (!ok) break;
      if (g.n > 0) {
        // Every S of this tile is done: the next one's Q can take Q's place,
        // and its first products run under this one's epilogue.
        ready = segment(sg + 1, g) && g.n > 0;
        if (ready) {
          row_stats(g, lse, delta, bound);
          ok = copy_q();
        }
        if (!ok) break;
        segment(sg, g);
        ok = c.wait(DONE, live++);
        if (!ok) break;
        tc_fence_after();
      }
      const bool some = g.n > 0 && limit > 0;
      float* part = p.part + (static_cast<long long>(g.slot) * kTile + r) * D + half * (D / 2);
      // checked builds: the rows of a part that this warp writes (a store by TMA stays inside its map)
      const bool fits = __all_sync(0xffffffffu, g.slot < 0 || in_span(part, 2 * D, p.sp_part, p.status));
      if (g.slot < 0) {
        // the store before has read the stage
        if (c.lane == 0) tma_store_wait_read();
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        float v[32];
        if (g.n > 0) {
          tmem_load32(tmem + kColDq + half * (D / 2) + 32 * i + lanes, v);
          tmem_wait_load(v);
          if (i == D / 64 - 1) c.arrive(ACC_FREE);
        }
        if (!fits) continue;
        if (g.slot >= 0)
          store_part<D>(part + 32 * i, v, grad_unlift<T>(lift), some, c.lane);
        else
          stage_cols<T, D / 2>(stage, 4 * i, v, p.scale * grad_unlift<T>(lift), some, c.lane);
      }
      if (g.slot < 0) {
        fence_async_shared();
        __syncwarp();
        // half of the columns: the second 64 of 128, or 32 of 64
        if (c.lane == 0 && row < p.seq_q)
          tma_store_box(&p.map_out, smem_addr(stage), D == 128 ? 0 : half * 32, row, D == 128 ? half : 0, g.h, g.b);
      }
    }
    if (c.lane == 0) tma_store_wait();
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Adds the parts of the tiles that were shared out, KV: of dk and dv (side by
// side in a slot, dv first), else of dq; a warp per row.
template <typename T, int D, bool KV>
__global__ void __launch_bounds__(256) attn_join_grad_kernel(const __grid_constant__ AttnParams p, int ctas) {
  constexpr int kRows = (KV ? 2 : 1) * kTile;     // rows of a slot
  const int item = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (item >= attn_cut_tiles(p) * kRows) return;
  const int r = item / kRows, q = item % kRows, which = q / kTile;
  const AttnParts parts(p, r, ctas);
  const AttnPlace at = attn_place(p, parts.tile, KV ? p.heads_k : p.heads_q, !KV);
  const int row = at.t * kTile + q % kTile, seq = KV ? p.seq_k : p.seq_q;
  if (row >= seq) return;
  float2 acc[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) acc[e] = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int i = 0; i < parts.count; ++i) {
    const float* src = p.part + (static_cast<long long>(parts.slot(i)) * kRows + q) * D;
    if (!in_span(src, 4 * D, p.sp_part, p.status)) continue;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = __fadd2_rn(acc[e], reinterpret_cast<const float2*>(src)[lane + 32 * e]);
  }
  const bool dv = KV && which == 0;
  const float f = dv ? 1.0f : p.scale;
  char* base = KV ? (dv ? p.dv : p.dk) : p.dq;
  const long long stride = KV ? (dv ? p.dv_stride : p.dk_stride) : p.dq_stride;
  char* dst = base + (static_cast<long long>(at.b) * seq + row) * stride + at.h * (D * 2);
  if (!in_span(dst, D * 2, KV ? (dv ? p.sp_dv : p.sp_dk) : p.sp_dq, p.status)) return;
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    reinterpret_cast<uint32_t*>(dst)[lane + 32 * e] = pack2<T>(__fmul_rn(acc[e].x, f), __fmul_rn(acc[e].y, f));
}

// ---------------------------------------------------------------------------
// backward, dk and dv: a tile is 128 keys of one key head, its iterations
// blocks of 128 queries of every head that shares it.  Per block, transposed
// so that P and dS come out as left operands: S^T = K Q^T, dP^T = V dO^T, dV
// += P^T dO, dK += dS^T Q.  A CTA keeps K and V while queries stream past, so
// nothing is added across CTAs but the parts of the last tiles.  Two warps
// issue, one for S and dV, one for dP and dK.  The whole backward pass of 4096
// x 24 x 128 takes 515 us, 1.0 PFLOP/s by the formulas (1.4 with S and dP,
// which both kernels work out): a block's exponentials, products and
// conversions on eight warps take about as long as its four products, and the
// accumulators leave tensor memory no room for a second block's scores.

namespace dkv {
constexpr int kQ = 3, kO = 2;                     // Q and dO tiles in flight
enum { K_FULL = 0, K_EMPTY, V_FULL, V_EMPTY, Q_FULL, Q_EMPTY = Q_FULL + kQ, O_FULL = Q_EMPTY + kQ,
       O_EMPTY = O_FULL + kO, S_FULL = O_EMPTY + kO, P_FULL, DP_FULL, DS_FULL, ROWS, ROWS_FREE = ROWS + 2,
       DONE = ROWS_FREE + 2, ACC_FREE, DRAIN, BARS = DRAIN + 2 };
__device__ __forceinline__ int arrivals(int i) {
  if (i == P_FULL || i == DS_FULL || i == ACC_FREE || (i >= ROWS_FREE && i < DONE)) return 8;
  // both chains are done with a tile, with the accumulators
  return (i >= Q_EMPTY && i < O_FULL) || (i >= O_EMPTY && i < S_FULL) || i == DONE ? 2 : 1;
}
constexpr int kRowBytes = 2 * 2 * kTile * 4 + 16; // two buffers of (lse, delta) of a tile's queries, and their lifts
template <int D>
constexpr int kCtl = (2 + kQ + kO) * kTileBytes<D> + kRowBytes;
template <int D>
constexpr int kSmem = kCtl<D> + 256;

struct Seg {
  int b, h, k0, slot;         // h: key head
  int q_len, k_len, diag;
  int first, end;             // query tiles [first, end) see one of these keys
  int n;                      // blocks
  int h0, t0;                 // head and query tile of the first
};
}  // namespace dkv

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_dkv_kernel(const __grid_constant__ AttnParams p) {
  using namespace dkv;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + kCtl<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  const AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
                  __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), arrivals(i));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  grid_dependency_wait();
  grid_dependents_launch();
  float* rows = reinterpret_cast<float*>(smem + (2 + kQ + kO) * kTileBytes<D>);   // [2][2][128]
  float* lifts = rows + 2 * 2 * kTile;            // [2]

  auto segment = [&](int s, Seg& g) {
    AttnWork w;
    if (!attn_work(p, s, w)) return false;
    const AttnPlace at = attn_place(p, w.tile, p.heads_k, false);
    g.b = at.b;
    g.h = at.h;
    g.k0 = at.t * kTile;
    g.slot = w.slot;
    g.q_len = clamp_len(p.q_lens, at.b, p.seq_q, p.sp_q_lens, p.status);
    g.k_len = clamp_len(p.k_lens, at.b, p.seq_k, p.sp_k_lens, p.status);
    g.diag = g.k_len - g.q_len;
    g.first = 0;
    g.end = (g.q_len + kTile - 1) / kTile;
    if (p.causal && g.k0 - g.diag > 0) g.first = (g.k0 - g.diag) / kTile;
    if (g.k0 >= g.k_len || g.first > g.end) g.first = g.end;
    const int per_head = g.end - g.first;
    int begin, end;
    attn_cut(w, per_head * p.group, begin, end);
    g.n = end - begin;
    g.h0 = g.h * p.group + (per_head ? begin / per_head : 0);
    g.t0 = g.first + (per_head ? begin % per_head : 0);
    return true;
  };
  const uint32_t sk = c.base, sv = c.base + kTileBytes<D>, sq = c.base + 2 * kTileBytes<D>,
                 sdo = c.base + (2 + kQ) * kTileBytes<D>;

  if (c.warp >= kAttnMmaWarp) fewer_registers<kAttnIssueRegs>();
  if (c.warp == kAttnLoadWarp) {
    if (c.lane == 0 && !(p.flags & 1u)) {         // test only: issue nothing
      RingPos<kQ> q;
      RingPos<kO> o;
      int uses = 0, vuses = 0, iq = 0, io = 0;
      bool ok = true;
      Seg g;
      for (int s = 0; ok && segment(s, g); ++s) {
        {
          Seg next;
          if (segment(s + 1, next) && next.n > 0) {
            tma_prefetch_tile(&p.map_k, next.k0, next.h, next.b);
            tma_prefetch_tile(&p.map_v, next.k0, next.h, next.b);
          }
        }
        if (g.n == 0) continue;
        ok = c.wait1(K_EMPTY, uses + 1);
        if (!ok) break;
        mbar_arrive_expect_tx(c.bar(K_FULL), kTileBytes<D>);
        tma_load_tile(sk, &p.map_k, g.k0, g.h, g.b, c.bar(K_FULL));
        ++uses;
        int h = g.h0, t = g.t0;
        for (int i = 0; i < g.n; ++i, q.step(), o.step()) {
          ok = c.wait1(Q_EMPTY + q.s, q.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(Q_FULL + q.s), kTileBytes<D>);
          tma_load_tile(sq + q.s * kTileBytes<D>, &p.map_q, t * kTile, h, g.b, c.bar(Q_FULL + q.s));
          ++iq;
          if (i == 0) {
            ok = c.wait1(V_EMPTY, uses);
            if (!ok) break;
            mbar_arrive_expect_tx(c.bar(V_FULL), kTileBytes<D>);
            tma_load_tile(sv, &p.map_v, g.k0, g.h, g.b, c.bar(V_FULL));
            ++vuses;
          }
          ok = c.wait1(O_EMPTY + o.s, o.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(O_FULL + o.s), kTileBytes<D>);
          tma_load_tile(sdo + o.s * kTileBytes<D>, &p.map_do, t * kTile, h, g.b, c.bar(O_FULL + o.s));
          ++io;
          if (++t == g.end) {
            t = g.first;
            ++h;
          }
        }
      }
      if (!ok || *abort_flag) {
        c.drain(Q_FULL, kQ, iq);
        c.drain(O_FULL, kO, io);
        c.drain(K_FULL, 1, uses);
        c.drain(V_FULL, 1, vuses);
      }
    }
    __syncwarp();
  } else if (c.warp == kAttnMmaWarp || c.warp == kAttnMma2Warp) {
    // Two chains of the same form: S(0), then per block dV += P^T dO, S(next);
    // dP(0), then per block dK += dS^T Q, dP(next).  (`a`: the tile of the
    // chain's first product, `b`: of its second.)
    const bool first_chain = c.warp == kAttnMmaWarp;
    RingPos<kQ> q;
    RingPos<kO> o;
    int done = 0, live = 0;                       // blocks and tiles so far
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      if (g.n == 0) continue;
      const int n = g.n;
      const bool ragged = g.q_len < p.seq_q;
      int t = g.t0;                               // the block's query tile
      // A tile that has landed: nothing past the sample's queries.  (Both
      // chains write the zeros: the same ones, before either gives the tile
      // back.)
      auto clean_q = [&](int tile) {
        if (ragged && (tile + 1) * kTile > g.q_len)
          zero_rows<D>(smem + (2 + q.s) * kTileBytes<D>, g.q_len - tile * kTile, c.lane);
      };
      auto clean_o = [&](int tile) {
        if (ragged && (tile + 1) * kTile > g.q_len)
          zero_rows<D>(smem + (2 + kQ + o.s) * kTileBytes<D>, g.q_len - tile * kTile, c.lane);
      };
      if (first_chain) {
        ok = c.wait(K_FULL, live) && c.wait(Q_FULL + q.s, q.phase);
        if (!ok) break;
        clean_q(t);
        if (elect_one()) {
          mma_rows<T, D>(tmem, sk, sq + q.s * kTileBytes<D>);
          mma_commit(c.bar(S_FULL));
          mma_commit(c.bar(Q_EMPTY + q.s));
          if (n == 1) mma_commit(c.bar(K_EMPTY));
        }
        q.step();
        for (int i = 0; i < n; ++i, ++done) {
          const bool more = i + 1 < n;
          const int next = t + 1 == g.end ? g.first : t + 1;
          // the accumulators have been read for the tile before
          ok = c.wait(O_FULL + o.s, o.phase) && (!more || c.wait(Q_FULL + q.s, q.phase));
          if (!ok) break;
          clean_o(t);
          if (more) clean_q(next);
          ok = (i > 0 || live == 0 || c.wait(ACC_FREE, live - 1)) && c.wait(P_FULL, done);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_cols<T, D, true>(tmem + 2 * kTile, tmem, sdo + o.s * kTileBytes<D>, i > 0);
            mma_commit(c.bar(O_EMPTY + o.s));
            if (!more) mma_commit(c.bar(DONE));
            if (more) {
              mma_rows<T, D>(tmem, sk, sq + q.s * kTileBytes<D>);
              mma_commit(c.bar(S_FULL));
              mma_commit(c.bar(Q_EMPTY + q.s));
              if (i + 2 == n) mma_commit(c.bar(K_EMPTY));
            }
          }
          o.step();
          if (more) q.step();
          t = next;
        }
      } else {
        ok = c.wait(V_FULL, live) && c.wait(O_FULL + o.s, o.phase);
        if (!ok) break;
        clean_o(t);
        if (elect_one()) {
          mma_rows<T, D>(tmem + kTile, sv, sdo + o.s * kTileBytes<D>);
          mma_commit(c.bar(DP_FULL));
          mma_commit(c.bar(O_EMPTY + o.s));
          if (n == 1) mma_commit(c.bar(V_EMPTY));
        }
        o.step();
        for (int i = 0; i < n; ++i, ++done) {
          const bool more = i + 1 < n;
          const int next = t + 1 == g.end ? g.first : t + 1;
          ok = c.wait(Q_FULL + q.s, q.phase) && (!more || c.wait(O_FULL + o.s, o.phase));
          if (!ok) break;
          clean_q(t);
          if (more) clean_o(next);
          ok = (i > 0 || live == 0 || c.wait(ACC_FREE, live - 1)) && c.wait(DS_FULL, done);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_cols<T, D, true>(tmem + 3 * kTile, tmem + kTile, sq + q.s * kTileBytes<D>, i > 0);
            mma_commit(c.bar(Q_EMPTY + q.s));
            if (!more) mma_commit(c.bar(DONE));
            if (more) {
              mma_rows<T, D>(tmem + kTile, sv, sdo + o.s * kTileBytes<D>);
              mma_commit(c.bar(DP_FULL));
              mma_commit(c.bar(O_EMPTY + o.s));
              if (i + 2 == n) mma_commit(c.bar(V_EMPTY));
            }
          }
          q.step();
          if (more) o.step();
          t = next;
        }
      }
      ++live;
    }
    if (!ok) c.drain_mma(DRAIN + (first_chain ? 0 : 1));
  } else if (c.warp == kAttnRowWarp) {
    // Warp 11 hands round kP - lse (log2) and -delta lift of the blocks'
    // queries, up to two blocks ahead.  A query past the length or with no
    // key gets -inf: p = 0.
    int done = 0;
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      int h = g.h0, t = g.t0;
      float lift = 1.0f;
      if (GradScale<T>::kFromData && g.n > 0) {
        // the largest bound among the queries of this key head
        const long long each = 4LL * p.q_tiles, n = p.group * each;
        const float* tops = p.ds_top + (static_cast<long long>(g.b) * p.heads_q + g.h * p.group) * each;
        float bound = 0.0f;
#pragma unroll 4
        for (long long i = c.lane; i < n; i += 32)
          if (in_span(tops + i, 4, p.sp_ds_top, p.status)) bound = fmaxf(bound, tops[i]);
        lift = grad_lift<T>(warp_max(bound));
      }
      for (int i = 0; i < g.n; ++i, ++done) {
        const long long at = (static_cast<long long>(g.b) * p.heads_q + h) * p.seq_q + t * kTile + c.lane;
        float l[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool valid = t * kTile + 32 * e + c.lane < g.q_len;
          l[e] = valid && in_span(p.lse + at + 32 * e, 4, p.sp_lse, p.status) ? p.lse[at + 32 * e] : -INFINITY;
          d[e] = valid && in_span(p.delta + at + 32 * e, 4, p.sp_delta, p.status) ? p.delta[at + 32 * e] : 0.0f;
        }
        // the block before last has been read
        ok = done < 2 || c.wait(ROWS_FREE + (done & 1), (done >> 1) - 1);
        if (!ok) break;
        float* out = rows + (done & 1) * 2 * kTile + c.lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          out[32 * e] = l[e] == -INFINITY ? -INFINITY : __fmaf_rn(l[e], -kLog2e, GradScale<T>::kP);
          out[kTile + 32 * e] = -d[e] * lift;
        }
        if (GradScale<T>::kFromData && c.lane == 0) lifts[done & 1] = lift;
        __syncwarp();
        if (c.lane == 0) mbar_arrive(c.bar(ROWS + (done & 1)));
        if (++t == g.end) {
          t = g.first;
          ++h;
        }
      }
    }
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // a thread per key and half of the block's queries
    const int half = c.warp >> 2, r = (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const uint32_t ts = tmem + half * 64 + lanes, tdp = tmem + kTile + half * 64 + lanes;
    const float2 SL = make_float2(p.scale_log2, p.scale_log2);
    int done = 0, live = 0;                       // blocks and tiles so far
    bool ok = true;
    Seg g;
    for (int sg = 0; ok && segment(sg, g); ++sg) {
      const int key = g.k0 + r;
      int t = g.t0;                               // the block's query tile
      float lift = 1.0f;
      for (int i = 0; i < g.n; ++i, ++done) {
        const float* mine = rows + (done & 1) * 2 * kTile;
        const float4* nl = reinterpret_cast<const float4*>(mine + half * 64);
        const float4* nd = reinterpret_cast<const float4*>(mine + kTile + half * 64);
        ok = c.wait(ROWS + (done & 1), done >> 1) && c.wait(S_FULL, done);
        if (!ok) break;
        tc_fence_after();
        if (GradScale<T>::kFromData) lift = lifts[done & 1];
        const float2 C = make_float2(lift, lift);
        float s[2][32];
        tmem_load32(ts, s[0]);
        tmem_load32(ts + 32, s[1]);
        tmem_wait_load(s[0]);
        tmem_loaded(s[1]);
        // query q0 + c sees this key when c >= from
        const int from = p.causal ? key - g.diag - t * kTile - half * 64 : 0;
        if (++t == g.end) t = g.first;
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
        ok = c.wait(DP_FULL, done);
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
        if (c.lane == 0) mbar_arrive(c.bar(ROWS_FREE + (done & 1)));
      }
      if (!ok) break;
      // the first group writes dv, the second dk
      if (g.n > 0) {
        ok = c.wait(DONE, live++);
        if (!ok) break;
        tc_fence_after();
      }
      const bool some = g.n > 0 && key < g.k_len;
      const float down = half ? grad_unlift<T>(lift) : grad_scale_down(GradScale<T>::kP), f = half ? p.scale * down : down;
      float* part = p.part + ((static_cast<long long>(g.slot) * 2 + half) * kTile + r) * D;
      char* dst = half ? p.dk + (static_cast<long long>(g.b) * p.seq_k + key) * p.dk_stride + g.h * (D * 2)
                       : p.dv + (static_cast<long long>(g.b) * p.seq_k + key) * p.dv_stride + g.h * (D * 2);
      const int there = p.seq_k - (key - c.lane);   // rows from the warp's first on
      const bool fits =
          __all_sync(0xffffffffu, g.slot >= 0 ? in_span(part, 4 * D, p.sp_part, p.status)
                                              : key >= p.seq_k || in_span(dst, D * 2, half ? p.sp_dk : p.sp_dv, p.status));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float v[32];
        if (g.n > 0) {
          tmem_load32(tmem + (2 + half) * kTile + 32 * i + lanes, v);
          tmem_wait_load(v);
          if (i == D / 32 - 1) c.arrive(ACC_FREE);
        }
        if (!fits) continue;
        if (g.slot >= 0)
          store_part<D>(part + 32 * i, v, down, some, c.lane);
        else
          store_cols<T>(dst + 64 * i, half ? p.dk_stride : p.dv_stride, there, v, f, some, c.lane);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace qknr
