// Layer norm, forward and backward, for sm_103a (formulas: qknr_ln.h).
//
// Both passes are bound by HBM: the forward reads x and writes y, the
// backward reads x and dy and writes dx.  Persistent CTAs, one per SM; their
// warps form groups that each take whole rows.  A group owns a ring of
// shared-memory stages that bulk copies fill some rows ahead (128 KB per SM
// in flight), reads a row into registers, and asks for the row after next
// into the same stage as soon as the group's first barrier says that every
// warp has its share.  Thread l of a group of W warps holds the 16-byte
// chunks l, l + 32 W, ... of every row it sees, so the row is unpacked once,
// the variance is a true second pass (squared deviations from the finished
// mean) without a second read, and what belongs to a column (gain, bias, the
// columns' sums) stays in registers from row to row.  At 2 x 4608 x 6144 with
// modulation the forward takes 40 us (5.6 TB/s), the backward 64 (5.3 TB/s,
// the sums over rows included); a call of few rows per SM has nothing to stream
// and takes the direct kernel, 2.4 us on the device at 256 x 1536.
//
// Every mbarrier wait is bounded.  A group decides together whether it goes
// on: each warp posts whether its wait succeeded with its part of the row's
// sums, so no warp is left at a named barrier for one that gave up.
#pragma once

#include "qknr_ptx.cuh"

namespace qknr {

struct LnParams {
  const char* x;
  char* y;
  const char* dy;
  char* dx;
  long long x_stride, y_stride, dy_stride, dx_stride;   // bytes per row
  long long tokens;
  long long rows_per_batch;
  const char* weight;
  const char* bias;
  long long param_stride;     // bytes between parameter rows
  int param_fp32;
  float* mean;
  float* rstd;
  float* dweight;
  float* dbias;
  float* parts;               // [units][2][hidden] partial sums (one unit per sample: null)
  float* row_sums;            // [T][2], rows too long for one CTA only
  int hidden;
  int group_warps;
  int groups;                 // row groups per CTA
  long long sets;             // parameter rows
  long long units_per_set;    // chunks of rows each parameter row's tokens are cut into
  long long unit_rows;        // rows per chunk
  int tiles;                  // column tiles a row is cut into
  int stages;                 // ring depth of a group
  unsigned row_bytes;         // hidden * 2
  unsigned flags;
  unsigned long long wait_limit_ns;
  float eps;
  float inv_c;
  float unit;                 // added to the weight
  int* status;
  MemSpan sp_x, sp_y, sp_dy, sp_dx, sp_weight, sp_bias, sp_mean, sp_rstd, sp_dweight, sp_dbias, sp_ws;
};

// the parameter row of a token row
__device__ __forceinline__ long long ln_set(const LnParams& p, long long row) {
  if (p.sets == 1) return 0;
  if (p.tokens <= 0xffffffffLL) return static_cast<unsigned>(row) / static_cast<unsigned>(p.rows_per_batch);
  return row / p.rows_per_batch;
}

// 16 bytes read once
__device__ __forceinline__ uint4 ln_load16(const char* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// 8 parameters of chunk k of a row as fp32 pairs
template <typename T>
__device__ __forceinline__ void ln_param8(const char* row, int k, int fp32, float2 (&m)[4]) {
  if (fp32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row) + 2 * k);
    const float4 b = __ldg(reinterpret_cast<const float4*>(row) + 2 * k + 1);
    m[0] = make_float2(a.x, a.y); m[1] = make_float2(a.z, a.w);
    m[2] = make_float2(b.x, b.y); m[3] = make_float2(b.z, b.w);
  } else {
    Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(row) + k), m);
  }
}

// the gain of chunk k: unit + weight, or 1
template <typename T>
__device__ __forceinline__ void ln_gain8(const LnParams& p, long long set, int k, float2 (&g)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = make_float2(1.0f, 1.0f);
  const int bytes = p.param_fp32 ? 32 : 16;
  const char* row = p.weight + set * p.param_stride;
  if (p.weight == nullptr || !in_span(row + k * bytes, bytes, p.sp_weight, p.status)) return;
  ln_param8<T>(row, k, p.param_fp32, g);
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = __fadd2_rn(g[j], make_float2(p.unit, p.unit));
}

// the bias of chunk k, or 0
template <typename T>
__device__ __forceinline__ void ln_bias8(const LnParams& p, long long set, int k, float2 (&b)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = make_float2(0.0f, 0.0f);
  const int bytes = p.param_fp32 ? 32 : 16;
  const char* row = p.bias + set * p.param_stride;
  if (p.bias && in_span(row + k * bytes, bytes, p.sp_bias, p.status)) ln_param8<T>(row, k, p.param_fp32, b);
}

// The sum of each of v's N (1, 2 or 4) values over a group's W <= MOST warps,
// the same in every thread: a shuffle tree inside each warp (the values share
// one tree, 32 / N lanes each once they have been folded), then the N * MOST
// slots of `red` that the group's warps fill are added in order; slots of
// absent warps hold zero.  Returns whether every thread's `ok` was true (the
// barrier's own reduction).  The caller uses two buffers `red` in turn, so
// the one barrier also keeps a fast warp from overwriting sums a slow one
// reads.
constexpr int kLnRedFloats = 32;

template <int N, int MOST>
__device__ __forceinline__ bool ln_group_sum(float (&v)[N], bool ok, int W, int gw, int lane, int bar_id, float* red) {
  static_assert(N * MOST <= kLnRedFloats && (N * MOST) % 4 == 0 && (N == 1 || N == 2 || N == 4), "slots");
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = v[i];
#pragma unroll
  for (int n = N, off = 16; off >= 1; off >>= 1) {
    if (n > 1) {
      // the lanes with bit `off` keep the second half of the values
      const bool upper = lane & off;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float keep = upper ? t[n / 2 + i] : t[i], give = upper ? t[i] : t[n / 2 + i];
        t[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, off));
      }
      n /= 2;
    } else {
      t[0] = __fadd_rn(t[0], __shfl_xor_sync(0xffffffffu, t[0], off));
    }
  }
  if (W == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t[0], i * (32 / N));
    return __all_sync(0xffffffffu, ok);
  }
  if (lane % (32 / N) == 0) red[N * gw + lane / (32 / N)] = t[0];
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(bar_id), "r"(32 * W)
      : "memory");
  const float4* r = reinterpret_cast<const float4*>(red);
  float2 lo = make_float2(0.0f, 0.0f), hi = lo;
#pragma unroll
  for (int i = 0; i < N * MOST / 4; ++i) {
    const float4 part = r[i];
    lo = __fadd2_rn(lo, make_float2(part.x, part.y));
    hi = __fadd2_rn(hi, make_float2(part.z, part.w));
  }
  if (N == 4) {
    v[0] = lo.x;
    v[N / 4] = lo.y;
    v[N / 2] = hi.x;
    v[N - 1] = hi.y;
  } else {
    const float2 s = __fadd2_rn(lo, hi);
    v[0] = N == 1 ? __fadd_rn(s.x, s.y) : s.x;
    if (N == 2) v[N - 1] = s.y;
  }
  return all != 0;
}

__device__ __forceinline__ float ln_hsum(const float2 (&v)[4]) {
  const float2 s = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
  return __fadd_rn(s.x, s.y);
}

// ---------------------------------------------------------------------------
// the rings

constexpr int kLnWarps = 16;                      // warps of the forward pass
constexpr int kLnThreads = 32 * kLnWarps;
constexpr int kLnMaxStages = 32;                  // all groups' together
// dynamic shared memory map (bytes)
constexpr int kLnOffBars = 0;                     // full[32]
constexpr int kLnOffAbort = 256;
constexpr int kLnOffRed = 512;                    // per group two buffers of kLnRedFloats
constexpr int kLnOffStages = kLnOffRed + kLnWarps * 2 * kLnRedFloats * 4;   // 4608
static_assert(kLnOffStages % 128 == 0, "shared memory map");

// One group's ring of `stages` stages.  Its rows come in the order in which
// the group's first thread put them.
struct LnRing {
  uint32_t bars, stage0;
  const unsigned char* ptr;
  unsigned stage_bytes;
  int stages;
  volatile int* abort_flag;
  int* status;
  unsigned long long limit;
  int s = 0;                  // next stage to read
  uint32_t phase = 0;
  int put_s = 0;              // next stage to fill (first thread)
  int in_flight = 0;

  __device__ __forceinline__ LnRing(unsigned char* smem, const LnParams& p, unsigned stage_bytes_, int grp)
      : bars(smem_addr(smem) + kLnOffBars + 8 * grp * p.stages),
        stage0(smem_addr(smem) + kLnOffStages + grp * p.stages * stage_bytes_),
        ptr(smem + kLnOffStages + grp * p.stages * stage_bytes_),
        stage_bytes(stage_bytes_),
        stages(p.stages),
        abort_flag(reinterpret_cast<volatile int*>(smem + kLnOffAbort)),
        status(p.status),
        limit(p.wait_limit_ns) {}

  // Row `a` (and `b` behind it) into the next stage, which has been read.
  __device__ __forceinline__ void put(const char* a, const MemSpan& sp_a, const char* b, const MemSpan& sp_b,
                                      unsigned bytes) {
    if (!in_span(a, bytes, sp_a, status) || (b && !in_span(b, bytes, sp_b, status))) {
      *abort_flag = 1;
      return;
    }
    const uint32_t dst = stage0 + put_s * stage_bytes, bar = bars + 8 * put_s;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the group's reads come before the copy
    mbar_arrive_expect_tx(bar, b ? 2 * bytes : bytes);
    bulk_load(dst, a, bytes, bar);
    if (b) bulk_load(dst + bytes, b, bytes, bar);
    if (++put_s == stages) put_s = 0;
    ++in_flight;
  }
  // The next row has landed (one thread's answer).
  __device__ __forceinline__ bool wait() const {
    return mbar_try_wait(bars + 8 * s, phase) || bounded_wait(bars + 8 * s, phase, limit, abort_flag, status);
  }
  __device__ __forceinline__ const uint4* row() const { return reinterpret_cast<const uint4*>(ptr + s * stage_bytes); }
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  // first thread, giving up: copies in flight end before the CTA leaves its
  // shared memory, those of the `given_up` rows before the next one included
  __device__ __forceinline__ void drain(int given_up) {
    const unsigned long long t0 = global_timer_ns();
    for (; given_up > 0; --given_up)
      if (--s < 0) {
        s = stages - 1;
        phase ^= 1u;
      }
    for (; in_flight > 0; --in_flight) {
      while (!mbar_try_wait(bars + 8 * s, phase) && global_timer_ns() - t0 < limit) {
      }
      next();
    }
  }
};

// the whole CTA: all groups' barriers and sum slots
__device__ __forceinline__ void ln_init_rings(unsigned char* smem, int n) {
  for (int i = threadIdx.x; i < kLnWarps * 2 * kLnRedFloats; i += blockDim.x)
    reinterpret_cast<float*>(smem + kLnOffRed)[i] = 0.0f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < n; ++i) mbar_init(smem_addr(smem) + kLnOffBars + 8 * i, 1);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + kLnOffAbort);
    flags[0] = flags[1] = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// forward

// Calls of a few rows per SM, and rows whose columns are too many for a
// thread to keep their parameters: a row is loaded straight into registers
// and held as read.
template <typename T, int CPT>
__device__ __forceinline__ void ln_forward_row(const LnParams& p, const uint4 (&raw)[CPT], long long row, int W, int gw,
                                               int lane, int bar, float* red) {
  const int l = gw * 32 + lane, step = 32 * W, n_chunks = p.hidden / 8;
  // mean: chunks past the row hold zeros
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float2 X[4];
    Elem<T>::unpack(raw[i], X);
    s = __fadd_rn(s, ln_hsum(X));
  }
  float t[1] = {s};
  ln_group_sum<1, kLnWarps>(t, true, W, gw, lane, bar, red);
  const float mean = __fmul_rn(t[0], p.inv_c);
  const float2 nm = make_float2(-mean, -mean);
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    if (l + i * step < n_chunks) {
      float2 X[4];
      Elem<T>::unpack(raw[i], X);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d = __fadd2_rn(X[j], nm);
        X[j] = __fmul2_rn(d, d);
      }
      s = __fadd_rn(s, ln_hsum(X));
    }
  }
  t[0] = s;
  ln_group_sum<1, kLnWarps>(t, true, W, gw, lane, bar, red + kLnRedFloats);
  const float var = __fmul_rn(t[0], p.inv_c);
  const float rstd = rsqrtf(__fadd_rn(var, p.eps));
  if (l == 0) {
    if (p.mean && in_span(p.mean + row, 4, p.sp_mean, p.status)) p.mean[row] = mean;
    if (p.rstd && in_span(p.rstd + row, 4, p.sp_rstd, p.status)) p.rstd[row] = rstd;
  }
  const long long set = ln_set(p, row);
  char* dst = p.y + row * p.y_stride;
  const bool fits = in_span(dst, p.row_bytes, p.sp_y, p.status);
  const float2 R = make_float2(rstd, rstd);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = l + i * step;
    if (fits && k < n_chunks) {
      float2 X[4], g[4], b[4];
      Elem<T>::unpack(raw[i], X);
      ln_gain8<T>(p, set, k, g);
      ln_bias8<T>(p, set, k, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) X[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(X[j], nm), R), g[j], b[j]);
      store16(dst + k * 16, Elem<T>::pack(X));
    }
  }
}

template <typename T, int CPT>
__global__ void __launch_bounds__(kLnThreads) ln_forward_direct_kernel(const __grid_constant__ LnParams p) {
  __shared__ __align__(16) float red[2 * kLnRedFloats];   // a CTA of several groups has groups of one warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W;
  const int l = gw * 32 + lane, n_chunks = p.hidden / 8;
  if (threadIdx.x < 2 * kLnRedFloats) red[threadIdx.x] = 0.0f;
  __syncthreads();
  grid_dependency_wait();
  const long long row = static_cast<long long>(blockIdx.x) * p.groups + grp;
  const char* src = p.x + row * p.x_stride;
  if (row < p.tokens && in_span(src, p.row_bytes, p.sp_x, p.status)) {
    uint4 raw[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * 32 * W;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (k < n_chunks) raw[i] = ln_load16(src + k * 16);
    }
    ln_forward_row<T, CPT>(p, raw, row, W, gw, lane, 1 + grp, red);
  }
  grid_dependents_launch();
}

// A group takes NR of its rows at a time: their sums share the shuffle trees
// and the barriers.
template <typename T, int CPT, int NR>
__global__ void __launch_bounds__(kLnThreads, 1) ln_forward_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W, l = gw * 32 + lane, n_chunks = p.hidden / 8;
  LnRing ring(smem, p, p.row_bytes, grp);
  ln_init_rings(smem, p.stages * p.groups);
  grid_dependency_wait();
  grid_dependents_launch();
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  long long row = static_cast<long long>(blockIdx.x) * p.groups + grp, ahead = row;
  const bool leader = gw == 0 && lane == 0 && !(p.flags & 1u);   // test only: issue nothing
  if (leader)
    for (int i = 0; i < p.stages && ahead < p.tokens; ++i, ahead += step)
      ring.put(p.x + ahead * p.x_stride, p.sp_x, nullptr, p.sp_x, p.row_bytes);
  float* red = reinterpret_cast<float*>(smem + kLnOffRed) + grp * 2 * kLnRedFloats;
  bool mine[CPT];
  float2 g[CPT][4], b[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) mine[i] = l + i * 32 * W < n_chunks;
  long long set_end = 0;                          // first row past the sample whose parameters are in g and b
  bool ok = true;
  while (row < p.tokens) {
    if (row >= set_end) {
      const long long set = ln_set(p, row);
      set_end = (set + 1) * p.rows_per_batch;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        if (!mine[i]) continue;
        ln_gain8<T>(p, set, l + i * 32 * W, g[i]);
        ln_bias8<T>(p, set, l + i * 32 * W, b[i]);
      }
    }
    // NR rows of the same sample, or one
    const long long most = set_end < p.tokens ? set_end : p.tokens;
    const int n = NR > 1 && row + step < most ? 2 : 1;
    float2 X[NR][CPT][4];
    float t[NR];
    bool landed = true;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      t[r] = 0.0f;
      if (r < n) {
        landed = ring.wait() && landed;
        const uint4* st = ring.row();
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          Elem<T>::unpack(mine[i] ? st[l + i * 32 * W] : make_uint4(0, 0, 0, 0), X[r][i]);
          t[r] = __fadd_rn(t[r], ln_hsum(X[r][i]));
        }
        ring.next();
      }
    }
    ok = ln_group_sum<NR, kLnWarps>(t, landed, W, gw, lane, 1 + grp, red);
    if (!ok) {
      if (leader) ring.drain(n);
      break;
    }
    if (leader)
      for (int r = 0; r < n; ++r) {
        --ring.in_flight;
        if (ahead < p.tokens) ring.put(p.x + ahead * p.x_stride, p.sp_x, nullptr, p.sp_x, p.row_bytes);
        ahead += step;
      }
    float mean[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      mean[r] = __fmul_rn(t[r], p.inv_c);
      const float2 nm = make_float2(-mean[r], -mean[r]);
      float2 q = make_float2(0.0f, 0.0f);
      if (r >= n) break;                          // there is no second row
#pragma unroll
      for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          X[r][i][j] = __fadd2_rn(X[r][i][j], nm);
          if (mine[i]) q = __ffma2_rn(X[r][i][j], X[r][i][j], q);
        }
      t[r] = __fadd_rn(q.x, q.y);
    }
    ln_group_sum<NR, kLnWarps>(t, true, W, gw, lane, 1 + grp, red + kLnRedFloats);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r >= n) break;
      const float rstd = rsqrtf(__fadd_rn(__fmul_rn(t[r], p.inv_c), p.eps));
      const long long at = row + r * step;
      if (l == 0) {
        if (p.mean && in_span(p.mean + at, 4, p.sp_mean, p.status)) p.mean[at] = mean[r];
        if (p.rstd && in_span(p.rstd + at, 4, p.sp_rstd, p.status)) p.rstd[at] = rstd;
      }
      const float2 R = make_float2(rstd, rstd);
      char* dst = p.y + at * p.y_stride + l * 16;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __ffma2_rn(__fmul2_rn(X[r][i][j], R), g[i][j], b[i][j]);
        if (mine[i] && in_span(dst + i * 512 * W, 16, p.sp_y, p.status)) store16(dst + i * 512 * W, Elem<T>::pack(o));
      }
    }
    row += n * step;
  }
}

// ---------------------------------------------------------------------------
// backward

// Eight warps of up to four chunks a thread: with 255 registers a thread
// holds its columns' sums, its gains and a row's xhat and dy, and the row's
// fixed costs (a shuffle tree, a barrier) are paid by few warps.
constexpr int kLnBwdWarps = 8;
constexpr int kLnBwdThreads = 32 * kLnBwdWarps;
constexpr int kLnBwdCpt = 4;
constexpr int kLnTile = 8 * 32 * kLnBwdWarps * kLnBwdCpt;   // 8192 columns: the longest row one CTA takes

// xhat and dy of one chunk
template <typename T>
__device__ __forceinline__ void ln_grad_values(const uint4& xr, const uint4& dr, float2 nm, float2 R, float2 (&xh)[4],
                                               float2 (&dy)[4]) {
  Elem<T>::unpack(xr, xh);
  Elem<T>::unpack(dr, dy);
#pragma unroll
  for (int j = 0; j < 4; ++j) xh[j] = __fmul2_rn(__fadd2_rn(xh[j], nm), R);
}

// one chunk's part of (sum g, sum g xhat)
__device__ __forceinline__ void ln_grad_sums(const float2 (&xh)[4], const float2 (&dy)[4], const float2 (&gain)[4],
                                             float2& s) {
  float2 a = make_float2(0.0f, 0.0f), c = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 g = __fmul2_rn(dy[j], gain[j]);
    a = __fadd2_rn(a, g);
    c = __ffma2_rn(g, xh[j], c);
  }
  s.x = __fadd_rn(s.x, __fadd_rn(a.x, a.y));
  s.y = __fadd_rn(s.y, __fadd_rn(c.x, c.y));
}

// Rows of more than kLnTile values: (mean_c g, mean_c g xhat) of each row,
// one CTA per row.
template <typename T>
__global__ void __launch_bounds__(256) ln_row_sums_kernel(const __grid_constant__ LnParams p) {
  __shared__ __align__(16) float red[2][kLnRedFloats];   // the sixteen read are written: eight warps, two values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_chunks = p.hidden / 8;
  grid_dependency_wait();
  int parity = 0;
  for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x, parity ^= 1) {
    const char* xs = p.x + row * p.x_stride;
    const char* ds = p.dy + row * p.dy_stride;
    float2 s = make_float2(0.0f, 0.0f);
    if (in_span(xs, p.row_bytes, p.sp_x, p.status) && in_span(ds, p.row_bytes, p.sp_dy, p.status) &&
        in_span(p.mean + row, 4, p.sp_mean, p.status) && in_span(p.rstd + row, 4, p.sp_rstd, p.status)) {
      const float2 nm = make_float2(-p.mean[row], -p.mean[row]), R = make_float2(p.rstd[row], p.rstd[row]);
      const long long set = ln_set(p, row);
      for (int k = threadIdx.x; k < n_chunks; k += 256) {
        float2 gain[4], xh[4], dy[4];
        ln_gain8<T>(p, set, k, gain);
        ln_grad_values<T>(*reinterpret_cast<const uint4*>(xs + k * 16), *reinterpret_cast<const uint4*>(ds + k * 16),
                          nm, R, xh, dy);
        ln_grad_sums(xh, dy, gain, s);
      }
    }
    float t[2] = {s.x, s.y};
    ln_group_sum<2, 8>(t, true, 8, warp, lane, 1, red[parity]);
    if (threadIdx.x == 0 && in_span(p.row_sums + 2 * row, 8, p.sp_ws, p.status)) {
      p.row_sums[2 * row] = __fmul_rn(t[0], p.inv_c);
      p.row_sums[2 * row + 1] = __fmul_rn(t[1], p.inv_c);
    }
  }
  grid_dependents_launch();
}

// dx, and the sums of dy and dy xhat over the rows.  A thread owns the same
// chunks of 8 columns for the whole launch, so those sums stay in its
// registers over all the rows of a unit (a chunk of one sample's rows); the
// CTA's row groups then add theirs in order through shared memory and write
// the unit's partial sums, or the result where a sample is one unit.  LONG:
// the row spans several CTAs (a column tile each) and its two sums come from
// ln_row_sums_kernel.
//
// NR rows go through the sums together (CPT <= 3: at four chunks a thread the
// registers hold one), which halves the shuffles, barriers and exposed
// latency per row.
template <typename T, int CPT, int NR, bool LONG>
__global__ void __launch_bounds__(kLnBwdThreads, 1) ln_backward_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps;
  const int tile = static_cast<int>(blockIdx.x % p.tiles), k0 = tile * (kLnTile / 8);
  const int n_chunks = p.hidden / 8 - k0 < kLnTile / 8 ? p.hidden / 8 - k0 : kLnTile / 8;   // of this tile
  const unsigned bytes = n_chunks * 16u;
  // two rows of the widest tile per stage
  const unsigned stage_bytes = 2 * (p.tiles > 1 ? kLnTile * 2u : p.row_bytes);
  const int grp = warp / W, gw = warp % W, l = gw * 32 + lane, cols = n_chunks * 8;
  LnRing ring(smem, p, stage_bytes, grp);
  volatile int* give_up = ring.abort_flag + 1;
  ln_init_rings(smem, p.stages * p.groups);
  grid_dependency_wait();
  grid_dependents_launch();
  const long long units = p.sets * p.units_per_set, unit_step = gridDim.x / p.tiles;
  // rows [first, last) of unit u
  auto rows_of = [&](long long u, long long& first, long long& last) {
    const long long set = u / p.units_per_set;
    const long long end = (set + 1) * p.rows_per_batch < p.tokens ? (set + 1) * p.rows_per_batch : p.tokens;
    first = set * p.rows_per_batch + (u - set * p.units_per_set) * p.unit_rows;
    last = first + p.unit_rows < end ? first + p.unit_rows : end;
    return set;
  };
  // the group's rows, some ahead of the one in work: unit, row, end of the unit
  long long a_unit = blockIdx.x / p.tiles, a_row = 0, a_last = 0;
  const bool leader = gw == 0 && lane == 0 && !(p.flags & 1u);   // test only: issue nothing
  auto put = [&]() {
    while (a_row >= a_last) {                     // the next unit with a row for this group
      if (a_unit >= units) return;
      rows_of(a_unit, a_row, a_last);
      a_row += grp;
      a_unit += unit_step;
    }
    ring.put(p.x + a_row * p.x_stride + k0 * 16, p.sp_x, p.dy + a_row * p.dy_stride + k0 * 16, p.sp_dy, bytes);
    a_row += p.groups;
  };
  if (leader)
    for (int i = 0; i < p.stages; ++i) put();

  float* acc = reinterpret_cast<float*>(smem + kLnOffStages + p.stages * p.groups * stage_bytes);   // [groups][2][columns]
  float* red = reinterpret_cast<float*>(smem + kLnOffRed) + grp * 2 * kLnRedFloats;
  bool mine[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) mine[i] = l + i * 32 * W < n_chunks;
  bool ok = true;
  int given_up = 0;
  // The two buffers alternate from one step to the next, from a unit's last to
  // the next unit's first too: a group alone in its CTA has no barrier between
  // units, and a slow warp may still read the sums of the step before.
  float* buf = red;
  for (long long u = blockIdx.x / p.tiles; u < units; u += unit_step) {
    long long first, last;
    const long long set = rows_of(u, first, last);
    float2 dw[CPT][4], db[CPT][4], gain[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = gain[i][j] = make_float2(0.0f, 0.0f);
      if (mine[i]) ln_gain8<T>(p, set, k0 + l + i * 32 * W, gain[i]);
    }
    // the statistics of the rows after those in work
    const float *at_mean = p.mean + first + grp, *at_rstd = p.rstd + first + grp;
    int left = last - first > grp ? static_cast<int>((last - first - grp + p.groups - 1) / p.groups) : 0;   // the group's rows
    float nmean[NR], nrstd[NR];
    auto stats = [&](int rows) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        nmean[r] = nrstd[r] = 0.0f;
        if (rows > r && in_span(at_mean, 4, p.sp_mean, p.status) && in_span(at_rstd, 4, p.sp_rstd, p.status)) {
          nmean[r] = *at_mean;
          nrstd[r] = *at_rstd;
        }
        at_mean += p.groups;
        at_rstd += p.groups;
      }
    };
    stats(left);
    char* dst = p.dx + (first + grp) * p.dx_stride + (k0 + l) * 16;
    const float2* sums = reinterpret_cast<const float2*>(p.row_sums) + first + grp;   // LONG
    for (; left > 0; left -= NR, buf = buf == red ? red + kLnRedFloats : red) {
      float2 xh[NR][CPT][4], dy[NR][CPT][4], R[NR];
      float t[2 * NR];
      bool landed = true;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 nm = make_float2(-nmean[r], -nmean[r]);
        R[r] = make_float2(nrstd[r], nrstd[r]);
        const bool some = r < left;               // an odd last row: its partner's dy is zero
        if (some) landed = ring.wait() && landed;
        const uint4* st = ring.row();
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          uint4 xr = make_uint4(0, 0, 0, 0), dr = xr;
          if (some && mine[i]) {
            xr = st[l + i * 32 * W];
            dr = st[n_chunks + l + i * 32 * W];
          }
          // past the row: dy = 0 and gain = 0, so xhat's value does not count
          ln_grad_values<T>(xr, dr, nm, R[r], xh[r][i], dy[r][i]);
          if (!LONG) ln_grad_sums(xh[r][i], dy[r][i], gain[i], s);
        }
        t[2 * r] = s.x;
        t[2 * r + 1] = s.y;
        if (some) ring.next();
      }
      stats(left - NR);
      ok = ln_group_sum<2 * NR, kLnBwdWarps>(t, landed, W, gw, lane, 1 + grp, buf);
      if (!ok) {
        given_up = left < NR ? left : NR;
        break;
      }
      if (leader)
        for (int r = 0; r < NR && r < left; ++r) {
          --ring.in_flight;
          put();
        }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float2 s = make_float2(__fmul_rn(t[2 * r], p.inv_c), __fmul_rn(t[2 * r + 1], p.inv_c));
        if (LONG && r < left && in_span(sums, 8, p.sp_ws, p.status)) s = *sums;
        const float2 c1 = make_float2(-s.x, -s.x), c2 = make_float2(-s.y, -s.y);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            db[i][j] = __fadd2_rn(db[i][j], dy[r][i][j]);
            dw[i][j] = __ffma2_rn(dy[r][i][j], xh[r][i][j], dw[i][j]);
            o[j] = __fmul2_rn(__ffma2_rn(xh[r][i][j], c2, __ffma2_rn(dy[r][i][j], gain[i][j], c1)), R[r]);
          }
          if (r < left && mine[i] && in_span(dst + i * 512 * W, 16, p.sp_dx, p.status))
            store16(dst + i * 512 * W, Elem<T>::pack(o));
        }
        dst += p.groups * p.dx_stride;
        sums += p.groups;
      }
    }
    // the groups' sums, added in order
    if (p.groups > 1) {
      float* slot = acc + grp * 2 * cols;
      named_barrier_sync(15, 32 * W * p.groups);   // the previous unit's sums have been read
#pragma unroll
      for (int i = 0; i < CPT; ++i)
        if (mine[i]) {
          float2* a = reinterpret_cast<float2*>(slot + (l + i * 32 * W) * 8);
          float2* b = reinterpret_cast<float2*>(slot + cols + (l + i * 32 * W) * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] = dw[i][j];
            b[j] = db[i][j];
          }
        }
      // one thread's view of the abort flag, for all to leave together
      if (threadIdx.x == 0) *give_up = *ring.abort_flag;
      named_barrier_sync(15, 32 * W * p.groups);
      if (*give_up) break;
      if (grp == 0)
        for (int g = 1; g < p.groups; ++g)
#pragma unroll
          for (int i = 0; i < CPT; ++i)
            if (mine[i]) {
              const float2* a = reinterpret_cast<const float2*>(acc + g * 2 * cols + (l + i * 32 * W) * 8);
              const float2* b = reinterpret_cast<const float2*>(acc + g * 2 * cols + cols + (l + i * 32 * W) * 8);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                dw[i][j] = __fadd2_rn(dw[i][j], a[j]);
                db[i][j] = __fadd2_rn(db[i][j], b[j]);
              }
            }
    } else if (!ok) {
      break;                                      // the group left its rows together
    }
    if (grp == 0) {
      const bool whole = p.units_per_set == 1;
      auto write = [&](float* out, const MemSpan& sp, const float2 (&v)[4]) {
        if (!in_span(out, 32, sp, p.status)) return;
        reinterpret_cast<float4*>(out)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        reinterpret_cast<float4*>(out)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
      };
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        if (!mine[i]) continue;
        const int c = (k0 + l + i * 32 * W) * 8;
        if (whole) {
          if (p.dweight) write(p.dweight + set * p.hidden + c, p.sp_dweight, dw[i]);
          if (p.dbias) write(p.dbias + set * p.hidden + c, p.sp_dbias, db[i]);
        } else {
          write(p.parts + u * 2 * p.hidden + c, p.sp_ws, dw[i]);
          write(p.parts + (u * 2 + 1) * p.hidden + c, p.sp_ws, db[i]);
        }
      }
    }
  }
  if (leader && *ring.abort_flag) ring.drain(given_up);   // this group or another gave up
}

}  // namespace qknr
