// Root-mean-square norm with the residual's addition, forward (into the
// activation dtype or 8 bits) and backward, for sm_103a (formulas:
// qknr_rms.h).
//
// Bound by HBM like layer norm, whose rings, row groups and sums it uses
// (ln_kernel.cuh): persistent CTAs, one per SM, whose warps form groups that
// each take whole rows; bulk copies bring a group's rows (x and residual, or
// the backward pass's two or three) some rows ahead; a row is read into
// registers once and the columns' gains and sums stay there from row to row.
// The forward pass needs one sum per row, so one barrier; a scale per row
// takes a second, a scale per 128 columns a shuffle tree over the 16 lanes
// that hold them.  At 2 x 4608 x 6144 with modulation and residual into 8 bits
// it takes 61.5 us (6.4 TB/s), the backward pass of 9216 x 6144 with dsum 75 (6.0
// TB/s, the sums over rows included).  A call of few rows per SM has nothing to
// stream and takes the direct kernel, 2.2 us on the device at 256 x 1536 (at 1001
// x 5120 9 us from the rings, 10.8 direct).
#pragma once

#include <cuda_fp8.h>

#include "ln_kernel.cuh"

namespace qknr {

struct RmsParams : LnParams {
  const char* residual;
  char* sum;
  const char* dsum;
  float* scales;
  long long residual_stride, sum_stride, dsum_stride;   // bytes per row
  MemSpan sp_residual, sp_sum, sp_dsum, sp_scales;
};

// what y is
enum { kRmsSame, kRmsRow8, kRmsBlock8 };
constexpr float kF8Max = 448.0f, kF8ScaleMin = 1.1754943508222875e-38f;   // 2^-126

// the larger, NaN where one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float abs_max(const float2 (&v)[4]) {
  float m = max_nan(fabsf(v[0].x), fabsf(v[0].y));
#pragma unroll
  for (int j = 1; j < 4; ++j) m = max_nan(m, max_nan(fabsf(v[j].x), fabsf(v[j].y)));
  return m;
}

// the scale of values up to m, and what they are multiplied by
__device__ __forceinline__ float f8_scale(float m) { return max_nan(__fdiv_rn(m, kF8Max), kF8ScaleMin); }

// Eight values times f in 8 bits.  f is the scale's reciprocal: with a division
// for each value the kernel takes 84 us instead of 63 at 2 x 4608 x 6144, and the
// results differ, by one 8-bit step, only next to the middle of two 8-bit values.
__device__ __forceinline__ uint2 pack_f8(const float2 (&v)[4], float f) {
  const float2 F = make_float2(f, f);
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(v[j], F), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// The largest of each of v's N values over a group's W warps (not negative; a
// NaN wins), the same in every thread.  Slots of absent warps hold zero.
template <int N>
__device__ __forceinline__ void rms_group_max(float (&v)[N], int W, int gw, int lane, int bar_id, float* red) {
  static_assert(N * kLnWarps <= kLnRedFloats, "slots");
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = max_nan(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
  if (W == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[N * gw + i] = v[i];
  named_barrier_sync(bar_id, 32 * W);
  const float4* r = reinterpret_cast<const float4*>(red);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < N * kLnWarps / 4; ++i) {
    const float4 part = r[i];
    v[0] = max_nan(v[0], part.x);
    v[1 % N] = max_nan(v[1 % N], part.y);
    v[0] = max_nan(v[0], part.z);
    v[1 % N] = max_nan(v[1 % N], part.w);
  }
}

// x + residual of one chunk
template <typename T>
__device__ __forceinline__ void rms_sum8(const uint4& x, bool more, const uint4& r, float2 (&h)[4]) {
  Elem<T>::unpack(x, h);
  if (!more) return;
  float2 b[4];
  Elem<T>::unpack(r, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __fadd2_rn(h[j], b[j]);
}

__device__ __forceinline__ float square_sum8(const float2 (&v)[4], float2 acc = make_float2(0.0f, 0.0f)) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __ffma2_rn(v[j], v[j], acc);
  return __fadd_rn(acc.x, acc.y);
}

// What a group does with NR rows (those at `at`, `at + step`, ... of which the
// first n are there) once their sums of squares are known: h and its gains in
// registers, everything written.  MINE(i): this thread has chunk l + 32 W i;
// GAIN(i): its gain.  The barriers of a scale per row use `red`.
template <typename T, int CPT, int NR, int OUT, typename MINE, typename GAIN>
__device__ __forceinline__ void rms_finish(const RmsParams& p, float2 (&X)[NR][CPT][4], const float (&squares)[NR], int n,
                                           long long at, long long step, int W, int gw, int lane, int bar, float* red,
                                           MINE mine, GAIN gain) {
  const int l = gw * 32 + lane;
  float top[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    top[r] = 0.0f;
    if (r >= n) break;
    const long long row = at + r * step;
    const float rstd = rsqrtf(__fadd_rn(__fmul_rn(squares[r], p.inv_c), p.eps));
    if (l == 0 && p.rstd && in_span(p.rstd + row, 4, p.sp_rstd, p.status)) p.rstd[row] = rstd;
    const float2 R = make_float2(rstd, rstd);
    char* dst = p.y + row * p.y_stride;
    char* sum = p.sum + row * p.sum_stride;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * 32 * W;
      if (p.sum && mine(i) && in_span(sum + k * 16, 16, p.sp_sum, p.status)) store16(sum + k * 16, Elem<T>::pack(X[r][i]));
      float2 g[4];
      gain(i, row, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) X[r][i][j] = __fmul2_rn(__fmul2_rn(X[r][i][j], R), g[j]);
      if (OUT == kRmsSame) {
        if (mine(i) && in_span(dst + k * 16, 16, p.sp_y, p.status)) store16(dst + k * 16, Elem<T>::pack(X[r][i]));
      } else if (OUT == kRmsRow8) {
        if (mine(i)) top[r] = max_nan(top[r], abs_max(X[r][i]));
      } else {
        // 128 columns are the chunks of 16 lanes
        float m = mine(i) ? abs_max(X[r][i]) : 0.0f;
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float scale = f8_scale(m);
        if (mine(i)) {
          const long long s = row * (p.hidden / 128) + k / 16;
          if (lane % 16 == 0 && in_span(p.scales + s, 4, p.sp_scales, p.status)) p.scales[s] = scale;
          if (in_span(dst + k * 8, 8, p.sp_y, p.status)) store8(dst + k * 8, pack_f8(X[r][i], __frcp_rn(scale)));
        }
      }
    }
  }
  if (OUT != kRmsRow8) return;
  rms_group_max<NR>(top, W, gw, lane, bar, red);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (r >= n) break;
    const long long row = at + r * step;
    const float scale = f8_scale(top[r]), f = __frcp_rn(scale);
    if (l == 0 && in_span(p.scales + row, 4, p.sp_scales, p.status)) p.scales[row] = scale;
    char* dst = p.y + row * p.y_stride;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * 32 * W;
      if (mine(i) && in_span(dst + k * 8, 8, p.sp_y, p.status)) store8(dst + k * 8, pack_f8(X[r][i], f));
    }
  }
}

// Calls of a few rows per SM, and rows whose columns are too many for a
// thread to keep their gains: a row is loaded straight into registers.
template <typename T, int CPT, int OUT>
__global__ void __launch_bounds__(kLnThreads) rms_forward_direct_kernel(const __grid_constant__ RmsParams p) {
  __shared__ __align__(16) float red[2 * kLnRedFloats];   // a CTA of several groups has groups of one warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W;
  const int l = gw * 32 + lane, n_chunks = p.hidden / 8;
  if (threadIdx.x < 2 * kLnRedFloats) red[threadIdx.x] = 0.0f;
  __syncthreads();
  grid_dependency_wait();
  const long long row = static_cast<long long>(blockIdx.x) * p.groups + grp;
  const char* src = p.x + row * p.x_stride;
  const char* res = p.residual + row * p.residual_stride;
  const bool more = p.residual != nullptr;
  if (row < p.tokens && in_span(src, p.row_bytes, p.sp_x, p.status) &&
      (!more || in_span(res, p.row_bytes, p.sp_residual, p.status))) {
    float2 X[1][CPT][4];
    uint4 raw[CPT], other[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * 32 * W;
      raw[i] = other[i] = make_uint4(0, 0, 0, 0);
      if (k < n_chunks) {
        raw[i] = ln_load16(src + k * 16);
        if (more) other[i] = ln_load16(res + k * 16);
      }
    }
    // what is not computed from x and residual is on its way while they come
    const long long set = ln_set(p, row);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      rms_sum8<T>(raw[i], more, other[i], X[0][i]);
      s = __fadd_rn(s, square_sum8(X[0][i]));
    }
    float t[1] = {s};
    ln_group_sum<1, kLnWarps>(t, true, W, gw, lane, 1 + grp, red);
    rms_finish<T, CPT, 1, OUT>(p, X, t, 1, row, 0, W, gw, lane, 1 + grp, red + kLnRedFloats,
                               [&](int i) { return l + i * 32 * W < n_chunks; },
                               [&](int i, long long, float2(&g)[4]) {
#pragma unroll
                                 for (int j = 0; j < 4; ++j) g[j] = make_float2(0.0f, 0.0f);
                                 if (l + i * 32 * W < n_chunks) ln_gain8<T>(p, set, l + i * 32 * W, g);
                               });
  }
  grid_dependents_launch();
}

// A group takes NR of its rows at a time: their sums share the shuffle trees
// and the barriers.
template <typename T, int CPT, int NR, int OUT>
__global__ void __launch_bounds__(kLnThreads, 1) rms_forward_kernel(const __grid_constant__ RmsParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W, l = gw * 32 + lane, n_chunks = p.hidden / 8;
  const bool more = p.residual != nullptr;
  LnRing ring(smem, p, more ? 2 * p.row_bytes : p.row_bytes, grp);
  ln_init_rings(smem, p.stages * p.groups);
  grid_dependency_wait();
  grid_dependents_launch();
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  long long row = static_cast<long long>(blockIdx.x) * p.groups + grp, ahead = row;
  const bool leader = gw == 0 && lane == 0 && !(p.flags & 1u);   // test only: issue nothing
  auto put = [&]() {
    ring.put(p.x + ahead * p.x_stride, p.sp_x, more ? p.residual + ahead * p.residual_stride : nullptr, p.sp_residual, p.row_bytes);
  };
  if (leader)
    for (int i = 0; i < p.stages && ahead < p.tokens; ++i, ahead += step) put();
  float* red = reinterpret_cast<float*>(smem + kLnOffRed) + grp * 2 * kLnRedFloats;
  float* buf = red;
  bool mine[CPT];
  float2 g[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    mine[i] = l + i * 32 * W < n_chunks;
#pragma unroll
    for (int j = 0; j < 4; ++j) g[i][j] = make_float2(0.0f, 0.0f);
  }
  long long set_end = 0;                          // first row past the sample whose gains are in g
  while (row < p.tokens) {
    if (row >= set_end) {
      const long long set = ln_set(p, row);
      set_end = (set + 1) * p.rows_per_batch;
#pragma unroll
      for (int i = 0; i < CPT; ++i)
        if (mine[i]) ln_gain8<T>(p, set, l + i * 32 * W, g[i]);
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
          uint4 a = make_uint4(0, 0, 0, 0), b = a;
          if (mine[i]) {
            a = st[l + i * 32 * W];
            if (more) b = st[n_chunks + l + i * 32 * W];
          }
          rms_sum8<T>(a, more, b, X[r][i]);
          t[r] = __fadd_rn(t[r], square_sum8(X[r][i]));
        }
        ring.next();
      }
    }
    const bool ok = ln_group_sum<NR, kLnWarps>(t, landed, W, gw, lane, 1 + grp, buf);
    // one barrier a step: the next one's sums go to the other buffer.  With a
    // scale per row the second barrier keeps the two apart.
    if (OUT != kRmsRow8) buf = buf == red ? red + kLnRedFloats : red;
    if (!ok) {
      if (leader) ring.drain(n);
      break;
    }
    if (leader)
      for (int r = 0; r < n; ++r) {
        --ring.in_flight;
        if (ahead < p.tokens) put();
        ahead += step;
      }
    rms_finish<T, CPT, NR, OUT>(p, X, t, n, row, step, W, gw, lane, 1 + grp, red + kLnRedFloats,
                                [&](int i) { return mine[i]; },
                                [&](int i, long long, float2(&v)[4]) {
#pragma unroll
                                  for (int j = 0; j < 4; ++j) v[j] = g[i][j];
                                });
    row += n * step;
  }
}

// ---------------------------------------------------------------------------
// backward

// Rows of more than kLnTile values: mean_c(g xhat) of each row, one CTA per row.
template <typename T>
__global__ void __launch_bounds__(256) rms_row_sums_kernel(const __grid_constant__ RmsParams p) {
  __shared__ __align__(16) float red[2][kLnRedFloats];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_chunks = p.hidden / 8;
  grid_dependency_wait();
  int parity = 0;
  for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x, parity ^= 1) {
    const char* xs = p.x + row * p.x_stride;
    const char* ds = p.dy + row * p.dy_stride;
    float2 s = make_float2(0.0f, 0.0f);
    if (in_span(xs, p.row_bytes, p.sp_x, p.status) && in_span(ds, p.row_bytes, p.sp_dy, p.status) &&
        in_span(p.rstd + row, 4, p.sp_rstd, p.status)) {
      const float2 R = make_float2(p.rstd[row], p.rstd[row]);
      const long long set = ln_set(p, row);
      for (int k = threadIdx.x; k < n_chunks; k += 256) {
        float2 gain[4], xh[4], dy[4];
        ln_gain8<T>(p, set, k, gain);
        ln_grad_values<T>(*reinterpret_cast<const uint4*>(xs + k * 16), *reinterpret_cast<const uint4*>(ds + k * 16),
                          make_float2(0.0f, 0.0f), R, xh, dy);
        ln_grad_sums(xh, dy, gain, s);
      }
    }
    float t[1] = {s.y};
    ln_group_sum<1, 8>(t, true, 8, warp, lane, 1, red[parity]);
    if (threadIdx.x == 0 && in_span(p.row_sums + row, 4, p.sp_ws, p.status)) p.row_sums[row] = __fmul_rn(t[0], p.inv_c);
  }
  grid_dependents_launch();
}

// One chunk's part of sum g xhat.
__device__ __forceinline__ float rms_grad_sum(const float2 (&xh)[4], const float2 (&dy)[4], const float2 (&gain)[4]) {
  float2 c = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __ffma2_rn(__fmul2_rn(dy[j], gain[j]), xh[j], c);
  return __fadd_rn(c.x, c.y);
}

// dx, and the sums of dy xhat over the rows, as ln_backward_kernel has them: a
// thread owns the same chunks of 8 columns for the whole launch and keeps
// their sums in registers over all the rows of a unit.  A stage holds a row of
// x, dy and, where it is given, dsum.
template <typename T, int CPT, int NR, bool LONG>
__global__ void __launch_bounds__(kLnBwdThreads, 1) rms_backward_kernel(const __grid_constant__ RmsParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps;
  const int tile = static_cast<int>(blockIdx.x % p.tiles), k0 = tile * (kLnTile / 8);
  const int n_chunks = p.hidden / 8 - k0 < kLnTile / 8 ? p.hidden / 8 - k0 : kLnTile / 8;   // of this tile
  const unsigned bytes = n_chunks * 16u;
  const bool more = p.dsum != nullptr;
  const unsigned stage_bytes = (more ? 3 : 2) * (p.tiles > 1 ? kLnTile * 2u : p.row_bytes);
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
    ring.put(p.x + a_row * p.x_stride + k0 * 16, p.sp_x, p.dy + a_row * p.dy_stride + k0 * 16, p.sp_dy, bytes,
             more ? p.dsum + a_row * p.dsum_stride + k0 * 16 : nullptr, p.sp_dsum);
    a_row += p.groups;
  };
  if (leader)
    for (int i = 0; i < p.stages; ++i) put();

  float* acc = reinterpret_cast<float*>(smem + kLnOffStages + p.stages * p.groups * stage_bytes);   // [groups][columns]
  float* red = reinterpret_cast<float*>(smem + kLnOffRed) + grp * 2 * kLnRedFloats;
  bool mine[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) mine[i] = l + i * 32 * W < n_chunks;
  bool ok = true;
  int given_up = 0;
  // The two buffers alternate from one step to the next, across units too: a
  // slow warp may still read the sums of the step before.
  float* buf = red;
  for (long long u = blockIdx.x / p.tiles; u < units; u += unit_step) {
    long long first, last;
    const long long set = rows_of(u, first, last);
    float2 dw[CPT][4], gain[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = gain[i][j] = make_float2(0.0f, 0.0f);
      if (mine[i]) ln_gain8<T>(p, set, k0 + l + i * 32 * W, gain[i]);
    }
    // the statistics of the rows after those in work
    const float* at_rstd = p.rstd + first + grp;
    int left = last - first > grp ? static_cast<int>((last - first - grp + p.groups - 1) / p.groups) : 0;   // the group's rows
    float nrstd[NR];
    auto stats = [&](int rows) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        nrstd[r] = 0.0f;
        if (rows > r && in_span(at_rstd, 4, p.sp_rstd, p.status)) nrstd[r] = *at_rstd;
        at_rstd += p.groups;
      }
    };
    stats(left);
    char* dst = p.dx + (first + grp) * p.dx_stride + (k0 + l) * 16;
    const float* sums = p.row_sums + first + grp; // LONG
    for (; left > 0; left -= NR, buf = buf == red ? red + kLnRedFloats : red) {
      float2 xh[NR][CPT][4], dy[NR][CPT][4], R[NR];
      uint4 past[NR][CPT];                        // dsum
      float t[NR];
      bool landed = true;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        R[r] = make_float2(nrstd[r], nrstd[r]);
        const bool some = r < left;               // an odd last row: its partner's dy is zero
        if (some) landed = ring.wait() && landed;
        const uint4* st = ring.row();
        t[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          uint4 xr = make_uint4(0, 0, 0, 0), dr = xr;
          past[r][i] = xr;
          if (some && mine[i]) {
            xr = st[l + i * 32 * W];
            dr = st[n_chunks + l + i * 32 * W];
            if (more) past[r][i] = st[2 * n_chunks + l + i * 32 * W];
          }
          ln_grad_values<T>(xr, dr, make_float2(0.0f, 0.0f), R[r], xh[r][i], dy[r][i]);
          if (!LONG) t[r] = __fadd_rn(t[r], rms_grad_sum(xh[r][i], dy[r][i], gain[i]));
        }
        if (some) ring.next();
      }
      stats(left - NR);
      ok = ln_group_sum<NR, kLnBwdWarps>(t, landed, W, gw, lane, 1 + grp, buf);
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
        float s = __fmul_rn(t[r], p.inv_c);
        if (LONG && r < left && in_span(sums, 4, p.sp_ws, p.status)) s = *sums;
        const float2 c = make_float2(-s, -s);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          float2 o[4], a[4];
          Elem<T>::unpack(past[r][i], a);         // zero where there is none
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i][j] = __ffma2_rn(dy[r][i][j], xh[r][i][j], dw[i][j]);
            o[j] = __ffma2_rn(__ffma2_rn(xh[r][i][j], c, __fmul2_rn(dy[r][i][j], gain[i][j])), R[r], a[j]);
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
      float* slot = acc + grp * cols;
      named_barrier_sync(15, 32 * W * p.groups);   // the previous unit's sums have been read
#pragma unroll
      for (int i = 0; i < CPT; ++i)
        if (mine[i]) {
          float2* a = reinterpret_cast<float2*>(slot + (l + i * 32 * W) * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = dw[i][j];
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
              const float2* a = reinterpret_cast<const float2*>(acc + g * cols + (l + i * 32 * W) * 8);
#pragma unroll
              for (int j = 0; j < 4; ++j) dw[i][j] = __fadd2_rn(dw[i][j], a[j]);
            }
    } else if (!ok) {
      break;                                      // the group left its rows together
    }
    if (grp == 0 && p.dweight) {
      // a sample of one unit: its sums are the result
      float* out = p.units_per_set == 1 ? p.dweight + set * p.hidden : p.parts + u * p.hidden;
      const MemSpan& sp = p.units_per_set == 1 ? p.sp_dweight : p.sp_ws;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float* at = out + (k0 + l + i * 32 * W) * 8;
        if (!mine[i] || !in_span(at, 32, sp, p.status)) continue;
        reinterpret_cast<float4*>(at)[0] = make_float4(dw[i][0].x, dw[i][0].y, dw[i][1].x, dw[i][1].y);
        reinterpret_cast<float4*>(at)[1] = make_float4(dw[i][2].x, dw[i][2].y, dw[i][3].x, dw[i][3].y);
      }
    }
  }
  if (leader && *ring.abort_flag) ring.drain(given_up);   // this group or another gave up
}

}  // namespace qknr
