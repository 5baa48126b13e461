// Layer norm, forward and backward, for sm_103a (formulas: qknr_ln.h).
//
// Both passes are bound by HBM: the forward reads x and writes y, the
// backward reads x and dy and writes dx.  A row lives in the registers of
// the warps that share it: thread l of a group of W warps holds the 16-byte
// chunks l, l + 32 W, ... of the row, so the variance is a true second pass
// (squared deviations from the finished mean) without a second read, and a
// group asks for its next row before it reduces the one it holds, which keeps
// the loads in flight across the reductions' latency.
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
  float eps;
  float inv_c;
  float unit;                 // added to the weight
  int* status;
  MemSpan sp_x, sp_y, sp_dy, sp_dx, sp_weight, sp_bias, sp_mean, sp_rstd, sp_dweight, sp_dbias, sp_ws;
};

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

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// The sum of `a` (and of `b`) over a group's W warps, the same in every
// thread: a shuffle tree inside each warp, then the warps' sums added in
// order from shared memory.  `red` alternates between two buffers, so the
// one barrier also keeps a fast warp from overwriting sums a slow one reads.
__device__ __forceinline__ float2 ln_group_sum(float2 v, int W, int gw, int lane, int bar_id, float2* red) {
  v.x = ln_warp_sum(v.x);
  v.y = ln_warp_sum(v.y);
  if (W == 1) return v;
  if (lane == 0) red[gw] = v;
  named_barrier_sync(bar_id, 32 * W);
  float2 s = red[0];
  for (int w = 1; w < W; ++w) s = __fadd2_rn(s, red[w]);
  return s;
}

__device__ __forceinline__ float ln_hsum(const float2 (&v)[4]) {
  const float2 s = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
  return __fadd_rn(s.x, s.y);
}

constexpr int kLnFwdThreads = 512;

template <typename T, int CPT>
__global__ void __launch_bounds__(kLnFwdThreads) ln_forward_kernel(const __grid_constant__ LnParams p) {
  __shared__ float2 red[2][kLnFwdThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W;
  const int l = gw * 32 + lane, step = 32 * W, n_chunks = p.hidden / 8;
  const long long stride = static_cast<long long>(gridDim.x) * p.groups;
  const unsigned row_bytes = p.hidden * 2u;
  grid_dependency_wait();

  uint4 next[CPT];
  long long row = static_cast<long long>(blockIdx.x) * p.groups + grp;
  auto fetch = [&](long long r) {
    const char* src = p.x + r * p.x_stride;
    const bool ok = r < p.tokens && in_span(src, row_bytes, p.sp_x, p.status);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * step;
      next[i] = make_uint4(0, 0, 0, 0);
      if (ok && k < n_chunks) next[i] = ln_load16(src + k * 16);
    }
  };
  fetch(row);
  for (; row < p.tokens; row += stride) {
    uint4 raw[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) raw[i] = next[i];
    fetch(row + stride);
    // mean: chunks past the row hold zeros
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float2 X[4];
      Elem<T>::unpack(raw[i], X);
      s = __fadd_rn(s, ln_hsum(X));
    }
    const int bar = 1 + grp;
    const float mean = __fmul_rn(ln_group_sum(make_float2(s, 0.0f), W, gw, lane, bar, red[0]).x, p.inv_c);
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
    const float var = __fmul_rn(ln_group_sum(make_float2(s, 0.0f), W, gw, lane, bar, red[1]).x, p.inv_c);
    const float rstd = rsqrtf(__fadd_rn(var, p.eps));
    if (l == 0) {
      if (p.mean && in_span(p.mean + row, 4, p.sp_mean, p.status)) p.mean[row] = mean;
      if (p.rstd && in_span(p.rstd + row, 4, p.sp_rstd, p.status)) p.rstd[row] = rstd;
    }
    const long long set = row / p.rows_per_batch;
    const char* brow = p.bias + set * p.param_stride;
    char* dst = p.y + row * p.y_stride;
    const bool ok = in_span(dst, row_bytes, p.sp_y, p.status) &&
                    (!p.bias || in_span(brow, static_cast<unsigned long long>(p.hidden) * (p.param_fp32 ? 4 : 2),
                                        p.sp_bias, p.status));
    const float2 R = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int k = l + i * step;
      if (ok && k < n_chunks) {
        float2 X[4], g[4], b[4];
        Elem<T>::unpack(raw[i], X);
        ln_gain8<T>(p, set, k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = make_float2(0.0f, 0.0f);
        if (p.bias) ln_param8<T>(brow, k, p.param_fp32, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) X[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(X[j], nm), R), g[j], b[j]);
        store16(dst + k * 16, Elem<T>::pack(X));
      }
    }
  }
  grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// backward

constexpr int kLnBwdWarps = 32;
constexpr int kLnBwdThreads = 32 * kLnBwdWarps;
constexpr int kLnTile = 8 * kLnBwdThreads;        // columns of one CTA: a chunk per thread
constexpr int kLnBwdRedBytes = 2 * kLnBwdWarps * 8;

// g * xhat and g of one chunk, summed into (sum g, sum g xhat)
template <typename T>
__device__ __forceinline__ void ln_grad_chunk(const uint4& xr, const uint4& dr, const float2 (&gain)[4], float2 nm,
                                              float2 R, float2 (&xh)[4], float2 (&dy)[4], float2& s) {
  Elem<T>::unpack(xr, xh);
  Elem<T>::unpack(dr, dy);
  float2 a = make_float2(0.0f, 0.0f), c = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xh[j] = __fmul2_rn(__fadd2_rn(xh[j], nm), R);
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
  __shared__ float2 red[2][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_chunks = p.hidden / 8;
  grid_dependency_wait();
  int parity = 0;
  for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x, parity ^= 1) {
    const char* xs = p.x + row * p.x_stride;
    const char* ds = p.dy + row * p.dy_stride;
    float2 s = make_float2(0.0f, 0.0f);
    if (in_span(xs, p.hidden * 2u, p.sp_x, p.status) && in_span(ds, p.hidden * 2u, p.sp_dy, p.status) &&
        in_span(p.mean + row, 4, p.sp_mean, p.status) && in_span(p.rstd + row, 4, p.sp_rstd, p.status)) {
      const float2 nm = make_float2(-p.mean[row], -p.mean[row]), R = make_float2(p.rstd[row], p.rstd[row]);
      const long long set = row / p.rows_per_batch;
      for (int k = threadIdx.x; k < n_chunks; k += 256) {
        float2 gain[4], xh[4], dy[4];
        ln_gain8<T>(p, set, k, gain);
        ln_grad_chunk<T>(*reinterpret_cast<const uint4*>(xs + k * 16), *reinterpret_cast<const uint4*>(ds + k * 16),
                         gain, nm, R, xh, dy, s);
      }
    }
    s = ln_group_sum(s, 8, warp, lane, 1, red[parity]);
    if (threadIdx.x == 0 && in_span(p.row_sums + 2 * row, 8, p.sp_ws, p.status)) {
      p.row_sums[2 * row] = __fmul_rn(s.x, p.inv_c);
      p.row_sums[2 * row + 1] = __fmul_rn(s.y, p.inv_c);
    }
  }
  grid_dependents_launch();
}

// dx, and the sums of dy and dy xhat over the rows.  A thread owns one chunk
// of 8 columns for the whole launch, so those sums stay in its registers
// over all the rows of a unit (a chunk of one sample's rows); the CTA's row
// groups then add theirs in order through shared memory and write the unit's
// partial sums, or the result where a sample is one unit.  LONG: the row
// spans several CTAs (a column tile each) and its two sums come from
// ln_row_sums_kernel.
template <typename T, bool LONG>
__global__ void __launch_bounds__(kLnBwdThreads) ln_backward_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ float2 red[];                 // [2][kLnBwdWarps], two buffers used in turn
  float* acc = reinterpret_cast<float*>(red + 2 * kLnBwdWarps);   // [groups][2][columns of the tile]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.group_warps, grp = warp / W, gw = warp % W;
  const int tile = static_cast<int>(blockIdx.x % p.tiles);
  const int k0 = tile * (kLnTile / 8), n_chunks = p.hidden / 8;
  const int k = k0 + gw * 32 + lane;              // this thread's chunk
  const int tile_cols = (n_chunks - k0 < kLnTile / 8 ? n_chunks - k0 : kLnTile / 8) * 8;
  const bool mine = k < n_chunks;
  const long long units = p.sets * p.units_per_set;
  grid_dependency_wait();

  for (long long u = blockIdx.x / p.tiles; u < units; u += gridDim.x / p.tiles) {
    const long long set = u / p.units_per_set;
    const long long set_end = (set + 1) * p.rows_per_batch < p.tokens ? (set + 1) * p.rows_per_batch : p.tokens;
    const long long first = set * p.rows_per_batch + (u % p.units_per_set) * p.unit_rows;
    const long long last = first + p.unit_rows < set_end ? first + p.unit_rows : set_end;
    float2 dw[4], db[4], gain[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = db[j] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) gain[j] = make_float2(0.0f, 0.0f);
    if (mine) ln_gain8<T>(p, set, k, gain);

    uint4 nx, nd;
    float nmean, nrstd;
    auto fetch = [&](long long r) {
      nx = nd = make_uint4(0, 0, 0, 0);
      nmean = nrstd = 0.0f;
      const char* xs = p.x + r * p.x_stride + k * 16;
      const char* ds = p.dy + r * p.dy_stride + k * 16;
      if (r < last && mine && in_span(xs, 16, p.sp_x, p.status) && in_span(ds, 16, p.sp_dy, p.status)) {
        nx = ln_load16(xs);
        nd = ln_load16(ds);
      }
      if (r < last && in_span(p.mean + r, 4, p.sp_mean, p.status) && in_span(p.rstd + r, 4, p.sp_rstd, p.status)) {
        nmean = p.mean[r];
        nrstd = p.rstd[r];
      }
    };
    fetch(first + grp);
    int parity = 0;
    for (long long row = first + grp; row < last; row += p.groups, parity ^= 1) {
      const uint4 xr = nx, dr = nd;
      const float2 nm = make_float2(-nmean, -nmean), R = make_float2(nrstd, nrstd);
      fetch(row + p.groups);
      float2 xh[4], dy[4], s = make_float2(0.0f, 0.0f);
      ln_grad_chunk<T>(xr, dr, gain, nm, R, xh, dy, s);
      if (LONG) {
        s = make_float2(0.0f, 0.0f);
        if (in_span(p.row_sums + 2 * row, 8, p.sp_ws, p.status))
          s = *reinterpret_cast<const float2*>(p.row_sums + 2 * row);
      } else {
        s = ln_group_sum(s, W, gw, lane, 1 + grp, red + parity * kLnBwdWarps + grp * W);
        s = __fmul2_rn(s, make_float2(p.inv_c, p.inv_c));
      }
      const float2 c1 = make_float2(-s.x, -s.x), c2 = make_float2(-s.y, -s.y);
      float2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        db[j] = __fadd2_rn(db[j], dy[j]);
        dw[j] = __ffma2_rn(dy[j], xh[j], dw[j]);
        o[j] = __fmul2_rn(__ffma2_rn(xh[j], c2, __ffma2_rn(dy[j], gain[j], c1)), R);
      }
      char* dst = p.dx + row * p.dx_stride + k * 16;
      if (mine && in_span(dst, 16, p.sp_dx, p.status)) store16(dst, Elem<T>::pack(o));
    }

    // the groups' sums, added in order
    const int c = (gw * 32 + lane) * 8;
    if (p.groups > 1) {
      float* slot = acc + grp * 2 * tile_cols;
      __syncthreads();                            // the previous unit's sums have been read
      if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<float2*>(slot + c + 2 * j) = dw[j];
          *reinterpret_cast<float2*>(slot + tile_cols + c + 2 * j) = db[j];
        }
      }
      __syncthreads();
      if (grp == 0 && mine) {
        for (int g = 1; g < p.groups; ++g) {
          const float* other = acc + g * 2 * tile_cols;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[j] = __fadd2_rn(dw[j], *reinterpret_cast<const float2*>(other + c + 2 * j));
            db[j] = __fadd2_rn(db[j], *reinterpret_cast<const float2*>(other + tile_cols + c + 2 * j));
          }
        }
      }
    }
    if (grp == 0 && mine) {
      const bool whole = p.units_per_set == 1;
      float* ow = whole ? p.dweight : p.parts;
      float* ob = whole ? p.dbias : p.parts;
      if (ow) {
        ow += whole ? set * p.hidden + k * 8 : u * 2 * p.hidden + k * 8;
        if (in_span(ow, 32, whole ? p.sp_dweight : p.sp_ws, p.status)) {
          reinterpret_cast<float4*>(ow)[0] = make_float4(dw[0].x, dw[0].y, dw[1].x, dw[1].y);
          reinterpret_cast<float4*>(ow)[1] = make_float4(dw[2].x, dw[2].y, dw[3].x, dw[3].y);
        }
      }
      if (ob) {
        ob += whole ? set * p.hidden + k * 8 : (u * 2 + 1) * p.hidden + k * 8;
        if (in_span(ob, 32, whole ? p.sp_dbias : p.sp_ws, p.status)) {
          reinterpret_cast<float4*>(ob)[0] = make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
          reinterpret_cast<float4*>(ob)[1] = make_float4(db[2].x, db[2].y, db[3].x, db[3].y);
        }
      }
    }
  }
  grid_dependents_launch();
}

}  // namespace qknr
