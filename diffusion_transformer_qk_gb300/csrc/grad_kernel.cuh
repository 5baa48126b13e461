// Backward pass of the fused QK-RMSNorm + RoPE for sm_103a (formulas:
// qknr_grad.h).
//
// Bound by HBM: x and the incoming gradient are read once, the gradient of x
// is written once.  A team of D/8 lanes takes one head of one token, 8 values
// a lane, so the two sums over the head are shuffles inside the team.  A lane
// holds 4 rotation pairs: the two members of a pair meet in one thread (16
// contiguous bytes when interleaved, two 8-byte pieces D/2 apart when
// rotated by halves) and neither is read twice or shuffled.  Teams walk the
// (token, head) items of Q, then of K, in strides of the whole grid, and ask
// for the next item before they reduce the one they hold.  Each lane's
// columns never change, so its share of dgamma stays in registers; a CTA's
// teams add theirs in order through shared memory and write one partial row.
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

// The 4 pairs of a lane: `f` the first members, `s` the second.
template <typename T, bool RH>
__device__ __forceinline__ void grad_split(const uint4& r, float (&f)[4], float (&s)[4]) {
  float2 X[4];
  Elem<T>::unpack(r, X);
  if (RH) {
    f[0] = X[0].x; f[1] = X[0].y; f[2] = X[1].x; f[3] = X[1].y;
    s[0] = X[2].x; s[1] = X[2].y; s[2] = X[3].x; s[3] = X[3].y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = X[i].x;
      s[i] = X[i].y;
    }
  }
}

// 16 bytes of a head: contiguous, or 8 + 8 bytes half a head apart
template <int D, bool RH>
__device__ __forceinline__ uint4 grad_load(const char* head, int lane) {
  if (!RH) return __ldcs(reinterpret_cast<const uint4*>(head) + lane);
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(head) + lane);
  const uint2 b = __ldcs(reinterpret_cast<const uint2*>(head + D) + lane);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// the same 8 values of a table row as (first, second) members
template <typename CT, int D, bool RH>
__device__ __forceinline__ void grad_table(const char* row, int lane, float (&f)[4], float (&s)[4]) {
  if (RH) {
    float2 a[2], b[2];
    load_table4<CT>(reinterpret_cast<const unsigned char*>(row) + lane * 4 * sizeof(CT), a);
    load_table4<CT>(reinterpret_cast<const unsigned char*>(row) + (D / 2 + lane * 4) * sizeof(CT), b);
    f[0] = a[0].x; f[1] = a[0].y; f[2] = a[1].x; f[3] = a[1].y;
    s[0] = b[0].x; s[1] = b[0].y; s[2] = b[1].x; s[3] = b[1].y;
  } else {
    float2 a[4];
    load_table8<CT>(reinterpret_cast<const unsigned char*>(row) + lane * 8 * sizeof(CT), a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i].x;
      s[i] = a[i].y;
    }
  }
}

template <typename T, typename CT, int D, bool RH>
__global__ void __launch_bounds__(kGradThreads) qk_grad_kernel(const __grid_constant__ GradParams p) {
  constexpr int L = D / 8;                        // lanes per team
  constexpr int TEAMS = kGradThreads / L;
  __shared__ float acc[TEAMS][D];
  const int team = threadIdx.x / L, lane = threadIdx.x % L;
  const long long step = static_cast<long long>(gridDim.x) * TEAMS;
  grid_dependency_wait();

#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const GradSide& sd = p.side[w];
    const int H = sd.heads;
    float gf[4], gs[4], wf[4], ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) gf[i] = gs[i] = wf[i] = ws[i] = 0.0f;
    if (H > 0 && in_span(sd.gamma, D * 4, sd.sp_gamma, p.status)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gf[i] = sd.gamma[RH ? lane * 4 + i : lane * 8 + 2 * i];
        gs[i] = sd.gamma[RH ? D / 2 + lane * 4 + i : lane * 8 + 2 * i + 1];
      }
    }
    const long long items = p.tokens * H;
    const long long step_t = H ? step / H : 0;
    const int step_h = H ? static_cast<int>(step % H) : 0;
    long long it = static_cast<long long>(blockIdx.x) * TEAMS + team;
    long long t = H ? it / H : 0;
    int h = H ? static_cast<int>(it % H) : 0;
    // table row of the item, t % cos_rows, kept by addition
    const long long step_row = step_t % p.cos_rows;
    long long row = t % p.cos_rows;
    uint4 nx = make_uint4(0, 0, 0, 0), nd = nx;
    auto fetch = [&](long long item, long long tok, int head) {
      if (item >= items) return;
      const char* xs = sd.x + tok * sd.x_stride + head * (D * 2);
      const char* ds = sd.dy + tok * sd.dy_stride + head * (D * 2);
      if (!in_span(xs, D * 2, sd.sp_x, p.status) || !in_span(ds, D * 2, sd.sp_dy, p.status)) return;
      nx = grad_load<D, RH>(xs, lane);
      nd = grad_load<D, RH>(ds, lane);
    };
    fetch(it, t, h);
    // the whole warp goes round together (the shuffles below), so a team
    // past the end walks along on zeros and stores nothing
    const long long warp_first = it - (threadIdx.x % 32) / L;
    for (long long base = warp_first; base < items; base += step) {
      const uint4 xr = nx, dr = nd;
      const long long tok = t;
      const int head = h;
      const long long off = row * p.table_stride + head * p.head_stride;
      const bool live = it < items;
      it += step;
      t += step_t;
      h += step_h;
      row += step_row;
      if (h >= H) {
        h -= H;
        ++t;
        ++row;
      }
      if (row >= p.cos_rows) row -= p.cos_rows;
      float cf[4], cs[4], sf[4], ss[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) cf[i] = cs[i] = sf[i] = ss[i] = 0.0f;
      if (live) {
        if (in_span(p.cos + off, D * sizeof(CT), p.sp_cos, p.status) &&
            in_span(p.sin + off, D * sizeof(CT), p.sp_sin, p.status)) {
          grad_table<CT, D, RH>(p.cos + off, lane, cf, cs);
          grad_table<CT, D, RH>(p.sin + off, lane, sf, ss);
        }
      }
      fetch(it, t, h);
      float xf[4], xs[4], df[4], ds[4];
      grad_split<T, RH>(xr, xf, xs);
      grad_split<T, RH>(dr, df, ds);
      float sq = 0.0f, gx = 0.0f;
      float yf[4], ys[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // o1 = y1 cos1 - y2 sin1, o2 = y2 cos2 + y1 sin2
        yf[i] = __fmaf_rn(df[i], cf[i], __fmul_rn(ds[i], ss[i]));
        ys[i] = __fmaf_rn(ds[i], cs[i], -__fmul_rn(df[i], sf[i]));
        sq = __fmaf_rn(xf[i], xf[i], __fmaf_rn(xs[i], xs[i], sq));
        gx = __fmaf_rn(__fmul_rn(yf[i], gf[i]), xf[i], __fmaf_rn(__fmul_rn(ys[i], gs[i]), xs[i], gx));
      }
#pragma unroll
      for (int off = L / 2; off >= 1; off >>= 1) {
        sq = __fadd_rn(sq, __shfl_xor_sync(0xffffffffu, sq, off));
        gx = __fadd_rn(gx, __shfl_xor_sync(0xffffffffu, gx, off));
      }
      const float r = rsqrtf(__fmaf_rn(sq, p.inv_d, p.eps));
      const float m = __fmul_rn(__fmul_rn(__fmul_rn(r, r), r), __fmul_rn(gx, p.inv_d));
      if (!live) continue;
      float of[4], os[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wf[i] = __fmaf_rn(yf[i], __fmul_rn(xf[i], r), wf[i]);
        ws[i] = __fmaf_rn(ys[i], __fmul_rn(xs[i], r), ws[i]);
        of[i] = __fmaf_rn(-xf[i], m, __fmul_rn(__fmul_rn(yf[i], gf[i]), r));
        os[i] = __fmaf_rn(-xs[i], m, __fmul_rn(__fmul_rn(ys[i], gs[i]), r));
      }
      char* dst = sd.dx + tok * sd.dx_stride + head * (D * 2);
      if (!in_span(dst, D * 2, sd.sp_dx, p.status)) continue;
      if (RH) {
        const float2 O[4] = {make_float2(of[0], of[1]), make_float2(of[2], of[3]), make_float2(os[0], os[1]),
                             make_float2(os[2], os[3])};
        const uint4 v = Elem<T>::pack(O);
        store8(dst + lane * 8, make_uint2(v.x, v.y));
        store8(dst + D + lane * 8, make_uint2(v.z, v.w));
      } else {
        const float2 O[4] = {make_float2(of[0], os[0]), make_float2(of[1], os[1]), make_float2(of[2], os[2]),
                             make_float2(of[3], os[3])};
        store16(dst + lane * 16, Elem<T>::pack(O));
      }
    }
    // this side's partial row
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[team][RH ? lane * 4 + i : lane * 8 + 2 * i] = wf[i];
      acc[team][RH ? D / 2 + lane * 4 + i : lane * 8 + 2 * i + 1] = ws[i];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.0f;
      for (int g = 0; g < TEAMS; ++g) s = __fadd_rn(s, acc[g][threadIdx.x]);
      float* out = p.parts + (static_cast<long long>(blockIdx.x) * 2 + w) * D + threadIdx.x;
      if (in_span(out, 4, p.sp_ws, p.status)) *out = s;
    }
  }

  // V's gradient, copied
  if (p.v_chunks > 0) {
    const long long items = p.tokens * p.v_chunks;
    for (long long it = static_cast<long long>(blockIdx.x) * kGradThreads + threadIdx.x; it < items;
         it += static_cast<long long>(gridDim.x) * kGradThreads) {
      const long long t = it / p.v_chunks, c = it % p.v_chunks;
      const char* src = p.dv + t * p.dv_stride + c * 16;
      char* dst = p.dv_out + t * p.dv_out_stride + c * 16;
      if (in_span(src, 16, p.sp_dv, p.status) && in_span(dst, 16, p.sp_dv_out, p.status))
        store16(dst, __ldcs(reinterpret_cast<const uint4*>(src)));
    }
  }
  grid_dependents_launch();
}

}  // namespace qknr
