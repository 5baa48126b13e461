// The second half of a sum over token rows: adds the partial sums that a
// kernel's CTAs left in the caller's workspace, in a fixed order.
#pragma once

#include "qknr_ptx.cuh"

namespace qknr {

struct PartsParams {
  const float* parts;         // [sets][units][2][cols]
  float* out[2];              // [sets][cols] each; null: not wanted
  int cols;                   // a multiple of 4
  long long units;
  MemSpan sp_parts, sp_out[2];
  int* status;
};

constexpr int kPartsCols = 128, kPartsRows = 16;

// out[i][s][c] = sum over u of parts[s][u][i][c]: 128 columns per CTA, four
// to a thread, 16 threads to a column that each take every 16th part, then a
// tree in a fixed order.  Bound by latency: the parts were just written and
// lie in L2.
static __global__ void __launch_bounds__(32 * kPartsRows) parts_kernel(const __grid_constant__ PartsParams p) {
  __shared__ float4 sm[kPartsRows][32];
  const int col_tiles = (p.cols + kPartsCols - 1) / kPartsCols;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x % col_tiles) * kPartsCols + 4 * tx;
  const int which = static_cast<int>(blockIdx.x / col_tiles % 2);
  const long long set = blockIdx.x / col_tiles / 2;
  auto add = [](float4 a, const float4& b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
  };
  grid_dependency_wait();
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < p.cols) {
    const float* src = p.parts + (set * p.units * 2 + which) * p.cols + c;
#pragma unroll 8
    for (long long u = ty; u < p.units; u += kPartsRows) {
      const float* at = src + u * 2 * p.cols;
      if (in_span(at, 16, p.sp_parts, p.status)) s = add(s, __ldcg(reinterpret_cast<const float4*>(at)));
    }
  }
  sm[ty][tx] = s;
  __syncthreads();
#pragma unroll
  for (int h = kPartsRows / 2; h >= 1; h >>= 1) {
    if (ty < h) sm[ty][tx] = add(sm[ty][tx], sm[ty + h][tx]);
    __syncthreads();
  }
  float* out = p.out[which];
  if (ty == 0 && c < p.cols && out) {
    out += set * p.cols + c;
    const float4 v = sm[0][tx];
    if (in_span(out, 16, p.sp_out[which], p.status)) {
      out[0] = v.x;
      out[1] = v.y;
      out[2] = v.z;
      out[3] = v.w;
    }
  }
  grid_dependents_launch();
}

inline long long parts_grid(const PartsParams& p, long long sets) {
  return sets * 2 * ((p.cols + kPartsCols - 1) / kPartsCols);
}

}  // namespace qknr
