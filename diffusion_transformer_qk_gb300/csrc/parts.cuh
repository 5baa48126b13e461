// The second half of a sum over token rows: adds the partial sums that a
// kernel's CTAs left in the caller's workspace, in a fixed order.
#pragma once

#include "qknr_ptx.cuh"

namespace qknr {

struct PartsParams {
  const float* parts;         // [sets][units][2][cols]
  float* out[2];              // [sets][cols] each; null: not wanted
  int cols;
  long long units;
  MemSpan sp_parts, sp_out[2];
  int* status;
};

constexpr int kPartsCols = 32, kPartsRows = 16;

// out[i][s][c] = sum over u of parts[s][u][i][c]: 32 columns per CTA, 16
// threads a column that each take every 16th part, then a tree in a fixed
// order.  Bound by latency: the parts were just written and lie in L2.
static __global__ void __launch_bounds__(kPartsCols* kPartsRows) parts_kernel(const __grid_constant__ PartsParams p) {
  __shared__ float sm[kPartsRows][kPartsCols + 1];
  const int col_tiles = (p.cols + kPartsCols - 1) / kPartsCols;
  const int tx = threadIdx.x % kPartsCols, ty = threadIdx.x / kPartsCols;
  const int c = static_cast<int>(blockIdx.x % col_tiles) * kPartsCols + tx;
  const int which = static_cast<int>(blockIdx.x / col_tiles % 2);
  const long long set = blockIdx.x / col_tiles / 2;
  grid_dependency_wait();
  float s = 0.0f;
  if (c < p.cols) {
    const float* src = p.parts + (set * p.units * 2 + which) * p.cols + c;
#pragma unroll 4
    for (long long u = ty; u < p.units; u += kPartsRows) {
      const float* at = src + u * 2 * p.cols;
      if (in_span(at, 4, p.sp_parts, p.status)) s = __fadd_rn(s, *at);
    }
  }
  sm[ty][tx] = s;
  __syncthreads();
#pragma unroll
  for (int h = kPartsRows / 2; h >= 1; h >>= 1) {
    if (ty < h) sm[ty][tx] = __fadd_rn(sm[ty][tx], sm[ty + h][tx]);
    __syncthreads();
  }
  float* out = p.out[which];
  if (ty == 0 && c < p.cols && out) {
    out += set * p.cols + c;
    if (in_span(out, 4, p.sp_out[which], p.status)) *out = sm[0][tx];
  }
  grid_dependents_launch();
}

inline long long parts_grid(const PartsParams& p, long long sets) {
  return sets * 2 * ((p.cols + kPartsCols - 1) / kPartsCols);
}

}  // namespace qknr
