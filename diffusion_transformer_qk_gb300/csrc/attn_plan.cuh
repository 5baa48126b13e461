// Work lists of attention over sequences whose lengths only the device knows
// (packed sequences; samples with lengths beside a shared prefix), for sm_103a.
//
// A head's tiles, of all sequences one after the other, form a line of items;
// a call's work is that line once per head.  An item's cost is its blocks (the
// iterations of its contraction) and one unit for its epilogue.  Every CTA
// gets an equal share of the whole cost, cut inside a tile where that is worth
// it: parts of a tile are joined in a fixed order by a second kernel.  So a
// batch of one long and many short sequences keeps all SMs busy to the end.
//
// attn_plan_kernel works the items and the CTAs' shares out, in one CTA (a
// scan over the sequences, one over the items, a search per CTA): 3 us for
// some tens of sequences, overlapped with the launch of the kernel that reads
// the plan.
#pragma once

#include "attn_kernel.cuh"

namespace qknr {

enum { kPlanQueries, kPlanKeys, kPlanFew };       // what a tile's rows are

struct AttnPlanJob {
  int kind;
  int rows;                   // rows of a tile (kPlanFew: of a key head's group * q_len)
  int heads, group, causal;
  int ctas;
  int whole;                  // tiles are not cut if none costs more than this
  int least;                  // units of a share at least
  int max_items;
  int batch, seq_q, seq_k;    // sequence b: rows b * seq .. of lens[b] (null: seq) rows,
  const int* q_lens;
  const int* k_lens;
  const int* q_starts;        // or, where these are given, rows starts[b] .. starts[b + 1] of seq rows in all
  const int* k_starts;
  AttnPlan plan;
  MemSpan sp_q_lens, sp_k_lens, sp_q_starts, sp_k_starts;
};

struct AttnPlanParams {
  AttnPlanJob job[2];
  int* status;
};

constexpr int kPlanThreads = 1024;

// Inclusive scan over the CTA's threads; `all`: over everybody.
template <typename V, typename OP>
__device__ __forceinline__ V plan_scan(V v, OP op, V* warps, V& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const V o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = op(o, v);
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    V w = warps[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const V o = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w = op(o, w);
    }
    warps[lane] = w;
  }
  __syncthreads();
  all = warps[31];
  return warp == 0 ? v : op(warps[warp - 1], v);
}

// The blocks of item t of a sequence.
__device__ __forceinline__ int plan_blocks(const AttnPlanJob& j, int t, int q_len, int k_len) {
  const int diag = k_len - q_len;
  if (j.kind == kPlanFew) return (k_len + kTile - 1) / kTile;
  if (j.kind == kPlanQueries) {
    const int last = min(t * j.rows + j.rows, q_len);
    const int keys = j.causal ? min(max(last + diag, 0), k_len) : k_len;
    return (keys + kTile - 1) / kTile;
  }
  const int k0 = t * j.rows, end = (q_len + kTile - 1) / kTile;
  const int first = j.causal && k0 - diag > 0 ? min((k0 - diag) / kTile, end) : 0;
  return (end - first) * j.group;
}

// One CTA per job.
static __global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnPlanParams p) {
  __shared__ long long warps[32];
  __shared__ int4 seqs[kPlanThreads];             // q row, q_len, k row, k_len
  __shared__ int firsts[kPlanThreads], tiles0[kPlanThreads], counts[kPlanThreads];
  const AttnPlanJob& j = p.job[blockIdx.x];
  const AttnPlan& out = j.plan;
  int* iwarps = reinterpret_cast<int*>(warps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const auto add = [](auto a, auto b) { return a + b; };
  const auto most = [](int a, int b) { return a > b ? a : b; };
  grid_dependency_wait();
  grid_dependents_launch();
  // Starts are clamped to the rows there are, and one that falls counts as the
  // largest before it: whatever they say, no row belongs to two sequences.
  auto start = [&](const int* starts, const MemSpan& sp, int b, int rows) {
    if (!in_span(starts + b, 4, sp, p.status)) return 0;
    return min(max(starts[b], 0), rows);
  };
  int items = 0, q_tiles = 0, q_at = 0, k_at = 0;
  if (j.q_starts) q_at = start(j.q_starts, j.sp_q_starts, 0, j.seq_q);
  if (j.k_starts) k_at = start(j.k_starts, j.sp_k_starts, 0, j.seq_k);
  const int k_first = k_at;
  for (int base = 0; base < j.batch; base += kPlanThreads) {
    const int b = base + tid;
    const bool there = b < j.batch;
    int4 s = make_int4(0, 0, 0, 0);
    int all;
    if (j.q_starts) {
      const int v = there ? start(j.q_starts, j.sp_q_starts, b + 1, j.seq_q) : 0;
      const int end = max(plan_scan<int>(v, most, iwarps, all), q_at);
      __syncthreads();
      firsts[tid] = end;
      __syncthreads();
      s.x = tid ? firsts[tid - 1] : q_at;
      s.y = there ? end - s.x : 0;
      q_at = max(q_at, all);
    } else if (there) {
      s.x = b * j.seq_q;
      s.y = clamp_len(j.q_lens, b, j.seq_q, j.sp_q_lens, p.status);
    }
    if (j.k_starts) {
      const int v = there ? start(j.k_starts, j.sp_k_starts, b + 1, j.seq_k) : 0;
      const int end = max(plan_scan<int>(v, most, iwarps, all), k_at);
      __syncthreads();
      firsts[tid] = end;
      __syncthreads();
      s.z = tid ? firsts[tid - 1] : k_at;
      s.w = there ? end - s.z : 0;
      k_at = max(k_at, all);
    } else if (there) {
      s.z = b * j.seq_k;
      s.w = clamp_len(j.k_lens, b, j.seq_k, j.sp_k_lens, p.status);
    }
    const int of = j.kind == kPlanKeys ? s.w : j.kind == kPlanFew ? s.y * j.group : s.y;
    const int n = there ? (of + j.rows - 1) / j.rows : 0, nq = there ? (s.y + kTile - 1) / kTile : 0;
    const int first = items + plan_scan<int>(n, add, iwarps, all) - n;
    items += all;
    const int first_q = q_tiles + plan_scan<int>(nq, add, iwarps, all) - nq;
    q_tiles += all;
    __syncthreads();
    seqs[tid] = s;
    firsts[tid] = first;
    tiles0[tid] = first_q;
    counts[tid] = n;
    if (there && out.seq_items && in_span(out.seq_items + b, 4, out.sp, p.status)) out.seq_items[b] = first;
    __syncthreads();
    // a warp per sequence
    for (int i = warp; i < kPlanThreads && base + i < j.batch; i += kPlanThreads / 32) {
      const int4 q = seqs[i];
      for (int t = lane; t < counts[i]; t += 32) {
        int4* at = out.items + 2LL * (firsts[i] + t);
        const int blocks = plan_blocks(j, t, q.y, q.w);
        if (firsts[i] + t >= j.max_items || !in_span(at, 32, out.sp, p.status)) continue;
        at[0] = q;
        at[1] = make_int4(t * j.rows, blocks, blocks + 1, tiles0[i]);
      }
    }
    __syncthreads();
  }
  // where each item's units begin, and the costliest
  long long units = 0;
  int costliest = 0;
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + tid;
    const int u = i < items && in_span(out.items + 2LL * i, 32, out.sp, p.status) ? out.items[2LL * i + 1].z : 0;
    long long all;
    const long long upto = units + plan_scan<long long>(u, add, warps, all);
    units += all;
    if (i < items && in_span(out.prefix + i, 8, out.sp, p.status)) out.prefix[i] = upto - u;
    int top;
    plan_scan<int>(u, most, iwarps, top);
    costliest = max(costliest, top);
    __syncthreads();
  }
  if (tid == 0 && in_span(out.head, 16, out.sp, p.status)) {
    out.head[0] = items;
    out.head[1] = k_first;
    out.head[2] = k_at;
  }
  __syncthreads();
  // where each CTA's share begins
  const long long work = units * j.heads;
  long long active = work / j.least;
  if (active > j.ctas) active = j.ctas;
  if (active < 1) active = 1;
  for (int c = tid; c <= j.ctas; c += kPlanThreads) {
    int2 at = make_int2(j.heads * items, 0);
    if (c < active && units > 0) {
      const long long x = work / active * c + work % active * c / active;
      const int h = static_cast<int>(x / units);
      const long long off = x - h * units;
      int lo = 0, hi = items - 1;                 // the last item that begins at or before `off`
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (out.prefix[mid] <= off) lo = mid;
        else hi = mid - 1;
      }
      int o = static_cast<int>(off - out.prefix[lo]);
      const int u = out.items[2LL * lo + 1].z;
      // no cut where it saves little: within two blocks of an end, or at all
      if (costliest <= j.whole || o < 2 || u - o < 3) {
        lo += 2 * o >= u;
        o = 0;
      }
      at = make_int2(h * items + lo, o);
    }
    if (in_span(out.spans + c, 8, out.sp, p.status)) out.spans[c] = at;
  }
}

// ---------------------------------------------------------------------------
// joining

// The parts of a tile: slots first, then every second one.
struct PlanParts {
  int c, cuts;                // the CTA that began it; how many times it was cut
  __device__ __forceinline__ int slot(int i) const { return i == 0 ? 2 * c + 1 : 2 * (c + i); }
};

// A whole warp: how the shares cut tile `tile`.
__device__ __forceinline__ PlanParts plan_parts(const AttnPlan& plan, int ctas, int tile, int lane, int* status) {
  int before = 0, cuts = 0;
  for (int c = lane; c - lane <= ctas; c += 32) {
    int2 at = make_int2(0x7fffffff, 0);
    if (c <= ctas && in_span(plan.spans + c, 8, plan.sp, status)) at = plan.spans[c];
    before += __popc(__ballot_sync(0xffffffffu, at.x < tile || (at.x == tile && at.y == 0)));
    cuts += __popc(__ballot_sync(0xffffffffu, at.x == tile && at.y > 0));
  }
  return PlanParts{before - 1, cuts};
}

// The tile that boundary c of the shares is the first to cut, or -1.
__device__ __forceinline__ int plan_cut_tile(const AttnPlan& plan, int c, int* status) {
  if (!in_span(plan.spans + c - 1, 16, plan.sp, status)) return -1;
  const int2 at = plan.spans[c], prev = plan.spans[c - 1];
  return at.y > 0 && (prev.x != at.x || prev.y == 0) ? at.x : -1;
}

constexpr int kPlanJoinCtas = 8;                  // CTAs that share a cut tile's rows

// o = sum_i w_i o_i / sum_i w_i l_i over the parts of one row, w_i =
// exp2((m_i - max m) scale): first all maxima, then the sums.
template <int D>
struct RowJoin {
  float m = -INFINITY, total = 0.0f;
  float2 acc[D / 64];
  __device__ __forceinline__ RowJoin() {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = make_float2(0.0f, 0.0f);
  }
  template <typename P>
  __device__ __forceinline__ void top(const P& p, long long k) {
    if (in_span(p.stats + 2 * k, 8, p.sp_stats, p.status)) m = fmaxf(m, p.stats[2 * k]);
  }
  template <typename P>
  __device__ __forceinline__ void add(const P& p, long long k, int lane) {
    if (!in_span(p.stats + 2 * k, 8, p.sp_stats, p.status) || !in_span(p.part + k * D, 4 * D, p.sp_part, p.status)) return;
    const float2 st = *reinterpret_cast<const float2*>(p.stats + 2 * k);
    // a part that saw no key has sum 0, maximum -inf and zeros
    const float w = st.x == m ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(st.x, m), p.scale_log2));
    total = __fmaf_rn(w, st.y, total);
    const float2* src = reinterpret_cast<const float2*>(p.part + k * D) + lane;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = __ffma2_rn(make_float2(w, w), src[32 * e], acc[e]);
  }
  // a warp's row of o and its lse
  template <typename T, typename P>
  __device__ __forceinline__ void write(const P& p, char* dst, float* lse, int lane) const {
    const bool some = total != 0.0f;
    const float inv = some ? __frcp_rn(total) : 0.0f;
    if (lane == 0 && in_span(lse, 4, p.sp_lse, p.status)) *lse = some ? __fmaf_rn(m, p.scale, log_sum<T>(total)) : -INFINITY;
    if (!in_span(dst, D * 2, p.sp_o, p.status)) return;
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      reinterpret_cast<uint32_t*>(dst)[lane + 32 * e] = some ? pack2<T>(__fmul_rn(acc[e].x, inv), __fmul_rn(acc[e].y, inv)) : 0u;
  }
};

// The cut tiles of the forward pass over packed sequences.  FEW: tiles of
// p.few_rows rows of a key head's group * q_len.
template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(256) plan_join_forward_kernel(const __grid_constant__ AttnParams p, int ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = 1 + static_cast<int>(blockIdx.x) / kPlanJoinCtas;
  const int rows = FEW ? p.few_rows : fwd::kRows;
  grid_dependency_wait();
  const int tile = plan_cut_tile(p.plan, c, p.status);
  if (tile < 0) return;
  const PlanParts parts = plan_parts(p.plan, ctas, tile, lane, p.status);
  const int n = p.plan.head[0], head = tile / n;
  const int4 s = p.plan.items[2LL * (tile - head * n)], w = p.plan.items[2LL * (tile - head * n) + 1];
  for (int r = (static_cast<int>(blockIdx.x) % kPlanJoinCtas) * 8 + warp; r < rows; r += 8 * kPlanJoinCtas) {
    const int x = w.x + r;
    if (x >= (FEW ? s.y * p.group : s.y)) return;
    const int h = FEW ? head * p.group + x / s.y : head;
    const long long row = s.x + (FEW ? x % s.y : x);
    RowJoin<D> j;
#pragma unroll 4
    for (int i = 0; i <= parts.cuts; ++i) j.top(p, static_cast<long long>(parts.slot(i)) * rows + r);
#pragma unroll 4
    for (int i = 0; i <= parts.cuts; ++i) j.add(p, static_cast<long long>(parts.slot(i)) * rows + r, lane);
    j.template write<T>(p, p.o + row * p.o_stride + h * (D * 2), p.lse + static_cast<long long>(h) * p.seq_q + row, lane);
  }
}

// and of the backward pass, KV: of dk and dv (side by side in a slot, dv
// first), else of dq.
template <typename T, int D, bool KV>
__global__ void __launch_bounds__(256) plan_join_grad_kernel(const __grid_constant__ AttnParams p, int ctas) {
  constexpr int kRows = (KV ? 2 : 1) * kTile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = 1 + static_cast<int>(blockIdx.x) / kPlanJoinCtas;
  grid_dependency_wait();
  const int tile = plan_cut_tile(p.plan, c, p.status);
  if (tile < 0) return;
  const PlanParts parts = plan_parts(p.plan, ctas, tile, lane, p.status);
  const int n = p.plan.head[0], h = tile / n;
  const int4 s = p.plan.items[2LL * (tile - h * n)], w = p.plan.items[2LL * (tile - h * n) + 1];
  for (int r = (static_cast<int>(blockIdx.x) % kPlanJoinCtas) * 8 + warp; r < kRows; r += 8 * kPlanJoinCtas) {
    const int x = w.x + r % kTile;
    if (x >= (KV ? s.w : s.y)) continue;
    float2 acc[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i <= parts.cuts; ++i) {
      const float* src = p.part + (static_cast<long long>(parts.slot(i)) * kRows + r) * D;
      if (!in_span(src, 4 * D, p.sp_part, p.status)) continue;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) acc[e] = __fadd2_rn(acc[e], reinterpret_cast<const float2*>(src)[lane + 32 * e]);
    }
    const bool dv = KV && r < kTile;
    const float f = dv ? 1.0f : p.scale;
    const long long row = (KV ? s.z : s.x) + x;
    char* dst = KV ? (dv ? p.dv + row * p.dv_stride : p.dk + row * p.dk_stride) : p.dq + row * p.dq_stride;
    dst += h * (D * 2);
    if (!in_span(dst, D * 2, KV ? (dv ? p.sp_dv : p.sp_dk) : p.sp_dq, p.status)) continue;
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      reinterpret_cast<uint32_t*>(dst)[lane + 32 * e] = pack2<T>(__fmul_rn(acc[e].x, f), __fmul_rn(acc[e].y, f));
  }
}

// Attention beside a shared prefix: the results of one pass, all in slots.
struct PrefixSide {
  AttnPlan plan;
  const float* part;
  const float* stats;
  int few;                    // tiles of few_rows rows of a key head, else of one head's queries
  int few_rows, slot_rows;
  int ctas;
  int there;                  // the pass was made
  float scale_log2;
  int* status;
  MemSpan sp_part, sp_stats;
};

struct PrefixJoinParams {
  PrefixSide side[2];         // the prefix (all rows one sequence), the samples' own keys
  char* o;
  float* lse;
  long long o_stride;
  const int* q_lens;
  int batch, seq_q, heads_q, group;
  float scale;
  int* status;
  MemSpan sp_o, sp_lse, sp_q_lens;
};

// A warp per query and head.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixJoinParams p) {
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  grid_dependents_launch();
  if (item >= static_cast<long long>(p.batch) * p.seq_q * p.heads_q) return;
  const int row = static_cast<int>(item / p.heads_q), h = static_cast<int>(item - static_cast<long long>(row) * p.heads_q);
  const int b = row / p.seq_q, i = row - b * p.seq_q, hk = h / p.group, hh = h - hk * p.group;
  const int q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
  RowJoin<D> j;
  if (i < q_len) {
    int r[2], tile[2];
    PlanParts parts[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const PrefixSide& s = p.side[k];
      if (!s.there) continue;
      // the row's place among its sequence's
      const int at = k == 0 ? row : i, rows = k == 0 ? p.batch * p.seq_q : q_len;
      int first = 0;
      if (k == 1 && in_span(s.plan.seq_items + b, 4, s.plan.sp, p.status)) first = s.plan.seq_items[b];
      const int x = s.few ? hh * rows + at : at, of = s.few ? s.few_rows : fwd::kRows;
      tile[k] = (s.few ? hk : h) * s.plan.head[0] + first + x / of;
      r[k] = x % of;
      parts[k] = plan_parts(s.plan, s.ctas, tile[k], lane, p.status);
    }
    auto each = [&](auto f) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const PrefixSide& s = p.side[k];
        if (!s.there) continue;
#pragma unroll 4
        for (int c = 0; c <= parts[k].cuts; ++c) {
          const int slot = parts[k].cuts ? parts[k].slot(c) : 2 * s.ctas + tile[k];
          f(s, static_cast<long long>(slot) * s.slot_rows + r[k]);
        }
      }
    };
    each([&](const PrefixSide& s, long long k) { j.top(s, k); });
    each([&](const PrefixSide& s, long long k) { j.add(s, k, lane); });
  }
  j.template write<T>(p, p.o + static_cast<long long>(row) * p.o_stride + h * (D * 2),
                      p.lse + (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + i, lane);
}

}  // namespace qknr
