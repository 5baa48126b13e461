// Work lists of attention over sequences whose lengths only the device knows
// (packed sequences; samples with lengths beside a shared prefix), for sm_103a.
//
// A head's tiles, of all sequences one after the other, form a line of items;
// a call's work is that line once per head.  An item's cost is its blocks (the
// iterations of its contraction) and one unit for its epilogue.  CTAs take the
// line's tiles in waves, neighbours next to each other, so that the keys of a
// few heads at a time are read from L2 (2 x 4608 x 48 x 128, whose keys and
// values are 226 MB: 3 GB from HBM and 785 us where each CTA walks a stretch of
// the line of its own instead).  The waves end where the CTA that they gave most
// has its share of the whole; what is left of the line is dealt out so that
// all shares are equal, cut inside a tile where that is worth it, and parts of
// a tile are joined in a fixed order by a second kernel.  So a batch of one
// long and many short sequences keeps all SMs busy to the end.
//
// attn_plan_kernel works the items and the shares out, in one CTA.
#pragma once

#include "attn_kernel.cuh"

namespace qknr {

struct AttnPlanJob {
  AttnSeqs seqs;
  int ctas;
  int whole;                  // tiles are not cut if none costs more than this
  int least;                  // units of a share at least
  int max_items;
  AttnPlan plan;
};

struct AttnPlanParams {
  AttnPlanJob job[2];
  int* status;
};

constexpr int kPlanThreads = 512;
constexpr int kPlanNear = 2048;                   // items whose sums stay in shared memory

// Inclusive scan over the CTA's threads; `all`: over everybody.
template <typename V, typename OP>
__device__ __forceinline__ V plan_scan(V v, OP op, V* warps, V& all) {
  constexpr int W = kPlanThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const V o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = op(o, v);
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums for itself
  V w = warps[lane < W ? lane : W - 1];
#pragma unroll
  for (int off = 1; off < W; off <<= 1) {
    const V o = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w = op(o, w);
  }
  all = __shfl_sync(0xffffffffu, w, W - 1);
  const V before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return warp == 0 ? v : op(before, v);
}

// One CTA per job.
static __global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnPlanParams p) {
  __shared__ long long warps[32];
  __shared__ int4 seqs[kPlanThreads];             // q row, q_len, k row, k_len
  __shared__ int firsts[kPlanThreads + 1], tiles0[kPlanThreads];
  __shared__ long long near[kPlanNear + 1];       // units before each item
  const AttnPlanJob& job = p.job[blockIdx.x];
  const AttnSeqs& j = job.seqs;
  const AttnPlan& out = job.plan;
  int* iwarps = reinterpret_cast<int*>(warps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const auto add = [](auto a, auto b) { return a + b; };
  const auto most = [](int a, int b) { return a > b ? a : b; };
  grid_dependency_wait();
  grid_dependents_launch();
  // A start that falls counts as the largest before it: whatever they say, no
  // row belongs to two sequences.
  int items = 0, q_tiles = 0, q_at = 0, k_at = 0;
  if (j.q_starts) q_at = plan_start(j.q_starts, j.sp_q_starts, 0, j.seq_q, p.status);
  if (j.k_starts) k_at = plan_start(j.k_starts, j.sp_k_starts, 0, j.seq_k, p.status);
  const int k_first = k_at;
  auto range = [&](const int* starts, const MemSpan& sp, int b, bool there, int rows, int& at, int& lo, int& len) {
    const int v = there ? plan_start(starts, sp, b + 1, rows, p.status) : 0;
    int all;
    const int end = max(plan_scan<int>(v, most, iwarps, all), at);
    __syncthreads();
    firsts[tid] = end;
    __syncthreads();
    lo = tid ? firsts[tid - 1] : at;
    len = there ? end - lo : 0;
    at = max(at, all);
  };
  for (int base = 0; base < j.batch; base += kPlanThreads) {
    const int b = base + tid;
    const bool there = b < j.batch;
    int4 s = make_int4(0, 0, 0, 0);
    if (j.q_starts) {
      range(j.q_starts, j.sp_q_starts, b, there, j.seq_q, q_at, s.x, s.y);
    } else if (there) {
      s.x = b * j.seq_q;
      s.y = clamp_len(j.q_lens, b, j.seq_q, j.sp_q_lens, p.status);
    }
    if (j.k_starts) {
      range(j.k_starts, j.sp_k_starts, b, there, j.seq_k, k_at, s.z, s.w);
    } else if (there) {
      s.z = b * j.seq_k;
      s.w = clamp_len(j.k_lens, b, j.seq_k, j.sp_k_lens, p.status);
    }
    // items and query tiles, scanned together
    const long long n = there ? (plan_rows(j, s.y, s.w) + j.rows - 1) / j.rows : 0, nq = there ? (s.y + kTile - 1) / kTile : 0;
    long long all;
    const long long upto = plan_scan<long long>(n | nq << 32, add, warps, all);
    const int first = items + static_cast<int>(upto) - static_cast<int>(n);
    seqs[tid] = s;
    firsts[tid] = first;
    tiles0[tid] = q_tiles + static_cast<int>(upto >> 32) - static_cast<int>(nq);
    if (tid == kPlanThreads - 1) firsts[kPlanThreads] = items + static_cast<int>(all);
    if (there && out.seq_items && in_span(out.seq_items + b, 4, out.sp, p.status)) out.seq_items[b] = first;
    items += static_cast<int>(all);
    q_tiles += static_cast<int>(all >> 32);
    __syncthreads();
    // a warp per sequence
    for (int i = warp; i < kPlanThreads && base + i < j.batch; i += kPlanThreads / 32) {
      const int4 q = seqs[i];
      const int from = firsts[i], count = firsts[i + 1] - from;
      for (int t = lane; t < count; t += 32) {
        int4* at = out.items + 2LL * (from + t);
        const int blocks = plan_blocks(j, t, q.y, q.w);
        if (from + t >= job.max_items || !in_span(at, 32, out.sp, p.status)) continue;
        at[0] = q;
        at[1] = make_int4(t * j.rows, blocks, blocks + 1, tiles0[i]);
        if (from + t < kPlanNear) near[from + t] = blocks + 1;
      }
    }
    __syncthreads();
  }
  // where each item's units begin, and the costliest
  auto unit_of = [&](int i) -> int { return in_span(out.items + 2LL * i, 32, out.sp, p.status) ? out.items[2LL * i + 1].z : 0; };
  long long units = 0;
  int costliest = 0;
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + tid;
    const int u = i >= items ? 0 : i < kPlanNear ? static_cast<int>(near[i]) : unit_of(i);
    long long all;
    const long long upto = units + plan_scan<long long>(u, add, warps, all);   // everybody has read their `near`
    units += all;
    costliest = max(costliest, u);
    if (i < items && i < kPlanNear) near[i] = upto - u;
    if (i < items && items > kPlanNear && in_span(out.prefix + i, 8, out.sp, p.status)) out.prefix[i] = upto - u;
  }
  if (tid == 0) {
    if (items <= kPlanNear) near[items] = units;
    else if (in_span(out.prefix + items, 8, out.sp, p.status)) out.prefix[items] = units;
  }
  int top;
  plan_scan<int>(costliest, most, iwarps, top);
  __syncthreads();
  auto before = [&](int i) -> long long { return items <= kPlanNear ? near[i] : out.prefix[i]; };
  // The waves: CTA c takes tile s * ctas + c, every other wave the other way
  // round, as long as nobody has more than an equal share of the whole.
  const long long work = units * j.heads, tiles = static_cast<long long>(items) * j.heads;
  long long active = work / job.least;
  if (active > job.ctas) active = job.ctas;
  if (active < 1) active = 1;
  const int c = tid;
  long long mine = 0, share = 0;                  // what the waves give CTA c; its share of the whole
  int waves = 0;
  if (c < active) share = work / active * (c + 1) + work % active * (c + 1) / active - (work / active * c + work % active * c / active);
  if (active == job.ctas && c < job.ctas) {
    for (waves = 0; (waves + 1LL) * job.ctas <= tiles; ++waves) {
      const long long tile = static_cast<long long>(waves) * job.ctas + (waves & 1 ? job.ctas - 1 - c : c);
      const int e = static_cast<int>(tile % items);
      mine += before(e + 1) - before(e);
      if (mine > share) break;
    }
  } else {
    waves = active == job.ctas ? 0x7fffffff : 0;  // no CTA: no say
  }
  {
    int least;
    plan_scan<int>(waves, [](int a, int b) { return a < b ? a : b; }, iwarps, least);
    waves = least;
  }
  mine = 0;
  if (c < job.ctas)
    for (int s = 0; s < waves; ++s) {
      const int e = static_cast<int>((static_cast<long long>(s) * job.ctas + (s & 1 ? job.ctas - 1 - c : c)) % items);
      mine += before(e + 1) - before(e);
    }
  // Behind them: CTA c's share begins where those before it end.
  long long all;
  const long long rest = c < active ? share - mine : 0, upto = plan_scan<long long>(rest, add, warps, all);
  if (c <= job.ctas) {
    int2 at = make_int2(j.heads * items, 0);
    if (c < active && units > 0) {
      const long long tile0 = static_cast<long long>(waves) * job.ctas, h0 = tile0 / items;
      const long long x = h0 * units + before(static_cast<int>(tile0 - h0 * items)) + upto - rest;
      const int h = static_cast<int>(x / units);
      const long long off = x - h * units;
      if (h < j.heads) {
        int lo = 0, hi = items - 1;               // the last item that begins at or before `off`
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (before(mid) <= off) lo = mid;
          else hi = mid - 1;
        }
        int o = static_cast<int>(off - before(lo));
        const int u = static_cast<int>(before(lo + 1) - before(lo));
        // no cut where it saves little: within two blocks of an end, or at all
        if (top <= job.whole || o < 2 || u - o < 3) {
          lo += 2 * o >= u;
          o = 0;
        }
        at = make_int2(h * items + lo, o);
      }
    }
    if (in_span(out.spans + c, 8, out.sp, p.status)) out.spans[c] = at;
  }
  if (tid == 0 && in_span(out.head, 16, out.sp, p.status)) *out.head = make_int4(items, k_first, k_at, waves);
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

// CTAs that share a cut tile's rows.
__host__ __device__ constexpr int plan_join_ctas(bool few) { return few ? 1 : 8; }

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
  constexpr int N = plan_join_ctas(FEW);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = 1 + static_cast<int>(blockIdx.x) / N;
  const int rows = FEW ? p.few_rows : fwd::kRows;
  grid_dependency_wait();
  const int tile = plan_cut_tile(p.plan, c, p.status);
  if (tile < 0) return;
  const PlanParts parts = plan_parts(p.plan, ctas, tile, lane, p.status);
  const int n = p.plan.head->x, head = tile / n;
  const int4 s = p.plan.items[2LL * (tile - head * n)], w = p.plan.items[2LL * (tile - head * n) + 1];
  for (int r = (static_cast<int>(blockIdx.x) % N) * 8 + warp; r < rows; r += 8 * N) {
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
  constexpr int kRows = (KV ? 2 : 1) * kTile, N = plan_join_ctas(false);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = 1 + static_cast<int>(blockIdx.x) / N;
  grid_dependency_wait();
  const int tile = plan_cut_tile(p.plan, c, p.status);
  if (tile < 0) return;
  const PlanParts parts = plan_parts(p.plan, ctas, tile, lane, p.status);
  const int n = p.plan.head->x, h = tile / n;
  const int4 s = p.plan.items[2LL * (tile - h * n)], w = p.plan.items[2LL * (tile - h * n) + 1];
  for (int r = (static_cast<int>(blockIdx.x) % N) * 8 + warp; r < kRows; r += 8 * N) {
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
  int few;                    // tiles of a key head's group * q_len rows, else of one head's queries
  int rows, slot_rows;        // of a tile, of a slot
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
      const int x = s.few ? hh * rows + at : at, of = s.rows;
      tile[k] = (s.few ? hk : h) * s.plan.head->x + first + x / of;
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
