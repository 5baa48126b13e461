// Work lists of attention over sequences whose lengths only the device knows
// (packed sequences; samples with lengths beside a shared prefix), for sm_103a.
//
// A head's tiles, of all sequences, are its items; an item's cost is its blocks
// (the iterations of its contraction) and some units for its beginning and end.  The
// call's tiles form a line: the costliest items first, those of one cost
// together, head by head.  CTAs take the line's tiles in waves, every other wave
// the other way round, so that neighbours read the same keys at the same time
// (2 x 4608 x 48 x 128, whose keys and values are 226 MB: 3 GB from HBM and 16 %
// more time where each CTA walks a stretch of the line of its own) and
// all get their part of the costly ones.  The waves end where a CTA would get
// more than its share of the whole; what is left of the line, its cheapest
// tiles, is dealt out so that all shares are equal, cut inside a tile where that
// is worth it, and a second kernel joins the parts of a tile in a fixed order.
// Where no tile is worth a cut, everything goes in waves.
//
// attn_plan_kernel works the items and the shares out, in one CTA.
#pragma once

#include "attn_kernel.cuh"

namespace qknr {

struct AttnPlanJob {
  AttnSeqs seqs;
  int ctas;
  int whole;                  // tiles are not cut if none costs more than this
  int cut;                    // units that cutting some costs
  int least;                  // units of a share at least
  int max_items;
  AttnPlan plan;
};

struct AttnPlanParams {
  AttnPlanJob job[2];
  int* status;
};

constexpr int kPlanThreads = 256;
constexpr int kPlanNear = 1024;                   // items that are sorted, of up to kPlanThreads sequences

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

// One CTA per job.  V: int for up to kPlanThreads sequences of up to kPlanNear
// items, all of whose units fit into it.  Others keep the sequences' order.
template <typename V>
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnPlanParams p) {
  constexpr bool kNear = sizeof(V) == 4;
  __shared__ long long warps[32];
  __shared__ int4 seqs[kPlanThreads];             // q row, q_len, k row, k_len
  __shared__ int firsts[kPlanThreads + 1], tiles0[kPlanThreads], ends[kPlanThreads];
  __shared__ __align__(16) int costs[kNear ? kPlanNear : 1];   // units of each item, in the sequences' order
  __shared__ int line[kNear ? kPlanNear + 1 : 1]; // in the line's order: units, then units before
  __shared__ int2 runs[kNear ? kPlanNear : 1];    // first and count of the items of the same cost
  const AttnPlanJob& job = p.job[blockIdx.x];
  const AttnSeqs& j = job.seqs;
  const AttnPlan& out = job.plan;
  int* iwarps = reinterpret_cast<int*>(warps);
  V* vwarps = reinterpret_cast<V*>(warps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ctas = job.ctas, H = j.heads;
  const auto add = [](auto a, auto b) { return a + b; };
  const auto most = [](int a, int b) { return a > b ? a : b; };
  grid_dependency_wait();
  grid_dependents_launch();
  // A start that falls counts as the largest before it: whatever they say, no
  // row belongs to two sequences.
  const bool same = j.q_starts && j.q_starts == j.k_starts && j.seq_q == j.seq_k;
  int items = 0, q_tiles = 0, q_at = 0, k_at = 0;
  if (j.q_starts) q_at = plan_start(j.q_starts, j.sp_q_starts, 0, j.seq_q, p.status);
  if (j.k_starts) k_at = plan_start(j.k_starts, j.sp_k_starts, 0, j.seq_k, p.status);
  auto range = [&](int v, bool there, int& at, int& lo, int& len) {
    int all;
    const int end = max(plan_scan<int>(v, most, iwarps, all), at);
    ends[tid] = end;                              // the scan before has been read: there was a barrier since
    __syncthreads();
    lo = tid ? ends[tid - 1] : at;
    len = there ? end - lo : 0;
    at = max(at, all);
  };
  auto record = [&](int i, int q, int t, int4 seq, int blocks, int2 run) {
    int4* at = out.items + 2LL * i;
    if (i >= job.max_items || !in_span(at, 32, out.sp, p.status) || !in_span(out.runs + i, 8, out.sp, p.status)) return;
    at[0] = seq;
    at[1] = make_int4(t * j.rows, blocks, blocks + j.over, tiles0[q]);
    out.runs[i] = run;
  };
  // the last sequence of the chunk that begins at or before item i
  auto sequence = [&](int i) {
    int q = 0;
#pragma unroll
    for (int step = kPlanThreads / 2; step >= 1; step >>= 1)
      if (firsts[q + step] <= i) q += step;
    return q;
  };
  int costliest = 0;
  for (int base = 0; base < j.batch; base += kPlanThreads) {
    const int b = base + tid;
    const bool there = b < j.batch;
    int4 s = make_int4(0, 0, 0, 0);
    const int vq = j.q_starts && there ? plan_start(j.q_starts, j.sp_q_starts, b + 1, j.seq_q, p.status) : 0;
    const int vk = j.k_starts && there && !same ? plan_start(j.k_starts, j.sp_k_starts, b + 1, j.seq_k, p.status) : 0;
    if (j.q_starts) {
      range(vq, there, q_at, s.x, s.y);
    } else if (there) {
      s.x = b * j.seq_q;
      s.y = clamp_len(j.q_lens, b, j.seq_q, j.sp_q_lens, p.status);
    }
    if (same) {
      s.z = s.x;
      s.w = s.y;
      k_at = q_at;
    } else if (j.k_starts) {
      range(vk, there, k_at, s.z, s.w);
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
    const int from_item = items;
    items += static_cast<int>(all);
    q_tiles += static_cast<int>(all >> 32);
    __syncthreads();
    for (int i = from_item + tid; i < items; i += kPlanThreads) {
      const int q = sequence(i), t = i - firsts[q], blocks = plan_blocks(j, t, seqs[q].y, seqs[q].w);
      costliest = max(costliest, blocks + j.over);
      if (kNear) {
        if (i < kPlanNear) costs[i] = blocks + j.over;
      } else {
        // without a causal mask a sequence's items cost the same
        record(i, q, t, seqs[q], blocks, j.causal ? make_int2(i, 1) : make_int2(firsts[q], firsts[q + 1] - firsts[q]));
        if (out.ranks && in_span(out.ranks + i, 4, out.sp, p.status)) out.ranks[i] = i;
      }
    }
    if (!kNear) __syncthreads();
  }
  if (kNear) {
    // an item's place: how many cost more, or as much and come before it
    if (items > kPlanNear) items = kPlanNear;     // the host has counted
    if (tid < 4 && items + tid < kPlanNear) costs[items + tid] = 0;
    __syncthreads();
    for (int i = tid; i < items; i += kPlanThreads) {
      const int mine = costs[i];
      int more = 0, equal = 0, before = 0;
      for (int k = 0; k < items; k += 4) {
        const int4 o = *reinterpret_cast<const int4*>(costs + k);
        more += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        const int e0 = o.x == mine, e1 = o.y == mine, e2 = o.z == mine, e3 = o.w == mine;
        equal += e0 + e1 + e2 + e3;
        before += (e0 & (k < i)) + (e1 & (k + 1 < i)) + (e2 & (k + 2 < i)) + (e3 & (k + 3 < i));
      }
      const int at = more + before, q = sequence(i);
      line[at] = mine;
      runs[at] = make_int2(more, equal);
      record(at, q, i - firsts[q], seqs[q], mine - j.over, make_int2(more, equal));
      if (out.ranks && in_span(out.ranks + i, 4, out.sp, p.status)) out.ranks[i] = at;
    }
    __syncthreads();
  }
  // where each item's units begin
  V units = 0;
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + tid;
    V u = 0, all;
    if (i < items) {
      if (kNear) u = line[i];
      else if (in_span(out.items + 2LL * i, 32, out.sp, p.status)) u = out.items[2LL * i + 1].z;
    }
    const V upto = units + plan_scan<V>(u, add, vwarps, all);   // everybody has read their `line`
    units += all;
    if (i < items) {
      if (kNear) line[i] = upto - u;
      else if (in_span(out.prefix + i, 8, out.sp, p.status)) out.prefix[i] = upto - u;
    }
  }
  if (tid == 0) {
    if (kNear) line[items] = units;
    else if (in_span(out.prefix + items, 8, out.sp, p.status)) out.prefix[items] = units;
  }
  costliest = __reduce_max_sync(0xffffffffu, costliest);
  __syncthreads();
  if (lane == 0) iwarps[warp] = costliest;
  __syncthreads();
  costliest = __reduce_max_sync(0xffffffffu, lane < kPlanThreads / 32 ? iwarps[lane] : 0);
  auto before = [&](int i) -> V { return kNear ? line[kNear ? i : 0] : static_cast<V>(out.prefix[i]); };
  auto run_of = [&](int i) { return kNear ? runs[kNear ? i : 0] : out.runs[i]; };
  const V work = units * H, tiles = static_cast<V>(items) * H;
  V active = work / job.least;
  if (active > ctas) active = ctas;
  if (active < 1) active = 1;
  const int c = tid;
  V mine = 0, share = 0;                          // what the waves give CTA c; its share of the whole
  const V each = work / active, over = work % active;
  if (c < active) share = each + (over * (c + 1) / active - over * c / active);
  // all in waves where that makes nobody later than the cuts would
  const int last = static_cast<int>((tiles + ctas - 1) / ctas);
  auto cost = [&](V tile) -> V { return before(static_cast<int>(tile / H) + 1) - before(static_cast<int>(tile / H)); };
  bool whole = costliest <= job.whole;
  int waves = whole ? last : 0;
  if (!whole && active == ctas) {
    V total = 0, last_but_one = 0;
    bool even = true;                             // nobody has more than its share
    int s = 0;
    for (; s < last; ++s) {
      const V tile = static_cast<V>(s) * ctas + (s & 1 ? ctas - 1 - c : c);
      if (c < ctas && tile < tiles) total += cost(tile);
      if (__syncthreads_or(c < ctas && total > share + job.cut)) break;
      if (even) even = !__syncthreads_or(c < ctas && total > share) && (s + 1LL) * ctas <= tiles;
      if (even) {
        last_but_one = mine;
        mine = total;
        waves = s + 1;
      }
    }
    whole = s == last;
    if (whole) waves = last;
    // what is left: no tile in more than three or so parts
    V left;
    plan_scan<V>(c < ctas ? share - mine : 0, add, vwarps, left);
    const V tile0 = static_cast<V>(waves) * ctas;
    if (!whole && waves > 0 && tile0 < tiles && 3LL * left < static_cast<long long>(cost(tile0)) * ctas) {
      mine = last_but_one;
      --waves;
    }
  }
  // Behind them: CTA c's share begins where those before it end.
  V all;
  const V rest = c < active ? share - mine : 0, upto = plan_scan<V>(rest, add, vwarps, all);
  if (c <= ctas) {
    int2 at = make_int2(static_cast<int>(tiles), 0);
    const V tile0 = static_cast<V>(waves) * ctas;
    if (c < active && !whole && tile0 < tiles) {
      const int i0 = static_cast<int>(tile0 / H), first0 = run_of(i0).x;
      const V x = before(first0) * H + (tile0 - static_cast<V>(first0) * H) * (before(i0 + 1) - before(i0)) + upto - rest;
      if (x < work) {
        int lo = 0, hi = items - 1;               // the last item whose run's units are at or before x
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (before(mid) * H <= x) lo = mid;
          else hi = mid - 1;
        }
        const int first = run_of(lo).x, u = static_cast<int>(before(lo + 1) - before(lo));
        const V off = x - before(first) * H;
        const int tile = first * H + static_cast<int>(off / u), o = share_cut(static_cast<int>(off % u), u, j.over);
        at = o == u ? make_int2(tile + 1, 0) : make_int2(tile, o);
      }
    }
    if (in_span(out.spans + c, 8, out.sp, p.status)) out.spans[c] = at;
  }
  if (tid == 0 && in_span(out.head, 8, out.sp, p.status)) *out.head = make_int2(items, waves);
}

// ---------------------------------------------------------------------------
// joining

// The parts of a tile: slots first, then every second one.
struct PlanParts {
  int c, cuts;                // the CTA that began it; how many times it was cut
  __device__ __forceinline__ int slot(int i) const { return i == 0 ? 2 * c + 1 : 2 * (c + i); }
};

// A whole warp: how the shares cut tile `tile`.  (MOST: CTAs at most.)
constexpr int kPlanMostCtas = 159;
template <typename F>
__device__ __forceinline__ PlanParts plan_parts(int ctas, int tile, int lane, F span) {
  int before = 0, cuts = 0;
#pragma unroll
  for (int i = 0; i <= kPlanMostCtas / 32; ++i) {
    const int c = 32 * i + lane;
    int2 at = make_int2(0x7fffffff, 0);
    if (c <= ctas) at = span(c);
    before += __popc(__ballot_sync(0xffffffffu, at.x < tile || (at.x == tile && at.y == 0)));
    cuts += __popc(__ballot_sync(0xffffffffu, at.x == tile && at.y > 0));
  }
  return PlanParts{before - 1, cuts};
}

__device__ __forceinline__ PlanParts plan_parts(const AttnPlan& plan, int ctas, int tile, int lane, int* status) {
  return plan_parts(ctas, tile, lane, [&](int c) {
    return in_span(plan.spans + c, 8, plan.sp, status) ? plan.spans[c] : make_int2(0x7fffffff, 0);
  });
}

// The tile that boundary c of the shares is the first to cut, or -1.
__device__ __forceinline__ int plan_cut_tile(const AttnPlan& plan, int c, int* status) {
  if (!in_span(plan.spans + c - 1, 16, plan.sp, status)) return -1;
  const int2 at = plan.spans[c], prev = plan.spans[c - 1];
  return at.y > 0 && (prev.x != at.x || prev.y == 0) ? at.x : -1;
}

// Partial results: rows of D sums and their (maximum, sum).
struct PartsView {
  const float* part;
  const float* stats;
  MemSpan sp_part, sp_stats;
};

// CTAs that share a cut tile's rows.
__host__ __device__ constexpr int plan_join_ctas(bool few) { return few ? 1 : 8; }

// o = sum_i w_i o_i / sum_i w_i l_i over the parts of one row, w_i =
// exp2((m_i - max m) scale), a warp per row.  32 parts' maxima and sums come at
// a time, a lane's each; `place(i, side)` is part i's row among `side`'s slots.
template <int D>
struct RowJoin {
  float m = -INFINITY, total = 0.0f;
  float2 acc[D / 64];
  __device__ __forceinline__ RowJoin() {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) acc[e] = make_float2(0.0f, 0.0f);
  }
  template <typename F>
  __device__ __forceinline__ void add(int n, int lane, float scale_log2, int* status, F place) {
    for (int base = 0; base < n; base += 32) {
      const PartsView* side = nullptr;
      long long k = 0;
      float2 st = make_float2(-INFINITY, 0.0f);
      if (base + lane < n) {
        k = place(base + lane, side);
        if (in_span(side->stats + 2 * k, 8, side->sp_stats, status)) st = *reinterpret_cast<const float2*>(side->stats + 2 * k);
      }
      const float top = fmaxf(m, warp_max(st.x));
      // a part that saw no key has sum 0, maximum -inf and zeros
      const float w = st.x == top ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(st.x, top), scale_log2));
      const float old = m == top ? 1.0f : exp2_approx(__fmul_rn(__fsub_rn(m, top), scale_log2));
      m = top;
      float l = __fmul_rn(w, st.y);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, off));
      total = __fmaf_rn(total, old, l);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) acc[e] = __fmul2_rn(acc[e], make_float2(old, old));
      const int count = n - base < 32 ? n - base : 32;
#pragma unroll 8
      for (int i = 0; i < count; ++i) {
        const PartsView* from = nullptr;
        const long long at = place(base + i, from);
        const float f = __shfl_sync(0xffffffffu, w, i);
        if (!in_span(from->part + at * D, 4 * D, from->sp_part, status)) continue;
        const float2* src = reinterpret_cast<const float2*>(from->part + at * D) + lane;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) acc[e] = __ffma2_rn(make_float2(f, f), src[32 * e], acc[e]);
      }
    }
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
  int head, item;
  if (FEW && p.from == kFromShares) {             // the CTA that began the tile has written it down
    item = parts.c;
    head = p.plan.items[2LL * item + 1].y;
  } else {
    const int2 at = plan_tile(p.plan, p.seqs.heads, tile);
    head = at.x;
    item = at.y;
  }
  const PartsView view{p.part, p.stats, p.sp_part, p.sp_stats};
  const int4 s = p.plan.items[2LL * item], w = p.plan.items[2LL * item + 1];
  for (int r = (static_cast<int>(blockIdx.x) % N) * 8 + warp; r < rows; r += 8 * N) {
    const int x = w.x + r;
    if (x >= (FEW ? s.y * p.group : s.y)) return;
    const int h = FEW ? head * p.group + x / s.y : head;
    const long long row = s.x + (FEW ? x % s.y : x);
    RowJoin<D> j;
    j.add(parts.cuts + 1, lane, p.scale_log2, p.status, [&](int i, const PartsView*& side) {
      side = &view;
      return static_cast<long long>(parts.slot(i)) * rows + r;
    });
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
  const int2 at = plan_tile(p.plan, p.seqs.heads, tile);
  const int h = at.x;
  const int4 s = p.plan.items[2LL * at.y], w = p.plan.items[2LL * at.y + 1];
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
  PartsView parts;
  int few;                    // tiles of a key head's group * q_len rows, else of one head's queries
  int rows, slot_rows;        // of a tile, of a slot
  int ctas, heads;            // lines of tiles
  int there;                  // the pass was made
  int from, over;             // kFrom...
  AttnUniform uniform;
};

struct PrefixJoinParams {
  PrefixSide side[2];         // the prefix (all rows one sequence), the samples' own keys
  char* o;
  float* lse;
  long long o_stride;
  const int* q_lens;
  int batch, seq_q, heads_q, group;
  float scale, scale_log2;
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
    int r[2] = {0, 0}, tile[2] = {0, 0}, n[2] = {0, 0};
    PlanParts parts[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const PrefixSide& s = p.side[k];
      if (!s.there) continue;
      // the row's place among its sequence's
      const int at = k == 0 ? row : i, rows = k == 0 ? p.batch * p.seq_q : q_len;
      const int x = s.few ? hh * rows + at : at;
      r[k] = x % s.rows;
      n[k] = 1;
      if (s.from >= kFromUniform) {
        const AttnUniform& u = s.uniform;
        tile[k] = (s.few ? hk : h) * u.items + (s.from == kFromSamples ? b * u.per_sample : 0) + x / s.rows;
        if (u.active) parts[k] = plan_parts(s.ctas, tile[k], lane, [&](int c) { return uniform_span(u, s.over, c); });
        n[k] += parts[k].cuts;
        continue;
      }
      int first = 0;
      if (k == 1 && in_span(s.plan.seq_items + b, 4, s.plan.sp, p.status)) first = s.plan.seq_items[b];
      const int e = first + x / s.rows;
      // the tile's place in the line
      const int i = in_span(s.plan.ranks + e, 4, s.plan.sp, p.status) ? s.plan.ranks[e] : 0;
      const int2 run = in_span(s.plan.runs + i, 8, s.plan.sp, p.status) ? s.plan.runs[i] : make_int2(i, 1);
      tile[k] = run.x * s.heads + (s.few ? hk : h) * run.y + i - run.x;
      parts[k] = plan_parts(s.plan, s.ctas, tile[k], lane, p.status);
      n[k] += parts[k].cuts;
    }
    // slot of part c of the first side, of the second
    const int slot0 = parts[0].cuts ? 2 * parts[0].c : 2 * p.side[0].ctas + tile[0];
    const int slot1 = parts[1].cuts ? 2 * parts[1].c : 2 * p.side[1].ctas + tile[1];
    const bool cut0 = parts[0].cuts > 0, cut1 = parts[1].cuts > 0;
    const int n0 = n[0], r0 = r[0], r1 = r[1];
    j.add(n[0] + n[1], lane, p.scale_log2, p.status, [&](int c, const PartsView*& side) {
      const bool second = c >= n0;
      const int i = second ? c - n0 : c;
      const int slot = (second ? slot1 : slot0) + ((second ? cut1 : cut0) ? (i == 0 ? 1 : 2 * i) : 0);
      side = second ? &p.side[1].parts : &p.side[0].parts;
      return static_cast<long long>(slot) * (second ? p.side[1].slot_rows : p.side[0].slot_rows) + (second ? r1 : r0);
    });
  }
  j.template write<T>(p, p.o + static_cast<long long>(row) * p.o_stride + h * (D * 2),
                      p.lse + (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + i, lane);
}

}  // namespace qknr
