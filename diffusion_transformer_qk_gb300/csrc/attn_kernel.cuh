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
//
// PLANNED instances take their tiles from a list that the device has worked
// out (attn_plan.cuh): sequences whose lengths the host does not know, their
// rows one after the other in q and k.  PREFIX instances (forward) read the
// blocks of a prefix, the same for every sample, before a sample's own.
#pragma once

#include "attn_share.cuh"
#include "tc.cuh"

namespace qknr {

// Sequences, and what their tiles are (attn_plan.cuh).
enum { kPlanQueries, kPlanKeys, kPlanFew };       // a tile's rows: a head's queries, a key head's keys, or its group * q_len queries
struct AttnSeqs {
  int kind;
  int rows;                   // rows of a tile
  int over;                   // units of a tile beside its blocks, one each
  int heads, group, causal;   // heads: lines of tiles
  int batch, seq_q, seq_k;    // sequence b: rows b * seq .. of lens[b] (null: seq) rows,
  const int* q_lens;
  const int* k_lens;
  const int* q_starts;        // or, where these are given, rows starts[b] .. starts[b + 1] of seq rows in all
  const int* k_starts;
  MemSpan sp_q_lens, sp_k_lens, sp_q_starts, sp_k_starts;
};

// A plan in the caller's workspace.
struct AttnPlan {
  int2* head;                 // items of a head, waves
  int2* spans;                // [CTAs + 1] where each CTA's share behind the waves begins: tile of the line, unit
  int4* items;                // [items][2] q row, q_len, k row, k_len; first row in its sequence, blocks, units, query tiles before
  int2* runs;                 // [items] first and count of the items of its cost
  int* ranks;                 // [items] the place of each in the line, in the sequences' order, or null
  long long* prefix;          // [items + 1] units before, of many items
  int* seq_items;             // [batch] first item of each sequence, or null
  MemSpan sp;
};

// The same for up to 32 sequences whose tiles all go out whole, worked out by
// each CTA in its shared memory: no plan, no kernel that makes it.
constexpr int kTableSeqs = 32;
struct AttnTable {
  int4 seqs[kTableSeqs];      // q row, q_len, k row, k_len
  int first[kTableSeqs + 1];  // items before
  int before[kTableSeqs + 1]; // query tiles before; a few queries: units of a head's items before
};

// Where no plan is needed either: one sequence whose tiles all cost the same
// (kFromUniform), or samples of a fixed number of rows whose tiles all go out
// whole, each working out its own lengths (kFromSamples; a few queries).
// kFromShares: the table's sequences in equal shares, cut inside a tile (a few
// queries): 7 % less time than with a plan at 16 x 1 query over up to 4096 keys of
// 24 heads x 128, 70 us.
enum { kFromPlan, kFromTable, kFromShares, kFromUniform, kFromSamples };
struct AttnUniform {
  int tiles, units;           // of the line; of each tile
  int active;                 // CTAs that get a share (0: tiles go out whole)
  int items;                  // tiles of a head (kFromSamples: of all samples, per_sample each)
  int per_sample;
};

// The pieces of a CTA's share as the forward and dq kernels' planning warp
// hands them round: the other roles read a piece from shared memory, a few
// tiles behind, instead of each working it out from global memory where a tile
// begins and ends (2 x 4608 x 48 x 128, forward: 5 % of its time).
constexpr int kPieces = 4;
struct AttnPieces {
  int4 at[kPieces][3];
};

// its place behind a CTA's barriers, abort flag and tensor memory address
constexpr int attn_table_at(int bars) { return (8 * bars + 8 + 15) / 16 * 16; }
constexpr int attn_pieces_at(int bars) { return attn_table_at(bars) + (static_cast<int>(sizeof(AttnTable)) + 15) / 16 * 16; }

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
  float* v_norm;              // PLANNED: [heads_k][seq_k] |v| of each row, and behind them [heads_k][blocks] the longest of 32 rows
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
      sp_v, sp_dout_norm, sp_v_top, sp_v_norm, sp_ds_top;
  // PLANNED (batch is 1, seq_q and seq_k are all rows)
  AttnPlan plan;
  AttnSeqs seqs;
  int from;                   // kFrom...: where tiles come from
  AttnUniform uniform;
  int few_rows, few_group;    // a few queries: rows of a tile, warps on a tile
  int least;                  // kFromShares: units of a share at least
  int beside;                 // forward: the launch before this one waited for all before it, and writes nothing this one
                              // reads: no wait at the start, and one at the end for those who wait for this launch
  int keep;                   // every tile's result goes to a slot: those that are not cut to 2 * CTAs + tile
  int slot_rows;              // forward: rows of a slot, 128 where no sequence has more queries, else 256
  // PREFIX
  CUtensorMap map_prefix_k, map_prefix_v;
  int prefix, prefix_blocks;  // keys, blocks of 128
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
  // PLANNED, forward and dq: the consumers' side of the pieces.  One thread or
  // (whole) a warp; false at the end, and where the wait ran out (`lost`).
  __device__ __forceinline__ bool piece(int full, int pieces_at, int s, bool whole, int4 (&v)[3], bool& lost) const {
    const int i = s % kPieces;
    const uint32_t phase = static_cast<uint32_t>(s / kPieces);
    if (!(whole ? wait(full + i, phase) : wait1(full + i, phase))) {
      lost = true;
      return false;
    }
    const uint32_t at = bars + pieces_at + i * 48;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                   : "r"(at + 16 * k)
                   : "memory");
    return v[2].w != 0;
  }
  // one thread, or (whole) a warp that has read what it needs of piece s
  __device__ __forceinline__ void release(int empty, int s, bool whole) const {
    if (whole) __syncwarp();
    if (!whole || lane == 0) mbar_arrive(bar(empty + s % kPieces));
  }
  // The planning warp: piece s (valid or the end) to the others.
  __device__ __forceinline__ bool hand_round(int full, int empty, int pieces_at, int s, int4 a, int4 b, int4 d) const {
    const int i = s % kPieces;
    AttnCta patient = *this;
    patient.limit = limit >> 53 ? ~0ull : limit << 10;   // a tile may take long; who waits for its parts sets the abort flag
    if (!patient.wait(empty + i, static_cast<uint32_t>(s / kPieces) ^ 1u)) return false;
    if (lane == 0) {
      const uint32_t at = bars + pieces_at + i * 48;
      asm volatile("st.shared.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w) : "memory");
      asm volatile("st.shared.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
      asm volatile("st.shared.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(at + 32), "r"(d.x), "r"(d.y), "r"(d.z), "r"(d.w) : "memory");
      mbar_arrive(bar(full + i));
    }
    __syncwarp();
    return true;
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

// The blocks of item t of a sequence.
__device__ __forceinline__ int plan_blocks(const AttnSeqs& j, int t, int q_len, int k_len) {
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

// Starts are clamped to the rows there are.
__device__ __forceinline__ int plan_start(const int* starts, const MemSpan& sp, int b, int rows, int* status) {
  return in_span(starts + b, 4, sp, status) ? min(max(starts[b], 0), rows) : 0;
}
__device__ __forceinline__ int plan_rows(const AttnSeqs& j, int q_len, int k_len) {
  return j.kind == kPlanKeys ? k_len : j.kind == kPlanFew ? q_len * j.group : q_len;
}

// One warp.  A start that falls counts as the largest before it: whatever they
// say, no row belongs to two sequences.
__device__ __forceinline__ void plan_table(const AttnSeqs& j, AttnTable& out, int lane, int* status) {
  auto ends = [&](const int* starts, const MemSpan& sp, int rows, int& lo) {
    int v = lane < j.batch ? plan_start(starts, sp, lane + 1, rows, status) : 0;
    const int first = plan_start(starts, sp, 0, rows, status);
    v = max(v, first);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, off));   // lanes below `off`: their own
    lo = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) lo = first;
    return v;
  };
  int4 s;
  s.y = ends(j.q_starts, j.sp_q_starts, j.seq_q, s.x) - s.x;
  s.w = ends(j.k_starts, j.sp_k_starts, j.seq_k, s.z) - s.z;
  int n = lane < j.batch ? (plan_rows(j, s.y, s.w) + j.rows - 1) / j.rows : 0, q = lane < j.batch ? (s.y + kTile - 1) / kTile : 0;
  const int mine_n = n, mine_q = q;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, n, off), b = __shfl_up_sync(0xffffffffu, q, off);
    if (lane >= off) {
      n += a;
      q += b;
    }
  }
  out.seqs[lane] = s;
  out.first[lane] = n - mine_n;
  if (lane == 31) out.first[32] = n;
  if (j.kind != kPlanFew) {
    out.before[lane] = q - mine_q;
    return;
  }
  const int mine_u = mine_n * (plan_blocks(j, 0, s.y, s.w) + j.over);
  int u = mine_u;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, u, off);
    if (lane >= off) u += a;
  }
  out.before[lane] = u - mine_u;
  if (lane == 31) out.before[32] = u;
}

// The last sequence of the table that begins at or before `at` (of first or before).
__device__ __forceinline__ int table_find(const int (&from)[kTableSeqs + 1], int at) {
  int b = 0;
#pragma unroll
  for (int step = kTableSeqs / 2; step >= 1; step >>= 1)
    if (from[b + step] <= at) b += step;
  return b;
}

// kFromShares: where CTA c's share begins, (tile, unit).  Shares are equal
// stretches of the line that has a head's items in the sequences' order: keys
// of a few queries are read once, so that neighbours have nothing to share.
__device__ __forceinline__ int2 table_span(const AttnTable& table, const AttnSeqs& j, int least, int ctas, int c) {
  const int items = table.first[kTableSeqs], units = table.before[kTableSeqs];
  const long long work = static_cast<long long>(units) * j.heads;
  const int tiles = items * j.heads;
  long long active = work / least;
  if (active > ctas) active = ctas;
  if (active < 1) active = 1;
  const long long x = c < active ? work / active * c + work % active * c / active : work;
  if (x >= work) return make_int2(tiles, 0);
  const int h = static_cast<int>(x / units), off = static_cast<int>(x - static_cast<long long>(h) * units);
  const int b = table_find(table.before, off), u = plan_blocks(j, 0, table.seqs[b].y, table.seqs[b].w) + j.over;
  const int tile = h * items + table.first[b] + (off - table.before[b]) / u, o = share_cut((off - table.before[b]) % u, u, j.over);
  return o == u ? make_int2(tile + 1, 0) : make_int2(tile, o);
}

// Where CTA c's share of a uniform line begins: (tile, unit).
__device__ __forceinline__ int2 uniform_span(const AttnUniform& u, int over, int c) {
  const long long work = static_cast<long long>(u.tiles) * u.units;
  if (c >= u.active) return make_int2(u.tiles, 0);
  const long long x = work / u.active * c + work % u.active * c / u.active;
  const int tile = static_cast<int>(x / u.units), o = share_cut(static_cast<int>(x - static_cast<long long>(tile) * u.units), u.units, over);
  return o == u.units ? make_int2(tile + 1, 0) : make_int2(tile, o);
}

// (head, item) of a tile of the line: items of one cost go head by head.
__device__ __forceinline__ int2 plan_tile(const AttnPlan& plan, int heads, int tile) {
  const int2 run = plan.runs[tile / heads];
  const int x = tile - run.x * heads, h = x / run.y;
  return make_int2(h, run.x + x - h * run.y);
}

// PLANNED: piece s of a CTA's share.
struct AttnPiece {
  int h, e, u0, u1, slot;     // head line, item; units [u0, u1) of its contraction
  int q_row, q_len, k_row, k_len, t0, blocks, tiles0;
};
// `share` (kFromShares): where it begins and ends.
template <bool FORWARD>
__device__ __forceinline__ bool attn_piece(const AttnParams& p, const AttnTable& table, const int2* share, int s, AttnPiece& w) {
  const int c = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  int tile = s * ctas + (s & 1 ? ctas - 1 - c : c);
  w.u0 = 0;
  w.slot = -1;
  if (p.from == kFromTable) {
    const int n = table.first[kTableSeqs];
    if (s * ctas >= n * p.seqs.heads) return false;
    if (tile >= n * p.seqs.heads) tile = 0, w.u0 = 1;           // nothing for this CTA in the last wave
    w.h = tile / n;
    w.e = tile - w.h * n;
    const int b = table_find(table.first, w.e);
    const int4 q = table.seqs[b];
    w.q_row = q.x;
    w.q_len = q.y;
    w.k_row = q.z;
    w.k_len = q.w;
    const int t = w.e - table.first[b];
    w.t0 = t * p.seqs.rows;
    w.blocks = plan_blocks(p.seqs, t, q.y, q.w);
    w.tiles0 = table.before[b];
    w.u1 = w.blocks + p.seqs.over;
    return w.u0 == 0;
  }
  if (FORWARD && share != nullptr && p.from == kFromShares) {
    const int2 from = share[0], to = share[1];
    tile = from.x + s;
    if (tile > to.x || (tile == to.x && to.y == 0)) return false;
    const int n = table.first[kTableSeqs];
    w.h = tile / n;
    w.e = tile - w.h * n;
    const int b = table_find(table.first, w.e);
    const int4 q = table.seqs[b];
    w.q_row = q.x;
    w.q_len = q.y;
    w.k_row = q.z;
    w.k_len = q.w;
    w.t0 = (w.e - table.first[b]) * p.seqs.rows;
    w.blocks = plan_blocks(p.seqs, 0, q.y, q.w);
    w.tiles0 = 0;
    if (s == 0) w.u0 = from.y;
    w.u1 = tile == to.x ? to.y : w.blocks + p.seqs.over;
    w.slot = w.u0 > 0 ? 2 * c : tile == to.x ? 2 * c + 1 : -1;
    return w.u0 <= w.u1;
  }
  if (FORWARD && p.from >= kFromUniform) {
    const AttnUniform& u = p.uniform;
    int end = 0;              // 0: the tile's
    tile = s * ctas + c;
    if (u.active) {
      const int2 from = uniform_span(u, p.seqs.over, c), to = uniform_span(u, p.seqs.over, c + 1);
      tile = from.x + s;
      if (tile > to.x || (tile == to.x && to.y == 0)) return false;
      if (s == 0) w.u0 = from.y;
      if (tile == to.x) end = to.y;
    }
    if (tile >= u.tiles) return false;
    w.h = tile / u.items;
    w.e = tile - w.h * u.items;
    int b = 0, t = w.e;
    if (p.from == kFromSamples) {
      b = w.e / u.per_sample;
      t = w.e - b * u.per_sample;
    }
    w.q_row = b * p.seqs.seq_q;
    w.k_row = b * p.seqs.seq_k;
    w.q_len = clamp_len(p.seqs.q_lens, b, p.seqs.seq_q, p.seqs.sp_q_lens, p.status);
    w.k_len = clamp_len(p.seqs.k_lens, b, p.seqs.seq_k, p.seqs.sp_k_lens, p.status);
    w.t0 = t * p.seqs.rows;
    if (w.t0 >= plan_rows(p.seqs, w.q_len, w.k_len)) w.k_len = 0;   // a sample with fewer rows: nothing in this tile
    w.blocks = plan_blocks(p.seqs, t, w.q_len, w.k_len);
    w.tiles0 = 0;
    w.u1 = end ? end : w.blocks + p.seqs.over;
    w.slot = w.u0 > 0 ? 2 * c : end ? 2 * c + 1 : p.keep ? 2 * ctas + tile : -1;
    return w.u0 <= w.u1;
  }
  if (!in_span(p.plan.spans + c, 16, p.plan.sp, p.status)) return false;
  const int2 head = *p.plan.head;
  int u1 = 0;                 // 0: to the end
  if (s >= head.y) {
    const int2 from = p.plan.spans[c], to = p.plan.spans[c + 1];
    tile = from.x + s - head.y;
    if (tile > to.x || (tile == to.x && to.y == 0)) return false;
    if (s == head.y) w.u0 = from.y;
    if (tile == to.x) u1 = to.y;
  }
  if (tile >= head.x * p.seqs.heads || !in_span(p.plan.runs + tile / p.seqs.heads, 8, p.plan.sp, p.status)) return false;
  const int2 at = plan_tile(p.plan, p.seqs.heads, tile);
  w.h = at.x;
  w.e = at.y;
  if (!in_span(p.plan.items + 2LL * w.e, 32, p.plan.sp, p.status)) return false;
  const int4 q = p.plan.items[2LL * w.e], x = p.plan.items[2LL * w.e + 1];
  w.q_row = q.x;
  w.q_len = q.y;
  w.k_row = q.z;
  w.k_len = q.w;
  w.t0 = x.x;
  w.blocks = x.y;
  w.tiles0 = x.w;
  w.u1 = u1 ? u1 : x.z;
  w.slot = w.u0 > 0 ? 2 * c : w.u1 < x.z ? 2 * c + 1 : p.keep ? 2 * ctas + tile : -1;
  return w.u0 <= w.u1;        // a share of nothing inside a tile: an empty part, which the join counts too
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
       S_FULL = V_EMPTY + kV, P_FULL = S_FULL + 2, O_DONE = P_FULL + 2, O_FREE = O_DONE + 2, DRAIN = O_FREE + 2,
       PIECE_FULL, PIECE_EMPTY = PIECE_FULL + kPieces, BARS = PIECE_EMPTY + kPieces };
__device__ __forceinline__ int arrivals(int i, bool grouped) {
  if (i >= PIECE_EMPTY) return 10;                // the loading and the issuing warp, eight of the softmax
  return (i >= P_FULL && i < O_DONE) || (i >= O_FREE && i < DRAIN) || (grouped && i < Q_EMPTY) ? 4 : 1;
}
constexpr int kStage = kOutRows * 128;            // a warp's staged rows: 64 columns
template <int D>
constexpr int kCtl = (2 + kK + kV) * kTileBytes<D> + 8 * kStage;
template <int D>
constexpr int kSmem = kCtl<D> + 256;
constexpr int kTableAt = attn_table_at(BARS);
constexpr int kPiecesAt = attn_pieces_at(BARS);
template <int D>
constexpr int kPlannedSmem = kCtl<D> + kPiecesAt + static_cast<int>(sizeof(AttnPieces));
static_assert(8 * BARS + 8 <= 256, "shared memory behind the tiles");
// The running maximum is only raised, and the accumulator rescaled, when the
// new one is more than 2^8 above: p stays below 2^8 (2^15 with kPLift), which
// 16-bit floats and the fp32 sums hold as exactly as values below one.
constexpr float kSlack = 8.0f;

struct Seg {
  int b, h, q0, slot;
  int q_row, k_row;           // PLANNED: the sequence's first rows
  int q_len, k_len, diag;     // causal: query i sees keys up to i + diag
  int begin;                  // first key block
  int nb[2];                  // key blocks of each half
  int blocks;
};
}  // namespace fwd

// GROUPED: a tile is 256 rows of a key head's group * q_len, query x % q_len of
// head x / q_len of its group, which the threads that own them fetch; all
// results go to slots, and there is no causal mask.
template <typename T, int D, bool PLANNED = false, bool PREFIX = false, bool GROUPED = false>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_forward_kernel(const __grid_constant__ AttnParams p) {
  using namespace fwd;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ctl = smem + kCtl<D>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * BARS);
  volatile uint32_t* tmem_word = reinterpret_cast<volatile uint32_t*>(ctl + 8 * BARS + 4);
  const AttnCta c{smem, smem_addr(smem), smem_addr(ctl), abort_flag, p.status, p.wait_limit_ns,
                  __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), static_cast<int>(threadIdx.x & 31)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(c.bar(i), arrivals(i, GROUPED));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (c.warp == kAttnMmaWarp) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_word)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_word;
  if (!(PLANNED && p.beside)) grid_dependency_wait();
  grid_dependents_launch();
  AttnTable& table = *reinterpret_cast<AttnTable*>(ctl + kTableAt);
  if (PLANNED && p.from == kFromTable) {
    if (c.warp == 0) plan_table(p.seqs, table, c.lane, p.status);
    __syncthreads();
  }

  auto work_out = [&](int s, Seg& g) {
    AttnWork w;
    AttnPiece piece;
    if (PLANNED) {
      if (!attn_piece<true>(p, table, nullptr, s, piece)) return false;
      g.b = 0;
      g.h = piece.h;
      g.q0 = piece.t0;
      g.slot = piece.slot;
      g.q_row = piece.q_row;
      g.k_row = piece.k_row;
      g.q_len = GROUPED ? piece.q_len * p.group : piece.q_len;
      g.k_len = piece.k_len;
    } else {
      if (!attn_work(p, s, w)) return false;
      const AttnPlace at = attn_place(p, w.tile, p.heads_q, true);
      g.b = at.b;
      g.h = at.h;
      g.q0 = at.t * kRows;
      g.slot = w.slot;
      g.q_row = g.k_row = 0;
      g.q_len = clamp_len(p.q_lens, at.b, p.seq_q, p.sp_q_lens, p.status);
      g.k_len = clamp_len(p.k_lens, at.b, p.seq_k, p.sp_k_lens, p.status);
    }
    g.diag = g.k_len - g.q_len;
    int nb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = g.q0 + t * kTile, last = first + kTile < g.q_len ? first + kTile : g.q_len;
      int keys = first >= g.q_len ? 0 : (!GROUPED && p.causal ? last + g.diag : g.k_len);
      keys = keys < 0 ? 0 : (keys > g.k_len ? g.k_len : keys);
      nb[t] = (keys + kTile - 1) / kTile;
      if (PREFIX && first < g.q_len) nb[t] += p.prefix_blocks;
    }
    int end;
    if (PLANNED) {
      g.begin = piece.u0 < piece.blocks ? piece.u0 : piece.blocks;
      end = piece.u1 < piece.blocks ? piece.u1 : piece.blocks;
    } else {
      attn_cut(w, nb[0] > nb[1] ? nb[0] : nb[1], g.begin, end);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int last = nb[t] < end ? nb[t] : end;
      g.nb[t] = last > g.begin ? last - g.begin : 0;
    }
    g.blocks = g.nb[0] > g.nb[1] ? g.nb[0] : g.nb[1];
    return true;
  };
  // piece s; `whole`: the warp asks together
  bool lost = false;
  auto segment = [&](int s, Seg& g, bool whole) {
    if (!PLANNED) return work_out(s, g);
    int4 v[3];
    if (!c.piece(PIECE_FULL, kPiecesAt, s, whole, v, lost)) return false;
    g.b = 0;
    g.h = v[0].x;
    g.q0 = v[0].y;
    g.slot = v[0].z;
    g.begin = v[0].w;
    g.q_row = v[1].x;
    g.q_len = v[1].y;
    g.k_row = v[1].z;
    g.k_len = v[1].w;
    g.nb[0] = v[2].x;
    g.nb[1] = v[2].y;
    g.diag = g.k_len - g.q_len;
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
      for (int s = 0; ok && segment(s, g, false); ++s) {
        if (!GROUPED) {
          // the next tile's queries come from HBM: on their way while this one's keys come from L2
          Seg next;
          if (segment(s + 1, next, false))
            for (int t = 0; t < 2; ++t)
              if (next.nb[t]) tma_prefetch_tile(&p.map_q, next.q_row + next.q0 + t * kTile, next.h, next.b);
        }
        for (int t = 0; t < 2 && ok; ++t) {
          if (GROUPED || g.nb[t] == 0) continue;
          ok = c.wait1(Q_EMPTY + t, uses[t] + 1);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(Q_FULL + t), kTileBytes<D>);
          tma_load_tile(c.base + t * kTileBytes<D>, &p.map_q, g.q_row + g.q0 + t * kTile, g.h, g.b, c.bar(Q_FULL + t));
          ++uses[t];
        }
        const int hk = GROUPED ? g.h : g.h / p.group;
        for (int j = 0; ok && j < g.blocks; ++j, k.step(), v.step()) {
          const bool shared = PREFIX && g.begin + j < p.prefix_blocks;
          const int row = g.k_row + (g.begin + j - (PREFIX && !shared ? p.prefix_blocks : 0)) * kTile, kb = shared ? 0 : g.b;
          ok = c.wait1(K_EMPTY + k.s, k.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(K_FULL + k.s), kTileBytes<D>);
          tma_load_tile(sk + k.s * kTileBytes<D>, shared ? &p.map_prefix_k : &p.map_k, row, hk, kb, c.bar(K_FULL + k.s));
          ++ik;
          ok = c.wait1(V_EMPTY + v.s, v.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(V_FULL + v.s), kTileBytes<D>);
          tma_load_tile(sv + v.s * kTileBytes<D>, shared ? &p.map_prefix_v : &p.map_v, row, hk, kb, c.bar(V_FULL + v.s));
          ++iv;
        }
        if (PLANNED) c.release(PIECE_EMPTY, s, false);
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
    for (int s = 0; ok && segment(s, g, true); ++s) {
      if (PLANNED) c.release(PIECE_EMPTY, s, true);
      if (g.blocks == 0) continue;
      const int n0 = g.nb[0], n1 = g.nb[1], blocks = g.blocks;
      // the block whose V has rows past the sample's keys (past a prefix's TMA reads zeros)
      const int ragged = (PLANNED || g.k_len < p.seq_k ? g.k_len / kTile - g.begin : blocks) + (PREFIX ? p.prefix_blocks : 0);
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
            if (j >= ragged) zero_rows<D>(smem + (2 + kK + v.s) * kTileBytes<D>, g.k_len - (g.begin + j - (PREFIX ? p.prefix_blocks : 0)) * kTile, c.lane);
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
    if (!ok || lost) c.drain_mma(DRAIN);
  } else if (PLANNED && c.warp == kAttnMma2Warp) {
    Seg g;
    for (int s = 0;; ++s) {
      const bool more = work_out(s, g);
      if (!c.hand_round(PIECE_FULL, PIECE_EMPTY, kPiecesAt, s, make_int4(g.h, g.q0, g.slot, g.begin),
                        make_int4(g.q_row, g.q_len, g.k_row, g.k_len), make_int4(g.nb[0], g.nb[1], 0, more)) || !more)
        break;
    }
  } else if (c.warp < kAttnMmaWarp) {
    more_registers<kAttnWorkRegs>();
    // softmax: a thread per query
    const int t = c.warp >> 2, r = (c.warp & 3) * 32 + c.lane;
    const uint32_t lanes = static_cast<uint32_t>(c.warp & 3) << 21;
    const uint32_t ts = tmem + t * kTile + lanes, to = tmem + 2 * kTile + t * kTile + lanes;
    unsigned char* stage = smem + (2 + kK + kV) * kTileBytes<D> + c.warp * kStage;
    const float sl = p.scale_log2, slack = kSlack / sl;
    int done = 0, fetched = 0;                    // blocks, tiles' queries so far
    bool ok = true;
    Seg g;
    for (int sg = 0; ok && segment(sg, g, true); ++sg) {
      const int n = t ? g.nb[1] : g.nb[0];
      if (GROUPED && n > 0) {
        ok = c.wait(Q_EMPTY + t, ++fetched);
        if (!ok) break;
        const int x = g.q0 + t * kTile + r, q_len = g.q_len / p.group;
        const char* src = p.q_in + static_cast<long long>(g.q_row + x % q_len) * p.q_stride + (g.h * p.group + x / q_len) * (D * 2);
        unsigned char* dst = smem + t * kTileBytes<D> + r * 128;
        const bool there = x < g.q_len && in_span(src, D * 2, p.sp_q, p.status);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {         // where the swizzle puts 16-byte chunk i of the row
          const uint4 w = there ? *reinterpret_cast<const uint4*>(src + 16 * i) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + (i >> 3) * (kTile * 128) + (((i & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_async_shared();
        __syncwarp();
        if (c.lane == 0) mbar_arrive(c.bar(Q_FULL + t));
      }
      int limit, shared = 0;                      // keys from the first block on that this query sees; PREFIX: of the prefix
      {
        const int row = g.q0 + t * kTile + r;
        limit = row < g.q_len ? (!GROUPED && p.causal ? row + g.diag + 1 : g.k_len) : 0;
        limit = (limit < 0 ? 0 : (limit > g.k_len ? g.k_len : limit)) - g.begin * kTile;
        if (PREFIX) {
          limit += p.prefix_blocks * kTile;
          shared = (row < g.q_len ? p.prefix : 0) - g.begin * kTile;
        }
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
        const int seen = (PREFIX && g.begin + j < p.prefix_blocks ? shared : limit) - j * kTile;
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
          // (unrolled, it spills registers of the loop around it where a piece's numbers take some)
#pragma unroll (PLANNED ? 1 : D / 16)
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
      segment(sg, g, true);                       // again: the loop above has no registers to keep it in
      const int row = g.q0 + t * kTile + r;
      const long long at = static_cast<long long>(g.slot) * (PLANNED ? p.slot_rows : kRows) + t * kTile + r;   // a part's row
      if (g.slot >= 0) {
        // a part of the keys: unnormalised, with its maximum and sum
        if ((!PLANNED || row < g.q_len) && in_span(p.stats + 2 * at, 8, p.sp_stats, p.status))
          *reinterpret_cast<float2*>(p.stats + 2 * at) = make_float2(m, total);
      } else {
        const long long l = (static_cast<long long>(g.b) * p.heads_q + g.h) * p.seq_q + g.q_row + row;
        if (row < (PLANNED ? g.q_len : p.seq_q) && in_span(p.lse + l, 4, p.sp_lse, p.status))
          p.lse[l] = some ? __fmaf_rn(m, p.scale, log_sum<T>(total)) : -INFINITY;
      }
      // PLANNED: rows behind a sequence's last one belong to the next, so that a warp's rows go one by one where some do
      const int there = g.q_len - (row - c.lane);
      const bool rows_end = PLANNED && g.slot < 0 && there < kOutRows;
      // checked builds: the rows of a part that this warp writes (a store by TMA stays inside its map)
      const bool fits = (!PLANNED || there > 0) &&
                        __all_sync(0xffffffffu, g.slot < 0 || in_span(p.part + at * D, 4 * D, p.sp_part, p.status));
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
        if (rows_end) {
          char* dst = p.o + static_cast<long long>(g.q_row + row) * p.o_stride + g.h * (D * 2) + 64 * i;
          if (__all_sync(0xffffffffu, c.lane >= there || in_span(dst, 64, p.sp_o, p.status)))
            store_cols<T>(dst, p.o_stride, there, o, inv, some, c.lane);
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
          if (c.lane == 0 && (PLANNED || row < p.seq_q)) tma_store_box(&p.map_out, smem_addr(stage), 0, g.q_row + row, i / 2, g.h, g.b);
        }
      }
      if (PLANNED) c.release(PIECE_EMPTY, sg, true);
    }
    if (c.lane == 0) tma_store_wait();
    tc_fence_before();
  }
  __syncthreads();
  if (c.warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  if (PLANNED && p.beside) grid_dependency_wait();
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
// and share the largest b.  Packed sequences, which may be other people's, each
// have a V of their own, and take |do| V + |delta|, which is no more than b and
// holds for an o over other keys too.  At 4096 x 24 x 128 the bounds cost 20 us (4 %), at
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

// Whether the probability of the one key that a query sees (2^kP times it: `p`)
// is 1 as far as fp32 can tell: the gradient of that score is then 0, and not
// what rounding leaves of dP - delta.  Score and log-sum are good to less than
// 2^-12 up to about 1000; a lse over other calls' keys too that leaves them less
// than that of the probability leaves this key's gradient below the rounding of
// o in delta (half a step of fp16: 2^-11).
template <typename T>
__device__ __forceinline__ bool only_key(float p) {
  return fabsf(__fmaf_rn(p, grad_scale_down(GradScale<T>::kP), -1.0f)) <= 0x1p-12f;
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

constexpr int kVBlock = 32;
__host__ __device__ constexpr int v_blocks(int rows) { return rows / kVBlock + (rows % kVBlock != 0); }

// A warp: the longest of rows [first, end) of v in a key head (PLANNED).
__device__ __forceinline__ float longest_v(const AttnParams& p, int h, int first, int end, int lane) {
  const float* rows = p.v_norm + h * static_cast<long long>(p.seq_k);
  const float* blocks = p.v_norm + p.heads_k * static_cast<long long>(p.seq_k) + h * static_cast<long long>(v_blocks(p.seq_k));
  const int b0 = v_blocks(first), b1 = end / kVBlock;            // whole blocks
  auto at = [&](const float* from, int i, int to) { return i < to && in_span(from + i, 4, p.sp_v_norm, p.status) ? from[i] : 0.0f; };
  // the rows before and behind them, and up to 4096 rows' blocks, on their way together
  const float head = at(rows, first + lane, b0 < b1 ? b0 * kVBlock : end), tail = at(rows, (b0 < b1 ? b1 * kVBlock : first + 32) + lane, end);
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = at(blocks, b0 + 32 * k + lane, b1);
  float top = fmaxf(fmaxf(fmaxf(head, tail), fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
#pragma unroll 4
  for (int i = b0 + 128 + lane; i < b1; i += 32) top = fmaxf(top, at(blocks, i, b1));
  return warp_max(top);
}

// delta = rowsum(do * o), one team of D/8 lanes per row.  Bound by HBM (50 us
// for 2 x 8190 x 40 x 128, 6.7 TB/s).  Worked out inside the dq kernel instead,
// whose tiles load do anyway, each tile waits for its rows of o: the same time
// there, 150 against 145 us at 3 x 1999 x 16 on 4 heads x 64, causal.
// fp16: also |do| of each row and a bound on the rows of v (GradScale); PLANNED:
// |v| of each row, of which the dq kernel takes a sequence's.
template <typename T, int D, bool PLANNED = false>
__global__ void __launch_bounds__(256, 8) attn_delta_kernel(const __grid_constant__ AttnParams p) {
  constexpr int L = D / 8, TEAMS = 256 / L;
  const int team = threadIdx.x / L, lane = threadIdx.x % L;
  const long long items = static_cast<long long>(p.batch) * p.seq_q * p.heads_q;
  // A plan lets this pass begin once all before it has ended, and runs beside
  // it (gradients of 9215 tokens x 16 on 4 x 64, 169 us: 5 more without).
  const bool beside_plan = PLANNED && p.from == kFromPlan;
  if (!beside_plan) grid_dependency_wait();
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
  if (PLANNED && GradScale<T>::kFromData) {
    // a warp per 32 rows of a key head
    constexpr int ROWS = 32 / L;                  // of a load
    const int blocks = v_blocks(p.seq_k), wl = threadIdx.x & 31;
    for (long long u = blockIdx.x * 8LL + (threadIdx.x >> 5); u < static_cast<long long>(blocks) * p.heads_k; u += gridDim.x * 8LL) {
      const int block = static_cast<int>(u / p.heads_k), h = static_cast<int>(u - static_cast<long long>(block) * p.heads_k);
      const int row0 = block * kVBlock, there = p.seq_k - row0;
      const char* src = p.v_in + (row0 + wl / L) * p.v_stride + h * (D * 2) + lane * 16;
      float mine = 0.0f;                          // of row row0 + wl
#pragma unroll 1
      for (int i = 0; i < L; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i * ROWS + wl / L < there && in_span(src, 16, p.sp_v, p.status)) x = *reinterpret_cast<const uint4*>(src);
        src += ROWS * p.v_stride;
        float2 y[4];
        Elem<T>::unpack(x, y);
        float n = square_sum(y);
#pragma unroll
        for (int off = L / 2; off >= 1; off >>= 1) n = __fadd_rn(n, __shfl_xor_sync(0xffffffffu, n, off));
        n = __shfl_sync(0xffffffffu, n, wl % ROWS * L);
        if (wl / ROWS == i) mine = n;
      }
      mine = wl < there ? __fsqrt_rn(mine) : 0.0f;
      float* at = p.v_norm + h * static_cast<long long>(p.seq_k) + row0 + wl;
      if (wl < there && in_span(at, 4, p.sp_v_norm, p.status)) *at = mine;
      mine = warp_max(mine);
      at = p.v_norm + p.heads_k * static_cast<long long>(p.seq_k) + h * static_cast<long long>(blocks) + block;
      if (wl == 0 && in_span(at, 4, p.sp_v_norm, p.status)) *at = mine;
    }
  }
  if (beside_plan) grid_dependency_wait();        // who waits for this pass has waited for the plan
  if (!PLANNED && GradScale<T>::kFromData) {
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
       PIECE_FULL = DRAIN + 2, PIECE_EMPTY = PIECE_FULL + kPieces, BARS = PIECE_EMPTY + kPieces };
__device__ __forceinline__ int arrivals(int i) {
  if (i >= PIECE_EMPTY) return 11;                // the loading warp, two issuing ones, eight workers
  return i == Q_READY || i == S_FREE || i == DP_FREE || i == DS_FULL || i == ACC_FREE ? 8 : 1;
}
template <int D>
constexpr int kStage = kOutRows * D;              // a warp's staged rows: D / 2 columns
template <int D>
constexpr int kCtl = (1 + kK + kV) * kTileBytes<D> + 8 * kStage<D>;
template <int D>
constexpr int kSmem = kCtl<D> + 256;
constexpr int kTableAt = attn_table_at(BARS);
constexpr int kPiecesAt = attn_pieces_at(BARS);
template <int D>
constexpr int kPlannedSmem = kCtl<D> + kPiecesAt + static_cast<int>(sizeof(AttnPieces));
static_assert(8 * BARS + 8 <= 256, "shared memory behind the tiles");

struct Seg {
  int b, h, q0, slot;
  int q_row, k_row;           // PLANNED: the sequence's first rows
  int q_len, k_len, diag;
  int top;                    // the tile's place in ds_top
  float v_top;                // PLANNED, fp16: no row of the sequence's v is longer
  int begin, n;               // key blocks [begin, begin + n)
  bool opens;                 // the tile's first piece
};
}  // namespace dq

template <typename T, int D, bool PLANNED = false>
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
  AttnTable& table = *reinterpret_cast<AttnTable*>(ctl + kTableAt);
  if (PLANNED && p.from == kFromTable) {
    if (c.warp == 0) plan_table(p.seqs, table, c.lane, p.status);
    __syncthreads();
  }

  auto work_out = [&](int s, Seg& g) {
    if (PLANNED) {
      AttnPiece piece;
      if (!attn_piece<false>(p, table, nullptr, s, piece)) return false;
      g.b = 0;
      g.h = piece.h;
      g.q0 = piece.t0;
      g.slot = piece.slot;
      g.opens = piece.u0 == 0;
      g.q_row = piece.q_row;
      g.k_row = piece.k_row;
      g.q_len = piece.q_len;
      g.k_len = piece.k_len;
      g.diag = g.k_len - g.q_len;
      g.top = piece.tiles0 + piece.t0 / kTile;
      g.begin = piece.u0 < piece.blocks ? piece.u0 : piece.blocks;
      g.n = (piece.u1 < piece.blocks ? piece.u1 : piece.blocks) - g.begin;
      return true;
    }
    AttnWork w;
    if (!attn_work(p, s, w)) return false;
    const AttnPlace at = attn_place(p, w.tile, p.heads_q, true);
    g.b = at.b;
    g.h = at.h;
    g.q0 = at.t * kTile;
    g.slot = w.slot;
    g.opens = w.u0 == 0;
    g.q_row = g.k_row = 0;
    g.top = at.t;
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
  // piece s; `whole`: the warp asks together
  bool lost = false;
  auto segment = [&](int s, Seg& g, bool whole) {
    if (!PLANNED) return work_out(s, g);
    int4 v[3];
    if (!c.piece(PIECE_FULL, kPiecesAt, s, whole, v, lost)) return false;
    g.b = 0;
    g.h = v[0].x;
    g.q0 = v[0].y;
    g.slot = v[0].z;
    g.begin = v[0].w;
    g.q_row = v[1].x;
    g.q_len = v[1].y;
    g.k_row = v[1].z;
    g.k_len = v[1].w;
    g.n = v[2].x;
    g.top = v[2].y;
    g.v_top = __int_as_float(v[2].z);
    g.opens = v[2].w & 2;
    g.diag = g.k_len - g.q_len;
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
      for (int s = 0; ok && segment(s, g, false); ++s) {
        {
          // the next tile's queries come from HBM: on their way while this one's keys come from L2
          Seg next;
          // (not before the first one's loads, which would wait for a second piece)
          if ((!PLANNED || s > 0) && segment(s + 1, next, false) && next.n > 0) {
            tma_prefetch_tile(&p.map_q, next.q_row + next.q0, next.h, next.b);
            tma_prefetch_tile(&p.map_do, next.q_row + next.q0, next.h, next.b);
          }
        }
        if (PLANNED) c.release(PIECE_EMPTY, s, false);
        if (g.n == 0) continue;
        const int hk = g.h / p.group;
        for (int j = -1; j < g.n; ++j) {
          // Q, then K blocks
          ok = c.wait1(K_EMPTY + k.s, k.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(K_FULL + k.s), kTileBytes<D>);
          if (j < 0)
            tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_q, g.q_row + g.q0, g.h, g.b, c.bar(K_FULL + k.s));
          else
            tma_load_tile(sk + k.s * kTileBytes<D>, &p.map_k, g.k_row + (g.begin + j) * kTile, hk, g.b, c.bar(K_FULL + k.s));
          ++ik;
          k.step();
          if (j < 0) continue;
          if (j == 0) {
            ok = c.wait1(O_EMPTY, io + 1);
            if (!ok) break;
            mbar_arrive_expect_tx(c.bar(O_FULL), kTileBytes<D>);
            tma_load_tile(sdo, &p.map_do, g.q_row + g.q0, g.h, g.b, c.bar(O_FULL));
            ++io;
          }
          ok = c.wait1(V_EMPTY + v.s, v.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(V_FULL + v.s), kTileBytes<D>);
          tma_load_tile(sv + v.s * kTileBytes<D>, &p.map_v, g.k_row + (g.begin + j) * kTile, hk, g.b, c.bar(V_FULL + v.s));
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
    for (int s = 0; ok && segment(s, g, true); ++s) {
      if (PLANNED) c.release(PIECE_EMPTY, s, true);
      if (g.n == 0) continue;
      const int n = g.n, ragged = PLANNED || g.k_len < p.seq_k ? g.k_len / kTile - g.begin : n;
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
    if (!ok || lost) c.drain_mma(DRAIN);
  } else if (c.warp == kAttnMma2Warp) {
    // dP of each block, when the block's before has been read
    RingPos<kV> v;
    int done = 0, live = 0;
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g, true); ++s) {
      if (PLANNED) c.release(PIECE_EMPTY, s, true);
      if (g.n == 0) continue;
      const int n = g.n, ragged = PLANNED || g.k_len < p.seq_k ? g.k_len / kTile - g.begin : n;
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
    if (!ok || lost) c.drain_mma(DRAIN + 1);
  } else if (PLANNED && c.warp == kAttnRowWarp) {
    Seg g;
    for (int s = 0;; ++s) {
      const bool more = work_out(s, g);
      // (A barrier of its own for the bound, which only the workers want, is no faster.  Gradients of 9215 tokens x 16 on 4
      // x 64, 169 us: 1 % more than with one bound for all sequences.)
      float v_top = 0.0f;
      if (GradScale<T>::kFromData && more && g.n > 0)
        v_top = longest_v(p, g.h / p.group, g.k_row, g.k_row + g.k_len, c.lane);
      if (!c.hand_round(PIECE_FULL, PIECE_EMPTY, kPiecesAt, s, make_int4(g.h, g.q0, g.slot, g.begin),
                        make_int4(g.q_row, g.q_len, g.k_row, g.k_len),
                        make_int4(g.n, g.top, __float_as_int(v_top), more ? (g.opens ? 3 : 1) : 0)) || !more)
        break;
    }
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
    if (!PLANNED && GradScale<T>::kFromData) {
#pragma unroll 4
      for (int i = c.lane; i < p.v_tops; i += 32)
        if (in_span(p.v_top + i, 4, p.sp_v_top, p.status)) v_top = fmaxf(v_top, p.v_top[i]);
      v_top = warp_max(v_top);
    }
    // a tile's row: log-sum, delta and the bound on |dP - delta|
    auto row_stats = [&](const Seg& g, float& lse, float& delta, float& bound) {
      const long long at = (static_cast<long long>(g.b) * p.heads_q + g.h) * p.seq_q + g.q_row + g.q0 + r;
      lse = delta = bound = 0.0f;
      if (g.q0 + r < (PLANNED ? g.q_len : p.seq_q) && in_span(p.lse + at, 4, p.sp_lse, p.status) && in_span(p.delta + at, 4, p.sp_delta, p.status)) {
        lse = p.lse[at];
        delta = p.delta[at];
        if (GradScale<T>::kFromData && in_span(p.dout_norm + at, 4, p.sp_dout_norm, p.status))
          bound = PLANNED ? __fmaf_rn(g.v_top, p.dout_norm[at], fabsf(delta)) : __fmul_rn(2.0f * v_top, p.dout_norm[at]);
      }
    };
    unsigned char* stage = smem + (1 + kK + kV) * kTileBytes<D> + c.warp * kStage<D>;
    float lse = 0.0f, delta = 0.0f, bound = 0.0f;
    int done = 0, live = 0;                       // blocks and tiles so far
    bool ok = true;
    Seg g;
    for (int sg = 0; ok && segment(sg, g, true); ++sg) {
      const int row = g.q0 + r;
      int limit = row < g.q_len ? (p.causal ? row + g.diag + 1 : g.k_len) : 0;
      limit = limit < 0 ? 0 : (limit > g.k_len ? g.k_len : limit);
      if (!ready) row_stats(g, lse, delta, bound);
      if (GradScale<T>::kFromData && half == 0 && g.opens) {
        // for dk, dv: the largest bound of these 32 queries
        const float top = warp_max(limit > 0 ? bound : 0.0f);
        float* at = p.ds_top + ((static_cast<long long>(g.b) * p.heads_q + g.h) * p.q_tiles + g.top) * 4 + c.warp;
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
        int seen = limit - (g.begin + j) * kTile - half * 64;
        if (__any_sync(0xffffffffu, seen < 64)) {
          if (PLANNED && limit == 1 && seen == 1 && only_key<T>(s[0][0])) seen = 0;
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
        ready = segment(sg + 1, g, true) && g.n > 0;
        if (ready) {
          row_stats(g, lse, delta, bound);
          ok = copy_q();
        }
        if (!ok) break;
        segment(sg, g, true);
        ok = c.wait(DONE, live++);
        if (!ok) break;
        tc_fence_after();
      }
      const bool some = g.n > 0 && limit > 0;
      float* part = p.part + (static_cast<long long>(g.slot) * kTile + r) * D + half * (D / 2);
      // checked builds: the rows of a part that this warp writes (a store by TMA stays inside its map)
      const bool fits = __all_sync(0xffffffffu, g.slot < 0 || in_span(part, 2 * D, p.sp_part, p.status));
      // PLANNED: rows behind a sequence's last one belong to the next, so that a warp's rows go one by one where some do
      const int there = g.q_len - (row - c.lane);
      const bool rows_end = PLANNED && g.slot < 0 && there < kOutRows;
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
        if (g.slot >= 0) {
          store_part<D>(part + 32 * i, v, grad_unlift<T>(lift), some, c.lane);
        } else if (rows_end) {
          char* dst = p.dq + static_cast<long long>(g.q_row + row) * p.dq_stride + g.h * (D * 2) + half * D + 64 * i;
          if (__all_sync(0xffffffffu, c.lane >= there || in_span(dst, 64, p.sp_dq, p.status)))
            store_cols<T>(dst, p.dq_stride, there, v, p.scale * grad_unlift<T>(lift), some, c.lane);
        } else
          stage_cols<T, D / 2>(stage, 4 * i, v, p.scale * grad_unlift<T>(lift), some, c.lane);
      }
      if (g.slot < 0 && !rows_end) {
        fence_async_shared();
        __syncwarp();
        // half of the columns: the second 64 of 128, or 32 of 64
        if (c.lane == 0 && (PLANNED || row < p.seq_q))
          tma_store_box(&p.map_out, smem_addr(stage), D == 128 ? 0 : half * 32, g.q_row + row, D == 128 ? half : 0, g.h, g.b);
      }
      if (PLANNED) c.release(PIECE_EMPTY, sg, true);
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
// At head_dim 64 they do (kTurns 2): products take turns on three buffers.  S of
// block j + 1 goes where dS of j - 1 was, and dP of j + 1 where P of j was, so
// that one warp issues dV and dP, the other dK and S two blocks ahead, and the
// eight warps find each product done when they come for it (whole backward pass
// of causal 8192 x 24 x 64: 723 us with S and dP each in one buffer, 645 so).

namespace dkv {
template <int D>
constexpr int kTurns = D == 64 ? 2 : 1;           // blocks whose scores, or dP, may be there at once
template <int D>
constexpr int kQ = D == 64 ? 4 : 3;               // Q tiles in flight
template <int D>
constexpr int kO = D == 64 ? 3 : 2;               // dO tiles in flight
template <int D>
constexpr int kBars = 4 + 2 * kQ<D> + 2 * kO<D> + 4 * kTurns<D> + 8;
constexpr int kRowBytes = 2 * 2 * kTile * 4 + 16; // two buffers of (lse, delta) of a tile's queries, and their lifts
template <int D>
constexpr int kCtl = (2 + kQ<D> + kO<D>) * kTileBytes<D> + kRowBytes;
template <int D>
constexpr int kTableAt = attn_table_at(kBars<D>);
template <int D>
constexpr int kSmem = kCtl<D> + kTableAt<D>;
template <int D>
constexpr int kPlannedSmem = kSmem<D> + static_cast<int>(sizeof(AttnTable));

struct Seg {
  int b, h, k0, slot;         // h: key head
  int q_row, k_row;           // PLANNED: the sequence's first rows
  int q_len, k_len, diag;
  int top, q_tiles;           // the sample's first place in ds_top of a head, its count
  int first, end;             // query tiles [first, end) see one of these keys
  int n;                      // blocks
  int h0, t0;                 // head and query tile of the first
};
}  // namespace dkv

template <typename T, int D, bool PLANNED = false>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_dkv_kernel(const __grid_constant__ AttnParams p) {
  using namespace dkv;
  constexpr int kQ = dkv::kQ<D>, kO = dkv::kO<D>, kTurns = dkv::kTurns<D>, kTableAt = dkv::kTableAt<D>;
  enum { K_FULL = 0, K_EMPTY, V_FULL, V_EMPTY, Q_FULL, Q_EMPTY = Q_FULL + kQ, O_FULL = Q_EMPTY + kQ,
         O_EMPTY = O_FULL + kO, S_FULL = O_EMPTY + kO, P_FULL = S_FULL + kTurns, DP_FULL = P_FULL + kTurns,
         DS_FULL = DP_FULL + kTurns, ROWS = DS_FULL + kTurns, ROWS_FREE = ROWS + 2, DONE = ROWS_FREE + 2, ACC_FREE,
         DRAIN, BARS = DRAIN + 2 };
  static_assert(BARS == kBars<D>, "barriers");
  auto arrivals = [](int i) {
    if ((i >= P_FULL && i < DP_FULL) || (i >= DS_FULL && i < ROWS) || i == ACC_FREE || (i >= ROWS_FREE && i < DONE)) return 8;
    // both chains are done with a tile (of one turn), with the accumulators
    const bool tile = (i >= Q_EMPTY && i < O_FULL) || (i >= O_EMPTY && i < S_FULL);
    return (kTurns == 1 && tile) || i == DONE ? 2 : 1;
  };
  // a block's barrier of kTurns, and its phase
  auto turn = [](int first, int block) { return kTurns == 1 ? first : first + (block & 1); };
  auto lap = [](int block) { return static_cast<uint32_t>(kTurns == 1 ? block : block >> 1); };
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
  AttnTable& table = *reinterpret_cast<AttnTable*>(ctl + kTableAt);
  if (PLANNED && p.from == kFromTable) {
    if (c.warp == 0) plan_table(p.seqs, table, c.lane, p.status);
    __syncthreads();
  }
  float* rows = reinterpret_cast<float*>(smem + (2 + kQ + kO) * kTileBytes<D>);   // [2][2][128]
  float* lifts = rows + 2 * 2 * kTile;            // [2]

  auto segment = [&](int s, Seg& g) {
    AttnWork w;
    AttnPiece piece;
    if (PLANNED) {
      if (!attn_piece<false>(p, table, nullptr, s, piece)) return false;
      g.b = 0;
      g.h = piece.h;
      g.k0 = piece.t0;
      g.slot = piece.slot;
      g.q_row = piece.q_row;
      g.k_row = piece.k_row;
      g.q_len = piece.q_len;
      g.k_len = piece.k_len;
      g.top = piece.tiles0;
      g.q_tiles = (g.q_len + kTile - 1) / kTile;
    } else {
      if (!attn_work(p, s, w)) return false;
      const AttnPlace at = attn_place(p, w.tile, p.heads_k, false);
      g.b = at.b;
      g.h = at.h;
      g.k0 = at.t * kTile;
      g.slot = w.slot;
      g.q_row = g.k_row = 0;
      g.q_len = clamp_len(p.q_lens, at.b, p.seq_q, p.sp_q_lens, p.status);
      g.k_len = clamp_len(p.k_lens, at.b, p.seq_k, p.sp_k_lens, p.status);
      g.top = 0;
      g.q_tiles = p.q_tiles;
    }
    g.diag = g.k_len - g.q_len;
    g.first = 0;
    g.end = (g.q_len + kTile - 1) / kTile;
    if (p.causal && g.k0 - g.diag > 0) g.first = (g.k0 - g.diag) / kTile;
    if (g.k0 >= g.k_len || g.first > g.end) g.first = g.end;
    const int per_head = g.end - g.first;
    int begin, end;
    if (PLANNED) {
      begin = piece.u0 < piece.blocks ? piece.u0 : piece.blocks;
      end = piece.u1 < piece.blocks ? piece.u1 : piece.blocks;
    } else {
      attn_cut(w, per_head * p.group, begin, end);
    }
    g.n = end - begin;
    g.h0 = g.h * p.group + (per_head ? begin / per_head : 0);
    g.t0 = g.first + (per_head ? begin % per_head : 0);
    return true;
  };
  const uint32_t sk = c.base, sv = c.base + kTileBytes<D>, sq = c.base + 2 * kTileBytes<D>,
                 sdo = c.base + (2 + kQ) * kTileBytes<D>;
  // dV's and dK's place
  const uint32_t acc_v = tmem + (kTurns == 1 ? 2 : 3) * kTile, acc_k = acc_v + (kTurns == 1 ? kTile : D);

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
            tma_prefetch_tile(&p.map_k, next.k_row + next.k0, next.h, next.b);
            tma_prefetch_tile(&p.map_v, next.k_row + next.k0, next.h, next.b);
          }
        }
        if (g.n == 0) continue;
        ok = c.wait1(K_EMPTY, uses + 1);
        if (!ok) break;
        mbar_arrive_expect_tx(c.bar(K_FULL), kTileBytes<D>);
        tma_load_tile(sk, &p.map_k, g.k_row + g.k0, g.h, g.b, c.bar(K_FULL));
        ++uses;
        int h = g.h0, t = g.t0;
        for (int i = 0; i < g.n; ++i, q.step(), o.step()) {
          ok = c.wait1(Q_EMPTY + q.s, q.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(Q_FULL + q.s), kTileBytes<D>);
          tma_load_tile(sq + q.s * kTileBytes<D>, &p.map_q, g.q_row + t * kTile, h, g.b, c.bar(Q_FULL + q.s));
          ++iq;
          if (i == 0) {
            ok = c.wait1(V_EMPTY, uses);
            if (!ok) break;
            mbar_arrive_expect_tx(c.bar(V_FULL), kTileBytes<D>);
            tma_load_tile(sv, &p.map_v, g.k_row + g.k0, g.h, g.b, c.bar(V_FULL));
            ++vuses;
          }
          ok = c.wait1(O_EMPTY + o.s, o.phase ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(c.bar(O_FULL + o.s), kTileBytes<D>);
          tma_load_tile(sdo + o.s * kTileBytes<D>, &p.map_do, g.q_row + t * kTile, h, g.b, c.bar(O_FULL + o.s));
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
  } else if (kTurns == 2 && (c.warp == kAttnMmaWarp || c.warp == kAttnMma2Warp)) {
    // Two chains: dP(0), then per block dV += P^T dO, dP(next) in P's place;
    // S(0), S(1), then per block dK += dS^T Q, S(the one after next) in dS's
    // place.  A chain's products run in the order of their issue, so that each
    // finds its place free.  (`ahead`: the tile of the chain's next S or dP,
    // `at`: of its next sum.)
    const bool v_chain = c.warp == kAttnMmaWarp;
    const int ring = v_chain ? kO : kQ, full = v_chain ? O_FULL : Q_FULL, empty = v_chain ? O_EMPTY : Q_EMPTY;
    const uint32_t left = v_chain ? sv : sk, tiles = v_chain ? sdo : sq, acc = v_chain ? acc_v : acc_k;
    const int score_full = v_chain ? DP_FULL : S_FULL, sum_full = v_chain ? P_FULL : DS_FULL;
    const int left_full = v_chain ? V_FULL : K_FULL, left_empty = v_chain ? V_EMPTY : K_EMPTY;
    const int lead = v_chain ? 1 : 2;             // blocks from a sum to the scores that take its place
    int ahead = 0, at = 0;
    uint32_t ahead_phase = 0;
    int done = 0, scores = 0, live = 0;           // blocks, scores issued and tiles so far
    // Block j's P^T and dS^T lie in buffers 2 j and 2 j + 1 (mod 3), and the
    // chain's scores of block j + lead after them.
    int place = v_chain ? 0 : 1;                  // of the next sum
    int score_place = v_chain ? 1 : 0;            // of the next scores
    bool ok = true;
    Seg g;
    for (int s = 0; ok && segment(s, g); ++s) {
      if (g.n == 0) continue;
      const int n = g.n;
      const bool ragged = PLANNED || g.q_len < p.seq_q;
      int t = g.t0, issued = 0;                   // the query tile of the next scores; scores of this tile so far
      // the next scores' tile has landed: nothing past the sample's queries
      auto arrived = [&]() {
        if (!c.wait(full + ahead, ahead_phase)) return false;
        if (ragged && (t + 1) * kTile > g.q_len) zero_rows<D>(smem + (tiles - c.base) + ahead * kTileBytes<D>, g.q_len - t * kTile, c.lane);
        return true;
      };
      auto issue = [&]() {                        // one thread
        mma_rows<T, D>(tmem + score_place * kTile, left, tiles + ahead * kTileBytes<D>);
        mma_commit(c.bar(turn(score_full, scores)));
        if (issued + 1 == n) mma_commit(c.bar(left_empty));
      };
      auto step = [&]() {
        ++scores;
        ++issued;
        score_place = score_place == 0 ? 2 : score_place - 1;   // + 2 mod 3
        if (++ahead == ring) {
          ahead = 0;
          ahead_phase ^= 1u;
        }
        if (++t == g.end) t = g.first;
      };
      ok = c.wait(left_full, live);
      while (ok && issued < lead && issued < n) {
        ok = arrived();
        if (!ok) break;
        if (elect_one()) issue();
        __syncwarp();
        step();
      }
      for (int i = 0; ok && i < n; ++i, ++done) {
        const bool more = issued < n;
        // the accumulators have been read for the tile before
        ok = (!more || arrived()) && (i > 0 || live == 0 || c.wait(ACC_FREE, live - 1)) &&
             c.wait(turn(sum_full, done), lap(done));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_cols<T, D, true>(acc, tmem + place * kTile, tiles + at * kTileBytes<D>, i > 0);
          mma_commit(c.bar(empty + at));
          if (i + 1 == n) mma_commit(c.bar(DONE));
          if (more) issue();
        }
        __syncwarp();
        place = place == 0 ? 2 : place - 1;
        if (++at == ring) at = 0;
        if (more) step();
      }
      ++live;
    }
    if (!ok) c.drain_mma(DRAIN + (v_chain ? 0 : 1));
  } else if (kTurns == 1 && (c.warp == kAttnMmaWarp || c.warp == kAttnMma2Warp)) {
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
      const bool ragged = PLANNED || g.q_len < p.seq_q;
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
        const long long each = 4LL * p.q_tiles, n = PLANNED ? 4LL * g.q_tiles : p.group * each;
        const float* tops = p.ds_top + (static_cast<long long>(g.b) * p.heads_q + g.h * p.group) * each + 4LL * g.top;
        float bound = 0.0f;
        for (int h = 0; h < (PLANNED ? p.group : 1); ++h, tops += each)
#pragma unroll 4
          for (long long i = c.lane; i < n; i += 32)
            if (in_span(tops + i, 4, p.sp_ds_top, p.status)) bound = fmaxf(bound, tops[i]);
        lift = grad_lift<T>(warp_max(bound));
      }
      for (int i = 0; i < g.n; ++i, ++done) {
        const long long at = (static_cast<long long>(g.b) * p.heads_q + h) * p.seq_q + g.q_row + t * kTile + c.lane;
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
    int s_at = 0, dp_at = 1;                      // the block's buffers
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
        const uint32_t ts = tmem + s_at * kTile + half * 64 + lanes, tdp = tmem + dp_at * kTile + half * 64 + lanes;
        ok = c.wait(ROWS + (done & 1), done >> 1) && c.wait(turn(S_FULL, done), lap(done));
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
        c.arrive(turn(P_FULL, done));
        ok = c.wait(turn(DP_FULL, done), lap(done));
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
        // A sequence of one key: dk is 0 too.  (Of several, what rounding leaves of the ds of a query that sees the first
        // alone, 2^-20 of dP, goes into a sum with other queries'.)
        if (PLANNED && g.k_len == 1) {
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (only_key<T>(s[a][e])) s[a][e] = 0.0f;
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
        c.arrive(turn(DS_FULL, done));
        if (c.lane == 0) mbar_arrive(c.bar(ROWS_FREE + (done & 1)));
        if (kTurns == 2) {
          const int next = 3 - s_at - dp_at;
          dp_at = s_at;
          s_at = next;
        }
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
      const int rows_k = PLANNED ? g.k_len : p.seq_k;
      char* dst = half ? p.dk + (static_cast<long long>(g.b) * p.seq_k + g.k_row + key) * p.dk_stride + g.h * (D * 2)
                       : p.dv + (static_cast<long long>(g.b) * p.seq_k + g.k_row + key) * p.dv_stride + g.h * (D * 2);
      const int there = rows_k - (key - c.lane);    // rows from the warp's first on
      const bool fits =
          __all_sync(0xffffffffu, g.slot >= 0 ? in_span(part, 4 * D, p.sp_part, p.status)
                                              : key >= rows_k || in_span(dst, D * 2, half ? p.sp_dk : p.sp_dv, p.status));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float v[32];
        if (g.n > 0) {
          tmem_load32((half ? acc_k : acc_v) + 32 * i + lanes, v);
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
