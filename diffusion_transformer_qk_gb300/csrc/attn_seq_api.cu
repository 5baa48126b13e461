// C-ABI launchers of attention over packed sequences, its backward pass, and
// attention beside a shared prefix.  No allocation, no synchronisation.
#include "../../include/qknr_pack.h"
#include "../../include/qknr_prefix.h"
#include "attn_few.cuh"
#include "attn_host.cuh"
#include "attn_plan.cuh"

namespace {

using namespace qknr_attn;

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// Takes pieces off a workspace, or only measures it.
struct Space {
  char* base;
  size_t used = 0;
  template <typename V>
  V* take(size_t n) {
    V* at = reinterpret_cast<V*>(base + used);   // base is null while measuring
    used += up16(n * sizeof(V));
    return at;
  }
};

// A job's items at most: a sequence leaves one tile partly filled.
long long max_items(long long rows, long long batch, int tile) { return rows / tile + batch; }

// Where a plan is in the workspace.
qknr::AttnPlan take_plan(Space* ws, long long items, long long batch, bool seq_items) {
  qknr::AttnPlan p;
  const size_t from = ws->used;
  char* const lo = ws->base + from;
  p.head = ws->take<int2>(1);
  p.spans = ws->take<int2>(kCtas + 1);
  p.items = ws->take<int4>(2 * items);
  p.runs = ws->take<int2>(items);
  p.ranks = seq_items ? ws->take<int>(items) : nullptr;
  p.prefix = ws->take<long long>(items + 1);
  p.seq_items = seq_items ? ws->take<int>(batch) : nullptr;
  p.sp = msp(span_of(lo, 1, 0, static_cast<long long>(ws->used - from)));
  return p;
}

constexpr int kLeastUnits = 6;                    // of a share
constexpr int kLeastFew = 4;

// One kind of tile of a call.
struct Job {
  int kind, rows, heads;
  long long items;            // at most
  long long units;            // of the costliest item, at most (job_of: its blocks)
  int slot_rows;              // fp32 rows of a partial result
  bool cuts;                  // some tile may be cut
  bool keep = false;
  int from = qknr::kFromPlan; // where the CTAs have their tiles from
  qknr::AttnUniform uniform{};
  int few_group = 0;          // a few queries: warps on a tile
  long long slots() const { return keep ? 2 * kCtas + heads * items : cuts ? 2 * kCtas : 0; }
};

bool is_few(const Job& j) { return j.kind == qknr::kPlanFew && j.rows <= qknr::kFewRows; }

// What a cut costs: partial results and the kernel that joins them, about six
// blocks' time at head_dim 128 and twelve at 64, so that tiles of twice as
// many go out whole (a share is then off by one tile at most).
int whole_units(const qknr_attn_args* a, const Job& j) {
  if (is_few(j)) return j.few_group < qknr::few_warps(j.rows) ? 12 : 5;
  return a->head_dim == 128 ? 12 : 24;
}

// What a tile costs beside its blocks, in blocks: its queries' way, the epilogue.
int over_units(const qknr_attn_args* a, const Job& j) { return is_few(j) ? 4 : a->head_dim == 128 ? 2 : 3; }

Job job_of(const qknr_attn_args* a, int kind, int rows, int heads, long long of_rows, long long batch, long long units,
           int slot_rows, int few_group = 0) {
  Job j{kind, rows, heads, max_items(of_rows, batch, rows), units, slot_rows, false};
  j.few_group = few_group;
  j.units += over_units(a, j);
  j.cuts = j.units > whole_units(a, j);
  return j;
}

// A few queries a sequence: the tiles that read keys once for 16 of their rows
// (attn_api.cu).  The host knows their mean only, and one form is the whole
// call's: any mix comes out right, but the rarer kind takes its time (one causal
// sequence of 4096 beside 300 single tokens that each see 1500 keys, 24 heads x 128:
// 2066 us, in two calls 91 and 806; beside 250, now in tiles, 1023 for 91 and 694).
bool few(long long rows, long long batch) { return rows <= qknr::kFewRows * batch; }

// Warps that share a tile of a few queries: all of a CTA's where there is much
// to read.  Over a few hundred keys a tile's beginning and end take longer than
// its steps: then three (of eight: four), so that more tiles are in work at a
// time (64 samples of 512 keys of 8 heads x 128 beside their prefix of 8190: 77 us
// with twelve, 59 with three; 128 x 1 query over up to 400 keys, 32 on 8 heads: 47
// against 31; over up to 4096 keys of 24 heads twelve take a tenth less than
// three).
constexpr long long kFewGroupKeys = 768;
int few_group(int rows, long long mean_keys) { return mean_keys > kFewGroupKeys ? qknr::few_warps(rows) : rows == 8 ? 3 : 4; }

// The forward pass's tiles of `rows` query rows in `batch` sequences over up to
// `keys` keys, `mean_keys` on average.
Job forward_job(const qknr_attn_args* a, long long rows, long long batch, int keys, long long mean_keys) {
  if (few(rows, batch)) {
    const long long group = a->n_heads_q / a->n_heads_k;
    const int tile = group * rows <= 8 * batch ? 8 : 16;
    return job_of(a, qknr::kPlanFew, tile, a->n_heads_k, group * rows, batch, blocks_of(keys), tile, few_group(tile, mean_keys));
  }
  return job_of(a, qknr::kPlanQueries, qknr::fwd::kRows, a->n_heads_q, rows, batch, blocks_of(keys), qknr::fwd::kRows);
}

struct Kernels {
  const void *fwd, *few[2], *grouped, *joint, *delta, *dq, *dkv, *join_fwd, *join_few, *join_dq, *join_dkv, *join_prefix, *join_halves;
  int planned_smem, joint_smem, dq_smem, dkv_smem;
};

template <typename T, int D>
Kernels kernels() {
  return Kernels{reinterpret_cast<const void*>(qknr::attn_forward_kernel<T, D, true>),
                 {reinterpret_cast<const void*>(qknr::attn_few_kernel<T, D, 1, true>),
                  reinterpret_cast<const void*>(qknr::attn_few_kernel<T, D, 2, true>)},
                 reinterpret_cast<const void*>(qknr::attn_forward_kernel<T, D, true, false, true>),
                 reinterpret_cast<const void*>(qknr::attn_forward_kernel<T, D, false, true>),
                 reinterpret_cast<const void*>(qknr::attn_delta_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::attn_dq_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::attn_dkv_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::plan_join_forward_kernel<T, D, false>),
                 reinterpret_cast<const void*>(qknr::plan_join_forward_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::plan_join_grad_kernel<T, D, false>),
                 reinterpret_cast<const void*>(qknr::plan_join_grad_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::prefix_join_kernel<T, D>),
                 reinterpret_cast<const void*>(qknr::attn_join_forward_kernel<T, D, false>),
                 qknr::fwd::kPlannedSmem<D>, qknr::fwd::kSmem<D>, qknr::dq::kPlannedSmem<D>,
                 qknr::dkv::kPlannedSmem<D>};
}

Kernels kernels_for(const qknr_attn_args* a) {
  if (a->dtype == QKNR_BF16) return a->head_dim == 64 ? kernels<__nv_bfloat16, 64>() : kernels<__nv_bfloat16, 128>();
  return a->head_dim == 64 ? kernels<__half, 64>() : kernels<__half, 128>();
}

qknr_status launch_plan(const qknr::AttnPlanParams& pp, const Job* of, int jobs, const qknr_attn_args* a, qknr_stream_t stream) {
  static_assert(kCtas <= qknr::kPlanMostCtas && kCtas < qknr::kPlanThreads, "a thread per share");
  qknr::AttnPlanParams copy = pp;
  void* kargs[] = {&copy};
  bool narrow = true;
  for (int i = 0; i < jobs; ++i)
    narrow = narrow && pp.job[i].max_items <= qknr::kPlanNear && pp.job[i].seqs.batch <= qknr::kPlanThreads &&
             static_cast<double>(pp.job[i].max_items) * static_cast<double>(of[i].units) * pp.job[i].seqs.heads < 2e9;
  const void* fn = narrow ? reinterpret_cast<const void*>(qknr::attn_plan_kernel<int>)
                          : reinterpret_cast<const void*>(qknr::attn_plan_kernel<long long>);
  return qknr_host::launch_kernel(fn, jobs, qknr::kPlanThreads, 0,
                                  reinterpret_cast<cudaStream_t>(stream), kargs, !(a->flags & QKNR_FLAG_NO_OVERLAP),
                                  "cudaLaunchKernelExC(attention plan)");
}

void fill_job(const qknr_attn_args* a, const Job& j, const qknr::AttnPlan& plan, qknr::AttnPlanJob* out) {
  out->seqs.kind = j.kind;
  out->seqs.rows = j.rows;
  out->seqs.heads = j.heads;
  out->seqs.group = a->n_heads_q / a->n_heads_k;
  out->seqs.causal = a->causal != 0;
  out->ctas = kCtas;
  out->seqs.over = over_units(a, j);
  out->whole = whole_units(a, j);
  out->cut = whole_units(a, j) / 2;
  out->least = is_few(j) ? kLeastFew : kLeastUnits;
  out->max_items = static_cast<int>(j.items);
  out->plan = plan;
}

// Partial results' place.
void take_parts(Space* ws, const qknr_attn_args* a, const Job& j, bool stats, qknr::AttnParams* kp) {
  const size_t n = static_cast<size_t>(j.slots()) * j.slot_rows;
  kp->part = ws->take<float>(n * a->head_dim);
  kp->stats = stats ? ws->take<float>(2 * n) : nullptr;
  kp->sp_part = msp(span_of(kp->part, 1, 0, static_cast<long long>(n * a->head_dim * 4)));
  kp->sp_stats = msp(span_of(kp->stats, 1, 0, static_cast<long long>(stats ? 8 * n : 0)));
}

// The pass over q rows by k rows whose tiles are `j`'s.
qknr_status launch_forward(const qknr_attn_args* a, const Job& j, const Kernels& fn, qknr::AttnParams* kp, int dev,
                           const qknr_host::DeviceInfo& di, qknr_stream_t stream) {
  if (is_few(j))
    return launch(fn.few[j.rows / 16], kCtas, 32 * qknr::few_warps(j.rows), qknr::few_planned_smem(j.rows, a->head_dim), a, kp, dev,
                  di, stream, "cudaLaunchKernelExC(attention, few queries)");
  return launch(j.kind == qknr::kPlanFew ? fn.grouped : fn.fwd, kCtas, qknr::kAttnThreads, fn.planned_smem, a, kp, dev, di, stream, "cudaLaunchKernelExC(attention)");
}

qknr_status launch_join(const void* fn, const Job& j, const qknr_attn_args* a, qknr::AttnParams* kp, qknr_stream_t stream,
                        const char* what) {
  if (!j.cuts) return QKNR_OK;
  int ctas = kCtas;
  void* kargs[] = {kp, &ctas};
  return qknr_host::launch_kernel(fn, (kCtas - 1) * qknr::plan_join_ctas(is_few(j)), 256, 0, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
}

// ---------------------------------------------------------------------------
// packed sequences

// The call as one sample of all rows.
qknr_attn_args one_sample(const qknr_pack_args* p) {
  qknr_attn_args a;
  memset(&a, 0, sizeof(a));
  a.abi_version = p->abi_version;
  a.dtype = p->dtype;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.o = p->o;
  a.lse = p->lse;
  a.batch = 1;
  a.seq_q = p->rows_q;
  a.seq_k = p->rows_k;
  a.n_heads_q = p->n_heads_q;
  a.n_heads_k = p->n_heads_k;
  a.head_dim = p->head_dim;
  a.scale = p->scale;
  a.causal = p->causal;
  a.workspace = p->workspace;
  a.workspace_bytes = p->workspace_bytes;
  a.dev_status = p->dev_status;
  a.flags = p->flags;
  a.wait_limit_ns = p->wait_limit_ns;
  return a;
}

qknr_status check_pack(const qknr_pack_args* p, qknr_attn_args* a) {
  if (!p) return fail(QKNR_ERR_NULL, "args is NULL");
  *a = one_sample(p);
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  if (p->batch < 0) return fail(QKNR_ERR_SHAPE, "negative batch");
  // items of the smallest tiles (8 rows of a key head), for every head
  const long long rows = p->rows_q > p->rows_k ? p->rows_q : p->rows_k;
  if ((rows / 8 + p->batch + 1) * p->n_heads_q > 0x7fffffffLL || rows * (p->n_heads_q / p->n_heads_k) > 0x7fffff00LL)
    return fail(QKNR_ERR_UNSUPPORTED, "more than 2^31 tiles");
  return QKNR_OK;
}

qknr_status check_starts(const qknr_pack_args* p) {
  if ((reinterpret_cast<uintptr_t>(p->q_starts) | reinterpret_cast<uintptr_t>(p->k_starts)) & 3u)
    return fail(QKNR_ERR_ALIGN, "q_starts or k_starts not 4-byte aligned");
  if (p->batch > 0 && !p->q_starts) return fail(QKNR_ERR_NULL, "q_starts is required");
  return QKNR_OK;
}

void pack_sequences(const qknr_pack_args* p, qknr::AttnSeqs* j) {
  j->batch = p->batch;
  j->seq_q = p->rows_q;
  j->seq_k = p->rows_k;
  j->q_starts = p->q_starts;
  j->k_starts = p->k_starts ? p->k_starts : p->q_starts;
  j->sp_q_starts = msp(span_of(j->q_starts, p->batch + 1LL, 4, 4));
  j->sp_k_starts = msp(span_of(j->k_starts, p->batch + 1LL, 4, 4));
}

// Whether every CTA can work its tiles out: few sequences, whose tiles go out
// whole and are too few to be worth an order (5 x 77 tokens of 16 heads: 8 us
// against 18 with a plan).
bool table_does(const Job& j, long long batch) {
  return !j.cuts && batch <= qknr::kTableSeqs && j.heads * j.items <= 2 * kCtas;
}

// What both passes put where.
struct PackSpace {
  Job job[2];
  qknr::AttnPlan plan[2] = {};
  float *delta, *dout_norm, *v_norm, *ds_top;
  size_t delta_n, v_norm_n, ds_top_n;
};

void pack_forward_space(const qknr_pack_args* p, const qknr_attn_args* a, Space* ws, PackSpace* s, qknr::AttnParams* kp) {
  s->job[0] = forward_job(a, p->rows_q, p->batch, p->rows_k, p->batch ? p->rows_k / p->batch : 0);
  Job& j = s->job[0];
  if (table_does(j, p->batch)) {
    j.from = qknr::kFromTable;
  } else if (is_few(j) && p->batch <= qknr::kTableSeqs && static_cast<double>(j.items) * static_cast<double>(j.units) < 2e9) {
    // Its spans and cut tiles' records take a plan's place.  Equal shares cut any tile that is long enough, whatever a cut
    // costs.
    j.from = qknr::kFromShares;
    j.cuts = qknr::share_cut(2, static_cast<int>(j.units), over_units(a, j)) == 2;
  }
  if (j.from != qknr::kFromTable) s->plan[0] = take_plan(ws, j.items > kCtas ? j.items : kCtas, p->batch, false);
  take_parts(ws, a, s->job[0], true, kp);
}

void pack_backward_space(const qknr_pack_args* p, const qknr_attn_args* a, Space* ws, PackSpace* s, qknr::AttnParams kp[2]) {
  const int group = a->n_heads_q / a->n_heads_k;
  s->job[0] = job_of(a, qknr::kPlanQueries, qknr::kTile, a->n_heads_q, p->rows_q, p->batch, blocks_of(p->rows_k), qknr::kTile);
  s->job[1] = job_of(a, qknr::kPlanKeys, qknr::kTile, a->n_heads_k, p->rows_k, p->batch, blocks_of(p->rows_q) * group,
                     2 * qknr::kTile);
  const bool table = table_does(s->job[0], p->batch) && table_does(s->job[1], p->batch);
  for (int i = 0; i < 2; ++i) {
    if (table) s->job[i].from = qknr::kFromTable;
    else s->plan[i] = take_plan(ws, s->job[i].items, p->batch, false);
  }
  s->delta_n = static_cast<size_t>(a->n_heads_q) * p->rows_q;
  s->delta = ws->take<float>(s->delta_n);
  // what fp16's dS takes its powers of two from
  const bool lifts = a->dtype == QKNR_FP16;
  s->ds_top_n = lifts ? static_cast<size_t>(a->n_heads_q) * s->job[0].items * 4 : 0;
  s->dout_norm = ws->take<float>(lifts ? s->delta_n : 0);
  s->v_norm_n = lifts ? a->n_heads_k * (static_cast<size_t>(p->rows_k) + qknr::v_blocks(p->rows_k)) : 0;
  s->v_norm = ws->take<float>(s->v_norm_n);
  s->ds_top = ws->take<float>(s->ds_top_n);
  // the parts one after the other in the same place
  Space here = *ws, end = *ws;
  for (int i = 0; i < 2; ++i) {
    here.used = ws->used;
    take_parts(&here, a, s->job[i], false, &kp[i]);
    if (here.used > end.used) end.used = here.used;
  }
  ws->used = end.used;
}

// ---------------------------------------------------------------------------
// a shared prefix

qknr_attn_args one_batch(const qknr_prefix_args* p) {
  qknr_attn_args a;
  memset(&a, 0, sizeof(a));
  a.abi_version = p->abi_version;
  a.dtype = p->dtype;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.o = p->o;
  a.lse = p->lse;
  a.batch = p->batch;
  a.seq_q = p->seq_q;
  a.seq_k = p->seq_k;
  a.n_heads_q = p->n_heads_q;
  a.n_heads_k = p->n_heads_k;
  a.head_dim = p->head_dim;
  a.q_lens = p->q_lens;
  a.k_lens = p->k_lens;
  a.scale = p->scale;
  a.causal = p->causal;
  a.workspace = p->workspace;
  a.workspace_bytes = p->workspace_bytes;
  a.dev_status = p->dev_status;
  a.flags = p->flags;
  a.wait_limit_ns = p->wait_limit_ns;
  return a;
}

qknr_status check_prefix(const qknr_prefix_args* p, qknr_attn_args* a) {
  if (!p) return fail(QKNR_ERR_NULL, "args is NULL");
  *a = one_batch(p);
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  if (p->prefix < 0) return fail(QKNR_ERR_SHAPE, "negative prefix");
  const long long rows = static_cast<long long>(p->batch) * p->seq_q;
  if ((rows / 8 + p->batch + 1) * p->n_heads_q > 0x7fffffffLL || rows * (p->n_heads_q / p->n_heads_k) > 0x7fffff00LL ||
      static_cast<long long>(p->prefix) + p->seq_k > 0x7fffff00LL)
    return fail(QKNR_ERR_UNSUPPORTED, "more than 2^31 rows or tiles");
  return QKNR_OK;
}

// Tiles of 128 rows.
long long halves(long long rows) { return (rows + qknr::kTile - 1) / qknr::kTile; }

// Estimated times in microseconds, from measurements of both forms at 120
// shapes (1 to 64 samples of 1 to 600 queries beside 100 to 16000 keys).
//
// Of a block of 128 keys for `rows` queries of a head, on all SMs: 256 of them
// at a time in 1.7 (head_dim 64: 1.0); 128 or fewer, whose scores, exponentials
// and products follow each other, in 1.8 (1.5).
double block_us(const qknr_attn_args* a, long long rows) {
  const double both = a->head_dim == 128 ? 1.7 : 1.0, one = a->head_dim == 128 ? 1.8 : 1.5;
  const long long rest = rows % qknr::fwd::kRows;
  return (static_cast<double>(rows / qknr::fwd::kRows) * both + (rest == 0 ? 0.0 : rest <= qknr::kTile ? one : both)) / kCtas;
}
// Of the batch's `rows` queries through the prefix together: as a few queries,
// 16 rows of a key head at a time with the keys read for each, or in tiles.  (16
// samples of 32 heads on 8 beside 32768 keys x 128: 98 us with four passes of a few
// queries, 68 in tiles.)
double few_prefix(const qknr_attn_args* a, long long rows, int prefix) {
  if (!few(rows, 1)) return 1e30;
  const double passes = std::ceil(static_cast<double>(a->n_heads_q / a->n_heads_k * rows) / 16.0);
  return passes * prefix * 4.0 * a->head_dim * a->n_heads_k / 6.2e6;
}
double tile_prefix(const qknr_attn_args* a, long long rows, int prefix) {
  const long long group = a->n_heads_q / a->n_heads_k;
  const double by_head = block_us(a, rows) * a->n_heads_q, by_group = block_us(a, group * rows) * a->n_heads_k;
  return 8.0 + (by_head < by_group ? by_head : by_group) * static_cast<double>(blocks_of(prefix));
}

// Whether the queries of the whole batch go through the prefix together, as
// one sequence, and then through their own keys.  Otherwise each sample's
// tiles go through both, cut and joined where they are few and long.
bool together(const qknr_attn_args* a, int prefix) {
  const double D = a->head_dim, B = a->batch, heads = a->n_heads_q, byte = 1.0 / 6.2e6;
  const long long rows = static_cast<long long>(a->batch) * a->seq_q;
  const long long np = blocks_of(prefix), nk = blocks_of(a->seq_k);
  const double block = B * heads * block_us(a, a->seq_q);
  const double apart = (np + nk > 12 ? 15.0 : 8.0) + block * static_cast<double>(np + nk);
  const double passes = std::ceil(heads / a->n_heads_k * a->seq_q / 16.0);
  const double own = few(a->seq_q, 1) ? passes * B * a->seq_k * 4.0 * D * a->n_heads_k * byte
                                     : 20.0 + block * static_cast<double>(nk);   // a plan, then tiles
  const double few_p = few_prefix(a, rows, prefix), tile_p = tile_prefix(a, rows, prefix);
  // a part of a row costs some 16 bytes for each value to write and read
  const double both = 6.0 + static_cast<double>(rows) * heads * D * 16.0 * byte + (few_p < tile_p ? few_p : tile_p) + own;
  // A call outside a graph takes as long as the host needs for three launches,
  // or for one: both times count.  (33 x 1 query beside 485 keys and 18, 4 heads x
  // 64: 30 against 21 us called one by one, much the same in a graph.)
  return both + std::fmax(both, 28.0) < apart + std::fmax(apart, 20.0);
}

struct PrefixSpace {
  bool split;                 // prefix and own keys in passes of their own
  Job job[2];                 // of the prefix, of the samples' keys
  qknr::AttnPlan plan[2] = {};
  Cut cut;                    // otherwise
};

void prefix_space(const qknr_prefix_args* p, const qknr_attn_args* a, Space* ws, PrefixSpace* s, qknr::AttnParams kp[2]) {
  s->split = together(a, p->prefix);
  if (!s->split) {
    const long long own = blocks_of(a->seq_k);
    qknr_attn_args even = *a;
    // a causal mask changes little where most of a tile's keys are the prefix
    even.causal = a->causal && blocks_of(p->prefix) < own / 2;
    s->cut = cut_tiles(&even, a->seq_q, a->n_heads_q, qknr::fwd::kRows, blocks_of(p->prefix) + own, qknr::fwd::kRows, true);
    ws->take<char>(s->cut.part_bytes + s->cut.stats_bytes);
    return;
  }
  const long long rows = static_cast<long long>(a->batch) * a->seq_q;
  const long long group = a->n_heads_q / a->n_heads_k;
  if (few_prefix(a, rows, p->prefix) <= tile_prefix(a, rows, p->prefix))
    s->job[0] = forward_job(a, rows, 1, p->prefix, p->prefix);
  else
    s->job[0] = job_of(a, qknr::kPlanQueries, qknr::fwd::kRows, a->n_heads_q, rows, 1, blocks_of(p->prefix), qknr::fwd::kRows);
  // the heads of a group in one tile where that leaves fewer rows of a tile empty
  if (s->job[0].kind == qknr::kPlanQueries && halves(group * rows) < group * halves(rows))
    s->job[0] = job_of(a, qknr::kPlanFew, qknr::fwd::kRows, a->n_heads_k, group * rows, 1, blocks_of(p->prefix), qknr::fwd::kRows);
  s->job[1] = forward_job(a, rows, a->batch, a->seq_k, a->seq_k);
  for (int i = 0; i < 2; ++i) {
    Job& j = s->job[i];
    j.keep = true;
    if (!is_few(j) && (i ? a->seq_q : j.kind == qknr::kPlanFew ? group * rows : rows) <= qknr::kTile) j.slot_rows = qknr::kTile;
    if ((i ? a->seq_k : p->prefix) == 0) j.keep = j.cuts = false;   // the pass is not made
    if (i == 0) {
      j.from = qknr::kFromUniform;
      j.items = ((j.kind == qknr::kPlanFew ? group * rows : rows) + j.rows - 1) / j.rows;
      const long long tiles = j.heads * j.items, most = tiles * j.units / (is_few(j) ? kLeastFew : kLeastUnits);
      const int active = j.cuts ? static_cast<int>(most < 1 ? 1 : most < kCtas ? most : kCtas) : 0;
      j.uniform = qknr::AttnUniform{static_cast<int>(tiles), static_cast<int>(j.units), active, static_cast<int>(j.items), 0};
    } else if (is_few(j) && !j.cuts) {
      j.from = qknr::kFromSamples;
      const int each = static_cast<int>((group * a->seq_q + j.rows - 1) / j.rows);
      j.items = static_cast<long long>(each) * a->batch;
      j.uniform = qknr::AttnUniform{static_cast<int>(j.heads * j.items), 0, 0, static_cast<int>(j.items), each};
    } else {
      s->plan[i] = take_plan(ws, j.items, a->batch, true);
    }
    take_parts(ws, a, j, true, &kp[i]);
  }
}

qknr_attn_args of_rows(const qknr_attn_args& a, int rows_q, int rows_k) {
  qknr_attn_args r = a;
  r.batch = 1;
  r.seq_q = rows_q;
  r.seq_k = rows_k;
  return r;
}

}  // namespace

extern "C" {

void qknr_pack_args_init(qknr_pack_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
}

size_t qknr_pack_sizeof_args(void) { return sizeof(qknr_pack_args); }

qknr_status qknr_pack_workspace_bytes(const qknr_pack_args* p, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  qknr_attn_args a;
  const qknr_status st = check_pack(p, &a);
  if (st != QKNR_OK) return st;
  Space ws{nullptr};
  PackSpace s;
  qknr::AttnParams kp;
  pack_forward_space(p, &a, &ws, &s, &kp);
  *bytes = ws.used;
  return QKNR_OK;
}

qknr_status qknr_pack_backward_workspace_bytes(const qknr_pack_args* p, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  qknr_attn_args a;
  const qknr_status st = check_pack(p, &a);
  if (st != QKNR_OK) return st;
  Space ws{nullptr};
  PackSpace s;
  qknr::AttnParams kp[2];
  pack_backward_space(p, &a, &ws, &s, kp);
  *bytes = ws.used;
  return QKNR_OK;
}

qknr_status qknr_pack_forward(const qknr_pack_args* p, qknr_stream_t stream) {
  qknr_attn_args a;
  qknr_status st = check_pack(p, &a);
  if (st != QKNR_OK) return st;
  Rows q{"q", p->q, p->q_stride, p->rows_q, p->n_heads_q}, k{"k", p->k, p->k_stride, p->rows_k, p->n_heads_k},
      v{"v", p->v, p->v_stride, p->rows_k, p->n_heads_k}, o{"o", p->o, p->o_stride, p->rows_q, p->n_heads_q};
  for (Rows* r : {&q, &k, &v, &o})
    if ((st = check_rows(&a, r)) != QKNR_OK) return st;
  qknr::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  if ((st = common(&a, &kp)) != QKNR_OK || (st = check_starts(p)) != QKNR_OK) return st;
  if (p->batch == 0 || p->rows_q == 0) return QKNR_OK;
  if (!p->lse) return fail(QKNR_ERR_NULL, "lse is required");
  Space ws{static_cast<char*>(p->workspace)};
  PackSpace s;
  pack_forward_space(p, &a, &ws, &s, &kp);
  if ((st = check_workspace(&a, ws.used)) != QKNR_OK) return st;
  qknr::AttnPlanParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.status = p->dev_status;
  fill_job(&a, s.job[0], s.plan[0], &pp.job[0]);
  pack_sequences(p, &pp.job[0].seqs);
  const Span space = span_of(p->workspace, 1, 0, static_cast<long long>(ws.used));
  const Span lse{static_cast<uintptr_t>(kp.sp_lse.lo), static_cast<uintptr_t>(kp.sp_lse.hi)};
  st = check_overlap(&a, {&o}, {&q, &k, &v}, {lse, space},
                     {span_of(p->q_starts, p->batch + 1LL, 4, 4), span_of(p->k_starts, p->batch + 1LL, 4, 4)});
  if (st != QKNR_OK) return st;
  if (qknr_host::overlaps(lse, space)) return fail(QKNR_ERR_OVERLAP, "lse and the workspace overlap");
  kp.plan = s.plan[0];
  kp.seqs = pp.job[0].seqs;
  kp.from = s.job[0].from;
  kp.few_rows = s.job[0].rows;
  kp.few_group = s.job[0].few_group;
  kp.least = kLeastFew;
  kp.slot_rows = s.job[0].slot_rows;
  kp.q_in = static_cast<const char*>(p->q);
  kp.q_stride = q.stride * 2;
  kp.sp_q = msp(q.span);
  kp.o = static_cast<char*>(p->o);
  kp.o_stride = o.stride * 2;
  kp.sp_o = msp(o.span);

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  const bool a_few = is_few(s.job[0]);
  const int box = a_few ? qknr::few_keys(a.head_dim) : qknr::kTile;
  if ((st = make_map(&kp.map_q, &a, p->q, q.stride, p->rows_q, p->n_heads_q)) != QKNR_OK) return st;
  if ((st = make_map(&kp.map_out, &a, p->o, o.stride, p->rows_q, p->n_heads_q, qknr::kOutRows, 64)) != QKNR_OK) return st;
  if (p->rows_k > 0) {   // without keys the kernels load nothing
    if ((st = make_map(&kp.map_k, &a, p->k, k.stride, p->rows_k, p->n_heads_k, box)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_v, &a, p->v, v.stride, p->rows_k, p->n_heads_k, box)) != QKNR_OK) return st;
  }
  const Kernels fn = kernels_for(&a);
  if (kp.from == qknr::kFromPlan && (st = launch_plan(pp, s.job, 1, &a, stream)) != QKNR_OK) return st;
  if ((st = launch_forward(&a, s.job[0], fn, &kp, dev, di, stream)) != QKNR_OK) return st;
  return launch_join(a_few ? fn.join_few : fn.join_fwd, s.job[0], &a, &kp, stream, "cudaLaunchKernelExC(attention, joining)");
}

qknr_status qknr_pack_backward(const qknr_pack_args* p, qknr_stream_t stream) {
  qknr_attn_args a;
  qknr_status st = check_pack(p, &a);
  if (st != QKNR_OK) return st;
  Rows q{"q", p->q, p->q_stride, p->rows_q, p->n_heads_q}, k{"k", p->k, p->k_stride, p->rows_k, p->n_heads_k},
      v{"v", p->v, p->v_stride, p->rows_k, p->n_heads_k}, o{"o", p->o, p->o_stride, p->rows_q, p->n_heads_q},
      g{"dout", p->dout, p->dout_stride, p->rows_q, p->n_heads_q}, dq{"dq", p->dq, p->dq_stride, p->rows_q, p->n_heads_q},
      dk{"dk", p->dk, p->dk_stride, p->rows_k, p->n_heads_k}, dv{"dv", p->dv, p->dv_stride, p->rows_k, p->n_heads_k};
  for (Rows* r : {&q, &k, &v, &o, &g, &dq, &dk, &dv})
    if ((st = check_rows(&a, r)) != QKNR_OK) return st;
  qknr::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  if ((st = common(&a, &kp)) != QKNR_OK || (st = check_starts(p)) != QKNR_OK) return st;
  if (p->batch == 0 || (p->rows_q == 0 && p->rows_k == 0)) return QKNR_OK;
  if (p->rows_q > 0 && !p->lse) return fail(QKNR_ERR_NULL, "lse is required");
  Space ws{static_cast<char*>(p->workspace)};
  PackSpace s;
  qknr::AttnParams parts[2];
  memset(parts, 0, sizeof(parts));
  pack_backward_space(p, &a, &ws, &s, parts);
  if ((st = check_workspace(&a, ws.used)) != QKNR_OK) return st;
  qknr::AttnPlanParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.status = p->dev_status;
  for (int i = 0; i < 2; ++i) {
    fill_job(&a, s.job[i], s.plan[i], &pp.job[i]);
    pack_sequences(p, &pp.job[i].seqs);
  }
  const Span space = span_of(p->workspace, 1, 0, static_cast<long long>(ws.used));
  const Span lse{static_cast<uintptr_t>(kp.sp_lse.lo), static_cast<uintptr_t>(kp.sp_lse.hi)};
  st = check_overlap(&a, {&dq, &dk, &dv}, {&q, &k, &v, &o, &g}, {space},
                     {lse, span_of(p->q_starts, p->batch + 1LL, 4, 4), span_of(p->k_starts, p->batch + 1LL, 4, 4)});
  if (st != QKNR_OK) return st;
  kp.o_in = static_cast<const char*>(p->o);
  kp.dout = static_cast<const char*>(p->dout);
  kp.dq = static_cast<char*>(p->dq);
  kp.dk = static_cast<char*>(p->dk);
  kp.dv = static_cast<char*>(p->dv);
  kp.o_stride = o.stride * 2;
  kp.dout_stride = g.stride * 2;
  kp.dq_stride = dq.stride * 2;
  kp.dk_stride = dk.stride * 2;
  kp.dv_stride = dv.stride * 2;
  kp.sp_o = msp(o.span);
  kp.sp_dout = msp(g.span);
  kp.sp_dq = msp(dq.span);
  kp.sp_dk = msp(dk.span);
  kp.sp_dv = msp(dv.span);
  kp.delta = s.delta;
  kp.sp_delta = msp(span_of(s.delta, 1, 0, static_cast<long long>(s.delta_n * 4)));
  if (a.dtype == QKNR_FP16) {
    kp.v_in = static_cast<const char*>(p->v);
    kp.v_stride = v.stride * 2;
    kp.sp_v = msp(v.span);
    kp.dout_norm = s.dout_norm;
    kp.v_norm = s.v_norm;
    kp.ds_top = s.ds_top;
    kp.q_tiles = static_cast<int>(s.job[0].items);
    kp.sp_dout_norm = msp(span_of(s.dout_norm, 1, 0, static_cast<long long>(s.delta_n * 4)));
    kp.sp_v_norm = msp(span_of(s.v_norm, 1, 0, static_cast<long long>(s.v_norm_n * 4)));
    kp.sp_ds_top = msp(span_of(s.ds_top, 1, 0, static_cast<long long>(s.ds_top_n * 4)));
  }

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  // a map of no rows is never loaded from
  if (p->rows_q > 0) {
    if ((st = make_map(&kp.map_q, &a, p->q, q.stride, p->rows_q, p->n_heads_q)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_do, &a, p->dout, g.stride, p->rows_q, p->n_heads_q)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_out, &a, p->dq, dq.stride, p->rows_q, p->n_heads_q, qknr::kOutRows, a.head_dim / 2)) != QKNR_OK)
      return st;
  }
  if (p->rows_k > 0) {
    if ((st = make_map(&kp.map_k, &a, p->k, k.stride, p->rows_k, p->n_heads_k)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_v, &a, p->v, v.stride, p->rows_k, p->n_heads_k)) != QKNR_OK) return st;
  }
  const Kernels fn = kernels_for(&a);
  kp.from = s.job[0].from;
  if (kp.from == qknr::kFromPlan && (st = launch_plan(pp, s.job, 2, &a, stream)) != QKNR_OK) return st;
  auto use = [&](int i) {
    kp.plan = s.plan[i];
    kp.seqs = pp.job[i].seqs;
    kp.part = parts[i].part;
    kp.sp_part = parts[i].sp_part;
  };
  if (p->rows_q > 0) {
    const long long teams = 256 / (a.head_dim / 8);
    long long grid = (static_cast<long long>(p->rows_q) * p->n_heads_q + teams - 1) / teams;
    if (a.dtype == QKNR_FP16) {
      const long long v_grid = (static_cast<long long>(p->rows_k) * p->n_heads_k + teams - 1) / teams;
      if (v_grid > grid) grid = v_grid;
    }
    if (grid > 8LL * di.num_sms) grid = 8LL * di.num_sms;
    use(0);
    void* kargs[] = {&kp};
    st = qknr_host::launch_kernel(fn.delta, static_cast<int>(grid), 256, 0, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a.flags & QKNR_FLAG_NO_OVERLAP), "cudaLaunchKernelExC(attention delta)");
    if (st != QKNR_OK) return st;
    st = launch(fn.dq, kCtas, qknr::kAttnThreads, fn.dq_smem, &a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention dq)");
    if (st != QKNR_OK) return st;
    st = launch_join(fn.join_dq, s.job[0], &a, &kp, stream, "cudaLaunchKernelExC(attention dq, joining)");
    if (st != QKNR_OK) return st;
  }
  if (p->rows_k == 0) return QKNR_OK;
  use(1);
  st = launch(fn.dkv, kCtas, qknr::kAttnThreads, fn.dkv_smem, &a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention dk, dv)");
  if (st != QKNR_OK) return st;
  return launch_join(fn.join_dkv, s.job[1], &a, &kp, stream, "cudaLaunchKernelExC(attention dk, dv, joining)");
}

void qknr_prefix_args_init(qknr_prefix_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
}

size_t qknr_prefix_sizeof_args(void) { return sizeof(qknr_prefix_args); }

qknr_status qknr_prefix_workspace_bytes(const qknr_prefix_args* p, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  qknr_attn_args a;
  const qknr_status st = check_prefix(p, &a);
  if (st != QKNR_OK) return st;
  Space ws{nullptr};
  PrefixSpace s;
  qknr::AttnParams kp[2];
  prefix_space(p, &a, &ws, &s, kp);
  *bytes = ws.used;
  return QKNR_OK;
}

qknr_status qknr_prefix_forward(const qknr_prefix_args* p, qknr_stream_t stream) {
  qknr_attn_args a;
  qknr_status st = check_prefix(p, &a);
  if (st != QKNR_OK) return st;
  Rows q{"q", p->q, p->q_stride, p->seq_q, p->n_heads_q}, k{"k", p->k, p->k_stride, p->seq_k, p->n_heads_k},
      v{"v", p->v, p->v_stride, p->seq_k, p->n_heads_k}, o{"o", p->o, p->o_stride, p->seq_q, p->n_heads_q};
  for (Rows* r : {&q, &k, &v, &o})
    if ((st = check_rows(&a, r)) != QKNR_OK) return st;
  const qknr_attn_args shared = of_rows(a, p->batch * p->seq_q, p->prefix);   // all queries as one sample of the prefix
  Rows pk{"prefix_k", p->prefix_k, p->prefix_k_stride, p->prefix, p->n_heads_k},
      pv{"prefix_v", p->prefix_v, p->prefix_v_stride, p->prefix, p->n_heads_k};
  for (Rows* r : {&pk, &pv})
    if ((st = check_rows(&shared, r)) != QKNR_OK) return st;
  qknr::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  if ((st = common(&a, &kp)) != QKNR_OK) return st;
  if (p->batch == 0 || p->seq_q == 0) return QKNR_OK;
  if (!p->lse) return fail(QKNR_ERR_NULL, "lse is required");
  Space ws{static_cast<char*>(p->workspace)};
  PrefixSpace s;
  qknr::AttnParams parts[2];
  memset(parts, 0, sizeof(parts));
  prefix_space(p, &a, &ws, &s, parts);
  if ((st = check_workspace(&a, ws.used)) != QKNR_OK) return st;
  const Span space = span_of(ws.used ? p->workspace : nullptr, 1, 0, static_cast<long long>(ws.used));
  const Span lse{static_cast<uintptr_t>(kp.sp_lse.lo), static_cast<uintptr_t>(kp.sp_lse.hi)};
  st = check_overlap(&a, {&o}, {&q, &k, &v, &pk, &pv}, {lse, space},
                     {span_of(p->q_lens, p->batch, 4, 4), span_of(p->k_lens, p->batch, 4, 4)});
  if (st != QKNR_OK) return st;
  if (qknr_host::overlaps(lse, space)) return fail(QKNR_ERR_OVERLAP, "lse and the workspace overlap");
  kp.q_in = static_cast<const char*>(p->q);
  kp.q_stride = q.stride * 2;
  kp.sp_q = msp(q.span);
  kp.o = static_cast<char*>(p->o);
  kp.o_stride = o.stride * 2;
  kp.sp_o = msp(o.span);

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  const Kernels fn = kernels_for(&a);
  if (!s.split) {
    apply(s.cut, &kp, p->workspace);
    kp.prefix = p->prefix;
    kp.prefix_blocks = static_cast<int>(blocks_of(p->prefix));
    if ((st = make_map(&kp.map_q, &a, p->q, q.stride, p->seq_q, p->n_heads_q)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_out, &a, p->o, o.stride, p->seq_q, p->n_heads_q, qknr::kOutRows, 64)) != QKNR_OK) return st;
    if (p->seq_k > 0) {   // without keys the kernel loads nothing
      if ((st = make_map(&kp.map_k, &a, p->k, k.stride, p->seq_k, p->n_heads_k)) != QKNR_OK) return st;
      if ((st = make_map(&kp.map_v, &a, p->v, v.stride, p->seq_k, p->n_heads_k)) != QKNR_OK) return st;
    }
    if (p->prefix > 0) {
      if ((st = make_map(&kp.map_prefix_k, &shared, p->prefix_k, pk.stride, p->prefix, p->n_heads_k)) != QKNR_OK) return st;
      if ((st = make_map(&kp.map_prefix_v, &shared, p->prefix_v, pv.stride, p->prefix, p->n_heads_k)) != QKNR_OK) return st;
    }
    st = launch(fn.joint, s.cut.ctas, qknr::kAttnThreads, fn.joint_smem, &a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention)");
    if (st != QKNR_OK) return st;
    return join(fn.join_halves, s.cut, qknr::fwd::kRows, &a, &kp, stream, "cudaLaunchKernelExC(attention, joining)");
  }

  qknr::AttnPlanParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.status = p->dev_status;
  qknr::PrefixJoinParams jp;
  memset(&jp, 0, sizeof(jp));
  const qknr_attn_args sides[2] = {shared, of_rows(a, p->batch * p->seq_q, p->batch * p->seq_k)};
  qknr::AttnParams pass[2];
  for (int i = 0; i < 2; ++i) {
    const Job& j = s.job[i];
    const qknr_attn_args& side = sides[i];
    fill_job(&a, j, s.plan[i], &pp.job[i]);
    qknr::AttnSeqs& pj = pp.job[i].seqs;
    pj.batch = i ? p->batch : 1;
    pj.seq_q = i ? p->seq_q : side.seq_q;
    pj.seq_k = i ? p->seq_k : p->prefix;
    if (i) {
      pj.q_lens = p->q_lens;
      pj.k_lens = p->k_lens;
      pj.sp_q_lens = kp.sp_q_lens;
      pj.sp_k_lens = kp.sp_k_lens;
    } else {
      pj.causal = 0;
    }
    qknr::AttnParams& w = pass[i];
    w = kp;
    w.q_lens = w.k_lens = nullptr;
    w.causal = pj.causal;
    w.batch = 1;
    w.seq_q = side.seq_q;
    w.seq_k = side.seq_k;
    w.plan = s.plan[i];
    w.seqs = pj;
    w.from = j.from;
    w.uniform = j.uniform;
    w.few_rows = j.rows;
    w.few_group = j.few_group;
    w.slot_rows = j.slot_rows;
    w.keep = 1;
    // Neither pass needs the other's results: the second's CTAs begin where
    // the first's have ended (4 samples' query beside 1000 keys and 100 of their
    // own, 24 x 128: 14.1 us on the device, 19.5 where they wait; 256 beside 4096
    // and 128, 32 on 8: 75 against 84; 64 x 32 queries beside 8192: 292 against 289).
    w.beside = i == 1 && sides[0].seq_k > 0;
    w.part = parts[i].part;
    w.stats = parts[i].stats;
    w.sp_part = parts[i].sp_part;
    w.sp_stats = parts[i].sp_stats;
    const int box = is_few(j) ? qknr::few_keys(a.head_dim) : qknr::kTile;
    if ((st = make_map(&w.map_q, &side, p->q, q.stride, side.seq_q, p->n_heads_q)) != QKNR_OK) return st;
    if (side.seq_k > 0) {
      const Rows &rk = i ? k : pk, &rv = i ? v : pv;
      if ((st = make_map(&w.map_k, &side, rk.base, rk.stride, side.seq_k, p->n_heads_k, box)) != QKNR_OK) return st;
      if ((st = make_map(&w.map_v, &side, rv.base, rv.stride, side.seq_k, p->n_heads_k, box)) != QKNR_OK) return st;
    }
    qknr::PrefixSide& js = jp.side[i];
    js.plan = s.plan[i];
    js.parts = qknr::PartsView{w.part, w.stats, w.sp_part, w.sp_stats};
    js.few = j.kind == qknr::kPlanFew;
    js.rows = j.rows;
    js.slot_rows = j.slot_rows;
    js.ctas = kCtas;
    js.heads = j.heads;
    js.from = j.from;
    js.over = pj.over;
    js.uniform = j.uniform;
    js.there = side.seq_k > 0;
  }
  jp.o = kp.o;
  jp.lse = kp.lse;
  jp.o_stride = kp.o_stride;
  jp.q_lens = p->q_lens;
  jp.batch = p->batch;
  jp.seq_q = p->seq_q;
  jp.heads_q = p->n_heads_q;
  jp.group = kp.group;
  jp.scale = kp.scale;
  jp.scale_log2 = kp.scale_log2;
  jp.status = p->dev_status;
  jp.sp_o = kp.sp_o;
  jp.sp_lse = kp.sp_lse;
  jp.sp_q_lens = kp.sp_q_lens;
  // only the samples' own keys may take a plan
  pp.job[0] = pp.job[1];
  if (s.job[1].from == qknr::kFromPlan && (st = launch_plan(pp, s.job + 1, 1, &a, stream)) != QKNR_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (sides[i].seq_k > 0 && (st = launch_forward(&a, s.job[i], fn, &pass[i], dev, di, stream)) != QKNR_OK) return st;
  const long long items = static_cast<long long>(p->batch) * p->seq_q * p->n_heads_q;
  void* kargs[] = {&jp};
  return qknr_host::launch_kernel(fn.join_prefix, static_cast<int>((items + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(stream),
                                  kargs, !(a.flags & QKNR_FLAG_NO_OVERLAP), "cudaLaunchKernelExC(attention, joining)");
}

}  // extern "C"
