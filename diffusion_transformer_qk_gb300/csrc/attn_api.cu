// C-ABI launchers of attention and its backward pass: launch planning and the
// launches.  No allocation, no synchronisation.
#include "attn_few.cuh"
#include "attn_host.cuh"

namespace {

using namespace qknr_attn;

// A few queries go without the 256-row tiles, which read a key head's keys for
// each of its query heads (us at 8 x 4096 keys of 24 heads x 128, few against
// tiles: 1 query 70 / 92, 16 queries 72 / 92, 1 query of 4 heads on a key head
// 72 / 298, of 16 heads 72 / 1115).
bool few(const qknr_attn_args* a) { return a->seq_q <= qknr::kFewRows; }

// Their tiles are up to kFewRows rows of a key head.  They go round to the
// CTAs, the last ones (or all, where they are fewer) cut along the keys.  Where
// all are cut, no more CTAs take part than leaves each 256 keys (a step of its
// warps is 128 to 384); what is left after whole tiles goes to all CTAs, down
// to a few keys each.  Below 1024 keys the second launch costs more than it
// saves.
Cut cut_few(const qknr_attn_args* a) {
  Cut c;
  const long long all = static_cast<long long>(a->seq_q) * (a->n_heads_q / a->n_heads_k);
  const long long rows = all < qknr::kFewRows ? all : qknr::kFewRows;
  c.tiles = static_cast<int>((all + qknr::kFewRows - 1) / qknr::kFewRows);
  const long long total = static_cast<long long>(a->n_heads_k) * a->batch * c.tiles;
  c.total = static_cast<int>(total);
  c.ctas = kCtas;
  const long long steps = a->seq_k < 1024 ? 1 : (static_cast<long long>(a->seq_k) + 255) / 256;
  if (total * steps < c.ctas) c.ctas = total * steps > 0 ? static_cast<int>(total * steps) : 1;
  c.waves = static_cast<int>(total / c.ctas);
  c.rem = static_cast<int>(total % c.ctas);
  if (c.rem > 0 && steps == 1) {
    ++c.waves;
    c.rem = 0;
  }
  if (c.rem > 0) {
    c.part_bytes = static_cast<size_t>(2 * c.ctas) * rows * a->head_dim * 4;
    c.stats_bytes = static_cast<size_t>(2 * c.ctas) * rows * 8;
  }
  return c;
}

Cut cut_forward(const qknr_attn_args* a) {
  if (few(a)) return cut_few(a);
  return cut_tiles(a, a->seq_q, a->n_heads_q, qknr::fwd::kRows, blocks_of(a->seq_k), qknr::fwd::kRows, true);
}
Cut cut_dq(const qknr_attn_args* a) {
  return cut_tiles(a, a->seq_q, a->n_heads_q, qknr::kTile, blocks_of(a->seq_k), qknr::kTile, false);
}
Cut cut_dkv(const qknr_attn_args* a) {
  return cut_tiles(a, a->seq_k, a->n_heads_k, qknr::kTile, blocks_of(a->seq_q) * (a->n_heads_q / a->n_heads_k),
                   2 * qknr::kTile, false);
}

// CTAs of the delta kernel at most: eight on each SM.
constexpr int kDeltaCtas = 8 * kCtas;

// What fp16's dS takes its powers of two from, behind delta: |do| of each row,
// a bound on v's rows per CTA of the delta kernel, four bounds per query tile.
size_t ds_top_bytes(const qknr_attn_args* a) {
  return static_cast<size_t>(a->batch) * a->n_heads_q * blocks_of(a->seq_q) * 16;
}
size_t lift_bytes(const qknr_attn_args* a) {
  return a->dtype == QKNR_FP16 ? delta_bytes(a) + kDeltaCtas * 4 + ds_top_bytes(a) : 0;
}

size_t backward_bytes(const qknr_attn_args* a) {
  const size_t q = cut_dq(a).part_bytes, kv = cut_dkv(a).part_bytes;
  return delta_bytes(a) + lift_bytes(a) + (q > kv ? q : kv);   // the parts one after the other in the same place
}

struct Kernels {
  const void *fwd, *few[2], *delta, *dq, *dkv, *join_fwd, *join_few, *join_dq, *join_dkv;
  int fwd_smem, dq_smem, dkv_smem;
};

template <typename T, int D>
Kernels kernels() {
  return Kernels{reinterpret_cast<const void*>(qknr::attn_forward_kernel<T, D>),
                 {reinterpret_cast<const void*>(qknr::attn_few_kernel<T, D, 1>),
                  reinterpret_cast<const void*>(qknr::attn_few_kernel<T, D, 2>)},
                 reinterpret_cast<const void*>(qknr::attn_delta_kernel<T, D>),
                 reinterpret_cast<const void*>(qknr::attn_dq_kernel<T, D>),
                 reinterpret_cast<const void*>(qknr::attn_dkv_kernel<T, D>),
                 reinterpret_cast<const void*>(qknr::attn_join_forward_kernel<T, D, false>),
                 reinterpret_cast<const void*>(qknr::attn_join_forward_kernel<T, D, true>),
                 reinterpret_cast<const void*>(qknr::attn_join_grad_kernel<T, D, false>),
                 reinterpret_cast<const void*>(qknr::attn_join_grad_kernel<T, D, true>),
                 qknr::fwd::kSmem<D>, qknr::dq::kSmem<D>, qknr::dkv::kSmem<D>};
}

Kernels kernels_for(const qknr_attn_args* a) {
  if (a->dtype == QKNR_BF16) return a->head_dim == 64 ? kernels<__nv_bfloat16, 64>() : kernels<__nv_bfloat16, 128>();
  return a->head_dim == 64 ? kernels<__half, 64>() : kernels<__half, 128>();
}

}  // namespace

extern "C" {

void qknr_attn_args_init(qknr_attn_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
}

size_t qknr_attn_sizeof_args(void) { return sizeof(qknr_attn_args); }

qknr_status qknr_attn_workspace_bytes(const qknr_attn_args* a, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const Cut c = cut_forward(a);
  *bytes = c.part_bytes + c.stats_bytes;
  return QKNR_OK;
}

qknr_status qknr_attn_backward_workspace_bytes(const qknr_attn_args* a, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  *bytes = backward_bytes(a);
  return QKNR_OK;
}

qknr_status qknr_attn_forward(const qknr_attn_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  qknr::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  Rows q{"q", a->q, a->q_stride, a->seq_q, a->n_heads_q}, k{"k", a->k, a->k_stride, a->seq_k, a->n_heads_k},
      v{"v", a->v, a->v_stride, a->seq_k, a->n_heads_k}, o{"o", a->o, a->o_stride, a->seq_q, a->n_heads_q};
  for (Rows* r : {&q, &k, &v, &o})
    if ((st = check_rows(a, r)) != QKNR_OK) return st;
  if ((st = common(a, &kp)) != QKNR_OK) return st;
  if (a->batch == 0 || a->seq_q == 0) return QKNR_OK;
  if (!a->lse) return fail(QKNR_ERR_NULL, "lse is required");
  const Cut cut = cut_forward(a);
  const size_t need = cut.part_bytes + cut.stats_bytes;
  if ((st = check_workspace(a, need)) != QKNR_OK) return st;
  const Span ws = span_of(need ? a->workspace : nullptr, 1, 0, static_cast<long long>(need));
  const Span lse{static_cast<uintptr_t>(kp.sp_lse.lo), static_cast<uintptr_t>(kp.sp_lse.hi)};
  st = check_overlap(a, {&o}, {&q, &k, &v}, {lse, ws}, {span_of(a->q_lens, a->batch, 4, 4), span_of(a->k_lens, a->batch, 4, 4)});
  if (st != QKNR_OK) return st;
  if (qknr_host::overlaps(lse, ws)) return fail(QKNR_ERR_OVERLAP, "lse and the workspace overlap");
  kp.o = static_cast<char*>(a->o);
  kp.o_stride = o.stride * 2;
  kp.sp_o = msp(o.span);
  apply(cut, &kp, a->workspace);

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  const Kernels fn = kernels_for(a);
  if (few(a)) {
    kp.q_in = static_cast<const char*>(a->q);
    kp.q_stride = q.stride * 2;
    kp.sp_q = msp(q.span);
    if (a->seq_k > 0) {
      if ((st = make_map(&kp.map_k, a, a->k, k.stride, a->seq_k, a->n_heads_k, qknr::few_keys(a->head_dim))) != QKNR_OK) return st;
      if ((st = make_map(&kp.map_v, a, a->v, v.stride, a->seq_k, a->n_heads_k, qknr::few_keys(a->head_dim))) != QKNR_OK) return st;
    }
    const int rows = a->seq_q * kp.group < qknr::kFewRows ? a->seq_q * kp.group : qknr::kFewRows, most = rows <= 8 ? 8 : 16;
    st = launch(fn.few[most / 16], cut.ctas, 32 * qknr::few_warps(most), qknr::few_smem(most, a->head_dim), a, &kp, dev, di, stream,
                "cudaLaunchKernelExC(attention, few queries)");
    if (st != QKNR_OK) return st;
    return join(fn.join_few, cut, rows, a, &kp, stream, "cudaLaunchKernelExC(attention, joining)");
  }
  if ((st = make_map(&kp.map_q, a, a->q, q.stride, a->seq_q, a->n_heads_q)) != QKNR_OK) return st;
  if (a->seq_k > 0) {   // without keys the kernel loads nothing
    if ((st = make_map(&kp.map_k, a, a->k, k.stride, a->seq_k, a->n_heads_k)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_v, a, a->v, v.stride, a->seq_k, a->n_heads_k)) != QKNR_OK) return st;
  }
  if ((st = make_map(&kp.map_out, a, a->o, o.stride, a->seq_q, a->n_heads_q, qknr::kOutRows, 64)) != QKNR_OK) return st;
  st = launch(fn.fwd, cut.ctas, qknr::kAttnThreads, fn.fwd_smem, a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention)");
  if (st != QKNR_OK) return st;
  return join(fn.join_fwd, cut, qknr::fwd::kRows, a, &kp, stream, "cudaLaunchKernelExC(attention, joining)");
}

qknr_status qknr_attn_backward(const qknr_attn_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  qknr::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  Rows q{"q", a->q, a->q_stride, a->seq_q, a->n_heads_q}, k{"k", a->k, a->k_stride, a->seq_k, a->n_heads_k},
      v{"v", a->v, a->v_stride, a->seq_k, a->n_heads_k}, o{"o", a->o, a->o_stride, a->seq_q, a->n_heads_q},
      g{"dout", a->dout, a->dout_stride, a->seq_q, a->n_heads_q}, dq{"dq", a->dq, a->dq_stride, a->seq_q, a->n_heads_q},
      dk{"dk", a->dk, a->dk_stride, a->seq_k, a->n_heads_k}, dv{"dv", a->dv, a->dv_stride, a->seq_k, a->n_heads_k};
  for (Rows* r : {&q, &k, &v, &o, &g, &dq, &dk, &dv})
    if ((st = check_rows(a, r)) != QKNR_OK) return st;
  if ((st = common(a, &kp)) != QKNR_OK) return st;
  if (a->batch == 0 || (a->seq_q == 0 && a->seq_k == 0)) return QKNR_OK;
  const size_t need = backward_bytes(a);
  if (a->seq_q > 0 && !a->lse) return fail(QKNR_ERR_NULL, "lse is required");
  if ((st = check_workspace(a, need)) != QKNR_OK) return st;
  const Span ws = span_of(need ? a->workspace : nullptr, 1, 0, static_cast<long long>(need));
  const Span lse{static_cast<uintptr_t>(kp.sp_lse.lo), static_cast<uintptr_t>(kp.sp_lse.hi)};
  st = check_overlap(a, {&dq, &dk, &dv}, {&q, &k, &v, &o, &g}, {ws},
                     {lse, span_of(a->q_lens, a->batch, 4, 4), span_of(a->k_lens, a->batch, 4, 4)});
  if (st != QKNR_OK) return st;
  kp.o_in = static_cast<const char*>(a->o);
  kp.dout = static_cast<const char*>(a->dout);
  kp.dq = static_cast<char*>(a->dq);
  kp.dk = static_cast<char*>(a->dk);
  kp.dv = static_cast<char*>(a->dv);
  kp.o_stride = o.stride * 2;
  kp.dout_stride = g.stride * 2;
  kp.dq_stride = dq.stride * 2;
  kp.dk_stride = dk.stride * 2;
  kp.dv_stride = dv.stride * 2;
  kp.delta = static_cast<float*>(a->workspace);
  kp.sp_o = msp(o.span);
  kp.sp_dout = msp(g.span);
  kp.sp_dq = msp(dq.span);
  kp.sp_dk = msp(dk.span);
  kp.sp_dv = msp(dv.span);
  kp.sp_delta = msp(span_of(kp.delta, 1, 0, static_cast<long long>(delta_bytes(a))));
  void* part = static_cast<char*>(a->workspace) + delta_bytes(a) + lift_bytes(a);
  if (a->dtype == QKNR_FP16) {
    kp.v_in = static_cast<const char*>(a->v);
    kp.v_stride = v.stride * 2;
    kp.sp_v = msp(v.span);
    kp.dout_norm = kp.delta + delta_bytes(a) / 4;
    kp.v_top = kp.dout_norm + delta_bytes(a) / 4;
    kp.ds_top = kp.v_top + kDeltaCtas;
    kp.q_tiles = static_cast<int>(blocks_of(a->seq_q));
    kp.sp_dout_norm = msp(span_of(kp.dout_norm, 1, 0, static_cast<long long>(delta_bytes(a))));
    kp.sp_v_top = msp(span_of(kp.v_top, 1, 0, 4LL * kDeltaCtas));
    kp.sp_ds_top = msp(span_of(kp.ds_top, 1, 0, static_cast<long long>(ds_top_bytes(a))));
  }

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  // a map of no rows is never loaded from
  if (a->seq_q > 0) {
    if ((st = make_map(&kp.map_q, a, a->q, q.stride, a->seq_q, a->n_heads_q)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_do, a, a->dout, g.stride, a->seq_q, a->n_heads_q)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_out, a, a->dq, dq.stride, a->seq_q, a->n_heads_q, qknr::kOutRows, a->head_dim / 2)) != QKNR_OK)
      return st;
  }
  if (a->seq_k > 0) {
    if ((st = make_map(&kp.map_k, a, a->k, k.stride, a->seq_k, a->n_heads_k)) != QKNR_OK) return st;
    if ((st = make_map(&kp.map_v, a, a->v, v.stride, a->seq_k, a->n_heads_k)) != QKNR_OK) return st;
  }
  const Kernels fn = kernels_for(a);
  if (a->seq_q > 0) {
    const long long rows = static_cast<long long>(a->batch) * a->seq_q * a->n_heads_q, teams = 256 / (a->head_dim / 8);
    long long grid = (rows + teams - 1) / teams;
    if (a->dtype == QKNR_FP16) {
      const long long v_grid = (static_cast<long long>(a->batch) * a->seq_k * a->n_heads_k + teams - 1) / teams;
      if (v_grid > grid) grid = v_grid;
    }
    if (grid > 8LL * di.num_sms) grid = 8LL * di.num_sms;
    if (grid > kDeltaCtas) grid = kDeltaCtas;
    kp.v_tops = static_cast<int>(grid);
    void* kargs[] = {&kp};
    st = qknr_host::launch_kernel(fn.delta, static_cast<int>(grid), 256, 0, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), "cudaLaunchKernelExC(attention delta)");
    if (st != QKNR_OK) return st;
    const Cut cut = cut_dq(a);
    apply(cut, &kp, part);
    st = launch(fn.dq, cut.ctas, qknr::kAttnThreads, fn.dq_smem, a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention dq)");
    if (st != QKNR_OK) return st;
    st = join(fn.join_dq, cut, qknr::kTile, a, &kp, stream, "cudaLaunchKernelExC(attention dq, joining)");
    if (st != QKNR_OK) return st;
  }
  if (a->seq_k == 0) return QKNR_OK;
  const Cut cut = cut_dkv(a);
  apply(cut, &kp, part);
  st = launch(fn.dkv, cut.ctas, qknr::kAttnThreads, fn.dkv_smem, a, &kp, dev, di, stream, "cudaLaunchKernelExC(attention dk, dv)");
  if (st != QKNR_OK) return st;
  return join(fn.join_dkv, cut, 2 * qknr::kTile, a, &kp, stream, "cudaLaunchKernelExC(attention dk, dv, joining)");
}

}  // extern "C"
