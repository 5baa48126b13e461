// C-ABI launchers of layer norm and its backward pass: validation, launch
// planning and the launches.  No allocation, no synchronisation.
#include <cuda_runtime.h>

#include <cstring>
#include <initializer_list>

#include "../../include/qknr_ln.h"
#include "ln_kernel.cuh"
#include "parts.cuh"
#include "qknr_host.h"

namespace {

using qknr_host::aligned16;
using qknr_host::fail;
using qknr_host::rows_overlap;
using qknr_host::RowSpan;
using qknr_host::Span;
using qknr_host::span_of;

// CTAs the backward pass's rows are cut for: one per SM of a GB300.
constexpr long long kCtas = 152;
constexpr int kMaxHidden = 32768;

// the instances with the fewest chunks per thread that hold the row
template <typename T>
const void* direct_fn(int cpt) {
  if (cpt <= 1) return reinterpret_cast<const void*>(qknr::ln_forward_direct_kernel<T, 1>);
  if (cpt <= 2) return reinterpret_cast<const void*>(qknr::ln_forward_direct_kernel<T, 2>);
  if (cpt <= 4) return reinterpret_cast<const void*>(qknr::ln_forward_direct_kernel<T, 4>);
  return reinterpret_cast<const void*>(qknr::ln_forward_direct_kernel<T, 8>);
}

template <typename T>
const void* forward_fn(int cpt) {
  switch (cpt) {
    case 1: return reinterpret_cast<const void*>(qknr::ln_forward_kernel<T, 1, 2>);
    case 2: return reinterpret_cast<const void*>(qknr::ln_forward_kernel<T, 2, 2>);
    default: return reinterpret_cast<const void*>(qknr::ln_forward_kernel<T, 3, 1>);
  }
}

template <typename T>
const void* backward_fn(int cpt, bool is_long) {
  if (is_long) return reinterpret_cast<const void*>(qknr::ln_backward_kernel<T, qknr::kLnBwdCpt, 1, true>);
  switch (cpt) {
    case 1: return reinterpret_cast<const void*>(qknr::ln_backward_kernel<T, 1, 2, false>);
    case 2: return reinterpret_cast<const void*>(qknr::ln_backward_kernel<T, 2, 2, false>);
    case 3: return reinterpret_cast<const void*>(qknr::ln_backward_kernel<T, 3, 2, false>);
    default: return reinterpret_cast<const void*>(qknr::ln_backward_kernel<T, 4, 1, false>);
  }
}

// The fewest warps, up to `most`, that leave a thread at most `cpt` of a
// row's chunks.
int warps_for(int n_chunks, int cpt, int most) {
  const int w = (n_chunks + 32 * cpt - 1) / (32 * cpt);
  return w < most ? w : most;
}

qknr::MemSpan msp(Span s) { return qknr::MemSpan{s.lo, s.hi}; }

// Rows that share a parameter row, of those that are there.
long long sample_rows(const qknr_ln_args* a) {
  return a->rows_per_batch && a->rows_per_batch < a->tokens ? a->rows_per_batch : a->tokens;
}

// How the backward pass cuts the rows (nothing here needs a device).
struct Cut {
  int tiles, group_warps, groups, cpt;
  long long sets, units_per_set, unit_rows, rows_per_batch;
  size_t sums_bytes, parts_bytes;
};

qknr_status check_shape(const qknr_ln_args* a) {
  if (!a) return fail(QKNR_ERR_NULL, "args is NULL");
  if (a->abi_version != QKNR_ABI_VERSION)
    return fail(QKNR_ERR_ABI, "abi_version %u, library expects %d", a->abi_version, QKNR_ABI_VERSION);
  if (a->dtype != QKNR_BF16 && a->dtype != QKNR_FP16)
    return fail(QKNR_ERR_UNSUPPORTED, "activation dtype must be BF16 or FP16");
  if (a->param_dtype != QKNR_FP32 && a->param_dtype != a->dtype)
    return fail(QKNR_ERR_UNSUPPORTED, "weight/bias dtype must be FP32 or the activation dtype");
  const int C = a->hidden;
  if (C < 8 || C % 8 || C > kMaxHidden)
    return fail(QKNR_ERR_UNSUPPORTED, "hidden %d (a multiple of 8, <= %d)", C, kMaxHidden);
  if (a->tokens < 0 || a->rows_per_batch < 0) return fail(QKNR_ERR_SHAPE, "negative tokens or rows_per_batch");
  if (!(a->eps >= 0.0f)) return fail(QKNR_ERR_SHAPE, "eps must be >= 0");
  return QKNR_OK;
}

// Ring depth of each of `groups` groups: 128 KB per SM in flight keep HBM
// busy, and at least two stages that fit beside `other` bytes.
int stages_for(const qknr_host::DeviceInfo& di, size_t stage_bytes, int groups, size_t other) {
  const size_t room = (di.smem_optin - qknr::kLnOffStages - other) / (stage_bytes * groups);
  size_t n = 128 * 1024 / (stage_bytes * groups);
  if (n < 2) n = 2;
  if (n > room) n = room;
  if (n > static_cast<size_t>(qknr::kLnMaxStages / groups)) n = qknr::kLnMaxStages / groups;
  return static_cast<int>(n);
}

Cut cut_rows(const qknr_ln_args* a) {
  Cut c;
  const long long T = a->tokens;
  const int n_chunks = a->hidden / 8;
  c.tiles = (a->hidden + qknr::kLnTile - 1) / qknr::kLnTile;
  c.group_warps = warps_for(n_chunks, qknr::kLnBwdCpt, qknr::kLnBwdWarps);
  c.groups = qknr::kLnBwdWarps / c.group_warps;   // groups of several warps: at most 8 named barriers
  c.cpt = (n_chunks + 32 * c.group_warps - 1) / (32 * c.group_warps);
  c.rows_per_batch = sample_rows(a);
  c.sets = T ? (T + c.rows_per_batch - 1) / c.rows_per_batch : 0;
  const long long rows = c.rows_per_batch;
  // One unit per CTA where the samples are few.  Where they are nearly as
  // many as the CTAs, four units per CTA, so that no CTA does twice
  // another's work; where they are more than that, a sample is a unit.
  const long long ctas = kCtas / c.tiles;
  long long ups = 1;
  if (c.sets && c.sets < 4 * ctas)
    ups = c.sets > ctas / 4 ? (4 * ctas + c.sets - 1) / c.sets : ctas / c.sets;
  const long long most = (rows + c.groups - 1) / c.groups;   // a row for each group
  if (ups > most) ups = most;
  if (ups < 1) ups = 1;
  c.unit_rows = rows ? (rows + ups - 1) / ups : 1;
  c.units_per_set = rows ? (rows + c.unit_rows - 1) / c.unit_rows : 1;
  c.sums_bytes = c.tiles > 1 ? (static_cast<size_t>(T) * 8 + 15) / 16 * 16 : 0;
  c.parts_bytes = c.units_per_set > 1 ? static_cast<size_t>(c.sets * c.units_per_set) * 2 * a->hidden * 4 : 0;
  return c;
}

// The fields both passes share, and the checks of x and the parameters.
qknr_status common(const qknr_ln_args* a, qknr::LnParams* kp) {
  const int C = a->hidden, es = 2, pes = a->param_dtype == QKNR_FP32 ? 4 : 2;
  const long long T = a->tokens;
  const long long xs = a->x_stride ? a->x_stride : C, ps = a->param_stride ? a->param_stride : C;
  const long long rpb = sample_rows(a);
  const long long sets = (T + rpb - 1) / rpb;
  if (!a->x) return fail(QKNR_ERR_NULL, "x is required");
  if (xs < C || ps < C) return fail(QKNR_ERR_SHAPE, "a stride is smaller than hidden");
  if (!aligned16(a->x) || !aligned16(a->weight) || !aligned16(a->bias) || (xs * es) % 16 || (ps * pes) % 16)
    return fail(QKNR_ERR_ALIGN, "x / weight / bias base or stride not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a->mean) | reinterpret_cast<uintptr_t>(a->rstd)) & 3u)
    return fail(QKNR_ERR_ALIGN, "mean / rstd not 4-byte aligned");
  memset(kp, 0, sizeof(*kp));
  kp->x = static_cast<const char*>(a->x);
  kp->x_stride = xs * es;
  kp->tokens = T;
  kp->rows_per_batch = rpb;
  kp->sets = sets;
  kp->weight = static_cast<const char*>(a->weight);
  kp->bias = static_cast<const char*>(a->bias);
  kp->param_stride = ps * pes;
  kp->param_fp32 = a->param_dtype == QKNR_FP32;
  kp->mean = a->mean;
  kp->rstd = a->rstd;
  kp->hidden = C;
  kp->eps = a->eps;
  kp->inv_c = 1.0f / static_cast<float>(C);
  kp->unit = a->flags & QKNR_LN_UNIT_OFFSET ? 1.0f : 0.0f;
  kp->row_bytes = static_cast<unsigned>(C) * 2;
  kp->flags = a->flags;
  kp->wait_limit_ns = a->wait_limit_ns ? a->wait_limit_ns : 2000000000ull;
  kp->status = a->dev_status;
  kp->sp_x = msp(span_of(a->x, T, xs * es, (long long)C * es));
  kp->sp_weight = msp(span_of(a->weight, sets, ps * pes, (long long)C * pes));
  kp->sp_bias = msp(span_of(a->bias, sets, ps * pes, (long long)C * pes));
  kp->sp_mean = msp(span_of(a->mean, T, 4, 4));
  kp->sp_rstd = msp(span_of(a->rstd, T, 4, 4));
  return QKNR_OK;
}

RowSpan rows_of(const qknr::MemSpan& s, long long stride, const qknr_ln_args* a) {
  return RowSpan{Span{static_cast<uintptr_t>(s.lo), static_cast<uintptr_t>(s.hi)}, stride, 2LL * a->hidden};
}

bool hits(Span out, std::initializer_list<qknr::MemSpan> ins) {
  for (const qknr::MemSpan& s : ins)
    if (qknr_host::overlaps(out, Span{static_cast<uintptr_t>(s.lo), static_cast<uintptr_t>(s.hi)})) return true;
  return false;
}

qknr_status run(const void* fn, long long grid, int block, size_t smem, const qknr_ln_args* a, void* kp,
                int dev, const qknr_host::DeviceInfo& di, qknr_stream_t stream, const char* what) {
  if (smem) {   // dynamic shared memory only
    int regs = 0;
    const qknr_status st = qknr_host::configure_kernel(fn, dev, di, &regs);
    if (st != QKNR_OK) return st;
  }
  void* kargs[] = {kp};
  return qknr_host::launch_kernel(fn, static_cast<int>(grid), block, smem, reinterpret_cast<cudaStream_t>(stream),
                                  kargs, !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
}

qknr_status device(int* dev, qknr_host::DeviceInfo* di) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaGetDevice");
  return qknr_host::device_info(*dev, di);
}

}  // namespace

extern "C" {

void qknr_ln_args_init(qknr_ln_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
  a->param_dtype = QKNR_FP32;
  a->eps = 1e-6f;
}

size_t qknr_ln_sizeof_args(void) { return sizeof(qknr_ln_args); }

qknr_status qknr_ln_forward(const qknr_ln_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK || a->tokens == 0) return st;
  qknr::LnParams kp;
  st = common(a, &kp);
  if (st != QKNR_OK) return st;
  const int C = a->hidden;
  const long long T = a->tokens;
  void* y = a->y ? a->y : const_cast<void*>(a->x);
  const long long xs = kp.x_stride / 2, ys = a->y_stride ? a->y_stride : xs;
  if (ys < C) return fail(QKNR_ERR_SHAPE, "a stride is smaller than hidden");
  if (!aligned16(y) || (ys * 2) % 16) return fail(QKNR_ERR_ALIGN, "y base or stride not 16-byte aligned");
  const Span so = span_of(y, T, ys * 2, 2LL * C);
  const bool in_place = y == a->x && ys == xs;
  if (!in_place && rows_overlap(rows_of(msp(so), ys * 2, a), rows_of(kp.sp_x, kp.x_stride, a)))
    return fail(QKNR_ERR_OVERLAP, "y overlaps x without being in place");
  if (hits(so, {kp.sp_weight, kp.sp_bias, kp.sp_mean, kp.sp_rstd}))
    return fail(QKNR_ERR_OVERLAP, "y overlaps a parameter, mean or rstd");
  const Span mean{static_cast<uintptr_t>(kp.sp_mean.lo), static_cast<uintptr_t>(kp.sp_mean.hi)};
  const Span rstd{static_cast<uintptr_t>(kp.sp_rstd.lo), static_cast<uintptr_t>(kp.sp_rstd.hi)};
  for (const Span& s : {mean, rstd})
    if (hits(s, {kp.sp_x, kp.sp_weight, kp.sp_bias})) return fail(QKNR_ERR_OVERLAP, "mean or rstd overlaps x or a parameter");
  if (qknr_host::overlaps(mean, rstd)) return fail(QKNR_ERR_OVERLAP, "mean and rstd overlap");
  kp.y = static_cast<char*>(y);
  kp.y_stride = ys * 2;
  kp.sp_y = msp(so);

  int dev = 0;
  qknr_host::DeviceInfo di;
  st = device(&dev, &di);
  if (st != QKNR_OK) return st;
  // Calls of a few rows per SM have nothing to stream: a CTA per row, its
  // chunks spread over as many warps as there are.  So do rows of more than
  // 12288 values, whose parameters do not fit in registers.
  const int n_chunks = C / 8, keep = 3;
  const bool bf = a->dtype == QKNR_BF16;
  if (T < 4LL * di.num_sms || n_chunks > 32 * keep * qknr::kLnWarps) {
    const int warps = warps_for(n_chunks, 1, qknr::kLnWarps);
    const int cpt = (n_chunks + 32 * warps - 1) / (32 * warps);
    kp.group_warps = warps;
    kp.groups = warps == 1 ? 4 : 1;               // rows of one warp: four to a CTA
    return run(bf ? direct_fn<__nv_bfloat16>(cpt) : direct_fn<__half>(cpt), (T + kp.groups - 1) / kp.groups,
               32 * warps * kp.groups, 0, a, &kp, dev, di, stream, "cudaLaunchKernelExC(layer norm)");
  }
  kp.groups = qknr::kLnWarps / warps_for(n_chunks, keep, qknr::kLnWarps);
  const int warps = qknr::kLnWarps / kp.groups, cpt = (n_chunks + 32 * warps - 1) / (32 * warps);
  kp.group_warps = warps;
  kp.stages = stages_for(di, kp.row_bytes, kp.groups, 0);
  return run(bf ? forward_fn<__nv_bfloat16>(cpt) : forward_fn<__half>(cpt), di.num_sms, 32 * warps * kp.groups,
             qknr::kLnOffStages + static_cast<size_t>(kp.stages) * kp.groups * kp.row_bytes, a, &kp, dev, di, stream,
             "cudaLaunchKernelExC(layer norm)");
}

qknr_status qknr_ln_workspace_bytes(const qknr_ln_args* a, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const Cut c = cut_rows(a);
  *bytes = c.sums_bytes + c.parts_bytes;
  return QKNR_OK;
}

qknr_status qknr_ln_backward(const qknr_ln_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const int C = a->hidden;
  const long long T = a->tokens;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if ((reinterpret_cast<uintptr_t>(a->dweight) | reinterpret_cast<uintptr_t>(a->dbias)) & 15u)
    return fail(QKNR_ERR_ALIGN, "dweight / dbias not 16-byte aligned");
  if (T == 0) {
    // the sum over no rows
    for (float* d : {a->dweight, a->dbias}) {
      if (!d || a->rows_per_batch) continue;
      const cudaError_t e = cudaMemsetAsync(d, 0, static_cast<size_t>(C) * 4, cs);
      if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaMemsetAsync(layer norm)");
    }
    return QKNR_OK;
  }
  qknr::LnParams kp;
  st = common(a, &kp);
  if (st != QKNR_OK) return st;
  if (!a->dy || !a->mean || !a->rstd) return fail(QKNR_ERR_NULL, "dy, mean and rstd are required");
  const long long ds = a->dy_stride ? a->dy_stride : C, os = a->dx_stride ? a->dx_stride : ds;
  void* dx = a->dx ? a->dx : const_cast<void*>(a->dy);
  if (ds < C || os < C) return fail(QKNR_ERR_SHAPE, "a stride is smaller than hidden");
  if (!aligned16(a->dy) || !aligned16(dx) || (ds * 2) % 16 || (os * 2) % 16)
    return fail(QKNR_ERR_ALIGN, "dy / dx base or stride not 16-byte aligned");
  const Cut c = cut_rows(a);
  const size_t need = c.sums_bytes + c.parts_bytes;
  if (need && !a->workspace) return fail(QKNR_ERR_NULL, "workspace is required");
  if (need && a->workspace_bytes < need)
    return fail(QKNR_ERR_SHAPE, "workspace of %zu bytes, %zu needed", a->workspace_bytes, need);
  if (!aligned16(a->workspace)) return fail(QKNR_ERR_ALIGN, "workspace not 16-byte aligned");
  kp.sp_dy = msp(span_of(a->dy, T, ds * 2, 2LL * C));
  const Span so = span_of(dx, T, os * 2, 2LL * C);
  const Span sw = span_of(a->dweight, c.sets, 4LL * C, 4LL * C), sb = span_of(a->dbias, c.sets, 4LL * C, 4LL * C);
  const Span sk = span_of(need ? a->workspace : nullptr, 1, 0, static_cast<long long>(need));
  const bool in_place = dx == a->dy && os == ds;
  const RowSpan out = rows_of(msp(so), os * 2, a);
  if (!in_place && rows_overlap(out, rows_of(kp.sp_dy, ds * 2, a)))
    return fail(QKNR_ERR_OVERLAP, "dx overlaps dy without being in place");
  if (rows_overlap(out, rows_of(kp.sp_x, kp.x_stride, a))) return fail(QKNR_ERR_OVERLAP, "dx overlaps x");
  const Span outs[] = {so, sw, sb, sk};
  for (int i = 0; i < 4; ++i) {
    if (hits(outs[i], {kp.sp_weight, kp.sp_mean, kp.sp_rstd}) || (i && hits(outs[i], {kp.sp_x, kp.sp_dy})))
      return fail(QKNR_ERR_OVERLAP, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (qknr_host::overlaps(outs[i], outs[j])) return fail(QKNR_ERR_OVERLAP, "two outputs overlap");
  }
  kp.dy = static_cast<const char*>(a->dy);
  kp.dx = static_cast<char*>(dx);
  kp.dy_stride = ds * 2;
  kp.dx_stride = os * 2;
  kp.dweight = a->dweight;
  kp.dbias = a->dbias;
  kp.row_sums = c.sums_bytes ? static_cast<float*>(a->workspace) : nullptr;
  kp.parts = c.parts_bytes ? reinterpret_cast<float*>(static_cast<char*>(a->workspace) + c.sums_bytes) : nullptr;
  kp.group_warps = c.group_warps;
  kp.groups = c.groups;
  kp.units_per_set = c.units_per_set;
  kp.unit_rows = c.unit_rows;
  kp.tiles = c.tiles;
  kp.sp_dx = msp(so);
  kp.sp_dweight = msp(sw);
  kp.sp_dbias = msp(sb);
  kp.sp_ws = msp(sk);

  int dev = 0;
  qknr_host::DeviceInfo di;
  st = device(&dev, &di);
  if (st != QKNR_OK) return st;
  const bool bf = a->dtype == QKNR_BF16;
  if (c.tiles > 1) {
    const void* fn = bf ? reinterpret_cast<const void*>(qknr::ln_row_sums_kernel<__nv_bfloat16>)
                        : reinterpret_cast<const void*>(qknr::ln_row_sums_kernel<__half>);
    const long long grid = T < 8LL * di.num_sms ? T : 8LL * di.num_sms;
    st = run(fn, grid, 256, 0, a, &kp, dev, di, stream, "cudaLaunchKernelExC(layer norm row sums)");
    if (st != QKNR_OK) return st;
  }
  const void* fn = bf ? backward_fn<__nv_bfloat16>(c.cpt, c.tiles > 1) : backward_fn<__half>(c.cpt, c.tiles > 1);
  const int cols = C < qknr::kLnTile ? C : qknr::kLnTile;
  const size_t sums = c.groups > 1 ? static_cast<size_t>(c.groups) * 2 * cols * 4 : 0;
  const size_t stage = 4 * static_cast<size_t>(cols);
  kp.stages = stages_for(di, stage, c.groups, sums);
  long long ctas = di.num_sms / c.tiles;
  if (ctas > c.sets * c.units_per_set) ctas = c.sets * c.units_per_set;
  st = run(fn, ctas * c.tiles, 32 * c.group_warps * c.groups, qknr::kLnOffStages + kp.stages * c.groups * stage + sums, a, &kp,
           dev, di, stream, "cudaLaunchKernelExC(layer norm backward)");
  if (st != QKNR_OK || !kp.parts || (!kp.dweight && !kp.dbias)) return st;
  qknr::PartsParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.sums = 2;
  pp.parts = kp.parts;
  pp.out[0] = kp.dweight;
  pp.out[1] = kp.dbias;
  pp.cols = C;
  pp.units = c.units_per_set;
  pp.sp_parts = kp.sp_ws;
  pp.sp_out[0] = kp.sp_dweight;
  pp.sp_out[1] = kp.sp_dbias;
  pp.status = a->dev_status;
  return run(reinterpret_cast<const void*>(qknr::parts_kernel), qknr::parts_grid(pp, c.sets),
             32 * qknr::kPartsRows, 0, a, &pp, dev, di, stream,
             "cudaLaunchKernelExC(layer norm parameter sums)");
}

}  // extern "C"
