// C-ABI launchers of the root-mean-square norm and its backward pass:
// validation, launch planning and the launches.  No allocation, no
// synchronisation.
#include <cuda_runtime.h>

#include <cstring>
#include <initializer_list>

#include "../../include/qknr_rms.h"
#include "parts.cuh"
#include "qknr_host.h"
#include "rms_kernel.cuh"

namespace {

using qknr_host::aligned16;
using qknr_host::fail;
using qknr_host::rows_overlap;
using qknr_host::RowSpan;
using qknr_host::Span;
using qknr_host::span_of;

// CTAs the backward pass's rows are cut for: one per SM of a GB300.
constexpr long long kCtas = 152;
constexpr int kMaxHidden = 32768, kBlock = 128;

// the instances with the fewest chunks per thread that hold the row
template <typename T, int OUT>
const void* direct_fn(int cpt) {
  if (cpt <= 1) return reinterpret_cast<const void*>(qknr::rms_forward_direct_kernel<T, 1, OUT>);
  if (cpt <= 2) return reinterpret_cast<const void*>(qknr::rms_forward_direct_kernel<T, 2, OUT>);
  if (cpt <= 4) return reinterpret_cast<const void*>(qknr::rms_forward_direct_kernel<T, 4, OUT>);
  return reinterpret_cast<const void*>(qknr::rms_forward_direct_kernel<T, 8, OUT>);
}

template <typename T, int OUT>
const void* ring_fn(int cpt) {
  switch (cpt) {
    case 1: return reinterpret_cast<const void*>(qknr::rms_forward_kernel<T, 1, 2, OUT>);
    case 2: return reinterpret_cast<const void*>(qknr::rms_forward_kernel<T, 2, 2, OUT>);
    default: return reinterpret_cast<const void*>(qknr::rms_forward_kernel<T, 3, 1, OUT>);
  }
}

template <typename T>
const void* forward_fn(bool direct, int out, int cpt) {
  using namespace qknr;
  if (out == kRmsSame) return direct ? direct_fn<T, kRmsSame>(cpt) : ring_fn<T, kRmsSame>(cpt);
  if (out == kRmsRow8) return direct ? direct_fn<T, kRmsRow8>(cpt) : ring_fn<T, kRmsRow8>(cpt);
  return direct ? direct_fn<T, kRmsBlock8>(cpt) : ring_fn<T, kRmsBlock8>(cpt);
}

template <typename T>
const void* backward_fn(int cpt, bool is_long) {
  if (is_long) return reinterpret_cast<const void*>(qknr::rms_backward_kernel<T, qknr::kLnBwdCpt, 1, true>);
  switch (cpt) {
    case 1: return reinterpret_cast<const void*>(qknr::rms_backward_kernel<T, 1, 2, false>);
    case 2: return reinterpret_cast<const void*>(qknr::rms_backward_kernel<T, 2, 2, false>);
    case 3: return reinterpret_cast<const void*>(qknr::rms_backward_kernel<T, 3, 2, false>);
    default: return reinterpret_cast<const void*>(qknr::rms_backward_kernel<T, 4, 1, false>);
  }
}

// The fewest warps, up to `most`, that leave a thread at most `cpt` of a
// row's chunks.
int warps_for(int n_chunks, int cpt, int most) {
  const int w = (n_chunks + 32 * cpt - 1) / (32 * cpt);
  return w < most ? w : most;
}

qknr::MemSpan msp(Span s) { return qknr::MemSpan{s.lo, s.hi}; }
Span span(const qknr::MemSpan& s) { return Span{static_cast<uintptr_t>(s.lo), static_cast<uintptr_t>(s.hi)}; }

// Rows that share a weight row, of those that are there.
long long sample_rows(const qknr_rms_args* a) {
  return a->rows_per_batch && a->rows_per_batch < a->tokens ? a->rows_per_batch : a->tokens;
}

qknr_status check_shape(const qknr_rms_args* a) {
  if (!a) return fail(QKNR_ERR_NULL, "args is NULL");
  if (a->abi_version != QKNR_ABI_VERSION)
    return fail(QKNR_ERR_ABI, "abi_version %u, library expects %d", a->abi_version, QKNR_ABI_VERSION);
  if (a->dtype != QKNR_BF16 && a->dtype != QKNR_FP16)
    return fail(QKNR_ERR_UNSUPPORTED, "activation dtype must be BF16 or FP16");
  if (a->param_dtype != QKNR_FP32 && a->param_dtype != a->dtype)
    return fail(QKNR_ERR_UNSUPPORTED, "weight dtype must be FP32 or the activation dtype");
  const int C = a->hidden;
  if (C < 8 || C % 8 || C > kMaxHidden)
    return fail(QKNR_ERR_UNSUPPORTED, "hidden %d (a multiple of 8, <= %d)", C, kMaxHidden);
  if (a->out != QKNR_RMS_OUT_SAME && a->out != QKNR_RMS_OUT_E4M3) return fail(QKNR_ERR_UNSUPPORTED, "out %d", a->out);
  if (a->scale_block != 0 && (a->scale_block != kBlock || a->out != QKNR_RMS_OUT_E4M3 || C % kBlock))
    return fail(QKNR_ERR_UNSUPPORTED, "scale_block %d (0, or %d for an 8-bit output of a multiple of %d columns)",
                a->scale_block, kBlock, kBlock);
  if (a->tokens < 0 || a->rows_per_batch < 0) return fail(QKNR_ERR_SHAPE, "negative tokens or rows_per_batch");
  if (!(a->eps >= 0.0f)) return fail(QKNR_ERR_SHAPE, "eps must be >= 0");
  return QKNR_OK;
}

// A tensor of token rows.
struct Rows {
  const char* name;
  const void* base;
  long long stride;           // elements
  int size;                   // bytes per element
  RowSpan span{};
};

// Fills in the default stride and checks one tensor.
qknr_status check_rows(const qknr_rms_args* a, Rows* r) {
  const long long C = a->hidden, align = r->size == 1 ? 8 : 16;
  if (r->stride == 0) r->stride = C;
  if (r->stride < C) return fail(QKNR_ERR_SHAPE, "%s_stride is smaller than hidden", r->name);
  if ((r->stride * r->size) % align || reinterpret_cast<uintptr_t>(r->base) % align)
    return fail(QKNR_ERR_ALIGN, "%s base or row stride not %lld-byte aligned", r->name, align);
  r->span = RowSpan{span_of(r->base, a->tokens, r->stride * r->size, C * r->size), r->stride * r->size, C * r->size};
  return QKNR_OK;
}

// Whether `out` may not be written while `in` is read: they share an element
// and are not the same rows.
bool clash(const Rows& out, const Rows& in, bool same_rows) {
  if (!out.base || !in.base) return false;
  if (same_rows && out.base == in.base && out.stride == in.stride && out.size == in.size) return false;
  return rows_overlap(out.span, in.span);
}

bool hits(Span out, std::initializer_list<Span> others) {
  for (const Span& s : others)
    if (qknr_host::overlaps(out, s)) return true;
  return false;
}

// The fields both passes share.
qknr_status common(const qknr_rms_args* a, qknr::RmsParams* kp) {
  const int C = a->hidden, pes = a->param_dtype == QKNR_FP32 ? 4 : 2;
  const long long T = a->tokens, ps = a->param_stride ? a->param_stride : C, rpb = sample_rows(a), sets = (T + rpb - 1) / rpb;
  if (ps < C) return fail(QKNR_ERR_SHAPE, "param_stride is smaller than hidden");
  if (!aligned16(a->weight) || (ps * pes) % 16) return fail(QKNR_ERR_ALIGN, "weight base or stride not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a->rstd) | reinterpret_cast<uintptr_t>(a->scales)) & 3u)
    return fail(QKNR_ERR_ALIGN, "rstd / scales not 4-byte aligned");
  memset(kp, 0, sizeof(*kp));
  kp->tokens = T;
  kp->rows_per_batch = rpb;
  kp->sets = sets;
  kp->weight = static_cast<const char*>(a->weight);
  kp->param_stride = ps * pes;
  kp->param_fp32 = a->param_dtype == QKNR_FP32;
  kp->rstd = a->rstd;
  kp->hidden = C;
  kp->eps = a->eps;
  kp->inv_c = 1.0f / static_cast<float>(C);
  kp->unit = a->flags & QKNR_RMS_UNIT_OFFSET ? 1.0f : 0.0f;
  kp->row_bytes = static_cast<unsigned>(C) * 2;
  kp->flags = a->flags;
  kp->wait_limit_ns = a->wait_limit_ns ? a->wait_limit_ns : 2000000000ull;
  kp->status = a->dev_status;
  kp->sp_weight = msp(span_of(a->weight, sets, ps * pes, static_cast<long long>(C) * pes));
  kp->sp_rstd = msp(span_of(a->rstd, T, 4, 4));
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

// How the backward pass cuts the rows (nothing here needs a device).
struct Cut {
  int tiles, group_warps, groups, cpt;
  long long sets, units_per_set, unit_rows;
  size_t sums_bytes, parts_bytes;
};

Cut cut_rows(const qknr_rms_args* a) {
  Cut c;
  const long long T = a->tokens, rows = sample_rows(a);
  const int n_chunks = a->hidden / 8;
  c.tiles = (a->hidden + qknr::kLnTile - 1) / qknr::kLnTile;
  c.group_warps = warps_for(n_chunks, qknr::kLnBwdCpt, qknr::kLnBwdWarps);
  c.groups = qknr::kLnBwdWarps / c.group_warps;
  c.cpt = (n_chunks + 32 * c.group_warps - 1) / (32 * c.group_warps);
  c.sets = T ? (T + rows - 1) / rows : 0;
  // One unit per CTA where the samples are few.  Where they are nearly as
  // many as the CTAs, four units per CTA, so that no CTA does twice
  // another's work; where they are more than that, a sample is a unit.
  const long long ctas = kCtas / c.tiles;
  long long ups = 1;
  if (c.sets && c.sets < 4 * ctas) ups = c.sets > ctas / 4 ? (4 * ctas + c.sets - 1) / c.sets : ctas / c.sets;
  const long long most = (rows + c.groups - 1) / c.groups;   // a row for each group
  if (ups > most) ups = most;
  if (ups < 1) ups = 1;
  c.unit_rows = rows ? (rows + ups - 1) / ups : 1;
  c.units_per_set = rows ? (rows + c.unit_rows - 1) / c.unit_rows : 1;
  c.sums_bytes = c.tiles > 1 ? (static_cast<size_t>(T) * 4 + 15) / 16 * 16 : 0;
  c.parts_bytes = c.units_per_set > 1 ? static_cast<size_t>(c.sets * c.units_per_set) * a->hidden * 4 : 0;
  return c;
}

qknr_status run(const void* fn, long long grid, int block, size_t smem, const qknr_rms_args* a, void* kp, int dev,
                const qknr_host::DeviceInfo& di, qknr_stream_t stream, const char* what) {
  if (grid > 0x7fffffffLL) return fail(QKNR_ERR_UNSUPPORTED, "more than 2^31 CTAs");
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

void qknr_rms_args_init(qknr_rms_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
  a->param_dtype = QKNR_FP32;
  a->eps = 1e-6f;
}

size_t qknr_rms_sizeof_args(void) { return sizeof(qknr_rms_args); }

qknr_status qknr_rms_forward(const qknr_rms_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK || a->tokens == 0) return st;
  const int C = a->hidden;
  const long long T = a->tokens;
  const bool small = a->out == QKNR_RMS_OUT_E4M3;
  if (!a->x || !a->y) return fail(QKNR_ERR_NULL, "x and y are required");
  if (small && !a->scales) return fail(QKNR_ERR_NULL, "scales is required");
  if (a->residual && !a->sum) return fail(QKNR_ERR_NULL, "sum is required with a residual");
  Rows x{"x", a->x, a->x_stride, 2}, r{"residual", a->residual, a->residual_stride, 2},
      sum{"sum", a->residual ? a->sum : nullptr, a->sum_stride, 2}, y{"y", a->y, a->y_stride, small ? 1 : 2};
  for (Rows* t : {&x, &r, &sum, &y})
    if ((st = check_rows(a, t)) != QKNR_OK) return st;
  qknr::RmsParams kp;
  if ((st = common(a, &kp)) != QKNR_OK) return st;
  const long long per_row = a->scale_block ? C / kBlock : 1;
  const Span scales = span_of(small ? a->scales : nullptr, T * per_row, 4, 4), rstd = span(kp.sp_rstd), weight = span(kp.sp_weight);
  if (clash(y, x, true) || clash(y, r, false)) return fail(QKNR_ERR_OVERLAP, "y overlaps x or residual without being x");
  if (clash(sum, x, true) || clash(sum, r, true)) return fail(QKNR_ERR_OVERLAP, "sum overlaps x or residual without being either");
  if (clash(sum, y, false)) return fail(QKNR_ERR_OVERLAP, "sum overlaps y");
  if (hits(y.span.span, {weight, rstd, scales}) || hits(sum.span.span, {weight, rstd, scales}))
    return fail(QKNR_ERR_OVERLAP, "y or sum overlaps weight, rstd or scales");
  if (hits(rstd, {x.span.span, r.span.span, weight, scales}) || hits(scales, {x.span.span, r.span.span, weight}))
    return fail(QKNR_ERR_OVERLAP, "rstd or scales overlaps another tensor");
  kp.x = static_cast<const char*>(a->x);
  kp.x_stride = x.stride * 2;
  kp.residual = static_cast<const char*>(a->residual);
  kp.residual_stride = r.stride * 2;
  kp.sum = static_cast<char*>(const_cast<void*>(sum.base));
  kp.sum_stride = sum.stride * 2;
  kp.y = static_cast<char*>(a->y);
  kp.y_stride = y.stride * y.size;
  kp.scales = small ? a->scales : nullptr;
  kp.sp_x = msp(x.span.span);
  kp.sp_residual = msp(r.span.span);
  kp.sp_sum = msp(sum.span.span);
  kp.sp_y = msp(y.span.span);
  kp.sp_scales = msp(scales);

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  // Calls of a few rows per SM have nothing to stream: a CTA per row, its
  // chunks spread over as many warps as there are.  So do rows of more than
  // 12288 values, whose gains do not fit in registers.
  const int n_chunks = C / 8, keep = 3, out = !small ? qknr::kRmsSame : a->scale_block ? qknr::kRmsBlock8 : qknr::kRmsRow8;
  const bool bf = a->dtype == QKNR_BF16;
  if (T < 4LL * di.num_sms || n_chunks > 32 * keep * qknr::kLnWarps) {
    const int warps = warps_for(n_chunks, 1, qknr::kLnWarps), cpt = (n_chunks + 32 * warps - 1) / (32 * warps);
    kp.group_warps = warps;
    kp.groups = warps == 1 ? 4 : 1;               // rows of one warp: four to a CTA
    return run(bf ? forward_fn<__nv_bfloat16>(true, out, cpt) : forward_fn<__half>(true, out, cpt),
               (T + kp.groups - 1) / kp.groups, 32 * warps * kp.groups, 0, a, &kp, dev, di, stream,
               "cudaLaunchKernelExC(RMS norm)");
  }
  kp.groups = qknr::kLnWarps / warps_for(n_chunks, keep, qknr::kLnWarps);
  const int warps = qknr::kLnWarps / kp.groups, cpt = (n_chunks + 32 * warps - 1) / (32 * warps);
  kp.group_warps = warps;
  const size_t stage = (a->residual ? 2 : 1) * static_cast<size_t>(kp.row_bytes);
  kp.stages = stages_for(di, stage, kp.groups, 0);
  return run(bf ? forward_fn<__nv_bfloat16>(false, out, cpt) : forward_fn<__half>(false, out, cpt), di.num_sms,
             32 * warps * kp.groups, qknr::kLnOffStages + kp.stages * kp.groups * stage, a, &kp, dev, di, stream,
             "cudaLaunchKernelExC(RMS norm)");
}

qknr_status qknr_rms_workspace_bytes(const qknr_rms_args* a, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const Cut c = cut_rows(a);
  *bytes = c.sums_bytes + c.parts_bytes;
  return QKNR_OK;
}

qknr_status qknr_rms_backward(const qknr_rms_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const int C = a->hidden;
  const long long T = a->tokens;
  if (!aligned16(a->dweight)) return fail(QKNR_ERR_ALIGN, "dweight not 16-byte aligned");
  if (T == 0) {
    // the sum over no rows
    if (!a->dweight || a->rows_per_batch) return QKNR_OK;
    const cudaError_t e = cudaMemsetAsync(a->dweight, 0, static_cast<size_t>(C) * 4, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QKNR_OK : qknr_host::cuda_fail(e, "cudaMemsetAsync(RMS norm)");
  }
  if (!a->x || !a->dy || !a->dx || !a->rstd) return fail(QKNR_ERR_NULL, "x, dy, dx and rstd are required");
  Rows x{"x", a->x, a->x_stride, 2}, dy{"dy", a->dy, a->dy_stride, 2}, ds{"dsum", a->dsum, a->dsum_stride, 2},
      dx{"dx", a->dx, a->dx_stride, 2};
  for (Rows* t : {&x, &dy, &ds, &dx})
    if ((st = check_rows(a, t)) != QKNR_OK) return st;
  qknr::RmsParams kp;
  if ((st = common(a, &kp)) != QKNR_OK) return st;
  const Cut c = cut_rows(a);
  const size_t need = c.sums_bytes + c.parts_bytes;
  if (need && !a->workspace) return fail(QKNR_ERR_NULL, "workspace is required");
  if (need && a->workspace_bytes < need)
    return fail(QKNR_ERR_SHAPE, "workspace of %zu bytes, %zu needed", a->workspace_bytes, need);
  if (!aligned16(a->workspace)) return fail(QKNR_ERR_ALIGN, "workspace not 16-byte aligned");
  const Span dw = span_of(a->dweight, c.sets, 4LL * C, 4LL * C),
             ws = span_of(need ? a->workspace : nullptr, 1, 0, static_cast<long long>(need)), rstd = span(kp.sp_rstd),
             weight = span(kp.sp_weight);
  if (clash(dx, dy, true) || clash(dx, ds, true)) return fail(QKNR_ERR_OVERLAP, "dx overlaps dy or dsum without being either");
  if (clash(dx, x, false)) return fail(QKNR_ERR_OVERLAP, "dx overlaps x");
  if (hits(dx.span.span, {weight, rstd, dw, ws})) return fail(QKNR_ERR_OVERLAP, "dx overlaps weight, rstd, dweight or the workspace");
  for (const Span& s : {dw, ws})
    if (hits(s, {x.span.span, dy.span.span, ds.span.span, weight, rstd})) return fail(QKNR_ERR_OVERLAP, "dweight or the workspace overlaps an input");
  if (qknr_host::overlaps(dw, ws)) return fail(QKNR_ERR_OVERLAP, "dweight and the workspace overlap");
  kp.x = static_cast<const char*>(a->x);
  kp.x_stride = x.stride * 2;
  kp.dy = static_cast<const char*>(a->dy);
  kp.dy_stride = dy.stride * 2;
  kp.dsum = static_cast<const char*>(a->dsum);
  kp.dsum_stride = ds.stride * 2;
  kp.dx = static_cast<char*>(a->dx);
  kp.dx_stride = dx.stride * 2;
  kp.dweight = a->dweight;
  kp.row_sums = c.sums_bytes ? static_cast<float*>(a->workspace) : nullptr;
  kp.parts = c.parts_bytes ? reinterpret_cast<float*>(static_cast<char*>(a->workspace) + c.sums_bytes) : nullptr;
  kp.group_warps = c.group_warps;
  kp.groups = c.groups;
  kp.units_per_set = c.units_per_set;
  kp.unit_rows = c.unit_rows;
  kp.tiles = c.tiles;
  kp.sp_x = msp(x.span.span);
  kp.sp_dy = msp(dy.span.span);
  kp.sp_dsum = msp(ds.span.span);
  kp.sp_dx = msp(dx.span.span);
  kp.sp_dweight = msp(dw);
  kp.sp_ws = msp(ws);

  int dev = 0;
  qknr_host::DeviceInfo di;
  if ((st = device(&dev, &di)) != QKNR_OK) return st;
  const bool bf = a->dtype == QKNR_BF16;
  if (c.tiles > 1) {
    const void* fn = bf ? reinterpret_cast<const void*>(qknr::rms_row_sums_kernel<__nv_bfloat16>)
                        : reinterpret_cast<const void*>(qknr::rms_row_sums_kernel<__half>);
    st = run(fn, T < 8LL * di.num_sms ? T : 8LL * di.num_sms, 256, 0, a, &kp, dev, di, stream,
             "cudaLaunchKernelExC(RMS norm row sums)");
    if (st != QKNR_OK) return st;
  }
  const void* fn = bf ? backward_fn<__nv_bfloat16>(c.cpt, c.tiles > 1) : backward_fn<__half>(c.cpt, c.tiles > 1);
  const int cols = C < qknr::kLnTile ? C : qknr::kLnTile;
  const size_t sums = c.groups > 1 ? static_cast<size_t>(c.groups) * cols * 4 : 0;
  const size_t stage = (a->dsum ? 6 : 4) * static_cast<size_t>(cols);
  kp.stages = stages_for(di, stage, c.groups, sums);
  long long ctas = di.num_sms / c.tiles;
  if (ctas > c.sets * c.units_per_set) ctas = c.sets * c.units_per_set;
  st = run(fn, ctas * c.tiles, 32 * c.group_warps * c.groups, qknr::kLnOffStages + kp.stages * c.groups * stage + sums, a, &kp,
           dev, di, stream, "cudaLaunchKernelExC(RMS norm backward)");
  if (st != QKNR_OK || !kp.parts || !kp.dweight) return st;
  qknr::PartsParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.sums = 1;
  pp.parts = kp.parts;
  pp.out[0] = kp.dweight;
  pp.cols = C;
  pp.units = c.units_per_set;
  pp.sp_parts = kp.sp_ws;
  pp.sp_out[0] = kp.sp_dweight;
  pp.status = a->dev_status;
  return run(reinterpret_cast<const void*>(qknr::parts_kernel), qknr::parts_grid(pp, c.sets), 32 * qknr::kPartsRows, 0, a, &pp,
             dev, di, stream, "cudaLaunchKernelExC(RMS norm weight sums)");
}

}  // extern "C"
