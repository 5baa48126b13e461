// C-ABI launcher of the backward pass of the fused QK-RMSNorm + RoPE:
// validation, launch planning and the launches.  No allocation, no
// synchronisation.
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/qknr_grad.h"
#include "grad_kernel.cuh"
#include "parts.cuh"
#include "qknr_host.h"

namespace {

using qknr_host::aligned16;
using qknr_host::fail;
using qknr_host::rows_overlap;
using qknr_host::RowSpan;
using qknr_host::Span;
using qknr_host::span_of;

// CTAs at most: the three of 256 threads that each SM of a GB300 holds.
constexpr long long kMaxCtas = 3 * 152;

template <typename T, typename CT>
const void* kernel(int D, bool rh) {
  if (D == 64)
    return rh ? reinterpret_cast<const void*>(qknr::qk_grad_kernel<T, CT, 64, true>)
              : reinterpret_cast<const void*>(qknr::qk_grad_kernel<T, CT, 64, false>);
  return rh ? reinterpret_cast<const void*>(qknr::qk_grad_kernel<T, CT, 128, true>)
            : reinterpret_cast<const void*>(qknr::qk_grad_kernel<T, CT, 128, false>);
}

qknr_status check_shape(const qknr_grad_args* a) {
  if (!a) return fail(QKNR_ERR_NULL, "args is NULL");
  if (a->abi_version != QKNR_ABI_VERSION)
    return fail(QKNR_ERR_ABI, "abi_version %u, library expects %d", a->abi_version, QKNR_ABI_VERSION);
  if (a->dtype != QKNR_BF16 && a->dtype != QKNR_FP16)
    return fail(QKNR_ERR_UNSUPPORTED, "activation dtype must be BF16 or FP16");
  if (a->cos_dtype != QKNR_FP32 && a->cos_dtype != QKNR_BF16)
    return fail(QKNR_ERR_UNSUPPORTED, "cos/sin dtype must be FP32 or BF16");
  if (a->cos_layout != QKNR_COS_SHARED_ROW && a->cos_layout != QKNR_COS_PER_HEAD_EXPANDED)
    return fail(QKNR_ERR_UNSUPPORTED, "unknown cos_layout %d", a->cos_layout);
  if (a->rope_style != QKNR_ROPE_INTERLEAVED && a->rope_style != QKNR_ROPE_ROTATE_HALF)
    return fail(QKNR_ERR_UNSUPPORTED, "unknown rope_style %d", a->rope_style);
  if (a->head_dim != 64 && a->head_dim != 128)
    return fail(QKNR_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", a->head_dim);
  if (a->tokens < 0 || a->cos_rows < 0) return fail(QKNR_ERR_SHAPE, "negative tokens or cos_rows");
  if (a->n_heads_q < 0 || a->n_heads_k < 0 || a->n_heads_v < 0) return fail(QKNR_ERR_SHAPE, "negative head count");
  if (!(a->eps >= 0.0f)) return fail(QKNR_ERR_SHAPE, "eps must be >= 0");
  if (a->cos_layout == QKNR_COS_PER_HEAD_EXPANDED && a->n_heads_q > 0 && a->n_heads_k > 0 &&
      a->n_heads_q != a->n_heads_k)
    return fail(QKNR_ERR_SHAPE, "per-head expanded tables need n_heads_q == n_heads_k");
  return QKNR_OK;
}

// CTAs of the launch: a head of Q, K for every team, until the device is full.
long long ctas(const qknr_grad_args* a) {
  const long long teams = qknr::kGradThreads / (a->head_dim / 8);
  const int heads = a->n_heads_q > a->n_heads_k ? a->n_heads_q : a->n_heads_k;
  long long n = (a->tokens * (heads > 0 ? heads : 1) + teams - 1) / teams;
  if (n > kMaxCtas) n = kMaxCtas;
  return n < 1 ? 1 : n;
}

size_t workspace(const qknr_grad_args* a) {
  return a->tokens ? static_cast<size_t>(ctas(a)) * 2 * a->head_dim * 4 : 0;
}

qknr::MemSpan msp(Span s) { return qknr::MemSpan{s.lo, s.hi}; }

}  // namespace

extern "C" {

void qknr_grad_args_init(qknr_grad_args* a) {
  if (!a) return;
  memset(a, 0, sizeof(*a));
  a->abi_version = QKNR_ABI_VERSION;
  a->dtype = QKNR_BF16;
  a->eps = 1e-6f;
  a->cos_dtype = QKNR_FP32;
  a->cos_layout = QKNR_COS_SHARED_ROW;
  a->rope_style = QKNR_ROPE_INTERLEAVED;
}

size_t qknr_sizeof_grad_args(void) { return sizeof(qknr_grad_args); }

qknr_status qknr_grad_workspace_bytes(const qknr_grad_args* a, size_t* bytes) {
  if (!bytes) return fail(QKNR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  const qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  *bytes = workspace(a);
  return QKNR_OK;
}

qknr_status qknr_backward(const qknr_grad_args* a, qknr_stream_t stream) {
  qknr_status st = check_shape(a);
  if (st != QKNR_OK) return st;
  const int D = a->head_dim, es = 2, ces = a->cos_dtype == QKNR_FP32 ? 4 : 2;
  const long long T = a->tokens;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if ((reinterpret_cast<uintptr_t>(a->dgamma_q) | reinterpret_cast<uintptr_t>(a->dgamma_k) |
       reinterpret_cast<uintptr_t>(a->gamma_q) | reinterpret_cast<uintptr_t>(a->gamma_k)) & 3u)
    return fail(QKNR_ERR_ALIGN, "gamma / dgamma not 4-byte aligned");
  if (T == 0) {
    // the sum over no rows
    for (float* d : {a->n_heads_q ? a->dgamma_q : nullptr, a->n_heads_k ? a->dgamma_k : nullptr}) {
      if (!d) continue;
      const cudaError_t e = cudaMemsetAsync(d, 0, static_cast<size_t>(D) * 4, cs);
      if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaMemsetAsync(dgamma)");
    }
    return QKNR_OK;
  }

  struct Side {
    const char* name;
    const void *x, *dy;
    void* dx;
    long long xs, ds, os;
    int heads;
    const float* gamma;
    float* dgamma;
  } sides[2] = {
      {"q", a->q, a->dq, a->dq_out, a->q_stride, a->dq_stride, a->dq_out_stride, a->n_heads_q, a->gamma_q, a->dgamma_q},
      {"k", a->k, a->dk, a->dk_out, a->k_stride, a->dk_stride, a->dk_out_stride, a->n_heads_k, a->gamma_k, a->dgamma_k}};
  qknr::GradParams kp;
  memset(&kp, 0, sizeof(kp));
  const bool expanded = a->cos_layout == QKNR_COS_PER_HEAD_EXPANDED;
  const int heads = a->n_heads_q > a->n_heads_k ? a->n_heads_q : a->n_heads_k;
  const long long cos_rows = a->cos_rows ? a->cos_rows : T;
  const long long table_row = heads ? (long long)(expanded ? heads : 1) * D * ces : 0;
  if (heads > 0 && (!a->cos || !a->sin)) return fail(QKNR_ERR_NULL, "cos and sin are required");
  if (heads > 0 && (!aligned16(a->cos) || !aligned16(a->sin)))
    return fail(QKNR_ERR_ALIGN, "cos / sin not 16-byte aligned");
  RowSpan ins[8];
  Span outs[3];
  int n_in = 0, n_out = 0;
  struct {
    RowSpan out, own;
    bool same;
  } grads[3];
  int n_grads = 0;
  auto flat = [](Span s) { return RowSpan{s, 0, 0}; };   // meets whatever its span meets
  for (int i = 0; i < 2; ++i) {
    Side& s = sides[i];
    qknr::GradSide& k = kp.side[i];
    if (s.heads == 0) continue;
    const long long row = (long long)s.heads * D;
    if (!s.x || !s.dy || !s.gamma)
      return fail(QKNR_ERR_NULL, "%s, d%s and gamma_%s are required when n_heads_%s > 0", s.name, s.name, s.name, s.name);
    void* dx = s.dx ? s.dx : const_cast<void*>(s.dy);
    const long long xs = s.xs ? s.xs : row, ds = s.ds ? s.ds : row, os = s.os ? s.os : ds;
    if (xs < row || ds < row || os < row)
      return fail(QKNR_ERR_SHAPE, "a stride of %s is smaller than n_heads_%s * head_dim", s.name, s.name);
    if (!aligned16(s.x) || !aligned16(s.dy) || !aligned16(dx) || (xs * es) % 16 || (ds * es) % 16 || (os * es) % 16)
      return fail(QKNR_ERR_ALIGN, "%s / d%s / d%s_out base or row stride not 16-byte aligned", s.name, s.name, s.name);
    const Span sx = span_of(s.x, T, xs * es, row * es), sd = span_of(s.dy, T, ds * es, row * es);
    const Span so = span_of(dx, T, os * es, row * es), sg = span_of(s.gamma, 1, 0, (long long)D * 4);
    k = qknr::GradSide{static_cast<const char*>(s.x), static_cast<const char*>(s.dy), static_cast<char*>(dx), xs * es,
                       ds * es, os * es, s.gamma, s.heads, msp(sx), msp(sd), msp(so), msp(sg)};
    ins[n_in++] = RowSpan{sx, xs * es, row * es};
    ins[n_in++] = flat(sg);
    grads[n_grads++] = {RowSpan{so, os * es, row * es}, RowSpan{sd, ds * es, row * es}, dx == s.dy && os == ds};
    if (s.dgamma) outs[n_out++] = span_of(s.dgamma, 1, 0, (long long)D * 4);
  }
  const long long vrow = (long long)a->n_heads_v * D;
  const long long vs = a->dv_stride ? a->dv_stride : vrow, vos = a->dv_out_stride ? a->dv_out_stride : vs;
  const bool copy_v = a->n_heads_v > 0 && a->dv_out && !(a->dv_out == a->dv && vos == vs);
  if (copy_v) {
    if (!a->dv) return fail(QKNR_ERR_NULL, "dv is required to copy it into dv_out");
    if (vs < vrow || vos < vrow) return fail(QKNR_ERR_SHAPE, "a stride of dv is too small");
    if (!aligned16(a->dv) || !aligned16(a->dv_out) || (vs * es) % 16 || (vos * es) % 16)
      return fail(QKNR_ERR_ALIGN, "dv / dv_out base or row stride not 16-byte aligned");
    const Span si = span_of(a->dv, T, vs * es, vrow * es), so = span_of(a->dv_out, T, vos * es, vrow * es);
    kp.dv = static_cast<const char*>(a->dv);
    kp.dv_out = static_cast<char*>(a->dv_out);
    kp.dv_stride = vs * es;
    kp.dv_out_stride = vos * es;
    kp.v_chunks = static_cast<int>(vrow * es / 16);
    kp.sp_dv = msp(si);
    kp.sp_dv_out = msp(so);
    grads[n_grads++] = {RowSpan{so, vos * es, vrow * es}, RowSpan{si, vs * es, vrow * es}, false};
  }
  const size_t need = workspace(a);
  const Span sk = span_of(a->workspace, 1, 0, static_cast<long long>(need));
  const Span sc = span_of(a->cos, heads ? cos_rows : 0, table_row, table_row);
  const Span ss = span_of(a->sin, heads ? cos_rows : 0, table_row, table_row);
  if (!a->workspace) return fail(QKNR_ERR_NULL, "workspace is required");
  if (a->workspace_bytes < need)
    return fail(QKNR_ERR_SHAPE, "workspace of %zu bytes, %zu needed", a->workspace_bytes, need);
  if (!aligned16(a->workspace)) return fail(QKNR_ERR_ALIGN, "workspace not 16-byte aligned");
  ins[n_in++] = flat(sc);
  ins[n_in++] = flat(ss);
  outs[n_out++] = sk;
  for (int i = 0; i < n_grads; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (rows_overlap(grads[i].out, ins[j])) return fail(QKNR_ERR_OVERLAP, "a gradient output overlaps an input");
    for (int j = 0; j < n_grads; ++j) {
      if ((j != i || !grads[i].same) && rows_overlap(grads[i].out, grads[j].own))
        return fail(QKNR_ERR_OVERLAP, "a gradient output overlaps an incoming gradient without being in place");
      if (j < i && rows_overlap(grads[i].out, grads[j].out)) return fail(QKNR_ERR_OVERLAP, "two gradient outputs overlap");
    }
  }
  for (int i = 0; i < n_out; ++i) {
    const RowSpan out = flat(outs[i]);
    for (int j = 0; j < n_in; ++j)
      if (rows_overlap(out, ins[j])) return fail(QKNR_ERR_OVERLAP, "dgamma or the workspace overlaps an input");
    for (int j = 0; j < n_grads; ++j)
      if (rows_overlap(out, grads[j].out) || rows_overlap(out, grads[j].own))
        return fail(QKNR_ERR_OVERLAP, "dgamma or the workspace overlaps a gradient");
    for (int j = 0; j < i; ++j)
      if (qknr_host::overlaps(outs[i], outs[j])) return fail(QKNR_ERR_OVERLAP, "two outputs overlap");
  }
  if (heads == 0 && !copy_v) return QKNR_OK;

  kp.tokens = T;
  kp.cos_rows = cos_rows;
  kp.cos = static_cast<const char*>(a->cos);
  kp.sin = static_cast<const char*>(a->sin);
  kp.table_stride = table_row;
  kp.head_stride = expanded ? D * ces : 0;
  kp.parts = static_cast<float*>(a->workspace);
  kp.eps = a->eps;
  kp.inv_d = 1.0f / static_cast<float>(D);
  kp.status = a->dev_status;
  kp.sp_cos = msp(sc);
  kp.sp_sin = msp(ss);
  kp.sp_ws = msp(sk);

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaGetDevice");
  qknr_host::DeviceInfo di;
  st = qknr_host::device_info(dev, &di);
  if (st != QKNR_OK) return st;
  const bool rh = a->rope_style == QKNR_ROPE_ROTATE_HALF, bt = a->cos_dtype == QKNR_BF16;
  const void* fn = a->dtype == QKNR_BF16
                       ? (bt ? kernel<__nv_bfloat16, __nv_bfloat16>(D, rh) : kernel<__nv_bfloat16, float>(D, rh))
                       : (bt ? kernel<__half, __nv_bfloat16>(D, rh) : kernel<__half, float>(D, rh));
  const bool overlap = !(a->flags & QKNR_FLAG_NO_OVERLAP);
  const long long n = ctas(a);
  void* kargs[] = {&kp};
  int regs = 0;
  st = qknr_host::configure_kernel(fn, dev, di, &regs);
  if (st != QKNR_OK) return st;
  st = qknr_host::launch_kernel(fn, static_cast<int>(n), qknr::kGradThreads, qknr::kGradSmem, cs, kargs, overlap,
                                "cudaLaunchKernelExC(QK backward)");
  if (st != QKNR_OK || (!a->dgamma_q && !a->dgamma_k)) return st;
  qknr::PartsParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.sums = 2;
  pp.parts = kp.parts;
  pp.out[0] = a->n_heads_q ? a->dgamma_q : nullptr;
  pp.out[1] = a->n_heads_k ? a->dgamma_k : nullptr;
  pp.cols = D;
  pp.units = n;
  pp.sp_parts = kp.sp_ws;
  pp.sp_out[0] = msp(span_of(pp.out[0], 1, 0, (long long)D * 4));
  pp.sp_out[1] = msp(span_of(pp.out[1], 1, 0, (long long)D * 4));
  pp.status = a->dev_status;
  void* pargs[] = {&pp};
  return qknr_host::launch_kernel(reinterpret_cast<const void*>(qknr::parts_kernel),
                                  static_cast<int>(qknr::parts_grid(pp, 1)), 32 * qknr::kPartsRows, 0, cs,
                                  pargs, overlap, "cudaLaunchKernelExC(dgamma)");
}

}  // extern "C"
