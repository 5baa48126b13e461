// Host side of the attention launchers: validation, tensor maps, how tiles go
// to CTAs, the launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "../../include/qknr_attn.h"
#include "attn_kernel.cuh"
#include "qknr_host.h"

namespace qknr_attn {

using qknr_host::aligned16;
using qknr_host::fail;
using qknr_host::Span;
using qknr_host::span_of;

inline qknr::MemSpan msp(Span s) { return qknr::MemSpan{s.lo, s.hi}; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor map encoder, looked up once.
inline qknr_status encoder(EncodeFn* out) {
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaGetDriverEntryPointByVersion");
    if (found != cudaDriverEntryPointSuccess || !sym)
      return fail(QKNR_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    fn = reinterpret_cast<EncodeFn>(sym);
    known.store(fn, std::memory_order_relaxed);
  }
  *out = fn;
  return QKNR_OK;
}

// Token rows as [batch][heads][D/64][rows][64], boxes of `box_rows` rows of
// one head, all its columns or `cols` of 64.  Rows past the sequence read as
// zero and are not written.
inline qknr_status make_map(CUtensorMap* map, const qknr_attn_args* a, const void* base, long long stride, int seq, int heads,
                     int box_rows = qknr::kTile, int cols = 0) {
  EncodeFn enc;
  const qknr_status st = encoder(&enc);
  if (st != QKNR_OK) return st;
  const cuuint64_t D = a->head_dim, row = static_cast<cuuint64_t>(stride) * 2;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(seq), D / 64, static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(a->batch)};
  const cuuint64_t strides[4] = {row, 128, D * 2, row * seq};
  const cuuint32_t box[5] = {cols ? static_cast<cuuint32_t>(cols) : 64, static_cast<cuuint32_t>(box_rows),
                             cols ? 1 : static_cast<cuuint32_t>(D / 64), 1, 1},
                   ones[5] = {1, 1, 1, 1, 1};
  const CUresult r = enc(map, a->dtype == QKNR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         5, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(QKNR_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
  return QKNR_OK;
}

inline qknr_status check_shape(const qknr_attn_args* a) {
  if (!a) return fail(QKNR_ERR_NULL, "args is NULL");
  if (a->abi_version != QKNR_ABI_VERSION)
    return fail(QKNR_ERR_ABI, "abi_version %u, library expects %d", a->abi_version, QKNR_ABI_VERSION);
  if (a->dtype != QKNR_BF16 && a->dtype != QKNR_FP16)
    return fail(QKNR_ERR_UNSUPPORTED, "activation dtype must be BF16 or FP16");
  if (a->head_dim != 64 && a->head_dim != 128)
    return fail(QKNR_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", a->head_dim);
  if (a->batch < 0 || a->seq_q < 0 || a->seq_k < 0) return fail(QKNR_ERR_SHAPE, "negative batch or sequence");
  if (a->n_heads_q < 1 || a->n_heads_k < 1 || a->n_heads_q % a->n_heads_k)
    return fail(QKNR_ERR_SHAPE, "n_heads_q %d must be a positive multiple of n_heads_k %d", a->n_heads_q, a->n_heads_k);
  if (a->scale != 0.0f && !(a->scale > 0.0f && std::isfinite(a->scale)))
    return fail(QKNR_ERR_SHAPE, "scale must be positive (0: 1 / sqrt(head_dim))");
  const long long q_tiles = (a->seq_q + 127LL) / 128, k_tiles = (a->seq_k + 127LL) / 128;
  if (q_tiles * a->n_heads_q * a->batch > 0x7fffffffLL || k_tiles * a->n_heads_k * a->batch > 0x7fffffffLL ||
      static_cast<long long>(a->seq_q) * a->batch > 0x7fffffffLL || static_cast<long long>(a->seq_k) * a->batch > 0x7fffffffLL)
    return fail(QKNR_ERR_UNSUPPORTED, "more than 2^31 rows or tiles");
  return QKNR_OK;
}

struct Rows {                 // a tensor of token rows
  const char* name;
  const void* base;
  long long stride;           // elements
  int seq, heads;
  Span span;
};

// Fills in the default stride and checks one tensor.  A NULL base is an
// error unless the tensor has no rows.
inline qknr_status check_rows(const qknr_attn_args* a, Rows* r) {
  const long long width = static_cast<long long>(r->heads) * a->head_dim, n = static_cast<long long>(a->batch) * r->seq;
  if (r->stride == 0) r->stride = width;
  if (r->stride < width) return fail(QKNR_ERR_SHAPE, "%s_stride is smaller than heads * head_dim", r->name);
  if (r->stride >= (1LL << 31)) return fail(QKNR_ERR_UNSUPPORTED, "%s_stride of 2^31 elements or more", r->name);
  if ((r->stride * 2) % 16 || !aligned16(r->base))
    return fail(QKNR_ERR_ALIGN, "%s base or row stride not 16-byte aligned", r->name);
  if (n > 0 && !r->base) return fail(QKNR_ERR_NULL, "%s is required", r->name);
  r->span = span_of(r->base, n, r->stride * 2, width * 2);
  return QKNR_OK;
}

inline qknr_host::RowSpan row_span(const qknr_attn_args* a, const Rows& r) {
  return qknr_host::RowSpan{r.span, r.stride * 2, 2LL * r.heads * a->head_dim};
}

// Outputs may interleave with inputs and with each other (column views of one
// packed buffer); `flat_outs` and `flat_ins` are the spans of what has no rows.
inline qknr_status check_overlap(const qknr_attn_args* a, std::initializer_list<const Rows*> outs,
                          std::initializer_list<const Rows*> ins, std::initializer_list<Span> flat_outs,
                          std::initializer_list<Span> flat_ins) {
  for (const Rows* o : outs) {
    for (const Rows* i : ins)
      if (qknr_host::rows_overlap(row_span(a, *o), row_span(a, *i)))
        return fail(QKNR_ERR_OVERLAP, "%s overlaps %s", o->name, i->name);
    for (const Rows* p : outs)
      if (p != o && qknr_host::rows_overlap(row_span(a, *o), row_span(a, *p)))
        return fail(QKNR_ERR_OVERLAP, "%s overlaps %s", o->name, p->name);
    for (const Span& s : flat_ins)
      if (qknr_host::overlaps(o->span, s)) return fail(QKNR_ERR_OVERLAP, "%s overlaps lse or the lengths", o->name);
  }
  for (const Span& f : flat_outs) {
    for (const Rows* r : ins)
      if (qknr_host::overlaps(f, r->span)) return fail(QKNR_ERR_OVERLAP, "%s overlaps lse or the workspace", r->name);
    for (const Rows* r : outs)
      if (qknr_host::overlaps(f, r->span)) return fail(QKNR_ERR_OVERLAP, "%s overlaps lse or the workspace", r->name);
    for (const Span& s : flat_ins)
      if (qknr_host::overlaps(f, s)) return fail(QKNR_ERR_OVERLAP, "lse, the lengths and the workspace overlap");
  }
  return QKNR_OK;
}

inline qknr_status check_workspace(const qknr_attn_args* a, size_t need) {
  if (need == 0) return QKNR_OK;
  if (!a->workspace) return fail(QKNR_ERR_NULL, "workspace is required");
  if (a->workspace_bytes < need)
    return fail(QKNR_ERR_SHAPE, "workspace of %zu bytes, %zu needed", a->workspace_bytes, need);
  if (!aligned16(a->workspace)) return fail(QKNR_ERR_ALIGN, "workspace not 16-byte aligned");
  return QKNR_OK;
}

// What both passes share, once the shapes are known to be good.
inline qknr_status common(const qknr_attn_args* a, qknr::AttnParams* kp) {
  if ((reinterpret_cast<uintptr_t>(a->lse) | reinterpret_cast<uintptr_t>(a->q_lens) | reinterpret_cast<uintptr_t>(a->k_lens)) & 3u)
    return fail(QKNR_ERR_ALIGN, "lse, q_lens or k_lens not 4-byte aligned");
  kp->batch = a->batch;
  kp->seq_q = a->seq_q;
  kp->seq_k = a->seq_k;
  kp->heads_q = a->n_heads_q;
  kp->heads_k = a->n_heads_k;
  kp->group = a->n_heads_q / a->n_heads_k;
  kp->causal = a->causal != 0;
  kp->scale = a->scale != 0.0f ? a->scale : 1.0f / std::sqrt(static_cast<float>(a->head_dim));
  kp->scale_log2 = kp->scale * qknr::kLog2e;
  kp->lse = a->lse;
  kp->q_lens = a->q_lens;
  kp->k_lens = a->k_lens;
  kp->flags = a->flags;
  kp->status = a->dev_status;
  kp->wait_limit_ns = a->wait_limit_ns ? a->wait_limit_ns : 2000000000ull;
  const long long n_lse = static_cast<long long>(a->batch) * a->n_heads_q * a->seq_q;
  kp->sp_lse = msp(span_of(a->lse, n_lse, 4, 4));
  kp->sp_q_lens = msp(span_of(a->q_lens, a->batch, 4, 4));
  kp->sp_k_lens = msp(span_of(a->k_lens, a->batch, 4, 4));
  return QKNR_OK;
}

inline size_t delta_bytes(const qknr_attn_args* a) {
  return (static_cast<size_t>(a->batch) * a->n_heads_q * a->seq_q * 4 + 15) / 16 * 16;
}

// How a kernel's tiles go to the CTAs, one on each SM of a GB300 (nothing here
// needs a device; on fewer SMs CTAs queue up, none waits for another).
constexpr int kCtas = 152;

struct Cut {
  int tiles = 0, total = 0, ctas = 0, halves = 0, waves = 0, rem = 0;
  size_t part_bytes = 0, stats_bytes = 0;
};

// `rows`: rows of a tile; `blocks`: its iterations at most; `slot_rows`: fp32
// rows of a partial result.
inline Cut cut_tiles(const qknr_attn_args* a, int seq, int heads, int rows, long long blocks, int slot_rows, bool stats) {
  Cut c;
  c.tiles = (seq + rows - 1) / rows;
  const long long total = static_cast<long long>(c.tiles) * heads * a->batch;
  c.total = static_cast<int>(total);
  c.ctas = kCtas;
  c.waves = static_cast<int>(total / c.ctas);
  c.rem = static_cast<int>(total % c.ctas);
  auto buffers = [&](long long slots) {
    c.part_bytes = static_cast<size_t>(slots) * slot_rows * a->head_dim * 4;
    c.stats_bytes = stats ? static_cast<size_t>(slots) * slot_rows * 8 : 0;
  };
  // A causal mask's tiles cost 1 to `blocks` iterations, so that equal shares
  // of the cheap ones left over gain nothing.  They go out whole, the costly
  // ones first, every other wave the other way round (backward of 3 x 1999 x 16
  // on 4 heads x 64: 133 us, 169 with the rest shared out); or all as two
  // halves, where a costly one alone takes longer than an even spread would:
  // by more than the 32 iterations that partial results of all tiles cost
  // (backward of 8192 x 24 on 3 heads x 128: 189 more, 980 against 1136 us;
  // forward of 8192 x 6 x 128: 24 more, 101 against 98), or by any where fewer
  // tiles than CTAs are cut anyway (backward of 4096 x 4 x 128: 81 against 91).
  const long long spread = total * blocks / (2 * c.ctas), half = blocks / 2 > spread ? blocks / 2 : spread;
  const long long other = c.waves > 0 ? blocks : blocks * total / c.ctas;
  if (a->causal && other - half > (c.waves > 0 ? 32 : 2)) {
    c.halves = 1;
    c.waves = static_cast<int>((2 * total + c.ctas - 1) / c.ctas);
    c.rem = 0;
    buffers(2 * total);
    return c;
  }
  if (c.rem == 0) return c;
  // Sharing the last tiles out saves most of a tile's time and costs the
  // partial results and a kernel that joins them, about as much as six
  // iterations at head_dim 128, twelve at 64.
  const long long cost = a->head_dim == 128 ? 6 : 12;
  const bool even = !(a->causal && c.waves > 0);
  if (even && blocks * (c.ctas - c.rem) > cost * c.ctas) {
    if (c.waves == 0) {
      // no smaller shares than two iterations
      const long long most = c.rem * blocks / 2;
      if (most < c.ctas) c.ctas = static_cast<int>(most > c.rem ? most : c.rem);
    }
    if (c.ctas > c.rem) {
      buffers(2 * c.ctas);
      return c;
    }
  }
  if (c.waves == 0) c.ctas = c.rem;
  ++c.waves;
  c.rem = 0;
  return c;
}

inline long long blocks_of(int seq) { return (static_cast<long long>(seq) + qknr::kTile - 1) / qknr::kTile; }

inline void apply(const Cut& c, qknr::AttnParams* kp, void* part) {
  kp->tiles = c.tiles;
  kp->total = c.total;
  kp->halves = c.halves;
  kp->waves = c.waves;
  kp->rem = c.rem;
  kp->part = static_cast<float*>(part);
  kp->stats = reinterpret_cast<float*>(static_cast<char*>(part) + c.part_bytes);
  kp->sp_part = msp(span_of(part, 1, 0, static_cast<long long>(c.part_bytes)));
  kp->sp_stats = msp(span_of(kp->stats, 1, 0, static_cast<long long>(c.stats_bytes)));
}

inline qknr_status launch(const void* fn, long long grid, int block, int smem, const qknr_attn_args* a, qknr::AttnParams* kp,
                   int dev, const qknr_host::DeviceInfo& di, qknr_stream_t stream, const char* what) {
  int regs = 0;
  const qknr_status st = qknr_host::configure_kernel(fn, dev, di, &regs);
  if (st != QKNR_OK) return st;
  void* kargs[] = {kp};
  return qknr_host::launch_kernel(fn, static_cast<int>(grid), block, smem, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
}

// The kernel that joins partial results: a warp per row of the tiles shared out.
inline qknr_status join(const void* fn, const Cut& c, int rows, const qknr_attn_args* a, qknr::AttnParams* kp, qknr_stream_t stream,
                 const char* what) {
  const long long cut = c.halves ? c.total : c.rem;
  if (cut == 0) return QKNR_OK;
  int ctas = c.ctas;
  void* kargs[] = {kp, &ctas};
  return qknr_host::launch_kernel(fn, static_cast<int>((cut * rows + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
}

inline qknr_status device(int* dev, qknr_host::DeviceInfo* di) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaGetDevice");
  return qknr_host::device_info(*dev, di);
}

}  // namespace qknr_attn
