// C-ABI launchers of attention and its backward pass: validation, tensor
// maps, launch planning and the launches.  No allocation, no synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "../../include/qknr_attn.h"
#include "attn_few.cuh"
#include "attn_kernel.cuh"
#include "qknr_host.h"

namespace {

using qknr_host::aligned16;
using qknr_host::fail;
using qknr_host::Span;
using qknr_host::span_of;

qknr::MemSpan msp(Span s) { return qknr::MemSpan{s.lo, s.hi}; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor map encoder, looked up once.
qknr_status encoder(EncodeFn* out) {
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
qknr_status make_map(CUtensorMap* map, const qknr_attn_args* a, const void* base, long long stride, int seq, int heads,
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

qknr_status check_shape(const qknr_attn_args* a) {
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
qknr_status check_rows(const qknr_attn_args* a, Rows* r) {
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

qknr_host::RowSpan row_span(const qknr_attn_args* a, const Rows& r) {
  return qknr_host::RowSpan{r.span, r.stride * 2, 2LL * r.heads * a->head_dim};
}

// Outputs may interleave with inputs and with each other (column views of one
// packed buffer); `flat_outs` and `flat_ins` are the spans of what has no rows.
qknr_status check_overlap(const qknr_attn_args* a, std::initializer_list<const Rows*> outs,
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

qknr_status check_workspace(const qknr_attn_args* a, size_t need) {
  if (need == 0) return QKNR_OK;
  if (!a->workspace) return fail(QKNR_ERR_NULL, "workspace is required");
  if (a->workspace_bytes < need)
    return fail(QKNR_ERR_SHAPE, "workspace of %zu bytes, %zu needed", a->workspace_bytes, need);
  if (!aligned16(a->workspace)) return fail(QKNR_ERR_ALIGN, "workspace not 16-byte aligned");
  return QKNR_OK;
}

// What both passes share, once the shapes are known to be good.
qknr_status common(const qknr_attn_args* a, qknr::AttnParams* kp) {
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

size_t delta_bytes(const qknr_attn_args* a) {
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
Cut cut_tiles(const qknr_attn_args* a, int seq, int heads, int rows, long long blocks, int slot_rows, bool stats) {
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
  // on 4 heads x 64: 147 us, 189 with the rest shared out); or all as two
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

long long blocks_of(int seq) { return (static_cast<long long>(seq) + qknr::kTile - 1) / qknr::kTile; }

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

void apply(const Cut& c, qknr::AttnParams* kp, void* part) {
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

qknr_status launch(const void* fn, long long grid, int block, int smem, const qknr_attn_args* a, qknr::AttnParams* kp,
                   int dev, const qknr_host::DeviceInfo& di, qknr_stream_t stream, const char* what) {
  int regs = 0;
  const qknr_status st = qknr_host::configure_kernel(fn, dev, di, &regs);
  if (st != QKNR_OK) return st;
  void* kargs[] = {kp};
  return qknr_host::launch_kernel(fn, static_cast<int>(grid), block, smem, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
}

// The kernel that joins partial results: a warp per row of the tiles shared out.
qknr_status join(const void* fn, const Cut& c, int rows, const qknr_attn_args* a, qknr::AttnParams* kp, qknr_stream_t stream,
                 const char* what) {
  const long long cut = c.halves ? c.total : c.rem;
  if (cut == 0) return QKNR_OK;
  int ctas = c.ctas;
  void* kargs[] = {kp, &ctas};
  return qknr_host::launch_kernel(fn, static_cast<int>((cut * rows + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(stream), kargs,
                                  !(a->flags & QKNR_FLAG_NO_OVERLAP), what);
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

qknr_status device(int* dev, qknr_host::DeviceInfo* di) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return qknr_host::cuda_fail(e, "cudaGetDevice");
  return qknr_host::device_info(*dev, di);
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
