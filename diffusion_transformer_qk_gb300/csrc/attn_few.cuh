// Attention of a few queries (a pooling token, a step of decoding) over many
// keys for sm_103a (formulas: qknr_attn.h).
//
// Bound by HBM: every key and value is read once, for up to 16 of the group *
// seq_q queries of a key head together.  A 256-row tile of attn_kernel.cuh
// would be almost empty and its CTA waits for its own softmax between two
// loads; here the warps run independently, each over 16 (head_dim 64: 32) keys
// at a time, which TMA brings to a ring of its own.  The products are warp-wide
// MMAs of 16 rows: the contraction's order is free, so a lane's 16 bytes of a
// key serve as two k-steps of Q K^T; and a lane's 16 bytes of four values,
// pairs of keys swapped together, as eight column tiles of P V.  A warp keeps
// the running maximum, sum and accumulator of each row; a CTA's warps join in
// order through shared memory, and CTAs share a key head's keys like the tiles'
// contraction in attn_kernel.cuh.
//
// 8 x 4096 keys of 24 heads x 128: 70 us for 1 to 8 rows (5.8 TB/s), 72 for 16;
// head_dim 64: 41 and 43.  Plain FMAs take 65 us for one row, but 79 for two
// and 132 for four; the same MMAs fed by loads to registers 75 us, by 16-byte
// asynchronous copies 85.
#pragma once

#include "attn_kernel.cuh"

namespace qknr {

// Keys of a warp's step: 8 KB of keys and values.
__host__ __device__ constexpr int few_keys(int d) { return 2048 / d; }
// Up to 8 rows: 12 warps with 168 registers a thread; up to 16: 8 with 255.
__host__ __device__ constexpr int few_warps(int rows) { return rows <= 8 ? 12 : 8; }
// Steps in flight: 192 KB of keys and values per SM.
__host__ __device__ constexpr int few_step_bytes(int d) { return 2 * few_keys(d) * d * 2; }
__host__ __device__ constexpr int few_stages(int rows, int d) { return 196608 / (few_warps(rows) * few_step_bytes(d)); }
// [warps][stages] steps, in whose place [warps] [rows][D] sums come after a
// key head's last step; [warps][rows] (maximum, sum); [warps][stages] barriers
__host__ __device__ constexpr int few_ring_bytes(int rows, int d) { return few_stages(rows, d) * few_step_bytes(d); }
__host__ __device__ constexpr int few_smem(int rows, int d) {
  return few_warps(rows) * (few_ring_bytes(rows, d) + rows * 8 + few_stages(rows, d) * 8) + 16;
}

// PLANNED: the table of sequences, and where the CTA's share of them begins and
// ends, behind that
__host__ __device__ constexpr int few_table(int rows, int d) { return (few_smem(rows, d) + 15) / 16 * 16; }
__host__ __device__ constexpr int few_planned_smem(int rows, int d) { return few_table(rows, d) + static_cast<int>(sizeof(AttnTable)) + 16; }

template <typename T>
__device__ __forceinline__ void few_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void few_mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void few_mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// H halves of 8 rows.  Lane (g, t) = (lane / 4, lane % 4) owns rows g and, with
// two halves, g + 8; of their accumulators columns 64 cc + 16 t + 0 .. 15.
// PLANNED: tiles of p.few_rows rows from the plan.  The warps form groups of
// p.few_group, each on a tile of its own: over a few hundred keys a tile's
// beginning and end take longer than its steps (64 samples of 512 keys of 8 heads x
// 128 beside their prefix of 8190: 77 us with all twelve warps on a tile, 59 with
// three).
template <typename T, int D, int H, bool PLANNED = false>
__global__ void __launch_bounds__(32 * few_warps(8 * H), 1) attn_few_kernel(const __grid_constant__ AttnParams p) {
  constexpr int ROWS = 8 * H, WARPS = few_warps(ROWS), KC = D / 32, VC = D / 64, STAGES = few_stages(ROWS, D);
  constexpr int kKeys = few_keys(D), KT = kKeys / 8;
  constexpr int kRing = few_ring_bytes(ROWS, D), kStep = few_step_bytes(D);
  static_assert(STAGES >= 2 && ROWS * D * 4 <= kRing, "a warp's share of shared memory");
  extern __shared__ __align__(1024) unsigned char smem[];
  auto sums = [&](int warp, int row) { return reinterpret_cast<float*>(smem + warp * kRing) + row * D; };
  float2(*stats)[ROWS] = reinterpret_cast<float2(*)[ROWS]>(smem + WARPS * kRing);   // (maximum, sum)
  unsigned char* ctl = smem + WARPS * (kRing + ROWS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * WARPS * STAGES);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, slot_rows = PLANNED ? p.few_rows : min(p.group * p.seq_q, kFewRows);
  const unsigned char* ring = smem + warp * kRing;
  // the warp's barriers
  const AttnCta cta{smem, smem_addr(ring), smem_addr(ctl) + 8 * warp * STAGES, abort_flag, p.status, p.wait_limit_ns, warp, lane};
  if (threadIdx.x == 0) {
    for (int i = 0; i < WARPS * STAGES; ++i) mbar_init(smem_addr(ctl) + 8 * i, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const bool beside = PLANNED && p.beside;
  if (!beside) grid_dependency_wait();
  grid_dependents_launch();
  AttnTable& table = *reinterpret_cast<AttnTable*>(smem + few_table(ROWS, D));
  int2* share = reinterpret_cast<int2*>(smem + few_table(ROWS, D) + sizeof(AttnTable));
  if (PLANNED && (p.from == kFromTable || p.from == kFromShares)) {
    if (warp == 0) plan_table(p.seqs, table, lane, p.status);
    __syncthreads();
    if (p.from == kFromShares) {
      if (threadIdx.x < 2) {
        const int c = static_cast<int>(blockIdx.x + threadIdx.x), ctas = static_cast<int>(gridDim.x);
        share[threadIdx.x] = table_span(table, p.seqs, p.least, ctas, c);
        // for the join: where the share begins (the last CTA: and ends)
        if ((threadIdx.x == 0 || c == ctas) && in_span(p.plan.spans + c, 8, p.plan.sp, p.status))
          p.plan.spans[c] = share[threadIdx.x];
      }
      __syncthreads();
    }
  }
  const int group = PLANNED ? p.few_group : WARPS, grp = PLANNED ? warp / group : 0, gw = warp - grp * group;
  const int groups = PLANNED ? WARPS / group : 1;
  RingPos<STAGES> at;         // the next step to read
  bool ok = true;
  AttnWork w;
  AttnPiece piece;
  for (int s = grp; ok && (PLANNED ? attn_piece<true>(p, table, share, s, piece) : attn_work(p, s, w)); s += groups) {
    // rows row0 + r, r < rows, of key head hk: query (row0 + r) % queries of head (row0 + r) / queries of its group
    int b, hk, row0, rows, q_len, k_len, queries;
    if (PLANNED) {
      b = 0;
      hk = piece.h;
      row0 = piece.t0;
      q_len = piece.q_len;
      queries = q_len > 0 ? q_len : 1;
      k_len = piece.k_len;
      rows = min(p.group * q_len - row0, p.few_rows);
      w.slot = piece.slot;
      if (p.from == kFromShares && gw == 0 && lane == 0 && w.slot == 2 * static_cast<int>(blockIdx.x) + 1) {
        // for the join: a tile that others end
        int4* at = p.plan.items + 2LL * blockIdx.x;
        if (in_span(at, 32, p.plan.sp, p.status)) {
          at[0] = make_int4(piece.q_row, piece.q_len, piece.k_row, piece.k_len);
          at[1] = make_int4(piece.t0, piece.h, 0, 0);
        }
      }
    } else {
      const int key_head = w.tile / p.tiles;
      b = key_head / p.heads_k;
      hk = key_head - b * p.heads_k;
      row0 = (w.tile - key_head * p.tiles) * kFewRows;
      queries = p.seq_q;
      rows = min(p.group * queries - row0, kFewRows);
      q_len = clamp_len(p.q_lens, b, p.seq_q, p.sp_q_lens, p.status);
      k_len = clamp_len(p.k_lens, b, p.seq_k, p.sp_k_lens, p.status);
    }
    const int q_row = PLANNED ? piece.q_row : 0, k_row = PLANNED ? piece.k_row : 0;
    // keys [0, limit) are seen; the last query sees the most
    const int n = q_len > 0 ? k_len : 0;
    int limit[H];
    uint4 q[H][KC];
    float m[H], l[H], acc[VC][8][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int r = g + 8 * h, i = (row0 + r) % queries, head = hk * p.group + (row0 + r) / queries;
      const bool mine = r < rows && i < q_len;
      m[h] = -INFINITY;
      l[h] = 0.0f;
      limit[h] = mine ? (p.causal ? min(max(i + k_len - q_len + 1, 0), k_len) : k_len) : 0;
      const char* src = p.q_in + (static_cast<long long>(b) * p.seq_q + q_row + i) * p.q_stride + head * (D * 2) + t * 32;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        q[h][c] = make_uint4(0, 0, 0, 0);
        const char* piece = src + (c >> 1) * 128 + (c & 1) * 16;
        if (mine && in_span(piece, 16, p.sp_q, p.status)) q[h][c] = *reinterpret_cast<const uint4*>(piece);
      }
    }
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][j][e] = 0.0f;
    int begin, end;
    if (PLANNED) {
      begin = min(piece.u0 * kTile, n);
      end = min(piece.u1 * kTile, n);
    } else {
      attn_cut(w, n, begin, end);
    }
    // lane 0: the next step's keys and values into the stage after those in flight
    const int kHop = group * kKeys;
    int ahead = begin + gw * kKeys, in_flight = 0;
    int put = at.s;
    auto fetch = [&]() {
      if (ahead >= end || (p.flags & 1u)) return;             // test only: issue nothing
      const uint32_t bar = cta.bar(put), dst = cta.base + put * kStep;
      mbar_arrive_expect_tx(bar, kStep);
      tma_load_tile(dst, &p.map_k, k_row + ahead, hk, b, bar);
      tma_load_tile(dst + kStep / 2, &p.map_v, k_row + ahead, hk, b, bar);
      put = put + 1 == STAGES ? 0 : put + 1;
      ahead += kHop;
      ++in_flight;
    };
    if (lane == 0)
      for (int i = 0; i < STAGES; ++i) fetch();
#pragma unroll 1
    for (int k0 = begin + gw * kKeys; k0 < end; k0 += kHop) {
      ok = cta.wait(at.s, at.phase);
      if (!ok) break;
      const unsigned char* in = ring + at.s * kStep;
      // scores of keys k0 + 8 i + 2t, + 1: [0], [1] of row g, [2], [3] of row g + 8
      float sc[KT][4];
#pragma unroll
      for (int i = 0; i < KT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 other = H > 1 ? q[H - 1][c] : make_uint4(0, 0, 0, 0);
          const uint32_t lo[4] = {q[0][c].x, other.x, q[0][c].y, other.y}, hi[4] = {q[0][c].z, other.z, q[0][c].w, other.w};
          // row 8 i + g, chunk 2 t + (c & 1) of its half
          const uint4 kr = *reinterpret_cast<const uint4*>(in + (c >> 1) * (kKeys * 128) + (8 * i + g) * 128 +
                                                           (((2 * t + (c & 1)) ^ g) << 4));
          few_mma<T>(sc[i], lo, kr.x, kr.y);
          few_mma<T>(sc[i], hi, kr.z, kr.w);
        }
      }
      uint32_t pr[KT / 2][4] = {};
      float old[H];
      bool raised = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float top = m[h];
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[i][2 * h + e];
            const int key = k0 + 8 * i + 2 * t + e;
            if (key >= end || key >= limit[h]) x = -INFINITY;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float base = top == -INFINITY ? 0.0f : top;   // no key so far: every p is zero
        old[h] = exp2_approx(__fmul_rn(__fsub_rn(m[h], base), p.scale_log2));
        raised |= top != m[h];
        m[h] = top;
        l[h] = __fmul_rn(l[h], old[h]);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const float a = exp2_approx(__fmaf_rn(__fsub_rn(sc[i][2 * h], base), p.scale_log2, kPLift<T>));
          const float c = exp2_approx(__fmaf_rn(__fsub_rn(sc[i][2 * h + 1], base), p.scale_log2, kPLift<T>));
          l[h] = __fadd_rn(l[h], __fadd_rn(a, c));
          pr[i / 2][i % 2 * 2 + h] = pack2<T>(a, c);   // 16 bits: the product's operand
        }
      }
      if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2 * H; ++e) acc[c][j][e] = __fmul_rn(acc[c][j][e], old[e >> 1]);
      }
#pragma unroll
      for (int u = 0; u < KT / 2; ++u)            // 16 keys at a time
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          uint32_t x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {           // keys 2t, 2t + 1, 2t + 8, 2t + 9; chunk g
            const int row = 16 * u + 2 * t + (i & 1) + 8 * (i >> 1);
            uint4 v = *reinterpret_cast<const uint4*>(in + kStep / 2 + c * (kKeys * 128) + row * 128 + ((g ^ (row & 7)) << 4));
            if (k0 + row >= end) v = make_uint4(0, 0, 0, 0);    // past a sample's length there may be anything
            x[i][0] = v.x;
            x[i][1] = v.y;
            x[i][2] = v.z;
            x[i][3] = v.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {           // column 64 c + 8 g + j of this lane's operand
            const uint32_t pick = j & 1 ? 0x7632u : 0x5410u;
            if (H == 1) acc[c][j][2] = acc[c][j][3] = 0.0f;
            few_mma<T>(acc[c][j], pr[u], __byte_perm(x[0][j / 2], x[1][j / 2], pick),
                       __byte_perm(x[2][j / 2], x[3][j / 2], pick));
          }
        }
      __syncwarp();
      at.step();
      if (lane == 0) {
        --in_flight;
        fetch();
      }
    }
    if (!ok && lane == 0) {                       // copies in flight end before the CTA leaves its shared memory
      const unsigned long long t0 = global_timer_ns();
      for (; in_flight > 0; --in_flight, at.step())
        while (!mbar_try_wait(cta.bar(at.s), at.phase) && global_timer_ns() - t0 < p.wait_limit_ns) {
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      l[h] = __fadd_rn(l[h], __shfl_xor_sync(0xffffffffu, l[h], 1));
      l[h] = __fadd_rn(l[h], __shfl_xor_sync(0xffffffffu, l[h], 2));
      const int r = g + 8 * h;
      if (t == 0) stats[warp][r] = make_float2(m[h], l[h]);
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4*>(sums(warp, r) + 64 * c + 16 * t + 8 * e + j) =
                make_float4(acc[c][j][2 * h + e], acc[c][j + 1][2 * h + e], acc[c][j + 2][2 * h + e], acc[c][j + 3][2 * h + e]);
    }
    if (PLANNED) named_barrier_sync(1 + grp, 32 * group);
    else __syncthreads();
    // the group's warps: a thread per two columns of a row
    const int first = grp * group, behind = first + group;
    for (int x = threadIdx.x - 32 * first; x < rows * (D / 2); x += 32 * group) {
      const int r = x / (D / 2), c = x % (D / 2) * 2;
      float top = -INFINITY;
#pragma unroll (PLANNED ? 4 : WARPS)
      for (int i = first; i < behind; ++i) top = fmaxf(top, stats[i][r].x);
      const float base = top == -INFINITY ? 0.0f : top;
      float total = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll (PLANNED ? 4 : WARPS)
      for (int i = first; i < behind; ++i) {
        const float f = exp2_approx(__fmul_rn(__fsub_rn(stats[i][r].x, base), p.scale_log2));
        total = __fmaf_rn(f, stats[i][r].y, total);
        o = __ffma2_rn(make_float2(f, f), *reinterpret_cast<const float2*>(sums(i, r) + c), o);
      }
      const int i = q_row + (row0 + r) % queries, h = hk * p.group + (row0 + r) / queries;
      if (w.slot >= 0) {
        const long long k = static_cast<long long>(w.slot) * slot_rows + r;
        if (in_span(p.part + k * D + c, 8, p.sp_part, p.status)) *reinterpret_cast<float2*>(p.part + k * D + c) = o;
        if (c == 0 && in_span(p.stats + 2 * k, 8, p.sp_stats, p.status))
          *reinterpret_cast<float2*>(p.stats + 2 * k) = make_float2(top, total);
      } else {
        const bool some = total != 0.0f;
        const float inv = some ? __frcp_rn(total) : 0.0f;
        char* dst = p.o + (static_cast<long long>(b) * p.seq_q + i) * p.o_stride + h * (D * 2) + c * 2;
        if (in_span(dst, 4, p.sp_o, p.status))
          *reinterpret_cast<uint32_t*>(dst) = some ? pack2<T>(__fmul_rn(o.x, inv), __fmul_rn(o.y, inv)) : 0u;
        float* lse = p.lse + (static_cast<long long>(b) * p.heads_q + h) * p.seq_q + i;
        if (c == 0 && in_span(lse, 4, p.sp_lse, p.status)) *lse = some ? __fmaf_rn(top, p.scale, log_sum<T>(total)) : -INFINITY;
      }
    }
    // the sums' place is TMA's again; a warp that gave up ends its group's work
    fence_async_shared();
    ok = PLANNED ? named_barrier_and(1 + grp, 32 * group, ok) : !__syncthreads_or(!ok);
  }
  if (beside) grid_dependency_wait();
}

}  // namespace qknr
