// Attention of one new token per sequence over a per-head key-value cache, for
// groups of 17 to 128 query heads per KV head (csa_kv_attn_decode; smaller groups
// and wide heads: kv_attention.cu).
//
// From 17 heads on a key costs more products than mma.sync has time for while it
// streams in (measured there: 64 heads on one KV head, 8 x 131072 slots of 128
// dims, 268 us at 128 TFLOP/s, mma.sync's rate; the bytes alone take 82 us), so
// the products go to tcgen05.  128 keys are the M side, up to 64 heads the N side:
//   S^T [128 keys x 64 heads]  = K [keys x dims] . Q^T         (A, B K-major)
//   O^T [dims x 64 heads]     += V^T [dims x keys] . P^T       (A, B MN-major)
// Keys and values come as TMA boxes of up to 128 rows into the 128-byte swizzle,
// a ring of half-steps (keys, values, keys, ..); where keys and values are the
// same memory (a shared-KV cache) one copy serves both products.
//
// Roles (one persistent CTA per SM; runs, pieces and joins as in kv_attention.cuh):
//   warps 0-7  softmax in two groups of four warps that split the heads: thread =
//              key.  The tile's exponents are formed against the running maxima
//              as they stand; only when some key exceeds its head's by more than
//              2^8 (a vote of the group, one barrier) are the maxima taken anew
//              (redux), and O^T and the sums rescaled.  P^T goes to shared memory
//              in the cache's type (fp16: times 2^7).  At the end of a segment thread = dim of O^T.
//   warp 8     TMEM, tcgen05.mma issue by one thread
//   warp 9     page ids and TMA
//   warp 10    the next segment's query heads, into the swizzled tile
// Waits are bounded; a wait that runs out is recorded and ends the CTA's work.
// What paces it: the issuing thread (64 heads over 8 x 131072 slots: 107 us, 5.0
// TB/s and 321 TFLOP/s; 32 heads on each of two: 174 us).  Stamps of a long run,
// of a copy with one commit more a tile, gave per 128-key tile about 900 cycles for the
// eight products of S^T, 1400 for those of P V with their commits, and 500 of
// waits; the softmax warps needed 2000 of those cycles and waited for the rest.
// The products themselves need less (96 KB of operands a tile, 770 cycles at 128
// bytes a cycle), so this is the issuing code's pace, not the chip's.  Four softmax
// groups of half the heads left it as it was (116 and 115 us at the time).
#include "kv_attention.cuh"

namespace csa {

using namespace kvattn;

namespace {

constexpr int kKeys = 128;                 // of a tile
constexpr int kHeads = 64;                 // MMA N
constexpr int kGroups = 2, kSmWarps = 8;   // softmax warps, in two groups
constexpr int kMmaWarp = 8, kLoadWarp = 9, kQueryWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kBlock = kKeys * 128;        // 64 columns of 128 rows
constexpr int kQBlock = kHeads * 128;
constexpr int kPTile = kKeys * 128;
constexpr int kTmemCols = 256;             // S^T twice, O^T
constexpr int kOkRing = 16;                // tiles whose row masks are kept
constexpr float kGrow = 8.f;               // log2: how far a score may exceed its head's maximum

template <int DP>
struct TcGeometry {
  static constexpr int BOXES = DP / 64;
  static constexpr int SLOT = BOXES * kBlock;                 // keys (or values) of a tile
  static constexpr int SLOTS = DP == 64 ? 9 : 5;
  // with 64 dims the second half of V^T's 128 rows is whatever follows the slot:
  // the last one needs something to follow it
  static constexpr int SMEM = 1024 + BOXES * kQBlock + 2 * kPTile + SLOTS * SLOT + (DP == 64 ? kBlock : 0);
};

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(v));
  return r;
}

// Barrier over a softmax group with an OR of `x` over its 128 threads.
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

// Ring slot and phase of the n-th use.
__device__ __forceinline__ uint32_t ring_slot(int64_t n, int slots) { return (uint32_t)(n % slots); }
__device__ __forceinline__ uint32_t ring_phase(int64_t n, int slots) { return (uint32_t)((n / slots) & 1); }

// HW heads per softmax group.
template <class T, int DP, int HW>
__global__ void __launch_bounds__(kThreads, 1)
kv_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ KvAttnArgs a, int box_rows, int shared_kv) {
  using Geo = TcGeometry<DP>;
  constexpr int SLOTS = Geo::SLOTS, BOXES = Geo::BOXES, HEADS = 2 * HW;
  constexpr int LIFT = lift<T>((int)kGrow);
  constexpr float DROP = 1.f / (1 << LIFT);
  constexpr bool kBf16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
  constexpr uint32_t kIdescS = kBf16 ? tc::idesc_bf16(128, kHeads) : tc::idesc_fp16(128, kHeads);
  constexpr uint32_t kIdescPV = kBf16 ? tc::idesc_bf16(128, kHeads, true, true) : tc::idesc_fp16(128, kHeads, true, true);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[SLOTS], kv_empty[SLOTS];
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full[2], p_empty[2], o_full, o_empty;
  __shared__ int64_t s_scan[kThreads / 32], s_first[2];
  __shared__ uint32_t s_tmem;
  __shared__ uint8_t s_rows[kOkRing];            // of a tile: bit i, rows 16 i .. 16 i + 15 lie on a page of the pool
  __shared__ int s_dead[kGroups];                // a wait of the group ran out
  __shared__ __align__(16) float s_max[kSmWarps][HW];      // per-warp maxima of a tile
  __shared__ __align__(16) float s_sum[kSmWarps][HW];      // per-warp sums of a segment
  __shared__ __align__(16) float s_off[kSmWarps][HW];      // each warp's copy: minus the running maxima
  __shared__ __align__(16) float s_fac[kSmWarps][HW];      // and factors
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t q_sm = smem_u32(smem), p_sm = q_sm + BOXES * kQBlock, kv_sm = p_sm + 2 * kPTile;
  const int G = a.H / a.n_kv_heads, blocks = (G + HEADS - 1) / HEADS, HZ = a.n_kv_heads * blocks;
  const int run = blockIdx.x / HZ, hz = blockIdx.x - run * HZ;
  const int kvh = hz / blocks, hb = hz - kvh * blocks;
  const int64_t hq = (int64_t)kvh * G;
  const int uses = shared_kv ? 1 : 2;   // ring slots of a tile

  if (warp == kLoadWarp && lane < 2) tc::prefetch_tmap(lane == 0 ? &map_k : &map_v);
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(smem_u32(&kv_full[i]), 1);
      mbar_init(smem_u32(&kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), kSmWarps);
      mbar_init(smem_u32(&p_full[i]), kSmWarps);
      mbar_init(smem_u32(&p_empty[i]), 1);
      s_dead[i] = 0;
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_empty), 1);
    mbar_init(smem_u32(&o_full), 1);
    mbar_init(smem_u32(&o_empty), kSmWarps);
    mbar_fence_init();
  }
  // the columns of P^T and rows of Q that no head has stay zero
  for (int i = tid; i < (2 * kPTile + BOXES * kQBlock) / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem_cta();
  if (warp == kMmaWarp) tc::tmem_alloc(smem_u32(&s_tmem), kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait();
  pdl_trigger();
  const uint32_t tm_s = s_tmem, tm_o = s_tmem + 2 * kHeads;
  Cursor c;
  bool more = begin_run<kKeys, kKeys, kThreads>(a, run, c, s_scan, s_first);
  bool continued = more && c.tile > 0;   // the unit began before this run

  // Query heads of a segment into the swizzled tile, by `n` threads.  Row r of the
  // tile: head r of group 0, r - 32 of group 1, HW of each.  Rolled, as all that
  // runs once: its instructions come from a cold cache.
  constexpr int kPieces = HEADS * BOXES * 8;   // of 16 bytes
  auto query_piece = [&](int32_t b, int idx) {
    const int h = hb * HEADS + idx / (BOXES * 8), piece = idx % (BOXES * 8);
    return h < G && piece * 8 < a.d ? *reinterpret_cast<const uint4*>(a.q + b * a.q_token + (hq + h) * a.q_head + piece * 16)
                                    : make_uint4(0, 0, 0, 0);
  };
  auto put_piece = [&](int idx, const uint4& v) {
    const int h = idx / (BOXES * 8), piece = idx % (BOXES * 8), r = h < HW ? h : 32 + h - HW;
    *reinterpret_cast<uint4*>(smem + (piece >> 3) * kQBlock + r * 128 + (((piece ^ r) & 7) << 4)) = v;
  };
  if (warp != kLoadWarp && more && c.s.tiles > 0) {   // the first segment's: everyone, while the first keys come
    constexpr int kOthers = kThreads - 32;
    const int t = warp < kLoadWarp ? tid : tid - 32;
    uint4 v[(kPieces + kOthers - 1) / kOthers];
#pragma unroll
    for (int i = 0; i < (kPieces + kOthers - 1) / kOthers; ++i)
      if (t + i * kOthers < kPieces) v[i] = query_piece(c.b, t + i * kOthers);
#pragma unroll
    for (int i = 0; i < (kPieces + kOthers - 1) / kOthers; ++i)
      if (t + i * kOthers < kPieces) put_piece(t + i * kOthers, v[i]);
    fence_async_smem_cta();
    named_barrier_sync(3, kOthers);
  }

  if (warp == kLoadWarp) {
    // ============================================================== keys, values
    const int boxes = kKeys / box_rows, step = box_rows / 16;   // row boxes of a tile, groups of 16 rows of a box
    const int box = lane % boxes, col = lane / boxes;           // what this lane copies
    const uint32_t whole = (1u << step) - 1u;
    int64_t tile = 0;                     // of the run
    bool ok = true;
    // lane i < 8: page of the tile's rows 16 i .. 16 i + 15; -1 also where nobody
    // sees any of them (behind the sequence, or before its window: those pages may
    // be gone)
    int32_t page = -1, row = 0, next_page, next_row;
    auto lookup = [&](const Cursor& x, int32_t& pg, int32_t& rw) {
      const int32_t s = x.s.start + x.tile * kKeys + 16 * lane;
      pg = lane < 8 && s < x.s.n && s + 16 > x.s.lo ? kv_page(a.kv, x.b, s, &rw, a.err) : -1;
    };
    Cursor x = c;
    bool live = more && c.s.tiles > 0;
    if (live) lookup(x, page, row);
    while (live && ok) {
      const Cursor now = x;
      next_page = -1;
      next_row = 0;
      if (++x.tile == x.end) live = next_segment<kKeys, kKeys>(a, x);
      if (live) lookup(x, next_page, next_row);
      const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
      if (lane == 0) s_rows[tile % kOkRing] = (uint8_t)mask;   // released by the arrivals below
      // a box with seen rows on a page of the pool lies on that page whole; its last
      // group looked up tells where it begins there
      const uint32_t groups = (mask >> (box * step)) & whole;
      const bool present = col < BOXES && groups != 0;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, present)) * box_rows * 128;
      const int last = groups ? 31 - __clz(groups) : 0;
      const int32_t pg = __shfl_sync(0xffffffffu, page, box * step + last);
      const int32_t rw = __shfl_sync(0xffffffffu, row, box * step + last) - 16 * last;
      for (int u = 0; u < uses; ++u) {
        const int64_t n = tile * uses + u;
        const uint32_t slot = ring_slot(n, SLOTS), bar = smem_u32(&kv_full[slot]);
        ok = mbar_wait(smem_u32(&kv_empty[slot]), ring_phase(n, SLOTS) ^ 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) report(a.err, kErrTimeout, now.b, 1);
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (present)
          tc::tma_load_4d(kv_sm + slot * Geo::SLOT + col * kBlock + box * box_rows * 128, u == 0 ? &map_k : &map_v, col * 64, kvh, rw,
                          pg, bar);
      }
      page = next_page;
      row = next_row;
      ++tile;
    }
    if (!ok)   // copies may still be under way: wait for them, within a limit
      for (int i = 0; i < SLOTS; ++i)
        for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(smem_u32(&kv_full[i]), ph, 100000000ll);
  } else if (warp == kQueryWarp) {
    // ============================================================== query heads
    Cursor x = c;
    bool ok = true;
    uint32_t seg = 0;
    for (bool go = more && c.s.tiles > 0; go && ok; ++seg) {
      if (seg > 0) {
        constexpr int kFlight = 8;   // pieces in flight per lane
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&q_empty), (seg & 1u) ^ 1u));
        if (!ok) {
          if (lane == 0) report(a.err, kErrTimeout, x.b, 2);
          break;
        }
#pragma unroll 1
        for (int i0 = lane; i0 < kPieces; i0 += 32 * kFlight) {
          uint4 v[kFlight];
#pragma unroll
          for (int i = 0; i < kFlight; ++i) v[i] = query_piece(x.b, i0 + i * 32);
#pragma unroll
          for (int i = 0; i < kFlight; ++i) put_piece(i0 + i * 32, v[i]);
        }
        fence_async_smem_cta();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(smem_u32(&q_full));
      x.tile = x.end;
      go = next_segment<kKeys, kKeys>(a, x);
    }
  } else if (warp == kMmaWarp) {
    // ============================================================== products
    if (lane == 0) {
      int64_t tile = 0;
      uint32_t seg = 0;
      bool ok = true;
      Cursor x = c;
      auto product_pv = [&](int64_t i, bool first) -> bool {
        const uint32_t pb = (uint32_t)(i & 1);
        const int64_t n = i * uses + (uses - 1);
        const uint32_t slot = ring_slot(n, SLOTS);
        if (!mbar_wait(smem_u32(&p_full[pb]), (uint32_t)((i >> 1) & 1))) return false;
        // the previous segment's O^T has been read
        if (first && !mbar_wait(smem_u32(&o_empty), (seg & 1u) ^ 1u)) return false;
        if (!mbar_wait(smem_u32(&kv_full[slot]), ring_phase(n, SLOTS))) return false;
        tc::fence_after_sync();
        // 16 keys are 2048 bytes: 128 on in a descriptor's address field
        const uint64_t v = tc::smem_desc_mn_sw128(kv_sm + slot * Geo::SLOT, kBlock);
        const uint64_t pt = tc::smem_desc_mn_sw128(p_sm + pb * kPTile, kPTile);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) tc::mma_bf16_ss(tm_o, v + kk * 128, pt + kk * 128, kIdescPV, !(first && kk == 0));
        tc::mma_commit(smem_u32(&kv_empty[slot]));
        tc::mma_commit(smem_u32(&p_empty[pb]));
        return true;
      };
      for (bool go = more && c.s.tiles > 0; go && ok; ++seg) {
        ok = mbar_wait(smem_u32(&q_full), seg & 1u);
        tc::fence_after_sync();
        const int64_t first = tile;
        for (; ok && x.tile < x.end; ++x.tile, ++tile) {
          const uint32_t sb = (uint32_t)(tile & 1);
          const int64_t n = tile * uses;
          const uint32_t slot = ring_slot(n, SLOTS);
          ok = mbar_wait(smem_u32(&kv_full[slot]), ring_phase(n, SLOTS)) &&
               mbar_wait(smem_u32(&s_empty[sb]), (uint32_t)(((tile >> 1) & 1) ^ 1));
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t k = tc::smem_desc_sw128(kv_sm + slot * Geo::SLOT), q = tc::smem_desc_sw128(q_sm);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            tc::mma_bf16_ss(tm_s + sb * kHeads, k + ((kk >> 2) * kBlock + (kk & 3) * 32) / 16,
                            q + ((kk >> 2) * kQBlock + (kk & 3) * 32) / 16, kIdescS, kk > 0);
          tc::mma_commit(smem_u32(&s_full[sb]));
          if (!shared_kv) tc::mma_commit(smem_u32(&kv_empty[slot]));
          if (x.tile + 1 == x.end) tc::mma_commit(smem_u32(&q_empty));
          if (tile > first) ok = product_pv(tile - 1, tile - 1 == first);
        }
        if (ok) ok = product_pv(tile - 1, tile - 1 == first);
        if (!ok) {
          report(a.err, kErrTimeout, x.b, 3);
          break;
        }
        tc::mma_commit(smem_u32(&o_full));
        go = next_segment<kKeys, kKeys>(a, x);
      }
    }
  } else {
    // ============================================================== softmax
    const int grp = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const int col = grp * 32;              // of S^T, P^T and O^T: the group's first
    const int h0 = hb * HEADS + grp * HW;  // its first head in the KV head's group
    const int bar = 1 + grp;
    const int hl = lane & (HW - 1);
    int64_t tile = 0;
    uint32_t seg = 0;
    auto fail = [&](int where) {
      s_dead[grp] = 1;
      report(a.err, kErrTimeout, c.b, where);
    };
    for (; more; ++seg) {
      float m_run = -INFINITY;   // lane hl: of head h0 + hl
      float sum[HW];
#pragma unroll
      for (int h = 0; h < HW; ++h) sum[h] = 0.f;
      bool unset = true;         // some head has no maximum yet
      const int32_t first_tile = c.tile;
      const int64_t bh = (int64_t)c.b * a.H + hq;
      bool alive = true;
      for (; c.tile < c.end; ++c.tile, ++tile) {
        const uint32_t sb = (uint32_t)(tile & 1);
        const int64_t nv = tile * uses + uses - 1;
        // The values' slot stays filled until this tile's product, so its phase can
        // still be asked for here (the keys' may have been filled again by now).
        bool ok = mbar_wait(smem_u32(&s_full[sb]), (uint32_t)((tile >> 1) & 1)) &&
                  mbar_wait(smem_u32(&kv_full[ring_slot(nv, SLOTS)]), ring_phase(nv, SLOTS));
        float y[HW];
        __syncwarp();
        tc::fence_after_sync();
        {
          uint32_t r[HW / 16][16];
#pragma unroll
          for (int i = 0; i < HW / 16; ++i) tc::tmem_ld16(tm_s + sb * kHeads + col + 16 * i + lanes, r[i]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < HW / 16; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) y[16 * i + j] = __uint_as_float(r[i][j]) * a.scale;
        }
        const int32_t key = c.s.start + c.tile * kKeys + row;
        const bool seen = key >= c.s.lo && key < c.s.n && ((s_rows[tile % kOkRing] >> (row >> 4)) & 1u);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_empty[sb]));
        if (!seen) {
#pragma unroll
          for (int h = 0; h < HW; ++h) y[h] = -INFINITY;
        }
        if (a.scores != nullptr && key < c.s.n) {
          float* sc = a.scores + (bh + h0) * a.score_stride + key;
#pragma unroll
          for (int h = 0; h < HW; ++h, sc += a.score_stride)
            if (h0 + h < G) *sc = y[h];
        }
        float over = -INFINITY;
        if (!unset) {
#pragma unroll
          for (int h = 0; h < HW; h += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&s_off[warp][h]);
            over = fmaxf(over, fmaxf(fmaxf(y[h] + m.x, y[h + 1] + m.y), fmaxf(y[h + 2] + m.z, y[h + 3] + m.w)));
          }
        }
        if (!ok) fail(4);
        const bool anew = group_any(bar, unset || over > kGrow || !ok);
        if (*(volatile int*)&s_dead[grp]) {
          alive = false;
          break;
        }
        if (anew) {   // take the maxima anew
          float mine = -INFINITY;
#pragma unroll
          for (int h = 0; h < HW; ++h) {
            const float v = redux_max(y[h]);
            if (hl == h) mine = v;
          }
          if (lane < HW) s_max[warp][lane] = mine;
          group_any(bar, false);
          const float top = fmaxf(fmaxf(s_max[4 * grp][hl], s_max[4 * grp + 1][hl]), fmaxf(s_max[4 * grp + 2][hl], s_max[4 * grp + 3][hl]));
          float f = 1.f;
          if (top > m_run + kGrow || (m_run == -INFINITY && top > -INFINITY)) {
            f = m_run == -INFINITY ? 0.f : ex2(m_run - top);
            m_run = top;
          }
          unset = __any_sync(0xffffffffu, m_run == -INFINITY);
          if (lane < HW) {
            s_off[warp][lane] = m_run == -INFINITY ? -INFINITY : -m_run;
            s_fac[warp][lane] = f;
          }
          __syncwarp();
#pragma unroll
          for (int h = 0; h < HW; ++h) sum[h] *= s_fac[warp][h];
          if (c.tile > first_tile && __any_sync(0xffffffffu, f != 1.f)) {
            // this warp's dims of O^T; every product so far must be done (the last
            // one's P buffer is then free; the one before it was waited for)
            if (!mbar_wait(smem_u32(&p_empty[sb ^ 1u]), (uint32_t)(((tile - 1) >> 1) & 1))) fail(5);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll
            for (int i = 0; i < HW / 16; ++i) {
              uint32_t r[16];
              tc::tmem_ld16(tm_o + col + 16 * i + lanes, r);
              tc::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * s_fac[warp][16 * i + j]);
              tc::tmem_st16(tm_o + col + 16 * i + lanes, r);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
          }
        }
        if (!mbar_wait(smem_u32(&p_empty[sb]), (uint32_t)(((tile >> 1) & 1) ^ 1))) fail(6);
        const uint32_t prow = p_sm + sb * kPTile + (uint32_t)row * 128;
#pragma unroll
        for (int i = 0; i < HW / 8; ++i) {
          const float4 m0 = *reinterpret_cast<const float4*>(&s_off[warp][8 * i]);
          const float4 m1 = *reinterpret_cast<const float4*>(&s_off[warp][8 * i + 4]);
          const float off[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int h = 8 * i + 2 * j;
            const float p0 = lifted<LIFT>(y[h] + off[2 * j]), p1 = lifted<LIFT>(y[h + 1] + off[2 * j + 1]);
            sum[h] += p0;
            sum[h + 1] += p1;
            pk[j] = pack2<T>(p0, p1);
          }
          const uint32_t chunk = col / 8 + i;
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(prow + (((chunk ^ row) & 7) << 4)), "r"(pk[0]), "r"(pk[1]),
                       "r"(pk[2]), "r"(pk[3])
                       : "memory");
        }
        if (grp == 0 && !seen) {   // 0 times what lies in an unseen value row may be NaN
          const uint32_t v = kv_sm + ring_slot(nv, SLOTS) * Geo::SLOT + row * 128;
          for (int i = 0; i < BOXES * 8; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(v + (i >> 3) * kBlock + (i & 7) * 16), "r"(0u) : "memory");
        }
        fence_async_smem_cta();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[sb]));
      }
      if (!alive) break;

      // ---- end of a segment: sums over keys, then O^T ------------------------------
      // A butterfly leaves lane h with the warp's sum of head h.
#pragma unroll
      for (int sh = HW / 2; sh >= 1; sh >>= 1) {
        const bool upper = (lane & sh) != 0;
#pragma unroll
        for (int j = 0; j < sh; ++j) {
          const float send = upper ? sum[j] : sum[j + sh];
          const float keep = upper ? sum[j + sh] : sum[j];
          sum[j] = keep + __shfl_xor_sync(0xffffffffu, send, sh);
        }
      }
      for (int o = HW; o < 32; o <<= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
      if (lane < HW) s_sum[warp][lane] = sum[0] * DROP;
      const bool any = c.end > first_tile;   // false: an empty sequence with a CTA to itself
      if (any && !mbar_wait(smem_u32(&o_full), seg & 1u)) fail(8);
      group_any(bar, false);
      if (*(volatile int*)&s_dead[grp]) break;
      const float l = (s_sum[4 * grp][hl] + s_sum[4 * grp + 1][hl]) + (s_sum[4 * grp + 2][hl] + s_sum[4 * grp + 3][hl]);
      const bool whole_unit = first_tile == 0 && c.tile == c.s.tiles;
      const int64_t piece = a.invariant ? ((int64_t)c.b * HZ + hz) * a.max_atoms + first_tile / a.atom
                                        : 2 * (int64_t)blockIdx.x + (continued ? 0 : 1);
      {
        const int h = h0 + hl;
        const Norm nm = normalise(m_run, l, a.sink && h < G ? a.sink[hq + h] * kLog2e : -INFINITY);
        if (wq == 0 && lane < HW) {
          if (!whole_unit) {
            *reinterpret_cast<float2*>(a.part_ml + (piece * HEADS + grp * HW + hl) * 2) = make_float2(m_run, l);
          } else if (h < G) {
            if (a.lse) a.lse[bh + h] = nm.lse2 * (1.f / kLog2e);
            if (a.lse2) a.lse2[bh + h] = nm.lse2;
          }
        }
        if (lane < HW) s_fac[warp][lane] = nm.scale * DROP;
      }
      __syncwarp();
      tc::fence_after_sync();
      const int heads = whole_unit && G - h0 < HW ? G - h0 : HW;   // beyond the group: nothing to write
      const int dims = whole_unit ? a.d : DP;
      float* acc = a.part_acc + (piece * HEADS + grp * HW) * DP + row;
      T* out = reinterpret_cast<T*>(a.out) + (bh + h0) * a.d + row;
#pragma unroll 1
      for (int i = 0; i < HW / 16; ++i) {
        uint32_t r[16];
        if (any) {
          tc::tmem_ld16(tm_o + col + 16 * i + lanes, r);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = 0u;
        }
        if (row < dims) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (16 * i + j < heads) {
              if (whole_unit) out[(16 * i + j) * (int64_t)a.d] = (T)(__uint_as_float(r[j]) * s_fac[warp][16 * i + j]);
              else acc[(16 * i + j) * DP] = __uint_as_float(r[j]) * DROP;
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (any && lane == 0) mbar_arrive(smem_u32(&o_empty));
      continued = false;
      more = next_segment<kKeys, kKeys>(a, c);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(s_tmem, kTmemCols);
}

template <class T, int DP, int HW>
cudaError_t launch_typed(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  using Geo = TcGeometry<DP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kv_attn_tc_kernel<T, DP, HW>, Geo::SMEM, done);
  if (e != cudaSuccess) return e;
  CUtensorMap map_k = {}, map_v = {};
  const KvRef& kv = a.kv;
  if (!tile_map(kv.k, kv.k_page, kv.k_slot, kv.k_head, a, p.box_rows, &map_k) ||
      !tile_map(kv.v, kv.v_page, kv.v_slot, kv.v_head, a, p.box_rows, &map_v))
    return cudaErrorInvalidValue;
  const int shared = kv.k == kv.v && kv.k_page == kv.v_page && kv.k_slot == kv.v_slot && kv.k_head == kv.v_head;
  L.begin(kKernelAttention);
  e = launch_kernel(kv_attn_tc_kernel<T, DP, HW>, dim3((unsigned)p.n_ctas), dim3(kThreads), Geo::SMEM, L.stream, true, map_k, map_v, a,
                    p.box_rows, shared);
  if (e != cudaSuccess) return e;
  e = L.end(kKernelAttention);
  if (e != cudaSuccess) return e;
  return launch_finish<T, DP, kKeys, kKeys, 2 * HW>(L, a, p);
}

template <class T>
cudaError_t launch_dims(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  if (p.dp == 64) return p.heads == 32 ? launch_typed<T, 64, 16>(L, a, p) : launch_typed<T, 64, 32>(L, a, p);
  return p.heads == 32 ? launch_typed<T, 128, 16>(L, a, p) : launch_typed<T, 128, 32>(L, a, p);
}

}  // namespace

// Rows of a box if this kernel takes caches of this geometry, else 0.
int kv_attn_tc_box_rows(const KvRef& kv, int32_t n_kv_heads) {
  const int64_t n[3] = {kv.n_pages, kv.page_size, n_kv_heads};
  const int64_t s[6] = {kv.k_page, kv.k_slot, kv.k_head, kv.v_page, kv.v_slot, kv.v_head};
  for (int i = 0; i < 6; ++i)
    if (n[i % 3] > 1 && (s[i] <= 0 || s[i] >= (int64_t(1) << 40))) return 0;
  if (kv.table == nullptr) return kKeys;
  for (int r = kKeys; r >= 16; r /= 2)
    if (kv.page_size % r == 0) return r;
  return 0;
}

cudaError_t launch_kv_attn_tc(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  return a.dtype == CSA_KV_FP16 ? launch_dims<__half>(L, a, p) : launch_dims<__nv_bfloat16>(L, a, p);
}

}  // namespace csa
