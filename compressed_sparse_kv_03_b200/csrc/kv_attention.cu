// Attention of one new token per sequence over a per-head key-value cache
// (csa_kv_attn_decode): groups of up to 16 query heads, and larger ones where
// the tcgen05 kernel (kv_attention_tc.cu) does not go.
//
// Work: every seen key and value is read once for the G query heads of its
// group; 4 G d flops per 4 d bytes, so HBM bounds it for G <= 16 and the
// mma.sync rate above (8 sequences x 131072 slots of 128 dims: 8 query heads on
// each of 8 KV heads 615 us, 16 on each of 4 325 us: 7.0 and 6.6 TB/s).  The
// layout follows from that:
//   * A unit is (sequence, KV head, block of up to 64 heads of its group, or 32 of
//     wide ones).  Its
//     slots are cut into tiles, and the tiles of all sequences, one after the
//     other, into equal runs, whatever the lengths.  A CTA takes one run of one
//     head (block) and streams through it without draining its copies between
//     sequences; a unit that spans several CTAs leaves partial (O, max, sum)
//     pieces that a second kernel joins in run order.
//   * CTAs of the same run and different heads are neighbours and keep pace, so
//     a 128-byte line that holds ends of two heads' rows (head dims that are no
//     multiple of 64) is fetched once: with a run over heads instead, 8 heads of
//     72 dims read 1.77 times their bytes from HBM.
//   * Keys are the M side of mma.m16n8k16, 16 a step, heads the N side, 8 or 16
//     a warp (mma.sync's rate on this chip is an eighth of tcgen05's, so the
//     columns matter).  Up to 16 heads (8 of more than 128 dims), the CTA's four
//     warps take the tile's keys apart, each with a ring of its own (no block
//     barrier in the loop); more heads put 2 and 4 warps side by side on the
//     same keys.  Rows come as TMA boxes of 16 rows (or, where 16 slots may lie
//     on several pages, by cp.async), page ids one step ahead of them.
//   * Softmax with a running maximum in base 2 and fp32; probabilities rounded
//     to the cache's type for P V (as every 16-bit tensor-core product needs; in
//     fp16 times 2^14), their sum taken before that rounding.
#include "kv_attention.cuh"

namespace csa {

using namespace kvattn;

namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 16;            // keys of a step

template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma_bf16_16816(d, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Resident CTAs per SM: registers (at most 128 a thread with 64 dims and 8 heads a
// warp, 255 otherwise) and the ring allow that many.
constexpr int ctas_per_sm(int dp, int nb, int wh) { return dp == 64 ? 4 / nb : dp == 128 || wh > 1 ? 2 : 1; }

// NB blocks of 8 heads per warp, WH warps side by side.
template <class T, int DP, int NB, int WH>
struct Geometry {
  static constexpr int NG = 4 / WH;                 // key groups of a CTA
  static constexpr int TILE = kKeys * NG;
  static constexpr int GROUP = 32 * WH;             // threads of a key group
  static constexpr int HEADS = 8 * NB * WH;         // of a unit
  static constexpr int BOXES = DP / 64;             // 128-byte column blocks of a row
  static constexpr int BOX = kKeys * 128;           // bytes of 16 rows of one
  static constexpr int STAGE = 2 * BOXES * BOX;     // a group's keys, then values
  static constexpr int CTAS = ctas_per_sm(DP, NB, WH);
  static constexpr int STAGES = DP == 64 && CTAS == 2 ? 6 : 3;
  static constexpr int SMEM = STAGES * STAGE * NG + 1024;   // + alignment
  // O of 16 heads fits a stage: joins go through the one that was just read
  static_assert(STAGE == 16 * DP * 4, "a stage holds a warp's O");
};

// Transposes an 8 x 8 matrix of 16-bit values held as (row lane/4, columns 2 (lane%4), +1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

template <class T, int DP, int NB, int WH>
__global__ void __launch_bounds__(kThreads, (Geometry<T, DP, NB, WH>::CTAS))
kv_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ KvAttnArgs a) {
  using Geo = Geometry<T, DP, NB, WH>;
  constexpr int LIFT = lift<T>(0);   // scores are at most the running maximum
  constexpr int NG = Geo::NG, TILE = Geo::TILE, S = Geo::STAGES, BOX = Geo::BOX, BOXES = Geo::BOXES, HEADS = Geo::HEADS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // the swizzle's atoms are 1024 bytes
  __shared__ int64_t s_scan[4];
  __shared__ int64_t s_first[2];
  __shared__ float2 s_ml[4][HEADS];
  __shared__ __align__(8) uint64_t s_bar[NG][S];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WH, wh = warp % WH;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.H / a.n_kv_heads;
  const int blocks = (G + HEADS - 1) / HEADS;
  const int HZ = a.n_kv_heads * blocks;   // units of a sequence
  const uint32_t ring = smem_u32(smem) + kg * (S * Geo::STAGE);
  const uint32_t bars = smem_u32(&s_bar[kg][0]);

  // ---- this CTA's run of atoms ------------------------------------------------
  const int run = blockIdx.x / HZ, hz = blockIdx.x - run * HZ;
  const int kvh = hz / blocks, hb = hz - kvh * blocks;
  Cursor c;
  if (!begin_run<TILE, kKeys, kThreads>(a, run, c, s_scan, s_first)) return;
  bool continued = c.tile > 0;   // the unit began before this run

  const bool producer = wh == 0;
  if (lane == 0 && producer) {
#pragma unroll
    for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, a.tiled ? 1 : 32);
    mbar_fence_init();
  }
  __syncthreads();

  // ---- copies -----------------------------------------------------------------
  // The first warp of a key group runs S-1 steps ahead of it, its page ids one
  // step more.  Tiled (16 keys lie on one page: page_size a multiple of 16, or
  // no page table): boxes of 16 rows by 128 bytes, one per lane; rows of the
  // page behind the sequence come with them and are masked.  Otherwise 16 bytes
  // a lane by cp.async, every row from its own page.
  Cursor p = c;
  bool p_live = c.s.tiles > 0;
  int32_t l_page = -1, l_row = 0;
  auto lookup = [&]() {
    int32_t s = p.s.start + p.tile * TILE + kg * kKeys;
    if (!a.tiled) s += lane & 15;
    l_page = s < p.s.n && (a.tiled || s >= p.s.lo) ? kv_page(a.kv, p.b, s, &l_row, a.err) : -1;
  };
  // Start the copies of the producer cursor's step into ring slot `st`; returns
  // the mask of its rows that the query sees.
  auto issue = [&](int st) -> uint32_t {
    const uint32_t bar = bars + 8 * st, dst = ring + st * Geo::STAGE;
    uint32_t rows = 0;
    if (a.tiled) {
      if (l_page >= 0) {
        const int32_t s0 = p.s.start + p.tile * TILE + kg * kKeys;
        rows = p.s.n - s0 >= kKeys ? 0xffffu : (1u << (p.s.n - s0)) - 1u;
        if (s0 < p.s.lo) rows &= 0xffffu << (p.s.lo - s0);   // at most 15: tiles start at lo rounded down
      }
      if (producer) {
        if (lane == 0) mbar_arrive_expect_tx(bar, l_page >= 0 ? Geo::STAGE : 0);
        __syncwarp();
        if (l_page >= 0 && lane < 2 * BOXES)
          tc::tma_load_4d(dst + lane * BOX, lane < BOXES ? &map_k : &map_v, (lane % BOXES) * 64, kvh, l_row, l_page, bar);
      }
    } else {
      rows = __ballot_sync(0xffffffffu, l_page >= 0) & 0xffffu;
      if (producer) {
        const int64_t page = l_page < 0 ? 0 : l_page;
        const int64_t ko = page * a.kv.k_page + l_row * a.kv.k_slot + kvh * a.kv.k_head;
        const int64_t vo = page * a.kv.v_page + l_row * a.kv.v_slot + kvh * a.kv.v_head;
#pragma unroll 4
        for (int i = 0; i < 4 * BOXES; ++i) {   // 16 rows of 8 BOXES pieces
          const int idx = i * 32 + lane, r = idx / (8 * BOXES), ch = idx % (8 * BOXES);
          const int64_t kro = __shfl_sync(0xffffffffu, ko, r), vro = __shfl_sync(0xffffffffu, vo, r);
          const bool ok = ((rows >> r) & 1u) && ch * 8 < a.d;
          const uint32_t at = dst + (ch >> 3) * BOX + r * 128 + (((ch ^ r) & 7) << 4);
          cp_async_16(at, ok ? a.kv.k + kro + 16 * ch : a.kv.k, ok);
          cp_async_16(at + BOXES * BOX, ok ? a.kv.v + vro + 16 * ch : a.kv.v, ok);
        }
        cp_async_mbar_arrive_noinc(bar);
      }
    }
    if (++p.tile == p.end) p_live = next_segment<TILE, kKeys>(a, p);
    if (p_live) lookup();
    return rows;
  };
  auto group_sync = [&]() {
    if (WH == 1) __syncwarp();
    else if (WH == 4) __syncthreads();
    else named_barrier_sync(1 + kg, Geo::GROUP);
  };

  uint32_t rows_q[S - 1];   // masks of the steps in flight, oldest first
  if (p_live) lookup();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) rows_q[i] = p_live ? issue(i) : 0u;

  // ---- segments -------------------------------------------------------------------
  // Scores are K Q^T and outputs V^T P^T: keys (then dims) on the 16 rows of an
  // mma, 8 heads on its columns, so up to 8 heads cost half of what 16 do.  A
  // lane holds keys g, g + 8 (dims g, g + 8 of each 16) of heads 2 t4, 2 t4 + 1
  // of each block of 8.
  int st = 0;   // ring slot of the current step
  uint32_t phase = 0;
  bool dead = false;   // a wait ran out: no more waiting, the result is void
  const int kmat = lane >> 3, kr = lane & 7;
  // ldmatrix rows: keys as (keys 0-7, 8-15) x (dims lo, hi), values transposed as
  // (dims lo, hi) x (keys 0-7, 8-15)
  const uint32_t k_lane = (kr + (kmat & 1) * 8) * 128 + (((kmat >> 1) ^ kr) << 4);
  const uint32_t v_lane = BOXES * BOX + (kr + (kmat >> 1) * 8) * 128 + (((kmat & 1) ^ kr) << 4);
  for (bool more = true; more;) {
    const int h0 = hb * HEADS + wh * (8 * NB);   // first head of the warp, in the group
    const int64_t hq = (int64_t)kvh * G, bh = (int64_t)c.b * a.H + hq;
    uint32_t q[NB][DP / 16][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int h = h0 + nb * 8 + g;
      const char* const qh = a.q + c.b * a.q_token + (hq + h) * a.q_head + 4 * t4;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        q[nb][ks][0] = h < G && ks * 16 < a.d ? *reinterpret_cast<const uint32_t*>(qh + ks * 32) : 0u;
        q[nb][ks][1] = h < G && ks * 16 + 8 < a.d ? *reinterpret_cast<const uint32_t*>(qh + ks * 32 + 16) : 0u;
      }
    }
    float o[NB][DP / 16][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nb][i][j] = 0.f;
    // running maxima (of scaled scores, base 2) and this lane's part of the sums
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
    }
    const int32_t first_tile = c.tile;
    for (; c.tile < c.end; ++c.tile) {
      if (!dead && !mbar_wait(bars + 8 * st, phase)) {
        dead = true;
        report(a.err, kErrTimeout, c.b, c.tile);
      }
      group_sync();   // everyone has left the slot that is filled next
      const uint32_t rows = rows_q[0];
#pragma unroll
      for (int i = 0; i + 1 < S - 1; ++i) rows_q[i] = rows_q[i + 1];
      rows_q[S - 2] = p_live ? issue(st == 0 ? S - 1 : st - 1) : 0u;
      const uint32_t base = ring + st * Geo::STAGE;
      if (++st == S) {
        st = 0;
        phase ^= 1u;
      }

      float s[NB][2][4] = {};   // even and odd k-steps: shorter chains
#pragma unroll
      for (int ks = 0; ks < DP / 16; ks += 2) {
        if (ks * 16 < a.d) {
          uint32_t k0[4], k1[4];
          ldmatrix_x4(k0, base + (ks >> 2) * BOX + (k_lane ^ ((ks & 3) * 32)));
          ldmatrix_x4(k1, base + (ks >> 2) * BOX + (k_lane ^ ((ks & 3) * 32 + 32)));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816<T>(s[nb][0], k0, q[nb][ks][0], q[nb][ks][1]);
            mma16816<T>(s[nb][1], k1, q[nb][ks + 1][0], q[nb][ks + 1][1]);
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nb][0][j] = (s[nb][0][j] + s[nb][1][j]) * a.scale;
      if (rows != 0xffffu) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((rows >> (g + (j >> 1) * 8)) & 1u)) s[nb][0][j] = -INFINITY;
        // 0 times what lies in an unseen value row may be NaN: clear those rows
        // (every warp of the group all of them, so that none waits for another)
        for (int i = lane; i < kKeys * BOXES * 8; i += 32) {
          const int r = (i >> 3) & (kKeys - 1);
          if (!((rows >> r) & 1u))
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(base + BOXES * BOX + i * 16), "r"(0u) : "memory");
        }
        fence_async_smem_cta();
        __syncwarp();
      }
      if (a.scores != nullptr) {
        const int32_t s0 = c.s.start + c.tile * TILE + kg * kKeys + g;
        float* const sc = a.scores + (bh + h0 + 2 * t4) * a.score_stride + s0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (s0 + (j >> 1) * 8 < c.s.n && h0 + nb * 8 + 2 * t4 + (j & 1) < G)
              sc[(nb * 8 + (j & 1)) * a.score_stride + (j >> 1) * 8] = s[nb][0][j];
      }
      bool grows = false;
      float x[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[nb][e] = fmaxf(s[nb][0][e], s[nb][0][e + 2]);
          grows |= x[nb][e] > m[nb][e];
        }
      if (__any_sync(0xffffffffu, grows)) {   // some head's maximum grows
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = x[nb][e];
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
            const float top = fmaxf(m[nb][e], v);
            const float f = top == -INFINITY ? 1.f : ex2(m[nb][e] - top);
            m[nb][e] = top;
            l[nb][e] *= f;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
              o[nb][i][e] *= f;
              o[nb][i][e + 2] *= f;
            }
          }
      }
      uint32_t pb[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float r0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0], r1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
        const float p0 = lifted<LIFT>(s[nb][0][0] - r0), p1 = lifted<LIFT>(s[nb][0][1] - r1);
        const float p2 = lifted<LIFT>(s[nb][0][2] - r0), p3 = lifted<LIFT>(s[nb][0][3] - r1);
        l[nb][0] += p0 + p2;
        l[nb][1] += p1 + p3;
        // (key, 2 heads) to (head, 2 keys)
        pb[nb][0] = transpose8x8(pack2<T>(p0, p1));
        pb[nb][1] = transpose8x8(pack2<T>(p2, p3));
      }
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        if (j * 16 < a.d) {
          uint32_t va[4];
          ldmatrix_x4_trans(va, base + (j >> 2) * BOX + (v_lane ^ ((j & 3) * 32)));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816<T>(o[nb][j], va, pb[nb][0], pb[nb][1]);
        }
      }
    }

    // ---- join the key groups, store --------------------------------------------
    // Everyone has read slot st - 1 to the end; the next step fills it.
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], off);
    if constexpr (LIFT > 0) {
      constexpr float DROP = 1.f / (1 << LIFT);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        l[nb][0] *= DROP;
        l[nb][1] *= DROP;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nb][i][j] *= DROP;
      }
    }
    const bool whole_unit = first_tile == 0 && c.tile == c.s.tiles;   // no other piece exists
    const int64_t piece = a.invariant ? ((int64_t)c.b * HZ + hz) * a.max_atoms + first_tile / a.atom
                                      : 2 * (int64_t)blockIdx.x + (continued ? 0 : 1);
    const int prev = st == 0 ? S - 1 : st - 1;
    auto sink_of = [&](int h) { return a.sink && h < G ? a.sink[hq + h] * kLog2e : -INFINITY; };
    auto store_ml = [&](int row, float top, float sum) {   // row: of the unit's heads
      const int h = hb * HEADS + row;
      if (!whole_unit) {
        *reinterpret_cast<float2*>(a.part_ml + (piece * HEADS + row) * 2) = make_float2(top, sum);
      } else if (h < G) {
        const Norm nm = normalise(top, sum, sink_of(h));
        if (a.lse) a.lse[bh + h] = nm.lse2 * (1.f / kLog2e);
        if (a.lse2) a.lse2[bh + h] = nm.lse2;
      }
    };
    if constexpr (NG > 1) {
      if (g == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) s_ml[kg][wh * (8 * NB) + nb * 8 + 2 * t4 + e] = make_float2(m[nb][e], l[nb][e]);
      }
    }
    if constexpr (NG == 4) {
      // every warp puts its O down, [head][dim], and sums a quarter of the columns of all four
      float* const mine = reinterpret_cast<float*>(smem + (kg * S + prev) * Geo::STAGE);
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)   // 8-float blocks permuted by head pair, off the bank conflicts
            mine[(nb * 8 + 2 * t4 + (j & 1)) * DP + ((i * 16 + (j >> 1) * 8 + g) ^ (t4 * 8))] = o[nb][i][j];
      __syncthreads();
      constexpr int F4 = DP / 16;   // float4 per row of a quarter
#pragma unroll
      for (int i = 0; i < HEADS * F4 / 32; ++i) {
        const int idx = i * 32 + lane, row = idx / F4, col = warp * (DP / 4) + (idx % F4) * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, s_ml[w][row].x);
        const float R = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 ml = s_ml[w][row];
          const float f = ex2(ml.x - R);
          sum = fmaf(ml.y, f, sum);
          const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + (w * S + prev) * Geo::STAGE) +
                                                            row * DP + (col ^ (((row >> 1) & 3) * 8)));
          acc.x = fmaf(y.x, f, acc.x);
          acc.y = fmaf(y.y, f, acc.y);
          acc.z = fmaf(y.z, f, acc.z);
          acc.w = fmaf(y.w, f, acc.w);
        }
        const int h = hb * HEADS + row;
        if (whole_unit) {
          if (h < G && col < a.d) {
            const float k = normalise(top, sum, sink_of(h)).scale;
            uint2 pk;
            pk.x = pack2<T>(acc.x * k, acc.y * k);
            pk.y = pack2<T>(acc.z * k, acc.w * k);
            *reinterpret_cast<uint2*>(a.out + ((bh + h) * a.d + col) * 2) = pk;
          }
        } else {
          *reinterpret_cast<float4*>(a.part_acc + (piece * HEADS + row) * DP + col) = acc;
        }
        if (col == 0) store_ml(row, top, sum);
      }
      fence_async_smem_cta();
      __syncthreads();   // the slots may be filled again
    } else {
      if constexpr (NG == 2) {   // group 1 hands its O to group 0 through both groups' slots
        float4* const buf = reinterpret_cast<float4*>(smem + (wh * S + prev) * Geo::STAGE) + lane;
        __syncthreads();   // and both groups have left their slots
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 other = s_ml[1 - kg][wh * (8 * NB) + nb * 8 + 2 * t4 + e];
            const float top = fmaxf(m[nb][e], other.x), R = top == -INFINITY ? 0.f : top;
            f[e] = ex2(m[nb][e] - R);
            l[nb][e] = l[nb][e] * f[e] + other.y * ex2(other.x - R);
            m[nb][e] = top;
          }
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) {
            o[nb][i][0] *= f[0];
            o[nb][i][1] *= f[1];
            o[nb][i][2] *= f[0];
            o[nb][i][3] *= f[1];
            if (kg == 1) buf[(nb * (DP / 16) + i) * 32] = make_float4(o[nb][i][0], o[nb][i][1], o[nb][i][2], o[nb][i][3]);
          }
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
              const float4 y = buf[(nb * (DP / 16) + i) * 32];
              o[nb][i][0] += y.x;
              o[nb][i][1] += y.y;
              o[nb][i][2] += y.z;
              o[nb][i][3] += y.w;
            }
        }
        fence_async_smem_cta();
        __syncthreads();
      }
      if (kg == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int row = wh * (8 * NB) + nb * 8 + 2 * t4;   // and row + 1
          if (g == 0) {
            store_ml(row, m[nb][0], l[nb][0]);
            store_ml(row + 1, m[nb][1], l[nb][1]);
          }
          if (whole_unit) {
            const int h = hb * HEADS + row + (g & 1);
            const float k0 = normalise(m[nb][0], l[nb][0], sink_of(hb * HEADS + row)).scale;
            const float k1 = normalise(m[nb][1], l[nb][1], sink_of(hb * HEADS + row + 1)).scale;
            char* const out = a.out + ((bh + h) * a.d + (g & 6)) * 2;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
              for (int half = 0; half < 2; ++half) {   // lanes of dims g, g ^ 1 trade heads for neighbours
                const float v0 = o[nb][i][2 * half] * k0, v1 = o[nb][i][2 * half + 1] * k1;
                const float y = __shfl_xor_sync(0xffffffffu, (g & 1) ? v0 : v1, 4);
                const int d0 = i * 16 + half * 8;
                if (h < G && d0 < a.d)
                  *reinterpret_cast<uint32_t*>(out + 2 * d0) = (g & 1) ? pack2<T>(y, v1) : pack2<T>(v0, y);
              }
          } else {
            float* const acc = a.part_acc + (piece * HEADS + row) * DP + g;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[(j & 1) * DP + i * 16 + (j >> 1) * 8] = o[nb][i][j];
          }
        }
      }
    }
    continued = false;
    more = next_segment<TILE, kKeys>(a, c);
  }
  if (dead) {   // copies may still be under way: wait for them, within a limit
    for (int i = 0; i < S; ++i) mbar_wait(bars + 8 * i, phase, 200000000ll);
  }
}

template <class T, int DP, int NB, int WH>
cudaError_t launch_typed(const Launch& L, const KvAttnArgs& args, const KvAttnPlan& p) {
  using Geo = Geometry<T, DP, NB, WH>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kv_attn_kernel<T, DP, NB, WH>, Geo::SMEM, done);
  if (e != cudaSuccess) return e;
  KvAttnArgs a = args;
  CUtensorMap map_k = {}, map_v = {};
  a.tiled = tile_map(a.kv.k, a.kv.k_page, a.kv.k_slot, a.kv.k_head, a, kKeys, &map_k) &&
            tile_map(a.kv.v, a.kv.v_page, a.kv.v_slot, a.kv.v_head, a, kKeys, &map_v);
  L.begin(kKernelAttention);
  e = launch_kernel(kv_attn_kernel<T, DP, NB, WH>, dim3((unsigned)p.n_ctas), dim3(kThreads), Geo::SMEM, L.stream, true, map_k,
                    map_v, a);
  if (e != cudaSuccess) return e;
  e = L.end(kKernelAttention);
  if (e != cudaSuccess) return e;
  return launch_finish<T, DP, Geo::TILE, kKeys, Geo::HEADS>(L, a, p);
}

template <class T, int DP>
cudaError_t launch_wh(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  if (p.nb == 1 && p.wh == 1) return launch_typed<T, DP, 1, 1>(L, a, p);
  if constexpr (DP <= 128)
    return p.wh == 1 ? launch_typed<T, DP, 2, 1>(L, a, p) : p.wh == 2 ? launch_typed<T, DP, 2, 2>(L, a, p) : launch_typed<T, DP, 2, 4>(L, a, p);
  else
    return p.wh == 2 ? launch_typed<T, DP, 1, 2>(L, a, p) : launch_typed<T, DP, 1, 4>(L, a, p);
}
template <class T>
cudaError_t launch_dp(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  switch (p.dp) {
    case 64: return launch_wh<T, 64>(L, a, p);
    case 128: return launch_wh<T, 128>(L, a, p);
    case 192: return launch_wh<T, 192>(L, a, p);
    default: return launch_wh<T, 256>(L, a, p);
  }
}

}  // namespace

// Which kernel, and how the work is cut.  Groups of more than 16 heads go to the
// tcgen05 kernel, except at head dims above 128 (its ring and TMEM are laid out
// for 64 and 128) and on pages that no 16-row box fits: 64 heads on one KV head,
// 8 x 131072 slots of 128 dims, 107 us there and 268 us here; 32 heads on each of
// two, 174 and 261 us; 17 heads on one, 100 and 140 us.
KvAttnPlan kv_attn_plan(const KvRef& kv, int32_t B, int32_t H, int32_t n_kv_heads, int32_t d, int64_t max_len,
                        int32_t window, bool invariant) {
  KvAttnPlan p{};
  const int G = H / n_kv_heads;
  p.invariant = invariant;
  p.dp = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256;
  p.box_rows = G > 16 && d <= 128 ? kv_attn_tc_box_rows(kv, n_kv_heads) : 0;
  if (p.dp <= 128) {
    p.nb = G <= 8 ? 1 : 2;
    p.wh = G <= 16 ? 1 : G <= 32 ? 2 : 4;
  } else {   // 16 heads of such rows would fill a warp's registers: side by side, and two CTAs an SM
    p.nb = 1;   // (16 heads of 256 dims on each of 4: 184 -> 97 us)
    p.wh = G <= 8 ? 1 : G <= 16 ? 2 : 4;
  }
  p.heads = p.box_rows ? (G <= 32 ? 32 : 64) : 8 * p.nb * p.wh;
  p.blocks = (G + p.heads - 1) / p.heads;
  p.tile = p.box_rows ? 128 : kKeys * 4 / p.wh;
  const int align = p.box_rows ? 128 : kKeys;   // a window may start that much early, less one
  int64_t most_slots = max_len;
  if (window > 0 && window + align - 1 < most_slots) most_slots = window + align - 1;
  const int64_t tiles = (most_slots + p.tile - 1) / p.tile;
  const int64_t units = (int64_t)B * n_kv_heads * p.blocks;
  p.atom = invariant ? kInvariantSlots / p.tile : 1;
  p.max_atoms = (tiles + p.atom - 1) / p.atom;
  p.whole = !invariant && most_slots <= 256;
  const int64_t per_run = (int64_t)n_kv_heads * p.blocks;   // CTAs of a run
  const int64_t most = (int64_t)kSms * (p.box_rows ? 1 : ctas_per_sm(p.dp, p.nb, p.wh));
  int64_t runs = most / per_run;
  // many heads may leave a good part of the SMs idle: several waves of shorter runs instead
  if (runs * per_run * 8 < most * 7) runs = (4 * most + per_run - 1) / per_run;
  if (runs > B * p.max_atoms) runs = B * p.max_atoms;
  if (runs < 1 || p.whole) runs = p.whole ? B : 1;
  p.runs = (int)runs;
  p.n_ctas = (int)(runs * per_run);
  p.pieces = p.whole ? 0 : invariant ? units * p.max_atoms : 2 * (int64_t)p.n_ctas;
  return p;
}

cudaError_t launch_kv_attn(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  if (p.box_rows) return launch_kv_attn_tc(L, a, p);
  return a.dtype == CSA_KV_FP16 ? launch_dp<__half>(L, a, p) : launch_dp<__nv_bfloat16>(L, a, p);
}

}  // namespace csa
