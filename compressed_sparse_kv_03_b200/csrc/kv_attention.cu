// Attention of one new token per sequence over a per-head key-value cache
// (csa_kv_attn_decode).
//
// Work: every seen key and value is read once for the G query heads of its
// group; 4 G d flops per 4 d bytes, so HBM bounds it for G <= 32 and the
// mma.sync rate above.  The layout follows from that:
//   * A unit is (sequence, KV head, block of up to 64 heads of its group).  Its
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
//     columns matter).  Up to 16 heads, the CTA's four warps take the tile's keys apart, each with a ring of its
//     own (no block barrier in the loop); 32 and 64 heads put 2 and 4 warps
//     side by side on the same keys.  Rows come as TMA boxes of 16 rows (or,
//     where 16 slots may lie on several pages, by cp.async), page ids one step
//     ahead of them.
//   * Softmax with a running maximum in base 2 and fp32; probabilities rounded
//     to the cache's type for P V (as every 16-bit tensor-core product needs),
//     their sum taken before that rounding.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv.cuh"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kSms = 148;
constexpr int kKeys = 16;            // keys of a step
constexpr int kInvariantSlots = 512;
constexpr int kMaxBlocks = 2;        // head blocks of a group: up to 128 heads, 64 at a time

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

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Slots that a query sees: [lo, n); tiles start at lo rounded down to 16, so
// that a step's 16 keys lie on one page wherever page_size is a multiple of 16.
struct Span {
  int32_t n, lo, start, tiles;
};
template <int TILE>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, int32_t b, WsHeader* err) {
  Span s;
  s.n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, err);
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.start = s.lo & ~(kKeys - 1);
  s.tiles = (s.n - s.start + TILE - 1) / TILE;
  return s;
}

template <int TILE>
__device__ __forceinline__ int64_t atoms_of(const KvAttnArgs& a, int32_t b) {   // of a unit of sequence b
  return (span_of<TILE>(a, b, nullptr).tiles + a.atom - 1) / a.atom;
}

// Sum over the block's 128 threads, and of the threads before this one.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* before, int64_t* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t up = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = up;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += scratch[w];
    all += scratch[w];
  }
  *before = base + up - x;
  return all;
}

// Atoms per run: equal shares.
__device__ __forceinline__ int64_t share_of(const KvAttnArgs& a, int64_t atoms) {
  return (atoms + a.runs - 1) / a.runs;
}

// Resident CTAs per SM: registers (at most 128 a thread with 8 heads a warp, 255
// with 16) and the ring allow that many.
constexpr int ctas_per_sm(int dp, int nb) { return dp == 64 ? 4 / nb : dp == 128 ? 2 : 1; }

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
  static constexpr int CTAS = ctas_per_sm(DP, NB);
  static constexpr int STAGES = DP == 64 && CTAS == 2 ? 6 : 3;
  static constexpr int SMEM = STAGES * STAGE * NG + 1024;   // + alignment
  // O of 16 heads fits a stage: joins go through the one that was just read
  static_assert(STAGE == 16 * DP * 4, "a stage holds a warp's O");
};

// A position in this CTA's run of tiles.  A segment is the part of a unit that
// the CTA takes in one go (in batch-invariant mode a slice): tiles [.., end).
struct Cursor {
  int32_t b, tile, end;
  int64_t left;   // atoms after this segment
  Span s;
};
__device__ __forceinline__ void open_segment(const KvAttnArgs& a, Cursor& c) {
  const int32_t rest = c.s.tiles - c.tile;
  if (a.whole) {
    c.end = c.s.tiles;
    c.left = 0;
  } else if (a.invariant) {
    c.end = c.tile + (rest < a.atom ? rest : a.atom);
    --c.left;
  } else {
    c.end = c.tile + (int32_t)(rest < c.left ? rest : c.left);
    c.left -= c.end - c.tile;
  }
}
// To the segment after the one that ends at c.tile; false: the run is over.
template <int TILE>
__device__ __forceinline__ bool next_segment(const KvAttnArgs& a, Cursor& c) {
  if (c.left <= 0) return false;
  if (c.tile == c.s.tiles) {
    c.tile = 0;
    do {
      if (++c.b >= a.B) return false;
      c.s = span_of<TILE>(a, c.b, a.err);
    } while (c.s.tiles == 0);
  }
  open_segment(a, c);
  return true;
}

// Transposes an 8 x 8 matrix of 16-bit values held as (row lane/4, columns 2 (lane%4), +1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Final scale and log-sum-exp (base 2) of a head from its maximum and sum.
struct Norm {
  float scale, lse2;
};
__device__ __forceinline__ Norm normalise(float m, float l, float z) {
  const float M = fmaxf(m, z), R = M == -INFINITY ? 0.f : M;
  const float f = exp2f(m - R);
  const float L = l * f + exp2f(z - R);
  return L == 0.f ? Norm{0.f, -INFINITY} : Norm{f / L, R + log2f(L)};
}

template <class T, int DP, int NB, int WH>
__global__ void __launch_bounds__(kThreads, (Geometry<T, DP, NB, WH>::CTAS))
kv_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ KvAttnArgs a) {
  using Geo = Geometry<T, DP, NB, WH>;
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
  if (a.whole) {
    c.b = run;
    c.s = span_of<TILE>(a, c.b, a.err);
    c.tile = 0;
  } else {
    // a stretch of sequences per thread; the one that holds atom `begin` finds it
    const int32_t per = (a.B + kThreads - 1) / kThreads, b0 = tid * per, b1 = b0 + per < a.B ? b0 + per : a.B;
    int64_t mine = 0, before;
    for (int32_t b = b0; b < b1; ++b) mine += atoms_of<TILE>(a, b);
    const int64_t all = block_scan(mine, &before, s_scan);
    const int64_t share = share_of(a, all), begin = run * share;
    c.left = all - begin < share ? all - begin : share;
    if (c.left <= 0) return;
    if (begin >= before && begin < before + mine) {
      int32_t b = b0;
      for (int64_t n; b + 1 < b1 && before + (n = atoms_of<TILE>(a, b)) <= begin; ++b) before += n;
      s_first[0] = b;
      s_first[1] = begin - before;
    }
    __syncthreads();
    c.b = (int32_t)s_first[0];
    c.s = span_of<TILE>(a, c.b, a.err);
    c.tile = (int32_t)(s_first[1] * a.atom);
  }
  open_segment(a, c);
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
    if (++p.tile == p.end) p_live = next_segment<TILE>(a, p);
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
        const float p0 = ex2(s[nb][0][0] - r0), p1 = ex2(s[nb][0][1] - r1);
        const float p2 = ex2(s[nb][0][2] - r0), p3 = ex2(s[nb][0][3] - r1);
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
    more = next_segment<TILE>(a, c);
  }
  if (dead) {   // copies may still be under way: wait for them, within a limit
    for (int i = 0; i < S; ++i) mbar_wait(bars + 8 * i, phase, 200000000ll);
  }
}

// ---- joining --------------------------------------------------------------------
// Pieces of a unit: its first, how many, and the step from one to the next.
struct Pieces {
  int64_t first, second;   // piece 0, and pieces 1, 2, .. from `second` on by `step`
  int64_t count;
  int step;
  __device__ __forceinline__ int64_t at(int64_t i) const { return i == 0 ? first : second + (i - 1) * step; }
};
template <int TILE>
__device__ Pieces pieces_of(const KvAttnArgs& a, int32_t b, int HZ, int hz, int64_t* scratch) {
  const int64_t atoms = atoms_of<TILE>(a, b);
  if (a.invariant) {
    const int64_t first = ((int64_t)b * HZ + hz) * a.max_atoms;
    return Pieces{first, first + 1, atoms, 1};
  }
  int64_t mine = 0, low = 0, x;
  for (int32_t i = threadIdx.x; i < a.B; i += kThreads) {
    const int64_t n = atoms_of<TILE>(a, i);
    mine += n;
    if (i < b) low += n;
  }
  const int64_t all = block_scan(mine, &x, scratch), base = block_scan(low, &x, scratch);
  if (atoms == 0) return Pieces{0, 0, 0, 0};
  const int64_t share = share_of(a, all);
  const int64_t r0 = base / share, r1 = (base + atoms - 1) / share;
  // it begins in run r0; the other runs begin in it
  return Pieces{2 * (r0 * HZ + hz) + 1, 2 * ((r0 + 1) * HZ + hz), r1 - r0 + 1, 2 * HZ};
}

// (max, sum) of two parts of one softmax.
__device__ __forceinline__ float2 join_ml(float2 x, float2 y) {
  const float M = fmaxf(x.x, y.x), R = M == -INFINITY ? 0.f : M;
  return make_float2(M, x.y * ex2(x.x - R) + y.y * ex2(y.x - R));
}

// Slots that a weighing block takes at a time: about 16 KB of scores.
constexpr int weigh_slots(int G) { return G <= 16 ? 512 : 128; }

// weights_out of one block of slots: the group's log-sum-exps from the pieces (or
// from the attention kernel, for units of one piece), then the probabilities of
// the scores, summed over the group in head order.  A lane takes four slots;
// for up to 16 heads each warp has slots of its own, beyond that the four warps
// take the heads of the same slots apart and their sums are added in warp order.
template <int TILE, int ROWS>
__device__ void weigh(const KvAttnArgs& a, int b, int kvh, int32_t n, int32_t s0, int32_t end, const Pieces* ps, int blocks) {
  __shared__ float2 s_part[kThreads];
  __shared__ float s_lse[128];
  __shared__ float4 s_sum[4][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.H / a.n_kv_heads;
  const int64_t bh = (int64_t)b * a.H + (int64_t)kvh * G;
  const int row = tid % ROWS, part = tid / ROWS;
  constexpr int PARTS = kThreads / ROWS;
  for (int hb = 0; hb < blocks; ++hb) {
    const int h = hb * ROWS + row;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (ps[hb].count > 1) {
#pragma unroll 4
      for (int64_t i = part; i < ps[hb].count; i += PARTS)
        ml = join_ml(ml, *reinterpret_cast<const float2*>(a.part_ml + (ps[hb].at(i) * ROWS + row) * 2));
      s_part[tid] = ml;
      __syncthreads();
      if (part == 0)
        for (int w = 1; w < PARTS; ++w) ml = join_ml(ml, s_part[w * ROWS + row]);
      __syncthreads();
    }
    if (part == 0 && h < G) {
      const float e = ps[hb].count > 1 ? normalise(ml.x, ml.y, a.sink ? a.sink[kvh * G + h] * kLog2e : -INFINITY).lse2
                                       : a.lse2[bh + h];
      s_lse[h] = e == -INFINITY ? INFINITY : e;   // a head without any weight (every slot on a bad page) adds nothing
    }
  }
  __syncthreads();
  const int64_t at = ((int64_t)b * a.n_kv_heads + kvh) * a.slots;
  const bool split = G > 16;
  if (end > n) end = n;
  for (; s0 < end; s0 += weigh_slots(G)) {
    const int32_t s = s0 + (split ? 0 : warp * 128) + 4 * lane;
    const float* const sc = a.scores + bh * a.score_stride + s;
    // slots in lane order: rows of weights need not be aligned
    const int32_t first = split ? s0 + tid : s0 + warp * 128 + lane;
    const int mine = split ? 1 : 4;
    float old[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) old[i] = a.weights && i < mine && first + i * 32 < end ? a.weights[at + first + i * 32] : 0.f;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s < end) {   // a row of scores ends on a multiple of 32
#pragma unroll 8
      for (int h = split ? warp : 0; h < G; h += split ? 4 : 1) {
        const float4 z = *reinterpret_cast<const float4*>(sc + h * a.score_stride);
        const float e = s_lse[h];
        w.x += ex2(z.x - e);
        w.y += ex2(z.y - e);
        w.z += ex2(z.z - e);
        w.w += ex2(z.w - e);
      }
    }
    s_sum[warp][lane] = w;
    const float* const sum = reinterpret_cast<const float*>(s_sum);
    if (split) __syncthreads();
    else __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = split ? (sum[tid] + sum[128 + tid]) + (sum[256 + tid] + sum[384 + tid]) : sum[warp * 128 + i * 32 + lane];
      if (i < mine && first + i * 32 < end) a.weights_out[at + first + i * 32] = old[i] + v;
    }
    if (split) __syncthreads();
    else __syncwarp();
  }
}

// Blocks x < join_blocks join the pieces of the units that have several (or
// none: an empty sequence; the attention kernel has written the others);
// `split` of the block's four warps share a head's pieces.  The other blocks, with
// weights_out, weigh.
template <class T, int DP, int NB, int WH>
__global__ void __launch_bounds__(kThreads) kv_finish_kernel(const __grid_constant__ KvAttnArgs a, int join_blocks, int split, int weigh_per) {
  using Geo = Geometry<T, DP, NB, WH>;
  constexpr int ROWS = Geo::HEADS, V = DP / 64;   // float2 per lane
  __shared__ int64_t s_scan[4];
  __shared__ float2 s_ml[4];
  __shared__ float2 s_acc[4][V][32];
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.n_kv_heads, blocks = (G + ROWS - 1) / ROWS, HZ = a.n_kv_heads * blocks;
  // the lengths do not come from the attention kernel: read them while it runs
  if ((int)blockIdx.x >= join_blocks) {
    const int32_t n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, nullptr);
    const int32_t s0 = (blockIdx.x - join_blocks) * weigh_per;
    Pieces ps[kMaxBlocks];
    if (s0 < n)
#pragma unroll
      for (int hb = 0; hb < kMaxBlocks; ++hb)
        ps[hb] = a.whole || hb >= blocks ? Pieces{0, 0, 1, 0} : pieces_of<Geo::TILE>(a, b, HZ, kvh * blocks + hb, s_scan);
    pdl_wait();
    pdl_trigger();
    if (s0 < n) weigh<Geo::TILE, ROWS>(a, b, kvh, n, s0, s0 + weigh_per, ps, blocks);
    return;
  }
  const int first = blockIdx.x * (4 / split);   // 4 / split heads, in one head block
  const int hb = first / ROWS;
  const Pieces ps = pieces_of<Geo::TILE>(a, b, HZ, kvh * blocks + hb, s_scan);
  pdl_wait();
  pdl_trigger();
  if (ps.count == 1) return;
  const int h = first + warp / split, part = warp % split, row = h - hb * ROWS;
  float2 ml = make_float2(-INFINITY, 0.f);
  float2 acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = make_float2(0.f, 0.f);
  if (h < G) {
    for (int64_t i = part + split * (int64_t)lane; i < ps.count; i += split * 32)
      ml.x = fmaxf(ml.x, a.part_ml[(ps.at(i) * ROWS + row) * 2]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ml.x = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, o));
    const float R = ml.x == -INFINITY ? 0.f : ml.x;
#pragma unroll 8
    for (int64_t i = part; i < ps.count; i += split) {
      const int64_t at = ps.at(i) * ROWS + row;
      const float2 p = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      const float f = ex2(p.x - R);
      ml.y = fmaf(p.y, f, ml.y);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 y = *reinterpret_cast<const float2*>(a.part_acc + at * DP + j * 64 + 2 * lane);
        acc[j].x = fmaf(y.x, f, acc[j].x);
        acc[j].y = fmaf(y.y, f, acc[j].y);
      }
    }
  }
  if (split > 1) {
    if (lane == 0) s_ml[warp] = ml;
#pragma unroll
    for (int j = 0; j < V; ++j) s_acc[warp][j][lane] = acc[j];
    __syncthreads();
    if (part != 0) return;
    const float own = ml.x;
    for (int w = 1; w < split; ++w) ml = join_ml(ml, s_ml[warp + w]);
    const float R = ml.x == -INFINITY ? 0.f : ml.x, f0 = ex2(own - R);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      acc[j].x *= f0;
      acc[j].y *= f0;
      for (int w = 1; w < split; ++w) {
        const float f = ex2(s_ml[warp + w].x - R);
        acc[j].x = fmaf(s_acc[warp + w][j][lane].x, f, acc[j].x);
        acc[j].y = fmaf(s_acc[warp + w][j][lane].y, f, acc[j].y);
      }
    }
  }
  if (h >= G) return;
  const int64_t bh = (int64_t)b * a.H + (int64_t)kvh * G + h;
  const Norm nm = normalise(ml.x, ml.y, a.sink ? a.sink[kvh * G + h] * kLog2e : -INFINITY);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j * 64 + 2 * lane < a.d)
      *reinterpret_cast<uint32_t*>(a.out + (bh * a.d + j * 64 + 2 * lane) * 2) = pack2<T>(acc[j].x * nm.scale, acc[j].y * nm.scale);
  if (lane == 0 && a.lse) a.lse[bh] = nm.lse2 * (1.f / kLog2e);
}

// Tensor map of a cache's keys or values, [page][slot][head][coordinate], if 16
// consecutive slots from a multiple of 16 on lie on one page and no dimension is
// broadcast (a stride of 0).
bool tile_map(const char* data, int64_t page_st, int64_t slot_st, int64_t head_st, const KvAttnArgs& a, CUtensorMap* map) {
  const KvRef& kv = a.kv;
  if (kv.table != nullptr && kv.page_size % kKeys != 0) return false;
  const uint64_t dims[4] = {(uint64_t)a.d, (uint64_t)a.n_kv_heads, (uint64_t)kv.page_size, (uint64_t)kv.n_pages};
  int64_t st[3] = {head_st, slot_st, page_st};
  for (int i = 0; i < 3; ++i) {
    if (dims[i + 1] == 1) st[i] = (int64_t)a.d * 2 + (-(int64_t)a.d * 2 & 15);   // never stepped over
    if (st[i] <= 0 || st[i] >= (int64_t(1) << 40)) return false;
  }
  const uint64_t strides[3] = {(uint64_t)st[0], (uint64_t)st[1], (uint64_t)st[2]};
  return make_tmap_16bit_4d(map, data, dims, strides, 64, kKeys);
}

template <class T, int DP, int NB, int WH>
cudaError_t launch_typed(const Launch& L, const KvAttnArgs& args, const KvAttnPlan& p) {
  using Geo = Geometry<T, DP, NB, WH>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kv_attn_kernel<T, DP, NB, WH>, Geo::SMEM, done);
  if (e != cudaSuccess) return e;
  KvAttnArgs a = args;
  CUtensorMap map_k = {}, map_v = {};
  a.tiled = tile_map(a.kv.k, a.kv.k_page, a.kv.k_slot, a.kv.k_head, a, &map_k) &&
            tile_map(a.kv.v, a.kv.v_page, a.kv.v_slot, a.kv.v_head, a, &map_v);
  L.begin(kKernelAttention);
  e = launch_kernel(kv_attn_kernel<T, DP, NB, WH>, dim3((unsigned)p.n_ctas), dim3(kThreads), Geo::SMEM, L.stream, true, map_k,
                    map_v, a);
  if (e != cudaSuccess) return e;
  e = L.end(kKernelAttention);
  if (e != cudaSuccess || (p.whole && a.weights_out == nullptr)) return e;
  const int G = a.H / a.n_kv_heads;
  const int split = (int64_t)a.B * a.n_kv_heads * p.blocks * 4 > p.n_ctas ? 1 : 4;   // 4 where a unit has many pieces
  const int join = p.whole ? 0 : (G * split + 3) / 4;
  // weighing blocks long enough that about eight an SM do it all: each first
  // finds its unit's pieces and sums (32 sequences of up to 8192 slots, 8 heads a group: 26 -> 19 us)
  const int64_t total = (int64_t)a.B * a.n_kv_heads * a.max_len / (8 * kSms) + 1;
  const int weigh_per = (int)((total + weigh_slots(G) - 1) / weigh_slots(G)) * weigh_slots(G);
  const int weigh = a.weights_out ? (int)((a.max_len + weigh_per - 1) / weigh_per) : 0;
  if (join + weigh == 0) return cudaSuccess;
  L.begin(kKernelMerge);
  e = launch_kernel(kv_finish_kernel<T, DP, NB, WH>, dim3((unsigned)(join + weigh), (unsigned)a.n_kv_heads, (unsigned)a.B),
                    dim3(kThreads), 0, L.stream, true, a, join, split, weigh_per);
  if (e != cudaSuccess) return e;
  return L.end(kKernelMerge);
}

template <class T, int DP>
cudaError_t launch_wh(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  if (p.nb == 1) return launch_typed<T, DP, 1, 1>(L, a, p);
  return p.wh == 1 ? launch_typed<T, DP, 2, 1>(L, a, p) : p.wh == 2 ? launch_typed<T, DP, 2, 2>(L, a, p) : launch_typed<T, DP, 2, 4>(L, a, p);
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

KvAttnPlan kv_attn_plan(int32_t B, int32_t H, int32_t n_kv_heads, int32_t d, int64_t max_len, int32_t window,
                        bool invariant) {
  KvAttnPlan p{};
  const int G = H / n_kv_heads;
  p.nb = G <= 8 ? 1 : 2;
  p.wh = G <= 16 ? 1 : G <= 32 ? 2 : 4;
  p.heads = 8 * p.nb * p.wh;
  p.blocks = (G + p.heads - 1) / p.heads;
  p.dp = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256;
  p.tile = kKeys * 4 / p.wh;
  const int64_t units = (int64_t)B * n_kv_heads * p.blocks;
  int64_t most_slots = max_len;
  if (window > 0 && window + kKeys - 1 < most_slots) most_slots = window + kKeys - 1;   // it may start up to 15 slots early
  const int64_t tiles = (most_slots + p.tile - 1) / p.tile;
  p.atom = invariant ? kInvariantSlots / p.tile : 1;
  p.max_atoms = (tiles + p.atom - 1) / p.atom;
  p.whole = !invariant && tiles <= 4;
  const int64_t per_run = (int64_t)n_kv_heads * p.blocks;   // CTAs of a run
  const int64_t most = (int64_t)kSms * ctas_per_sm(p.dp, p.nb);
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
  return a.dtype == CSA_KV_FP16 ? launch_dp<__half>(L, a, p) : launch_dp<__nv_bfloat16>(L, a, p);
}

}  // namespace csa
