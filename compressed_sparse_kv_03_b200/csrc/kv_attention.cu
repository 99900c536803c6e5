// Attention of one new token per sequence over a per-head key-value cache
// (csa_kv_attn_decode).
//
// Work: every seen key and value is read once for the G query heads of its
// group; 4 G d flops per 4 d bytes, so HBM bounds it for G <= 32 and the
// mma.sync rate above.  The layout follows from that:
//   * A unit is (sequence, KV head, block of up to 64 heads of its group).  Its
//     slots are cut into tiles, and the tiles of the whole batch, unit after
//     unit, into one equal run per CTA, whatever the lengths.  A CTA streams
//     through its run without draining its copies between units; a unit that
//     spans several CTAs leaves partial (O, max, sum) pieces that a second
//     kernel joins in CTA order.
//   * 16 heads are the M side of mma.m16n8k16, 16 keys a step.  Up to 16 heads,
//     the CTA's four warps take the tile's keys apart, each with a ring of its
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

// Atoms before sequence `b` and in the whole batch, per unit of a sequence;
// every thread of the block gets both (128 threads).
template <int TILE>
__device__ int64_t atoms_before(const KvAttnArgs& a, int32_t b, int64_t* all, int64_t* scratch) {
  int64_t before = 0, total = 0;
  for (int32_t i = threadIdx.x; i < a.B; i += kThreads) {
    const int64_t t = (span_of<TILE>(a, i, nullptr).tiles + a.atom - 1) / a.atom;
    total += t;
    if (i < b) before += t;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    scratch[threadIdx.x >> 5] = before;
    scratch[4 + (threadIdx.x >> 5)] = total;
  }
  __syncthreads();
  *all = scratch[4] + scratch[5] + scratch[6] + scratch[7];
  return scratch[0] + scratch[1] + scratch[2] + scratch[3];
}

// Atoms per CTA: equal shares.
__device__ __forceinline__ int64_t share_of(const KvAttnArgs& a, int64_t atoms) {
  return (atoms + a.n_ctas - 1) / a.n_ctas;
}

template <class T, int DP, int WH>
struct Geometry {
  static constexpr int NG = 4 / WH;                 // key groups of a CTA
  static constexpr int TILE = kKeys * NG;
  static constexpr int GROUP = 32 * WH;             // threads of a key group
  static constexpr int BOXES = DP / 64;             // 128-byte column blocks of a row
  static constexpr int BOX = kKeys * 128;           // bytes of 16 rows of one
  static constexpr int STAGE = 2 * BOXES * BOX;     // a group's keys, then values
  static constexpr int STAGES = DP == 64 ? 6 : 3;
  static constexpr int SMEM = STAGES * STAGE * NG + 1024;   // + alignment
  static constexpr int CTAS = DP <= 128 ? 2 : 1;    // resident per SM
  // O of 16 heads fits a stage: joins go through the one that was just read
  static_assert(STAGE == 16 * DP * 4, "a stage holds a warp's O");
};

// A position in this CTA's run of tiles.  A segment is the part of a unit that
// the CTA takes in one go (in batch-invariant mode a slice): tiles [.., end).
struct Cursor {
  int32_t b, hz, tile, end;
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
__device__ __forceinline__ bool next_segment(const KvAttnArgs& a, Cursor& c, int HZ) {
  if (c.left <= 0) return false;
  if (c.tile == c.s.tiles) {
    c.tile = 0;
    if (++c.hz == HZ) {
      c.hz = 0;
      do {
        if (++c.b >= a.B) return false;
        c.s = span_of<TILE>(a, c.b, a.err);
      } while (c.s.tiles == 0);
    }
  }
  open_segment(a, c);
  return true;
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

template <class T, int DP, int WH>
__global__ void __launch_bounds__(kThreads, (Geometry<T, DP, WH>::CTAS))
kv_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ KvAttnArgs a) {
  using Geo = Geometry<T, DP, WH>;
  constexpr int NG = Geo::NG, TILE = Geo::TILE, S = Geo::STAGES, BOX = Geo::BOX, BOXES = Geo::BOXES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // the swizzle's atoms are 1024 bytes
  __shared__ int64_t s_scan[8];
  __shared__ int64_t s_first[2];
  __shared__ float2 s_ml[4][16];
  __shared__ __align__(8) uint64_t s_bar[NG][S];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WH, wh = warp % WH;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.H / a.n_kv_heads;
  const int blocks = (G + 16 * WH - 1) / (16 * WH);
  const int HZ = a.n_kv_heads * blocks;   // units of a sequence
  const uint32_t ring = smem_u32(smem) + kg * (S * Geo::STAGE);
  const uint32_t bars = smem_u32(&s_bar[kg][0]);

  // ---- this CTA's run of atoms ------------------------------------------------
  Cursor c;
  if (a.whole) {
    c.b = blockIdx.x / HZ;
    c.hz = blockIdx.x - c.b * HZ;
    c.s = span_of<TILE>(a, c.b, a.err);
    c.tile = 0;
  } else {
    int64_t all;
    atoms_before<TILE>(a, 0, &all, s_scan);
    all *= HZ;
    const int64_t share = share_of(a, all), begin = (int64_t)blockIdx.x * share;
    c.left = all - begin < share ? all - begin : share;
    if (c.left <= 0) return;
    if (warp == 0) {   // the sequence that holds atom `begin`
      int64_t base = 0;
      for (int32_t b0 = 0; b0 < a.B; b0 += 32) {
        int64_t t = 0;
        if (b0 + lane < a.B)
          t = (int64_t)((span_of<TILE>(a, b0 + lane, nullptr).tiles + a.atom - 1) / a.atom) * HZ;
        int64_t up = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, base + up > begin);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            s_first[0] = b0 + lane;
            s_first[1] = begin - (base + up - t);
          }
          break;
        }
        base += __shfl_sync(0xffffffffu, up, 31);
      }
    }
    __syncthreads();
    c.b = (int32_t)s_first[0];
    c.s = span_of<TILE>(a, c.b, a.err);
    const int64_t per_unit = (c.s.tiles + a.atom - 1) / a.atom;
    c.hz = (int32_t)(s_first[1] / per_unit);
    c.tile = (int32_t)((s_first[1] - c.hz * per_unit) * a.atom);
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
    const int h = p.hz / blocks;
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
          tc::tma_load_4d(dst + lane * BOX, lane < BOXES ? &map_k : &map_v, (lane % BOXES) * 64, h, l_row, l_page, bar);
      }
    } else {
      rows = __ballot_sync(0xffffffffu, l_page >= 0) & 0xffffu;
      if (producer) {
        const int64_t page = l_page < 0 ? 0 : l_page;
        const int64_t ko = page * a.kv.k_page + l_row * a.kv.k_slot + h * a.kv.k_head;
        const int64_t vo = page * a.kv.v_page + l_row * a.kv.v_slot + h * a.kv.v_head;
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
    if (++p.tile == p.end) p_live = next_segment<TILE>(a, p, HZ);
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
  int st = 0;   // ring slot of the current step
  uint32_t phase = 0;
  bool dead = false;   // a wait ran out: no more waiting, the result is void
  const int kmat = lane >> 3, kr = lane & 7;
  // ldmatrix rows: keys in non-transposed pairs (dims lo, hi of 8 keys), values in
  // transposed ones (keys 0-7, 8-15 of 8 dims)
  const uint32_t k_lane = (kr + (kmat >> 1) * 8) * 128 + (((kmat & 1) ^ kr) << 4);
  const uint32_t v_lane = BOXES * BOX + (kr + (kmat & 1) * 8) * 128 + (((kmat >> 1) ^ kr) << 4);
  for (bool more = true; more;) {
    const int kvh = c.hz / blocks, hb = c.hz - kvh * blocks;
    const int h_lo = hb * 16 * WH + wh * 16 + g;    // heads of the group that this lane's rows are
    const int h_hi = h_lo + 8;
    const int64_t hq = (int64_t)kvh * G;
    uint32_t q[DP / 16][4];
    {
      const char* const q_lo = a.q + c.b * a.q_token + (hq + h_lo) * a.q_head;
      const char* const q_hi = q_lo + 8 * a.q_head;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        const int d0 = ks * 16 + 2 * t4;
        q[ks][0] = h_lo < G && d0 < a.d ? *reinterpret_cast<const uint32_t*>(q_lo + 2 * d0) : 0u;
        q[ks][1] = h_hi < G && d0 < a.d ? *reinterpret_cast<const uint32_t*>(q_hi + 2 * d0) : 0u;
        q[ks][2] = h_lo < G && d0 + 8 < a.d ? *reinterpret_cast<const uint32_t*>(q_lo + 2 * d0 + 16) : 0u;
        q[ks][3] = h_hi < G && d0 + 8 < a.d ? *reinterpret_cast<const uint32_t*>(q_hi + 2 * d0 + 16) : 0u;
      }
    }
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    // running maxima (of scaled scores, base 2) and this lane's part of the sums
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
    const int32_t first_tile = c.tile;
    float* sc = nullptr;
    if (a.scores != nullptr)
      sc = a.scores + (c.b * (int64_t)a.H + hq + h_lo) * a.score_stride + c.s.start + c.tile * TILE + kg * kKeys + 2 * t4;
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

      float sa[2][4] = {}, sb[2][4] = {};   // even and odd k-steps: shorter chains
#pragma unroll
      for (int ks = 0; ks < DP / 16; ks += 2) {
        uint32_t k0[4], k1[4];
        ldmatrix_x4(k0, base + (ks >> 2) * BOX + (k_lane ^ ((ks & 3) * 32)));
        ldmatrix_x4(k1, base + (ks >> 2) * BOX + (k_lane ^ ((ks & 3) * 32 + 32)));
        mma16816<T>(sa[0], q[ks], k0[0], k0[1]);
        mma16816<T>(sa[1], q[ks], k0[2], k0[3]);
        mma16816<T>(sb[0], q[ks + 1], k1[0], k1[1]);
        mma16816<T>(sb[1], q[ks + 1], k1[2], k1[3]);
      }
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] = (sa[nt][j] + sb[nt][j]) * a.scale;
      if (rows != 0xffffu) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((rows >> (nt * 8 + 2 * t4 + (j & 1))) & 1u)) s[nt][j] = -INFINITY;
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
        const int32_t s0 = c.s.start + c.tile * TILE + kg * kKeys + 2 * t4;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          if (s0 + nt * 8 < c.s.n) {   // rows hold an even number of slots
            if (h_lo < G) *reinterpret_cast<float2*>(sc + nt * 8) = make_float2(s[nt][0], s[nt][1]);
            if (h_hi < G) *reinterpret_cast<float2*>(sc + 8 * a.score_stride + nt * 8) = make_float2(s[nt][2], s[nt][3]);
          }
        }
        sc += TILE;
      }
      float x_lo = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x_hi = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (__any_sync(0xffffffffu, x_lo > m_lo || x_hi > m_hi)) {   // some row's maximum grows
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
          x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, off));
          x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, off));
        }
        const float n_lo = fmaxf(m_lo, x_lo), n_hi = fmaxf(m_hi, x_hi);
        const float f_lo = n_lo == -INFINITY ? 1.f : ex2(m_lo - n_lo);
        const float f_hi = n_hi == -INFINITY ? 1.f : ex2(m_hi - n_hi);
        m_lo = n_lo;
        m_hi = n_hi;
        l_lo *= f_lo;
        l_hi *= f_hi;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          o[i][0] *= f_lo;
          o[i][1] *= f_lo;
          o[i][2] *= f_hi;
          o[i][3] *= f_hi;
        }
      }
      const float r_lo = m_lo == -INFINITY ? 0.f : m_lo, r_hi = m_hi == -INFINITY ? 0.f : m_hi;
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float p0 = ex2(s[nt][0] - r_lo), p1 = ex2(s[nt][1] - r_lo);
        const float p2 = ex2(s[nt][2] - r_hi), p3 = ex2(s[nt][3] - r_hi);
        l_lo += p0 + p1;
        l_hi += p2 + p3;
        pa[2 * nt] = pack2<T>(p0, p1);
        pa[2 * nt + 1] = pack2<T>(p2, p3);
      }
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        uint32_t vb[4];
        ldmatrix_x4_trans(vb, base + (j >> 2) * BOX + (v_lane ^ ((j & 3) * 32)));
        mma16816<T>(o[2 * j], pa, vb[0], vb[1]);
        mma16816<T>(o[2 * j + 1], pa, vb[2], vb[3]);
      }
    }

    // ---- join the key groups, store --------------------------------------------
    // Everyone has read slot st - 1 to the end; the next step fills it.
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, off);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, off);
    }
    const bool whole_unit = first_tile == 0 && c.tile == c.s.tiles;   // no other piece exists
    const int64_t bh = (int64_t)c.b * a.H + hq;
    const int64_t piece = a.invariant ? ((int64_t)c.b * HZ + c.hz) * a.max_atoms + first_tile / a.atom
                                      : 2 * (int64_t)blockIdx.x + (continued ? 0 : 1);
    // Stores 4 (or 2) neighbouring columns of a row of heads.
    auto store_ml = [&](int row, float m, float l) {   // row: of the head block
      const int h = hb * 16 * WH + row;
      if (!whole_unit) {
        *reinterpret_cast<float2*>(a.part_ml + (piece * (16 * WH) + row) * 2) = make_float2(m, l);
      } else if (h < G) {
        const Norm nm = normalise(m, l, a.sink ? a.sink[hq + h] * kLog2e : -INFINITY);
        if (a.lse) a.lse[bh + h] = nm.lse2 * (1.f / kLog2e);
        if (a.lse2) a.lse2[bh + h] = nm.lse2;
      }
    };
    if constexpr (NG == 4) {
      // every warp puts its O down and sums a quarter of the columns of all four
      const int prev = st == 0 ? S - 1 : st - 1;
      float* const mine = reinterpret_cast<float*>(smem + (kg * S + prev) * Geo::STAGE);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        // 8-float blocks permuted by row, off the bank conflicts
        const int at = ((i ^ (g & 3)) * 8) + 2 * t4;
        *reinterpret_cast<float2*>(mine + g * DP + at) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(mine + (g + 8) * DP + at) = make_float2(o[i][2], o[i][3]);
      }
      if (t4 == 0) {
        s_ml[warp][g] = make_float2(m_lo, l_lo);
        s_ml[warp][g + 8] = make_float2(m_hi, l_hi);
      }
      __syncthreads();
      constexpr int F4 = DP / 16;   // float4 per row of a quarter
#pragma unroll
      for (int i = 0; i < 16 * F4 / 32; ++i) {
        const int idx = i * 32 + lane, row = idx / F4, col = warp * (DP / 4) + (idx % F4) * 4;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, s_ml[w][row].x);
        const float R = m == -INFINITY ? 0.f : m;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 ml = s_ml[w][row];
          const float f = ex2(ml.x - R);
          l = fmaf(ml.y, f, l);
          const float4 x = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + (w * S + prev) * Geo::STAGE) + row * DP + (col ^ ((row & 3) * 8)));
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
        const int h = hb * 16 + row;
        if (whole_unit) {
          if (h < G && col < a.d) {
            const float k = normalise(m, l, a.sink ? a.sink[hq + h] * kLog2e : -INFINITY).scale;
            uint2 pk;
            pk.x = pack2<T>(acc.x * k, acc.y * k);
            pk.y = pack2<T>(acc.z * k, acc.w * k);
            *reinterpret_cast<uint2*>(a.out + ((bh + h) * a.d + col) * 2) = pk;
          }
        } else {
          *reinterpret_cast<float4*>(a.part_acc + (piece * 16 + row) * DP + col) = acc;
        }
        if (col == 0) store_ml(row, m, l);
      }
      fence_async_smem_cta();
      __syncthreads();   // the slots may be filled again
    } else {
      if constexpr (NG == 2) {   // group 1 hands its O to group 0 through both groups' slots
        const int prev = st == 0 ? S - 1 : st - 1;
        float2* const buf = reinterpret_cast<float2*>(smem + (wh * S + prev) * Geo::STAGE) + lane;
        if (t4 == 0) {
          s_ml[warp][g] = make_float2(m_lo, l_lo);
          s_ml[warp][g + 8] = make_float2(m_hi, l_hi);
        }
        __syncthreads();   // and both groups have left their slots
        const float2 x_lo = s_ml[(1 - kg) * WH + wh][g], x_hi = s_ml[(1 - kg) * WH + wh][g + 8];
        const float M_lo = fmaxf(m_lo, x_lo.x), M_hi = fmaxf(m_hi, x_hi.x);
        const float R_lo = M_lo == -INFINITY ? 0.f : M_lo, R_hi = M_hi == -INFINITY ? 0.f : M_hi;
        const float f_lo = ex2(m_lo - R_lo), f_hi = ex2(m_hi - R_hi);
        l_lo = l_lo * f_lo + x_lo.y * ex2(x_lo.x - R_lo);
        l_hi = l_hi * f_hi + x_hi.y * ex2(x_hi.x - R_hi);
        m_lo = M_lo;
        m_hi = M_hi;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          o[i][0] *= f_lo;
          o[i][1] *= f_lo;
          o[i][2] *= f_hi;
          o[i][3] *= f_hi;
          if (kg == 1) {
            buf[(2 * i) * 32] = make_float2(o[i][0], o[i][1]);
            buf[(2 * i + 1) * 32] = make_float2(o[i][2], o[i][3]);
          }
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const float2 x = buf[(2 * i) * 32], y = buf[(2 * i + 1) * 32];
            o[i][0] += x.x;
            o[i][1] += x.y;
            o[i][2] += y.x;
            o[i][3] += y.y;
          }
        }
        fence_async_smem_cta();
        __syncthreads();
      }
      if (kg == 0) {
        const int row = wh * 16 + g;
        if (t4 == 0) {
          store_ml(row, m_lo, l_lo);
          store_ml(row + 8, m_hi, l_hi);
        }
        if (whole_unit) {
          const float k_lo = h_lo < G ? normalise(m_lo, l_lo, a.sink ? a.sink[hq + h_lo] * kLog2e : -INFINITY).scale : 0.f;
          const float k_hi = h_hi < G ? normalise(m_hi, l_hi, a.sink ? a.sink[hq + h_hi] * kLog2e : -INFINITY).scale : 0.f;
          char* const out_lo = a.out + (bh + h_lo) * a.d * 2;
          char* const out_hi = out_lo + 8 * a.d * 2;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const int d0 = i * 8 + 2 * t4;
            if (d0 < a.d) {
              if (h_lo < G) *reinterpret_cast<uint32_t*>(out_lo + 2 * d0) = pack2<T>(o[i][0] * k_lo, o[i][1] * k_lo);
              if (h_hi < G) *reinterpret_cast<uint32_t*>(out_hi + 2 * d0) = pack2<T>(o[i][2] * k_hi, o[i][3] * k_hi);
            }
          }
        } else {
          float* const acc = a.part_acc + (piece * (16 * WH) + row) * DP;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            *reinterpret_cast<float2*>(acc + i * 8 + 2 * t4) = make_float2(o[i][0], o[i][1]);
            *reinterpret_cast<float2*>(acc + 8 * DP + i * 8 + 2 * t4) = make_float2(o[i][2], o[i][3]);
          }
        }
      }
    }
    continued = false;
    more = next_segment<TILE>(a, c, HZ);
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
  const int32_t tiles = span_of<TILE>(a, b, nullptr).tiles;
  const int64_t atoms = (tiles + a.atom - 1) / a.atom;
  Pieces r;
  if (a.invariant) {
    r.first = ((int64_t)b * HZ + hz) * a.max_atoms;
    r.second = r.first + 1;
    r.count = atoms;
    r.step = 1;
    return r;
  }
  int64_t all;
  const int64_t base = atoms_before<TILE>(a, b, &all, scratch) * HZ + hz * atoms;
  const int64_t share = share_of(a, all * HZ);
  if (atoms == 0) {
    r.first = r.second = r.count = 0;
    r.step = 2;
    return r;
  }
  const int64_t c0 = base / share, c1 = (base + atoms - 1) / share;
  r.first = 2 * c0 + 1;   // it begins in c0's run; the others' runs begin in it
  r.second = 2 * (c0 + 1);
  r.count = c1 - c0 + 1;
  r.step = 2;
  return r;
}

constexpr int kWeighSlots = 1024;   // slots of a weighing block

// Blocks x < join_blocks: one warp per head joins that head's pieces (count 1:
// the attention kernel has written the result; 0: an empty sequence).  The
// others, with weights_out: the log-sum-exps of the group from the pieces,
// then the probabilities of the scores, summed over the group in head order.
template <class T, int DP, int WH>
__global__ void __launch_bounds__(kThreads) kv_finish_kernel(KvAttnArgs a, int join_blocks) {
  constexpr int TILE = Geometry<T, DP, WH>::TILE, ROWS = 16 * WH;
  __shared__ int64_t s_scan[8];
  __shared__ float s_lse[128];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.n_kv_heads, blocks = (G + ROWS - 1) / ROWS, HZ = a.n_kv_heads * blocks;
  const int64_t bh = (int64_t)b * a.H + (int64_t)kvh * G;

  if ((int)blockIdx.x < join_blocks) {
    if (a.whole) return;
    const int h = blockIdx.x * 4 + warp;
    const int hb = (blockIdx.x * 4) / ROWS;   // 4 divides the heads of a block
    const Pieces ps = pieces_of<TILE>(a, b, HZ, kvh * blocks + hb, s_scan);
    if (h >= G || ps.count == 1) return;
    const int row = h - hb * ROWS;
    const float z = a.sink ? a.sink[kvh * G + h] * kLog2e : -INFINITY;
    float M = z;
    for (int64_t i = lane; i < ps.count; i += 32) M = fmaxf(M, a.part_ml[(ps.at(i) * ROWS + row) * 2]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float R = M == -INFINITY ? 0.f : M;
    float den = z == -INFINITY ? 0.f : exp2f(z - R);
    float2 acc[DP / 64];
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) acc[j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int64_t i = 0; i < ps.count; ++i) {
      const int64_t at = ps.at(i) * ROWS + row;
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      const float f = exp2f(ml.x - R);
      den += ml.y * f;
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        const float2 x = *reinterpret_cast<const float2*>(a.part_acc + at * DP + j * 64 + 2 * lane);
        acc[j].x = fmaf(x.x, f, acc[j].x);
        acc[j].y = fmaf(x.y, f, acc[j].y);
      }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j)
      if (j * 64 + 2 * lane < a.d)
        *reinterpret_cast<uint32_t*>(a.out + ((bh + h) * a.d + j * 64 + 2 * lane) * 2) =
            pack2<T>(acc[j].x * inv, acc[j].y * inv);
    if (lane == 0 && a.lse) a.lse[bh + h] = den == 0.f ? -INFINITY : (R + log2f(den)) * (1.f / kLog2e);
    return;
  }

  const int32_t n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, nullptr);
  const int32_t s0 = (blockIdx.x - join_blocks) * kWeighSlots;
  if (s0 >= n) return;
  for (int hb = 0; hb < blocks; ++hb) {
    Pieces ps{0, 0, 1, 1};
    if (!a.whole) ps = pieces_of<TILE>(a, b, HZ, kvh * blocks + hb, s_scan);
    const int end = G - hb * ROWS < ROWS ? G - hb * ROWS : ROWS;
    for (int r = warp; r < end; r += 4) {
      const int h = hb * ROWS + r;
      float e;
      if (ps.count == 1) {
        e = a.lse2[bh + h];
      } else {
        const float z = a.sink ? a.sink[kvh * G + h] * kLog2e : -INFINITY;
        float M = z;
        for (int64_t i = lane; i < ps.count; i += 32) M = fmaxf(M, a.part_ml[(ps.at(i) * ROWS + r) * 2]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float R = M == -INFINITY ? 0.f : M;
        float den = 0.f;
        for (int64_t i = lane; i < ps.count; i += 32) {
          const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (ps.at(i) * ROWS + r) * 2);
          den += ml.y * exp2f(ml.x - R);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        if (z != -INFINITY) den += exp2f(z - R);
        e = R + log2f(den);
      }
      // a head without any weight (every slot on a bad page) adds nothing
      if (lane == 0) s_lse[h] = e == -INFINITY ? INFINITY : e;
    }
  }
  __syncthreads();
  const float* const sc = a.scores + bh * a.score_stride;
  const int64_t at = ((int64_t)b * a.n_kv_heads + kvh) * a.slots;
  const int32_t end = s0 + kWeighSlots < n ? s0 + kWeighSlots : n;
  for (int32_t s = s0 + threadIdx.x; s < end; s += kThreads) {
    float w = 0.f;
#pragma unroll 8
    for (int h = 0; h < G; ++h) w += exp2f(sc[h * a.score_stride + s] - s_lse[h]);
    a.weights_out[at + s] = a.weights ? a.weights[at + s] + w : w;
  }
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

template <class T, int DP, int WH>
cudaError_t launch_typed(const Launch& L, const KvAttnArgs& args, const KvAttnPlan& p) {
  using Geo = Geometry<T, DP, WH>;
  cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<T, DP, WH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::SMEM);
  if (e != cudaSuccess) return e;
  KvAttnArgs a = args;
  CUtensorMap map_k = {}, map_v = {};
  a.tiled = tile_map(a.kv.k, a.kv.k_page, a.kv.k_slot, a.kv.k_head, a, &map_k) &&
            tile_map(a.kv.v, a.kv.v_page, a.kv.v_slot, a.kv.v_head, a, &map_v);
  L.begin(kKernelAttention);
  e = launch_kernel(kv_attn_kernel<T, DP, WH>, dim3((unsigned)p.n_ctas), dim3(kThreads), Geo::SMEM, L.stream, true, map_k,
                    map_v, a);
  if (e != cudaSuccess) return e;
  e = L.end(kKernelAttention);
  if (e != cudaSuccess || (p.whole && a.weights_out == nullptr)) return e;
  const int G = a.H / a.n_kv_heads;
  const int join = p.whole ? 0 : (G + 3) / 4;
  const int weigh = a.weights_out ? (int)((a.max_len + kWeighSlots - 1) / kWeighSlots) : 0;
  L.begin(kKernelMerge);
  e = launch_kernel(kv_finish_kernel<T, DP, WH>, dim3((unsigned)(join + weigh), (unsigned)a.n_kv_heads, (unsigned)a.B),
                    dim3(kThreads), 0, L.stream, true, a, join);
  if (e != cudaSuccess) return e;
  return L.end(kKernelMerge);
}

template <class T, int DP>
cudaError_t launch_wh(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  return p.wh == 1 ? launch_typed<T, DP, 1>(L, a, p) : p.wh == 2 ? launch_typed<T, DP, 2>(L, a, p) : launch_typed<T, DP, 4>(L, a, p);
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
  p.wh = G <= 16 ? 1 : G <= 32 ? 2 : 4;
  p.blocks = (G + 16 * p.wh - 1) / (16 * p.wh);
  p.dp = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256;
  p.tile = kKeys * 4 / p.wh;
  const int64_t units = (int64_t)B * n_kv_heads * p.blocks;
  int64_t most_slots = max_len;
  if (window > 0 && window + kKeys - 1 < most_slots) most_slots = window + kKeys - 1;   // it may start up to 15 slots early
  const int64_t tiles = (most_slots + p.tile - 1) / p.tile;
  p.atom = invariant ? kInvariantSlots / p.tile : 1;
  p.max_atoms = (tiles + p.atom - 1) / p.atom;
  p.whole = !invariant && tiles <= 4;
  const int64_t most = (int64_t)kSms * (p.dp <= 128 ? 2 : 1);
  if (p.whole) {
    p.n_ctas = (int)units;
    p.pieces = 0;
  } else {
    const int64_t want = units * p.max_atoms;
    p.n_ctas = (int)(want < most ? want : most);
    p.pieces = invariant ? units * p.max_atoms : 2 * (int64_t)p.n_ctas;
  }
  return p;
}

cudaError_t launch_kv_attn(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  return a.dtype == CSA_KV_FP16 ? launch_dp<__half>(L, a, p) : launch_dp<__nv_bfloat16>(L, a, p);
}

}  // namespace csa
