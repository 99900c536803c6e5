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
//     side by side on the same keys.  Rows come by 16-byte cp.async into
//     XOR-swizzled shared memory, page ids one step ahead of the copies.
//   * Softmax with a running maximum in base 2 and fp32; probabilities rounded
//     to the cache's type for P V (as every 16-bit tensor-core product needs),
//     their sum taken before that rounding.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv.cuh"

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

// A position in the batch's list of tiles.
struct Cursor {
  int32_t b, hz, tile;
  Span s;
};

// To the next sequence that has slots (a run's atoms lie on such sequences
// only: there is one while atoms are left).
template <int TILE>
__device__ __forceinline__ bool next_sequence(const KvAttnArgs& a, Cursor& c) {
  while (++c.b < a.B) {
    c.s = span_of<TILE>(a, c.b, a.err);
    if (c.s.tiles > 0) return true;
  }
  return false;
}

template <class T, int DP, int WH>
struct Geometry {
  static constexpr int NG = 4 / WH;                 // key groups of a CTA
  static constexpr int TILE = kKeys * NG;
  static constexpr int GROUP = 32 * WH;             // threads of a key group
  static constexpr int CH = DP / 8;                 // 16-byte pieces of a row
  static constexpr int ROW = DP * 2;
  static constexpr int STAGE = kKeys * ROW * 2;     // a group's keys and values
  static constexpr int STAGES = DP == 64 ? 5 : DP == 128 ? 3 : DP == 192 ? 4 : 3;
  static constexpr int RING = STAGES * STAGE * NG;
  static constexpr int JOIN = NG > 1 ? NG / 2 * WH * 16 * DP * 4 : 0;
  static constexpr int SMEM = RING + JOIN;
  static constexpr int CTAS = DP <= 128 ? 2 : 1;    // resident per SM
};

template <class T, int DP, int WH>
__global__ void __launch_bounds__(kThreads, (Geometry<T, DP, WH>::CTAS)) kv_attn_kernel(KvAttnArgs a) {
  using Geo = Geometry<T, DP, WH>;
  constexpr int NG = Geo::NG, TILE = Geo::TILE, S = Geo::STAGES, CH = Geo::CH, ROW = Geo::ROW;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_scan[8];
  __shared__ int64_t s_first[2];
  __shared__ float2 s_ml[4][16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WH, wh = warp % WH, gtid = tid % Geo::GROUP;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.H / a.n_kv_heads;
  const int blocks = (G + 16 * WH - 1) / (16 * WH);
  const int HZ = a.n_kv_heads * blocks;   // units of a sequence
  const uint32_t ring = smem_u32(smem) + kg * (S * Geo::STAGE);
  float* const s_join = reinterpret_cast<float*>(smem + Geo::RING);

  // ---- this CTA's run of atoms ------------------------------------------------
  Cursor c;
  int64_t atoms_left;
  int64_t first_atom = 0;   // of the unit the run begins in, relative to that unit
  if (a.whole) {
    c.b = blockIdx.x / HZ;
    c.hz = blockIdx.x - c.b * HZ;
    c.s = span_of<TILE>(a, c.b, a.err);
    c.tile = 0;
    atoms_left = 1;
  } else {
    int64_t all;
    atoms_before<TILE>(a, 0, &all, s_scan);
    all *= HZ;
    const int64_t share = share_of(a, all), begin = (int64_t)blockIdx.x * share;
    atoms_left = all - begin < share ? all - begin : share;
    if (atoms_left <= 0) return;
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
    first_atom = s_first[1] - c.hz * per_unit;
    c.tile = (int32_t)(first_atom * a.atom);
  }

  // ---- copies -----------------------------------------------------------------
  // The producer cursor runs S-1 steps ahead; the page ids of the step after
  // that are already on their way.
  Cursor p = c;
  int64_t p_left = a.whole ? (c.s.tiles > 0 ? 1 : 0) : atoms_left;
  const bool one_page = a.kv.table == nullptr || a.kv.page_size % kKeys == 0;
  int32_t l_page = -1, l_row = 0;   // lookup of the producer cursor's step
  auto lookup = [&]() {
    const int32_t s0 = p.s.start + p.tile * TILE + kg * kKeys;
    l_page = -1;
    if (one_page) {
      if (s0 < p.s.n) l_page = kv_page(a.kv, p.b, s0, &l_row, a.err);
    } else {
      const int32_t s = s0 + (lane & 15);
      if (s >= p.s.lo && s < p.s.n) l_page = kv_page(a.kv, p.b, s, &l_row, a.err);
    }
  };
  auto ends_atom = [&](const Cursor& x) {
    return x.tile + 1 == x.s.tiles || (x.tile + 1) % a.atom == 0;
  };
  // Issue the copies of the producer cursor's step into ring slot `st`; returns
  // the mask of its rows that exist.
  auto issue = [&](int st) -> uint32_t {
    const int32_t s0 = p.s.start + p.tile * TILE + kg * kKeys;
    uint32_t rows = 0;
    if (one_page) {
      if (l_page >= 0) {
        const int32_t end = p.s.n - s0;
        rows = end >= 16 ? 0xffffu : (1u << end) - 1u;
        if (s0 < p.s.lo) rows &= p.s.lo - s0 >= 16 ? 0u : 0xffffu << (p.s.lo - s0);
      }
    } else {
      rows = __ballot_sync(0xffffffffu, l_page >= 0) & 0xffffu;
    }
    const int h = p.hz / blocks;
    const char* const kb = a.kv.k + h * a.kv.k_head;
    const char* const vb = a.kv.v + h * a.kv.v_head;
    const int64_t page = l_page < 0 ? 0 : l_page;
    int64_t ko = page * a.kv.k_page + l_row * a.kv.k_slot;
    int64_t vo = page * a.kv.v_page + l_row * a.kv.v_slot;
    const uint32_t dst = ring + st * Geo::STAGE;
#pragma unroll
    for (int i = 0; i < 16 * CH / Geo::GROUP; ++i) {
      const int idx = i * Geo::GROUP + gtid, r = idx / CH, ch = idx % CH;
      int64_t kro, vro;
      if (one_page) {
        kro = ko + r * a.kv.k_slot;
        vro = vo + r * a.kv.v_slot;
      } else {
        kro = __shfl_sync(0xffffffffu, ko, r);
        vro = __shfl_sync(0xffffffffu, vo, r);
      }
      const bool ok = ((rows >> r) & 1u) && ch * 8 < a.d;
      const uint32_t at = dst + r * ROW + ((ch ^ (r & 7)) << 4);
      cp_async_16(at, ok ? kb + kro + 16 * ch : a.kv.k, ok);
      cp_async_16(at + kKeys * ROW, ok ? vb + vro + 16 * ch : a.kv.v, ok);
    }
    // step on
    if (ends_atom(p)) {
      if (a.whole ? p.tile + 1 == p.s.tiles : --p_left == 0) p_left = 0;
    }
    if (p_left > 0) {
      if (++p.tile == p.s.tiles) {
        p.tile = 0;
        if (++p.hz == HZ) {
          p.hz = 0;
          if (!next_sequence<TILE>(a, p)) p_left = 0;
        }
      }
      if (p_left > 0) lookup();
    }
    return rows;
  };
  auto group_sync = [&]() {
    if (WH == 1) __syncwarp();
    else if (WH == 4) __syncthreads();
    else named_barrier_sync(1 + kg, Geo::GROUP);
  };

  uint32_t rows_q[S - 1];   // masks of the steps in flight, oldest first
  if (p_left > 0) lookup();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    rows_q[i] = p_left > 0 ? issue(i) : 0u;
    cp_async_commit();
  }

  // ---- units --------------------------------------------------------------------
  int st = 0;   // ring slot of the current step
  bool continued = first_atom > 0;   // the unit began before this run
  const int kmat = lane >> 3, kr = lane & 7;
  // ldmatrix rows: keys are non-transposed pairs (dims lo, hi of 8 keys), values
  // transposed pairs (keys 0-7, 8-15 of 8 dims)
  const uint32_t k_lane = (kr + (kmat >> 1) * 8) * ROW + (((kmat & 1) ^ kr) << 4);
  const uint32_t v_lane = kKeys * ROW + (kr + (kmat & 1) * 8) * ROW + (((kmat >> 1) ^ kr) << 4);
  bool more = a.whole || atoms_left > 0;
  while (more) {
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
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
    const int32_t first_tile = c.tile;
    bool unit_done = c.s.tiles == 0;
    if (unit_done) more = false;   // an empty sequence with a CTA to itself
    while (!unit_done) {
      cp_async_wait<S - 2>();
      group_sync();   // the step's rows are in place, and everyone has left the slot that is filled next
      const uint32_t rows = rows_q[0];
#pragma unroll
      for (int i = 0; i + 1 < S - 1; ++i) rows_q[i] = rows_q[i + 1];
      {
        const int nst = st == 0 ? S - 1 : st - 1;
        rows_q[S - 2] = p_left > 0 ? issue(nst) : 0u;
        cp_async_commit();
      }
      const uint32_t base = ring + st * Geo::STAGE;
      st = st + 1 == S ? 0 : st + 1;

      float s[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        uint32_t kb[4];
        ldmatrix_x4(kb, base + (ks >> 2) * 128 + (k_lane ^ ((ks & 3) * 32)));
        mma16816<T>(s[0], q[ks], kb[0], kb[1]);
        mma16816<T>(s[1], q[ks], kb[2], kb[3]);
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = nt * 8 + 2 * t4 + (j & 1);
          s[nt][j] = (rows >> key) & 1u ? s[nt][j] * a.scale : -INFINITY;
        }
      if (a.scores != nullptr) {
        const int32_t s0 = c.s.start + c.tile * TILE + kg * kKeys + 2 * t4;
        float* const w = a.scores + (c.b * (int64_t)a.H + hq) * a.score_stride + s0;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          if (s0 + nt * 8 < c.s.n) {   // rows hold an even number of slots
            if (h_lo < G) *reinterpret_cast<float2*>(w + h_lo * a.score_stride + nt * 8) = make_float2(s[nt][0], s[nt][1]);
            if (h_hi < G) *reinterpret_cast<float2*>(w + h_hi * a.score_stride + nt * 8) = make_float2(s[nt][2], s[nt][3]);
          }
        }
      }
      float x_lo = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x_hi = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int off = 1; off <= 2; off <<= 1) {
        x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, off));
        x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, off));
      }
      if (__any_sync(0xffffffffu, x_lo > m_lo || x_hi > m_hi)) {
        const float n_lo = fmaxf(m_lo, x_lo), n_hi = fmaxf(m_hi, x_hi);
        const float f_lo = n_lo == -INFINITY ? 1.f : exp2f(m_lo - n_lo);
        const float f_hi = n_hi == -INFINITY ? 1.f : exp2f(m_hi - n_hi);
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
        const float p0 = exp2f(s[nt][0] - r_lo), p1 = exp2f(s[nt][1] - r_lo);
        const float p2 = exp2f(s[nt][2] - r_hi), p3 = exp2f(s[nt][3] - r_hi);
        l_lo += p0 + p1;
        l_hi += p2 + p3;
        pa[2 * nt] = pack2<T>(p0, p1);
        pa[2 * nt + 1] = pack2<T>(p2, p3);
      }
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        uint32_t vb[4];
        ldmatrix_x4_trans(vb, base + (j >> 2) * 128 + (v_lane ^ ((j & 3) * 32)));
        mma16816<T>(o[2 * j], pa, vb[0], vb[1]);
        mma16816<T>(o[2 * j + 1], pa, vb[2], vb[3]);
      }

      // next tile
      const bool last = c.tile + 1 == c.s.tiles;
      const bool atom_end = last || (c.tile + 1) % a.atom == 0;
      if (a.whole) {
        unit_done = last;
        more = !last;
      } else {
        if (atom_end) --atoms_left;
        unit_done = last || atoms_left == 0 || (a.invariant && atom_end);
        more = atoms_left > 0;
      }
      ++c.tile;
    }

    // ---- join the key groups, store --------------------------------------------
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, off);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, off);
    }
    if constexpr (NG > 1) {
      if (t4 == 0) {
        s_ml[warp][g] = make_float2(m_lo, l_lo);
        s_ml[warp][g + 8] = make_float2(m_hi, l_hi);
      }
      __syncthreads();
      float M_lo = -INFINITY, M_hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        M_lo = fmaxf(M_lo, s_ml[i * WH + wh][g].x);
        M_hi = fmaxf(M_hi, s_ml[i * WH + wh][g + 8].x);
      }
      const float R_lo = M_lo == -INFINITY ? 0.f : M_lo, R_hi = M_hi == -INFINITY ? 0.f : M_hi;
      l_lo = l_hi = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const float2 x = s_ml[i * WH + wh][g], y = s_ml[i * WH + wh][g + 8];
        l_lo += x.y * exp2f(x.x - R_lo);
        l_hi += y.y * exp2f(y.x - R_hi);
      }
      const float f_lo = exp2f(m_lo - R_lo), f_hi = exp2f(m_hi - R_hi);
      m_lo = M_lo;
      m_hi = M_hi;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        o[i][0] *= f_lo;
        o[i][1] *= f_lo;
        o[i][2] *= f_hi;
        o[i][3] *= f_hi;
      }
      // groups half, half+1, .. hand theirs down, log2(NG) times
#pragma unroll
      for (int half = NG / 2; half >= 1; half >>= 1) {
        float4* const buf = reinterpret_cast<float4*>(s_join) + (((kg % half) * WH + wh) * (DP / 8)) * 32 + lane;
        if (kg >= half && kg < 2 * half) {
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) buf[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
        __syncthreads();
        if (kg < half) {
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const float4 x = buf[i * 32];
            o[i][0] += x.x;
            o[i][1] += x.y;
            o[i][2] += x.z;
            o[i][3] += x.w;
          }
        }
        if (half > 1) __syncthreads();
      }
    }
    const bool whole_unit = first_tile == 0 && c.tile == c.s.tiles;   // no other piece exists
    if (kg == 0) {
      const int64_t bh = (int64_t)c.b * a.H + hq;
      if (whole_unit) {
        const float z_lo = a.sink && h_lo < G ? a.sink[hq + h_lo] * kLog2e : -INFINITY;
        const float z_hi = a.sink && h_hi < G ? a.sink[hq + h_hi] * kLog2e : -INFINITY;
        const float M_lo = fmaxf(m_lo, z_lo), M_hi = fmaxf(m_hi, z_hi);
        const float R_lo = M_lo == -INFINITY ? 0.f : M_lo, R_hi = M_hi == -INFINITY ? 0.f : M_hi;
        const float f_lo = exp2f(m_lo - R_lo), f_hi = exp2f(m_hi - R_hi);
        const float L_lo = l_lo * f_lo + exp2f(z_lo - R_lo), L_hi = l_hi * f_hi + exp2f(z_hi - R_hi);
        const float i_lo = L_lo == 0.f ? 0.f : f_lo / L_lo, i_hi = L_hi == 0.f ? 0.f : f_hi / L_hi;
        if (t4 == 0) {
          const float e_lo = L_lo == 0.f ? -INFINITY : R_lo + log2f(L_lo);
          const float e_hi = L_hi == 0.f ? -INFINITY : R_hi + log2f(L_hi);
          if (a.lse) {
            if (h_lo < G) a.lse[bh + h_lo] = e_lo * (1.f / kLog2e);
            if (h_hi < G) a.lse[bh + h_hi] = e_hi * (1.f / kLog2e);
          }
          if (a.lse2) {
            if (h_lo < G) a.lse2[bh + h_lo] = e_lo;
            if (h_hi < G) a.lse2[bh + h_hi] = e_hi;
          }
        }
        char* const out_lo = a.out + (bh + h_lo) * a.d * 2;
        char* const out_hi = out_lo + 8 * a.d * 2;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const int d0 = i * 8 + 2 * t4;
          if (d0 < a.d) {
            if (h_lo < G) *reinterpret_cast<uint32_t*>(out_lo + 2 * d0) = pack2<T>(o[i][0] * i_lo, o[i][1] * i_lo);
            if (h_hi < G) *reinterpret_cast<uint32_t*>(out_hi + 2 * d0) = pack2<T>(o[i][2] * i_hi, o[i][3] * i_hi);
          }
        }
      } else {
        const int64_t unit = (int64_t)c.b * HZ + c.hz;
        const int64_t piece = a.invariant ? unit * a.max_atoms + first_tile / a.atom
                                          : 2 * (int64_t)blockIdx.x + (continued ? 0 : 1);
        const int row = wh * 16 + g;
        float* const acc = a.part_acc + (piece * (16 * WH) + row) * DP;
        float* const ml = a.part_ml + (piece * (16 * WH) + row) * 2;
        if (t4 == 0) {
          *reinterpret_cast<float2*>(ml) = make_float2(m_lo, l_lo);
          *reinterpret_cast<float2*>(ml + 16) = make_float2(m_hi, l_hi);
        }
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          *reinterpret_cast<float2*>(acc + i * 8 + 2 * t4) = make_float2(o[i][0], o[i][1]);
          *reinterpret_cast<float2*>(acc + 8 * DP + i * 8 + 2 * t4) = make_float2(o[i][2], o[i][3]);
        }
      }
    }
    continued = false;
    if (more) {
      if (c.tile == c.s.tiles) {
        c.tile = 0;
        if (++c.hz == HZ) {
          c.hz = 0;
          if (!next_sequence<TILE>(a, c)) more = false;
        }
      }
    }
  }
  cp_async_wait<0>();
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

template <class T, int DP, int WH>
cudaError_t launch_typed(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  using Geo = Geometry<T, DP, WH>;
  cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<T, DP, WH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::SMEM);
  if (e != cudaSuccess) return e;
  L.begin(kKernelAttention);
  e = launch_kernel(kv_attn_kernel<T, DP, WH>, dim3((unsigned)p.n_ctas), dim3(kThreads), Geo::SMEM, L.stream, true, a);
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
