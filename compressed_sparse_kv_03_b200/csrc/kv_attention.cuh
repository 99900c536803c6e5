// What the two kernels of csa_kv_attn_decode share (kv_attention.cu for groups of
// up to 16 query heads and for wide heads, kv_attention_tc.cu for larger groups):
// how the batch is cut into runs, and the kernel that joins and weighs.
#pragma once

#include <cuda_fp16.h>

#include "kernels.h"
#include "kv.cuh"
#include "tc.cuh"

namespace csa {
namespace kvattn {

constexpr int kFinishThreads = 128;
constexpr int kSms = 148;
constexpr int kInvariantSlots = 512;
// Head blocks that a group may have: up to 128 heads, 64 at a time, or 32 wide ones.
constexpr int max_blocks(int dp, int rows) { return dp > 128 ? (rows == 32 ? 4 : 1) : rows == 64 ? 2 : 1; }

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

// fp16 ends at 2^-14 (2^-24 with fewer bits), and the probabilities of a long cache
// can lie below that and still make the output together; they are rounded to the
// type as p * 2^LIFT, with sums and O on that scale until the segment's end (powers
// of two: exact).  `top` is log2 of the largest p that occurs; fp16 holds 2^15.
// bf16 has the exponents of fp32 and needs none.
template <class T>
constexpr int lift(int top) { return __is_same(T, __half) ? (top > 0 ? 15 - top : 14) : 0; }

// Slots that a query sees: [lo, n); tiles start at lo rounded down to ALIGN, so
// that ALIGN slots from there lie on one page wherever page_size is a multiple of it.
struct Span {
  int32_t n, lo, start, tiles;
};
template <int TILE, int ALIGN>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, int32_t b, WsHeader* err) {
  Span s;
  s.n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, err);
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.start = s.lo & ~(ALIGN - 1);
  s.tiles = (s.n - s.start + TILE - 1) / TILE;
  return s;
}

template <int TILE, int ALIGN>
__device__ __forceinline__ int64_t atoms_of(const KvAttnArgs& a, int32_t b) {   // of a unit of sequence b
  return (span_of<TILE, ALIGN>(a, b, nullptr).tiles + a.atom - 1) / a.atom;
}

// Sum over the block's THREADS threads, and of the threads before this one.
template <int THREADS>
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
  for (int w = 0; w < THREADS / 32; ++w) {
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
template <int TILE, int ALIGN>
__device__ __forceinline__ bool next_segment(const KvAttnArgs& a, Cursor& c) {
  if (c.left <= 0) return false;
  if (c.tile == c.s.tiles) {
    c.tile = 0;
    do {
      if (++c.b >= a.B) return false;
      c.s = span_of<TILE, ALIGN>(a, c.b, a.err);
    } while (c.s.tiles == 0);
  }
  open_segment(a, c);
  return true;
}

// The position that run `run` of the batch begins at (all THREADS threads; false:
// it is empty).  Each thread has a stretch of sequences; the one that holds the
// run's first atom finds it.
template <int TILE, int ALIGN, int THREADS>
__device__ __forceinline__ bool begin_run(const KvAttnArgs& a, int run, Cursor& c, int64_t* scratch, int64_t* found) {
  if (a.whole) {
    c.b = run;
    c.s = span_of<TILE, ALIGN>(a, c.b, a.err);
    c.tile = 0;
  } else {
    const int32_t per = (a.B + THREADS - 1) / THREADS, b0 = threadIdx.x * per, b1 = b0 + per < a.B ? b0 + per : a.B;
    int64_t mine = 0, before;
    for (int32_t b = b0; b < b1; ++b) mine += atoms_of<TILE, ALIGN>(a, b);
    const int64_t all = block_scan<THREADS>(mine, &before, scratch);
    const int64_t share = share_of(a, all), begin = run * share;
    c.left = all - begin < share ? all - begin : share;
    if (c.left <= 0) return false;
    if (begin >= before && begin < before + mine) {
      int32_t b = b0;
      for (int64_t n; b + 1 < b1 && before + (n = atoms_of<TILE, ALIGN>(a, b)) <= begin; ++b) before += n;
      found[0] = b;
      found[1] = begin - before;
    }
    __syncthreads();
    c.b = (int32_t)found[0];
    c.s = span_of<TILE, ALIGN>(a, c.b, a.err);
    c.tile = (int32_t)(found[1] * a.atom);
  }
  open_segment(a, c);
  return true;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// p * 2^LIFT of log2 p (multiplied, not added to the exponent, whose bits it would cost)
template <int LIFT>
__device__ __forceinline__ float lifted(float x) {
  return ex2(x) * (float)(1 << LIFT);
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

// ---- joining --------------------------------------------------------------------
// Pieces of a unit: its first, how many, and the step from one to the next.
struct Pieces {
  int64_t first, second;   // piece 0, and pieces 1, 2, .. from `second` on by `step`
  int64_t count;
  int step;
  __device__ __forceinline__ int64_t at(int64_t i) const { return i == 0 ? first : second + (i - 1) * step; }
};
template <int TILE, int ALIGN>
__device__ Pieces pieces_of(const KvAttnArgs& a, int32_t b, int HZ, int hz, int64_t* scratch) {
  const int64_t atoms = atoms_of<TILE, ALIGN>(a, b);
  if (a.invariant) {
    const int64_t first = ((int64_t)b * HZ + hz) * a.max_atoms;
    return Pieces{first, first + 1, atoms, 1};
  }
  int64_t mine = 0, low = 0, x;
  for (int32_t i = threadIdx.x; i < a.B; i += kFinishThreads) {
    const int64_t n = atoms_of<TILE, ALIGN>(a, i);
    mine += n;
    if (i < b) low += n;
  }
  const int64_t all = block_scan<kFinishThreads>(mine, &x, scratch), base = block_scan<kFinishThreads>(low, &x, scratch);
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
template <int ROWS, int BLOCKS>
__device__ void weigh(const KvAttnArgs& a, int b, int kvh, int32_t n, int32_t s0, int32_t end, const Pieces* ps, int blocks) {
  __shared__ float2 s_part[kFinishThreads];
  __shared__ float s_lse[128];
  __shared__ float4 s_sum[4][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.H / a.n_kv_heads;
  const int64_t bh = (int64_t)b * a.H + (int64_t)kvh * G;
  const int row = tid % ROWS, part = tid / ROWS;
  constexpr int PARTS = kFinishThreads / ROWS;
#pragma unroll
  for (int hb = 0; hb < BLOCKS; ++hb) {
    if (hb >= blocks) break;
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
#pragma unroll 4
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
template <class T, int DP, int TILE, int ALIGN, int ROWS>
__global__ void __launch_bounds__(kFinishThreads) kv_finish_kernel(const __grid_constant__ KvAttnArgs a, int join_blocks, int split, int weigh_per) {
  constexpr int V = DP / 64;   // float2 per lane
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
    constexpr int BLOCKS = max_blocks(DP, ROWS);
    Pieces ps[BLOCKS];
    if (s0 < n)
#pragma unroll
      for (int hb = 0; hb < BLOCKS; ++hb)
        ps[hb] = a.whole || hb >= blocks ? Pieces{0, 0, 1, 0} : pieces_of<TILE, ALIGN>(a, b, HZ, kvh * blocks + hb, s_scan);
    pdl_wait();
    pdl_trigger();
    if (s0 < n) weigh<ROWS, BLOCKS>(a, b, kvh, n, s0, s0 + weigh_per, ps, blocks);
    return;
  }
  const int first = blockIdx.x * (4 / split);   // 4 / split heads, in one head block
  const int hb = first / ROWS;
  const Pieces ps = pieces_of<TILE, ALIGN>(a, b, HZ, kvh * blocks + hb, s_scan);
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
#pragma unroll 4
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

// Tensor map of a cache's keys or values, [page][slot][head][coordinate], in boxes
// of `rows` slots, if `rows` consecutive slots from a multiple of it on lie on one
// page and no dimension is broadcast (a stride of 0).
inline bool tile_map(const char* data, int64_t page_st, int64_t slot_st, int64_t head_st, const KvAttnArgs& a, int rows,
                     CUtensorMap* map) {
  const KvRef& kv = a.kv;
  if (kv.table != nullptr && kv.page_size % rows != 0) return false;
  const uint64_t dims[4] = {(uint64_t)a.d, (uint64_t)a.n_kv_heads, (uint64_t)kv.page_size, (uint64_t)kv.n_pages};
  int64_t st[3] = {head_st, slot_st, page_st};
  for (int i = 0; i < 3; ++i) {
    if (dims[i + 1] == 1) st[i] = (int64_t)a.d * 2 + (-(int64_t)a.d * 2 & 15);   // never stepped over
    if (st[i] <= 0 || st[i] >= (int64_t(1) << 40)) return false;
  }
  const uint64_t strides[3] = {(uint64_t)st[0], (uint64_t)st[1], (uint64_t)st[2]};
  return make_tmap_16bit_4d(map, data, dims, strides, 64, rows);
}

// The second launch: joins, and with weights_out weighs.
template <class T, int DP, int TILE, int ALIGN, int ROWS>
cudaError_t launch_finish(const Launch& L, const KvAttnArgs& a, const KvAttnPlan& p) {
  if (p.whole && a.weights_out == nullptr) return cudaSuccess;
  const int G = a.H / a.n_kv_heads;
  // warps of a head: 4 where a unit has many pieces.  The order of the sums follows
  // it, so with fixed slices it is fixed as well
  const int split = !a.invariant && (int64_t)a.B * a.n_kv_heads * p.blocks * 4 > p.n_ctas ? 1 : 4;
  const int join = p.whole ? 0 : (G * split + 3) / 4;
  // weighing blocks long enough that about eight an SM do it all: each first
  // finds its unit's pieces and sums (32 sequences of up to 8192 slots, 8 heads a group: 26 -> 19 us)
  const int64_t total = (int64_t)a.B * a.n_kv_heads * a.max_len / (8 * kSms) + 1;
  const int weigh_per = (int)((total + weigh_slots(G) - 1) / weigh_slots(G)) * weigh_slots(G);
  const int weigh = a.weights_out ? (int)((a.max_len + weigh_per - 1) / weigh_per) : 0;
  if (join + weigh == 0) return cudaSuccess;
  L.begin(kKernelMerge);
  const cudaError_t e = launch_kernel(kv_finish_kernel<T, DP, TILE, ALIGN, ROWS>, dim3((unsigned)(join + weigh), (unsigned)a.n_kv_heads, (unsigned)a.B),
                    dim3(kFinishThreads), 0, L.stream, true, a, join, split, weigh_per);
  if (e != cudaSuccess) return e;
  return L.end(kKernelMerge);
}

}  // namespace kvattn
}  // namespace csa
