// Eviction from a per-head key-value cache by accumulated attention weight
// (csa_kv_evict).
//
// Per (sequence, KV head) with n slots: an exact select of the `budget` best
// keys (held slots first, then the weight), then every slot below the budget
// that lost its row takes the row of a staying slot above it.  Filling holes
// moves at most min(n - budget, budget) rows; compacting in order would move
// nearly every kept row (256 slots over a budget of 2048: 2048 rows a head
// instead of about 256).
//
// One cluster of CTAs per (sequence, head).  Each warp owns a run of consecutive
// slots, so ranks are prefix sums over warps and a ballot within a warp:
//   1. keys from weights and positions, kept in shared memory while they fit;
//   2. radix select, 8 bits a pass: a histogram per CTA, summed over the
//      cluster through distributed shared memory;
//   3. equal keys ranked by slot; the staying slots above the budget and the
//      holes below it are numbered in order and listed;
//   4. all CTAs of the cluster copy the listed rows, 16 bytes a thread.
// Sources lie at or above the budget and targets below it, so the copies need
// no order.
#include <cooperative_groups.h>

#include "kernels.h"
#include "kv.cuh"

namespace cg = cooperative_groups;

namespace csa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxCachedKeys = 24576;   // 96 KB of keys per CTA
constexpr int kUnroll = 4;              // row pieces in flight per thread
constexpr uint32_t kHeld = 0xffffffffu;

__device__ __forceinline__ uint32_t slot_key(const KvEvictArgs& a, int64_t at, int32_t newest) {
  const int32_t p = a.slot_pos[at];
  if ((int64_t)p > (int64_t)newest - a.recent || p < a.keep_first) return kHeld;
  const float w = a.weights[at];
  return w != w ? kHeld - 1 : score_key(w);   // +inf is below kHeld - 1
}

struct Shared {
  uint32_t hist[4][256];
  int32_t warp_eq[kWarps], warp_hole[kWarps], warp_move[kWarps];
  int32_t cta_eq, cta_hole, cta_move;
  uint32_t bin, above, count;
};

__global__ void __launch_bounds__(kThreads) kv_evict_kernel(KvEvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t unit = blockIdx.x / cs;
  const int b = (int)(unit / a.n_kv_heads), h = (int)(unit - (int64_t)b * a.n_kv_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t base = unit * a.slots;      // of weights and slot_pos
  const int32_t n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, a.err);
  const int32_t budget = a.budget;
  const int32_t left = n < budget ? n : budget;
  const bool inplace = a.weights_out == a.weights;
  const bool pos_inplace = a.slot_pos_out == a.slot_pos;

  if (h == 0 && rank == 0 && tid == 0 && a.lens_out != a.lens) a.lens_out[b] = left;
  // beyond the old length both arrays are zero
  for (int64_t j = n + rank * kThreads + tid; j < a.max_len; j += (int64_t)cs * kThreads) {
    a.weights_out[base + j] = 0.f;
    a.slot_pos_out[base + j] = 0;
  }
  if (a.src_out)
    for (int64_t j = left + rank * kThreads + tid; j < budget; j += (int64_t)cs * kThreads)
      a.src_out[unit * budget + j] = -1;
  if (n <= budget) {   // nothing leaves (the whole cluster takes this branch)
    for (int j = rank * kThreads + tid; j < n; j += cs * kThreads) {
      if (!inplace) a.weights_out[base + j] = a.weights[base + j];
      if (!pos_inplace) a.slot_pos_out[base + j] = a.slot_pos[base + j];
      if (a.src_out) a.src_out[unit * budget + j] = j;
    }
    return;
  }

  const int32_t newest = __ldg(a.pos + b);
  // runs of whole 32-slot rows, one per warp of the cluster
  const int32_t run = (int32_t)((((int64_t)n + cs * kWarps - 1) / (cs * kWarps) + 31) / 32 * 32);
  const int64_t cta0 = (int64_t)rank * kWarps * run;
  const int64_t w0 = cta0 + (int64_t)warp * run;
  const int32_t w_end = (int32_t)(w0 + run < n ? w0 + run : n);
  const bool cached = (int64_t)run * kWarps <= a.key_cap;

  for (int i = tid; i < 4 * 256; i += kThreads) (&s.hist[0][0])[i] = 0;
  __syncthreads();

  auto key_at = [&](int32_t j) -> uint32_t {
    return cached ? s_keys[j - cta0] : slot_key(a, base + j, newest);
  };

  // ---- the budget-th largest key -------------------------------------------
  uint32_t prefix = 0;
  uint32_t need = (uint32_t)budget, equal = 0;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int32_t j = (int32_t)w0 + lane; j < w_end; j += 32) {
      uint32_t key;
      if (pass == 0) {
        key = slot_key(a, base + j, newest);
        if (cached) s_keys[j - cta0] = key;
      } else {
        key = key_at(j);
      }
      if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&s.hist[pass][(key >> shift) & 255u], 1u);
    }
    cluster.sync();
    if (warp < 8) {   // 8 warps, one bin per thread, bins in descending order
      const int bin = 255 - tid;
      uint32_t c = 0;
      for (int r = 0; r < cs; ++r) c += *cluster.map_shared_rank(&s.hist[pass][bin], r);
      uint32_t up = c;   // keys in this bin and the higher ones of the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      if (lane == 31) s.warp_eq[warp] = (int32_t)up;
      named_barrier_sync(1, 256);
      for (int w = 0; w < warp; ++w) up += (uint32_t)s.warp_eq[w];
      if (up >= need && up - c < need) {
        s.bin = (uint32_t)bin;
        s.above = up - c;
        s.count = c;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | s.bin;
    need -= s.above;
    equal = s.count;
  }
  const uint32_t cut = prefix;   // keys above it stay, and the `need` lowest slots of the `equal` on it

  // ---- ranks of the equal keys ---------------------------------------------
  int32_t eq_before = 0;
  if (need < equal) {
    int32_t c = 0;
    for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32) {
      const int32_t j = j0 + lane;
      c += __popc(__ballot_sync(0xffffffffu, j < w_end && key_at(j) == cut));
    }
    if (lane == 0) s.warp_eq[warp] = c;
    __syncthreads();
    if (tid == 0) {
      int32_t t = 0;
      for (int w = 0; w < kWarps; ++w) t += s.warp_eq[w];
      s.cta_eq = t;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) eq_before += *cluster.map_shared_rank(&s.cta_eq, r);
    for (int w = 0; w < warp; ++w) eq_before += s.warp_eq[w];
  }
  // Calls f(j, stays) for the warp's slots, a 32-slot row at a time (j >= w_end: none).
  auto walk = [&](auto f) {
    int32_t rank_eq = eq_before;
    for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32) {
      const int32_t j = j0 + lane;
      const uint32_t key = j < w_end ? key_at(j) : 0u;
      const bool eq = j < w_end && key == cut;
      bool stays = j < w_end && key > cut;
      if (need < equal) {
        const uint32_t m = __ballot_sync(0xffffffffu, eq);
        stays |= eq && (uint32_t)(rank_eq + __popc(m & ((1u << lane) - 1u))) < need;
        rank_eq += __popc(m);
      } else {
        stays |= eq;
      }
      f(j, stays);
    }
  };
  // ---- number the holes and the movers -------------------------------------
  int32_t holes = 0, moves = 0;
  walk([&](int32_t j, bool stays) {
    holes += __popc(__ballot_sync(0xffffffffu, j < w_end && j < budget && !stays));
    moves += __popc(__ballot_sync(0xffffffffu, j >= budget && stays));
  });
  if (lane == 0) {
    s.warp_hole[warp] = holes;
    s.warp_move[warp] = moves;
  }
  __syncthreads();
  if (tid == 0) {
    int32_t x = 0, y = 0;
    for (int w = 0; w < kWarps; ++w) x += s.warp_hole[w], y += s.warp_move[w];
    s.cta_hole = x;
    s.cta_move = y;
  }
  cluster.sync();
  int32_t hole_at = 0, move_at = 0, total = 0;
  for (int r = 0; r < cs; ++r) {
    const int32_t x = *cluster.map_shared_rank(&s.cta_hole, r);
    if (r < rank) {
      hole_at += x;
      move_at += *cluster.map_shared_rank(&s.cta_move, r);
    }
    total += x;   // as many holes as movers: exactly `budget` slots stay
  }
  for (int w = 0; w < warp; ++w) hole_at += s.warp_hole[w], move_at += s.warp_move[w];

  // ---- list them; the slots that keep or lose what they hold ----------------
  int32_t* const to = a.list + unit * 2 * a.list_len;
  int32_t* const from = to + a.list_len;
  walk([&](int32_t j, bool stays) {
    const uint32_t below = (1u << lane) - 1u;
    const bool hole = j < w_end && j < budget && !stays, mover = j >= budget && stays;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole) to[hole_at + __popc(mh & below)] = j;
    if (mover) from[move_at + __popc(mm & below)] = j;
    hole_at += __popc(mh);
    move_at += __popc(mm);
    if (j < w_end && j < budget && stays) {
      if (!inplace) a.weights_out[base + j] = a.weights[base + j];
      if (!pos_inplace) a.slot_pos_out[base + j] = a.slot_pos[base + j];
      if (a.src_out) a.src_out[unit * budget + j] = j;
    }
    if (j < w_end && j >= budget) {   // in place a mover's are cleared once they have been read
      if (!inplace || !mover) a.weights_out[base + j] = 0.f;
      if (!pos_inplace || !mover) a.slot_pos_out[base + j] = 0;
    }
  });
  cluster.sync();   // the lists are complete (and no CTA leaves while its counts are read)

  // ---- move rows -------------------------------------------------------------
  const uint32_t per_row = a.shared ? a.chunks : 2 * a.chunks;   // 16-byte pieces of a key and a value
  const uint32_t items = (uint32_t)total * per_row;   // budget <= 2^24: below 2^30
  const uint32_t step = cs * kThreads;
  for (uint32_t i0 = rank * kThreads + tid; i0 < items; i0 += step * kUnroll) {
    uint4 val[kUnroll];
    char* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      dst[u] = nullptr;
      if (i >= items) continue;
      const uint32_t pair = i / per_row;
      const int p = (int)(i - pair * per_row);
      const int32_t d_slot = to[pair], s_slot = from[pair];
      if (p == 0) {
        a.weights_out[base + d_slot] = a.weights[base + s_slot];
        a.slot_pos_out[base + d_slot] = a.slot_pos[base + s_slot];
        if (inplace) a.weights_out[base + s_slot] = 0.f;
        if (pos_inplace) a.slot_pos_out[base + s_slot] = 0;
        if (a.src_out) a.src_out[unit * budget + d_slot] = s_slot;
      }
      int32_t d_row, s_row;
      const int32_t d_page = kv_page(a.kv, b, d_slot, &d_row, a.err);
      const int32_t s_page = kv_page(a.kv, b, s_slot, &s_row, a.err);
      if (d_page < 0 || s_page < 0) continue;
      if (p < a.chunks) {
        const int64_t off = h * a.kv.k_head + 16 * p;
        val[u] = *reinterpret_cast<const uint4*>(a.kv.k + s_page * a.kv.k_page + s_row * a.kv.k_slot + off);
        dst[u] = a.kv.k + d_page * a.kv.k_page + d_row * a.kv.k_slot + off;
      } else {
        const int64_t off = h * a.kv.v_head + 16 * (p - a.chunks);
        val[u] = *reinterpret_cast<const uint4*>(a.kv.v + s_page * a.kv.v_page + s_row * a.kv.v_slot + off);
        dst[u] = a.kv.v + d_page * a.kv.v_page + d_row * a.kv.v_slot + off;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = val[u];
  }
}

// lens in place: after every block has read them.
__global__ void __launch_bounds__(256) kv_evict_lengths_kernel(KvEvictArgs a) {
  const int32_t b = blockIdx.x * 256 + threadIdx.x;
  if (b >= a.B) return;
  const int32_t n = kv_clamp_len(a.lens[b], a.max_len, b, nullptr);
  a.lens_out[b] = n < a.budget ? n : a.budget;
}

}  // namespace

cudaError_t launch_kv_evict(const Launch& L, const KvEvictArgs& args) {
  KvEvictArgs a = args;
  const int64_t units = (int64_t)a.B * a.n_kv_heads;
  int cs = 1;
  while (cs < kMaxCluster && a.max_len > 512 * cs && (a.max_len > 4096 * cs || units * cs * 2 <= 148)) cs *= 2;
  const int64_t run = ((a.max_len + cs * kWarps - 1) / (cs * kWarps) + 31) / 32 * 32;
  a.key_cap = (int32_t)(run * kWarps <= kMaxCachedKeys ? run * kWarps : kMaxCachedKeys);
  const size_t smem = (size_t)a.key_cap * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxCachedKeys * (int)sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  L.begin(kKernelKvEvict);
  e = cudaLaunchKernelEx(&cfg, kv_evict_kernel, a);
  if (e != cudaSuccess) return e;
  e = L.end(kKernelKvEvict);
  if (e != cudaSuccess || a.lens_out != a.lens) return e;
  kv_evict_lengths_kernel<<<(unsigned)((a.B + 255) / 256), 256, 0, L.stream>>>(a);
  return L.end(kKernelKvEvict);
}

}  // namespace csa
