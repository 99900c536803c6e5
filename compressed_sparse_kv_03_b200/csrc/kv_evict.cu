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
// One cluster of CTAs per (sequence, head), of one CTA where the sequences and
// heads fill the GPU by themselves.  Each warp owns a run of consecutive slots, so
// ranks are prefix sums over warps and a ballot within a warp:
//   1. keys from weights and positions, kept in shared memory while they fit;
//   2. radix select, 8 bits a pass: a histogram per CTA, summed over the
//      cluster through distributed shared memory, until the bin that holds the
//      budget-th key is wholly kept, or holds at most 64 keys, which are ranked
//      directly by (key, slot); where more than 64 equal keys (slots that were
//      never looked at) straddle the budget, they are ranked by slot;
//   3. the staying slots above the budget and the holes below it are numbered
//      in order and listed;
//   4. a thread per listed row looks its pages up and moves its weight and
//      position, then all threads copy the rows, 16 bytes each: in the same launch
//      by a CTA that lists at most 512 rows, else by a second one whose CTAs take
//      64 rows each (a prompt cut from 65536 slots to 4096 in 16 heads: 55 -> 47 us).
// Sources lie at or above the budget and targets below it, so the copies need
// no order.  Bound by latency (a chain of about five loads and ten barriers)
// until some hundred rows move, then by HBM.
#include <cooperative_groups.h>

#include "kernels.h"
#include "kv.cuh"

namespace cg = cooperative_groups;

namespace csa {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxCachedKeys = 24576;   // 96 KB of keys per CTA
constexpr int kUnroll = 4;              // row pieces in flight per thread
constexpr int kLoads = 9;               // weights and positions in flight per thread
constexpr int kFew = 64;                // keys of a bin that are ranked directly
constexpr int kSmemList = 512;          // moves listed in shared memory (clusters of one)
constexpr int kMoveThreads = 256, kMoveRows = 64;   // of a CTA of the second launch
constexpr uint32_t kHeld = 0xffffffffu;

__device__ __forceinline__ uint32_t slot_key(const KvEvictArgs& a, float w, int32_t p, int32_t newest) {
  if ((int64_t)p > (int64_t)newest - a.recent || p < a.keep_first) return kHeld;
  return w != w ? kHeld - 1 : score_key(w);   // +inf is below kHeld - 1
}

template <int WARPS>
struct Shared {
  uint32_t hist[4][256];
  int32_t warp_a[WARPS], warp_b[WARPS];
  int32_t cta_a, cta_b;
  uint32_t bin, above, count;
  uint32_t few_n;
  uint64_t few[kFew];                 // the cluster's keys of the bin: key, then the lower slot first
  uint64_t least[WARPS], cta_least;
  uint32_t key_and[4], key_or[4];     // of a pass's candidates
  uint32_t cut;
  int32_t cut_slot;
  int32_t list[2 * kSmemList];
  int4 pages[kSmemList];
};

// Rows first .. first + count - 1 of the unit's lists; `pages`: shared memory for
// count entries.
template <int THREADS>
__device__ __forceinline__ void move_rows(const KvEvictArgs& a, int64_t unit, int b, int h, const int32_t* to, const int32_t* from,
                                          int first, int count, int4* pages) {
  const int64_t base = unit * a.slots;
  const int tid = threadIdx.x;
  for (int i = tid; i < count; i += THREADS) {
    const int32_t d_slot = to[first + i], s_slot = from[first + i];
    a.weights_out[base + d_slot] = a.weights[base + s_slot];
    a.slot_pos_out[base + d_slot] = a.slot_pos[base + s_slot];
    if (a.weights_out == a.weights) a.weights_out[base + s_slot] = 0.f;
    if (a.slot_pos_out == a.slot_pos) a.slot_pos_out[base + s_slot] = 0;
    if (a.src_out) a.src_out[unit * a.budget + d_slot] = s_slot;
    int4 pg;   // (from page, row, to page, row); from page -1: not copied
    pg.x = kv_page(a.kv, b, s_slot, &pg.y, a.err);
    pg.z = kv_page(a.kv, b, d_slot, &pg.w, a.err);
    if (pg.z < 0) pg.x = -1;
    pages[i] = pg;
  }
  __syncthreads();
  const uint32_t per_row = a.shared ? a.chunks : 2 * a.chunks;   // 16-byte pieces of a key and a value
  const uint32_t items = (uint32_t)count * per_row;
  for (uint32_t i0 = tid; i0 < items; i0 += THREADS * kUnroll) {
    uint4 val[kUnroll];
    char* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * THREADS;
      const uint32_t row = i / per_row;
      const int4 pg = i < items ? pages[row] : make_int4(-1, 0, 0, 0);
      const int p = (int)(i - row * per_row);
      const bool is_v = p >= a.chunks;
      const int64_t off = is_v ? h * a.kv.v_head + 16 * (p - a.chunks) : h * a.kv.k_head + 16 * p;
      const int64_t page_st = is_v ? a.kv.v_page : a.kv.k_page, slot_st = is_v ? a.kv.v_slot : a.kv.k_slot;
      char* const data = (is_v ? a.kv.v : a.kv.k) + off;
      dst[u] = pg.x >= 0 ? data + pg.z * page_st + pg.w * slot_st : nullptr;
      if (pg.x >= 0) val[u] = *reinterpret_cast<const uint4*>(data + pg.x * page_st + pg.y * slot_st);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = val[u];
  }
}

// CLUSTER: several CTAs per unit (without, all that reaches across them is left
// out: the kernel runs once through cold code).
template <int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_evict_kernel(const __grid_constant__ KvEvictArgs a) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ uint32_t s_keys[];
  __shared__ Shared<WARPS> s;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  auto sync = [&]() {
    if constexpr (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  // a value of CTA r of the cluster
  auto of = [&](auto* p, int r) {
    if constexpr (CLUSTER) return *cluster.map_shared_rank(p, r);
    else return *p;
  };
  const int64_t unit = blockIdx.x / cs;
  const int b = (int)(unit / a.n_kv_heads), h = (int)(unit - (int64_t)b * a.n_kv_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t base = unit * a.slots;      // of weights and slot_pos
  const int32_t newest = __ldg(a.pos + b);
  const int32_t n = kv_clamp_len(__ldg(a.lens + b), a.max_len, b, a.err);
  const int32_t budget = a.budget;
  const int32_t left = n < budget ? n : budget;
  const bool inplace = a.weights_out == a.weights;
  const bool pos_inplace = a.slot_pos_out == a.slot_pos;

  if (h == 0 && rank == 0 && tid == 0 && a.lens_out != a.lens) a.lens_out[b] = left;
  // arrays of their own are zero beyond the old length
  if (!inplace || !pos_inplace)
    for (int64_t j = n + rank * THREADS + tid; j < a.max_len; j += (int64_t)cs * THREADS) {
      if (!inplace) a.weights_out[base + j] = 0.f;
      if (!pos_inplace) a.slot_pos_out[base + j] = 0;
    }
  if (a.src_out)
    for (int64_t j = left + rank * THREADS + tid; j < budget; j += (int64_t)cs * THREADS)
      a.src_out[unit * budget + j] = -1;
  const bool near = cs == 1 && a.list_len <= kSmemList;   // the rows are moved here
  if (n <= budget) {   // nothing leaves (the whole cluster takes this branch)
    if (!near && rank == 0 && tid == 0) a.moves[unit] = 0;
#pragma unroll 4
    for (int j = rank * THREADS + tid; j < n; j += cs * THREADS) {
      if (!inplace) a.weights_out[base + j] = a.weights[base + j];
      if (!pos_inplace) a.slot_pos_out[base + j] = a.slot_pos[base + j];
      if (a.src_out) a.src_out[unit * budget + j] = j;
    }
    return;
  }

  // runs of whole 32-slot rows, one per warp of the cluster
  const int32_t run = (int32_t)((((int64_t)n + cs * WARPS - 1) / (cs * WARPS) + 31) / 32 * 32);
  const int64_t cta0 = (int64_t)rank * WARPS * run;
  const int64_t w0 = cta0 + (int64_t)warp * run;
  const int32_t w_end = (int32_t)(w0 + run < n ? w0 + run : n);
  const bool cached = (int64_t)run * WARPS <= a.key_cap;

  for (int i = tid; i < 4 * 256; i += THREADS) (&s.hist[0][0])[i] = 0;
  if (tid < 4) {
    s.key_and[tid] = 0xffffffffu;
    s.key_or[tid] = 0u;
  }
  if (tid == 0) s.few_n = 0;
  __syncthreads();

  auto key_at = [&](int32_t j) -> uint32_t {
    return cached ? s_keys[j - cta0] : slot_key(a, a.weights[base + j], a.slot_pos[base + j], newest);
  };

  // One slot too many (a step at the budget): no threshold is needed, only the
  // least (key, higher slot first).
  const bool one = n - budget == 1;
  uint64_t least = ~0ull;

  // ---- the budget-th largest (key, lower slot first) ---------------------------
  uint32_t prefix = 0, need = (uint32_t)budget, cut = 0;
  int32_t cut_slot = 0x7fffffff;   // slots on the cut stay up to this one
  int last_shift = 0;
  bool few = false, ties = false;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    if (pass == 0) {
      uint32_t held = 0;   // one shared address for all of them: counted per thread
      for (int32_t j0 = (int32_t)w0 + lane; j0 < w_end; j0 += 32 * kLoads) {
        float w[kLoads];
        int32_t sp[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int32_t j = j0 + 32 * u;
          w[u] = j < w_end ? a.weights[base + j] : 0.f;
          sp[u] = j < w_end ? a.slot_pos[base + j] : 0;
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int32_t j = j0 + 32 * u;
          if (j >= w_end) break;
          const uint32_t key = slot_key(a, w[u], sp[u], newest);
          if (cached) s_keys[j - cta0] = key;
          if (one) {
            const uint64_t x = (uint64_t)key << 32 | (uint32_t)~j;
            least = x < least ? x : least;
          } else if (key == kHeld) {
            ++held;
          } else {
            atomicAdd(&s.hist[0][key >> 24], 1u);
          }
          // as if every slot below the budget stayed: the holes are overwritten
          if (!inplace) a.weights_out[base + j] = j < budget ? w[u] : 0.f;
          if (!pos_inplace) a.slot_pos_out[base + j] = j < budget ? sp[u] : 0;
          if (a.src_out && j < budget) a.src_out[unit * budget + j] = j;
        }
      }
      if (one) break;
      held = __reduce_add_sync(0xffffffffu, held);
      if (lane == 0 && held) atomicAdd(&s.hist[0][255], held);
    } else {
      uint32_t all_and = 0xffffffffu, all_or = 0u;
#pragma unroll 4
      for (int32_t j = (int32_t)w0 + lane; j < w_end; j += 32) {
        const uint32_t key = key_at(j);
        if ((key >> (shift + 8)) != prefix) continue;
        atomicAdd(&s.hist[pass][(key >> shift) & 255u], 1u);
        all_and &= key;
        all_or |= key;
      }
      all_and = __reduce_and_sync(0xffffffffu, all_and);
      all_or = __reduce_or_sync(0xffffffffu, all_or);
      if (lane == 0 && all_or != 0u) {
        atomicAnd(&s.key_and[pass], all_and);
        atomicOr(&s.key_or[pass], all_or);
      }
    }
    sync();
    if (warp < 8) {   // one bin per thread, bins in descending order
      const int bin = 255 - tid;
      uint32_t c = 0;
      if (cs == 1) {
        c = s.hist[pass][bin];
      } else {
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) c += r < cs ? of(&s.hist[pass][bin], r) : 0u;
      }
      uint32_t up = c;   // keys in this bin and the higher ones of the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      if (lane == 31) s.warp_a[warp] = (int32_t)up;
      named_barrier_sync(1, 256);
      for (int w = 0; w < warp; ++w) up += (uint32_t)s.warp_a[w];
      if (up >= need && up - c < need) {
        s.bin = (uint32_t)bin;
        s.above = up - c;
        s.count = c;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | s.bin;
    need -= s.above;
    const uint32_t count = s.count;
    cut = prefix << shift;
    last_shift = shift;
    if (need == count) break;          // the whole bin stays
    if (count <= kFew) {
      few = true;
      break;
    }
    if (pass > 0) {
      uint32_t all_and = s.key_and[pass], all_or = s.key_or[pass];
      for (int r = 0; cs > 1 && r < cs; ++r) all_and &= of(&s.key_and[pass], r), all_or |= of(&s.key_or[pass], r);
      if (all_and == all_or) {         // all candidates are one key
        cut = all_and;
        ties = true;
        break;
      }
    }
    ties = pass == 3;                  // all of the bin's are
  }
  if (few) {   // rank the bin's keys: they gather in every CTA, in any order
    for (int32_t j = (int32_t)w0 + lane; j < w_end; j += 32) {
      const uint32_t key = key_at(j);
      if ((key >> last_shift) != prefix) continue;
      const uint64_t x = (uint64_t)key << 32 | (uint32_t)~j;
      if (cs == 1) {
        s.few[atomicAdd(&s.few_n, 1u)] = x;
      } else {
        const uint32_t at = atomicAdd(cluster.map_shared_rank(&s.few_n, 0), 1u);
        for (int r = 0; r < cs; ++r) *cluster.map_shared_rank(&s.few[at], r) = x;
      }
    }
    sync();
    if (warp < kFew / 32) {
      const int m = (int)s.count;
      const uint64_t mine = tid < m ? s.few[tid] : 0;
      uint32_t above = 0;
#pragma unroll 16
      for (int k = 0; k < kFew; ++k) above += k < m && s.few[k] > mine;
      if (tid < m && above == need - 1) {
        s.cut = (uint32_t)(mine >> 32);
        s.cut_slot = (int32_t)~(uint32_t)mine;
      }
    }
    __syncthreads();
    cut = s.cut;
    cut_slot = s.cut_slot;
  }
  if (ties) {   // the need-th lowest slot of those on the cut
    int32_t c = 0;
    for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32)
      c += __popc(__ballot_sync(0xffffffffu, j0 + lane < w_end && key_at(j0 + lane) == cut));
    if (lane == 0) s.warp_a[warp] = c;
    __syncthreads();
    const int32_t x = lane < WARPS ? s.warp_a[lane] : 0;
    int32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
    if (cs > 1) {
      const int32_t sum = __reduce_add_sync(0xffffffffu, x);
      if (tid == 0) s.cta_a = sum;
      cluster.sync();
      before += __reduce_add_sync(0xffffffffu, lane < rank ? *cluster.map_shared_rank(&s.cta_a, lane) : 0);
    }
    if (before < (int32_t)need && before + c >= (int32_t)need) {   // in this warp's run
      for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32) {
        const bool eq = j0 + lane < w_end && key_at(j0 + lane) == cut;
        const uint32_t m = __ballot_sync(0xffffffffu, eq);
        if (eq && before + __popc(m & ((2u << lane) - 1u)) == (int32_t)need) {
          if (cs == 1) s.cut_slot = j0 + lane;
          else
            for (int r = 0; r < cs; ++r) *cluster.map_shared_rank(&s.cut_slot, r) = j0 + lane;
        }
        before += __popc(m);
      }
    }
    sync();
    cut_slot = s.cut_slot;
  }

  // ---- number the holes and the movers -------------------------------------
  int32_t* const to = near ? s.list : a.list + unit * 2 * a.list_len;
  int32_t* const from = near ? s.list + kSmemList : to + a.list_len;
  auto stays = [&](int32_t j) {
    const uint32_t key = key_at(j);
    return key > cut || (key == cut && j <= cut_slot);
  };
  int32_t total = 0;
  if (one) {
    auto warp_least = [](uint64_t x) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, x, o);
        x = y < x ? y : x;
      }
      return x;
    };
    least = warp_least(least);
    if (lane == 0) s.least[warp] = least;
    __syncthreads();
    least = warp_least(lane < WARPS ? s.least[lane] : ~0ull);
    if (cs > 1) {
      if (tid == 0) s.cta_least = least;
      cluster.sync();
      least = warp_least(lane < cs ? *cluster.map_shared_rank(&s.cta_least, lane) : ~0ull);
    }
    const int32_t out = (int32_t)~(uint32_t)least;
    total = out < budget;   // the slot above the budget takes its place, or leaves itself
    if (rank == 0 && tid == 0) {
      if (total) {
        to[0] = out;
        from[0] = budget;
      } else {
        if (inplace) a.weights_out[base + budget] = 0.f;
        if (pos_inplace) a.slot_pos_out[base + budget] = 0;
      }
    }
  } else {
    int32_t holes = 0, moves = 0;
#pragma unroll 4
    for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32) {
      const int32_t j = j0 + lane;
      const bool in = j < w_end, st = in && stays(j);
      holes += __popc(__ballot_sync(0xffffffffu, in && j < budget && !st));
      moves += __popc(__ballot_sync(0xffffffffu, j >= budget && st));
    }
    __syncthreads();   // warp_a may still be read
    if (lane == 0) {
      s.warp_a[warp] = holes;
      s.warp_b[warp] = moves;
    }
    __syncthreads();
    const int32_t wa = lane < WARPS ? s.warp_a[lane] : 0, wb = lane < WARPS ? s.warp_b[lane] : 0;
    int32_t hole_at = __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    int32_t move_at = __reduce_add_sync(0xffffffffu, lane < warp ? wb : 0);
    total = __reduce_add_sync(0xffffffffu, wa);   // as many holes as movers: exactly `budget` slots stay
    if (cs > 1) {
      const int32_t y = __reduce_add_sync(0xffffffffu, wb);
      if (tid == 0) {
        s.cta_a = total;
        s.cta_b = y;
      }
      cluster.sync();
      const int32_t ra = lane < cs ? *cluster.map_shared_rank(&s.cta_a, lane) : 0;
      const int32_t rb = lane < rank ? *cluster.map_shared_rank(&s.cta_b, lane) : 0;
      hole_at += __reduce_add_sync(0xffffffffu, lane < rank ? ra : 0);
      move_at += __reduce_add_sync(0xffffffffu, rb);
      total = __reduce_add_sync(0xffffffffu, ra);
    }

    // ---- list them -------------------------------------------------------------
#pragma unroll 4
    for (int32_t j0 = (int32_t)w0; j0 < w_end; j0 += 32) {
      const int32_t j = j0 + lane;
      const uint32_t below = (1u << lane) - 1u;
      const bool in = j < w_end, st = in && stays(j);
      const bool hole = in && j < budget && !st, mover = st && j >= budget;
      const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
      if (hole) to[hole_at + __popc(mh & below)] = j;
      if (mover) from[move_at + __popc(mm & below)] = j;
      hole_at += __popc(mh);
      move_at += __popc(mm);
      if (in && j >= budget && !mover) {   // in place a mover's are cleared once they have been read
        if (inplace) a.weights_out[base + j] = 0.f;
        if (pos_inplace) a.slot_pos_out[base + j] = 0;
      }
    }
  }
  sync();   // the lists are complete (and no CTA leaves while its counts are read)

  // ---- move rows, or leave that to the next launch --------------------------------
  if (near) {
    move_rows<THREADS>(a, unit, b, h, to, from, 0, total, s.pages);
  } else if (rank == 0 && tid == 0) {
    a.moves[unit] = total;
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const __grid_constant__ KvEvictArgs a) {
  __shared__ int4 s_pages[kMoveRows];
  pdl_wait();
  const int64_t unit = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (unit >= (int64_t)a.B * a.n_kv_heads) return;
  const int first = blockIdx.x * kMoveRows;
  const int total = a.moves[unit];
  if (first >= total) return;
  const int b = (int)(unit / a.n_kv_heads), h = (int)(unit - (int64_t)b * a.n_kv_heads);
  const int32_t* const to = a.list + unit * 2 * a.list_len;
  move_rows<kMoveThreads>(a, unit, b, h, to, to + a.list_len, first, total - first < kMoveRows ? total - first : kMoveRows, s_pages);
}

// lens in place: after every block has read them.
__global__ void __launch_bounds__(256) kv_evict_lengths_kernel(KvEvictArgs a) {
  const int32_t b = blockIdx.x * 256 + threadIdx.x;
  if (b >= a.B) return;
  const int32_t n = kv_clamp_len(a.lens[b], a.max_len, b, nullptr);
  a.lens_out[b] = n < a.budget ? n : a.budget;
}

}  // namespace

template <int THREADS, bool CLUSTER>
static cudaError_t launch_threads(const Launch& L, KvEvictArgs& a, int cs) {
  const int64_t units = (int64_t)a.B * a.n_kv_heads;
  const int per = cs * THREADS;   // slots a run advances by
  const int64_t run = ((a.max_len + per / 32 - 1) / (per / 32) + 31) / 32 * 32 * (THREADS / 32);
  a.key_cap = (int32_t)(run <= kMaxCachedKeys ? run : kMaxCachedKeys);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kv_evict_kernel<THREADS, CLUSTER>, kMaxCachedKeys * (int)sizeof(uint32_t), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)a.key_cap * sizeof(uint32_t);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  L.begin(kKernelKvEvict);
  e = cudaLaunchKernelEx(&cfg, kv_evict_kernel<THREADS, CLUSTER>, a);
  if (e != cudaSuccess) return e;
  return L.end(kKernelKvEvict);
}

// CTAs per (sequence, head) and their threads (64 registers each): all resident at
// once.  Up to 296 units take 512 threads, and clusters of up to eight while a CTA
// keeps 1024 slots and two CTAs an SM hold them all (clusters of 1024-thread CTAs
// did not all find room in the GPU's processing clusters and ran in two waves).
cudaError_t launch_kv_evict(const Launch& L, const KvEvictArgs& args) {
  KvEvictArgs a = args;
  const int64_t units = (int64_t)a.B * a.n_kv_heads;
  int cs = 1;
  while (cs < kMaxCluster && a.max_len > 1024 * cs && (units * cs * 2 <= 296 || a.max_len > (int64_t)kMaxCachedKeys * cs)) cs *= 2;
  cudaError_t e = cs > 1 ? launch_threads<512, true>(L, a, cs)
                  : units <= 296 ? launch_threads<512, false>(L, a, cs) : launch_threads<256, false>(L, a, cs);
  if (e != cudaSuccess) return e;
  if (a.list_len > 0 && (cs > 1 || a.list_len > kSmemList)) {
    const unsigned y = (unsigned)(units < 32768 ? units : 32768);
    L.begin(kKernelKvEvict);
    e = launch_kernel(kv_evict_move_kernel, dim3((unsigned)((a.list_len + kMoveRows - 1) / kMoveRows), y, (unsigned)((units + y - 1) / y)),
                      dim3(kMoveThreads), 0, L.stream, true, a);
    if (e == cudaSuccess) e = L.end(kKernelKvEvict);
    if (e != cudaSuccess) return e;
  }
  if (a.lens_out != a.lens) return e;
  L.begin(kKernelKvEvict);
  kv_evict_lengths_kernel<<<(unsigned)((a.B + 255) / 256), 256, 0, L.stream>>>(a);
  return L.end(kKernelKvEvict);
}

}  // namespace csa
