// Appending tokens to a per-head key-value cache (csa_kv_append).
//
// A copy: every 16-byte piece of every new row is read once and written once to
// the page that its slot lies on.  Bound by HBM for prompts and by the launch
// and three dependent loads (length, page id, row) for a decode step.
//
// A token is a (sequence, index) pair.  Threads take the 16-byte pieces of a
// run of tokens in order, so that a warp reads and writes whole rows; each
// looks its token's slot up itself (the lookups of a row's threads hit the
// same line).  Lengths are written by the same launch when they go to an array
// of their own; in place they are written by a second one, since the first
// one's blocks read them at any time.
#include "kernels.h"
#include "kv.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;   // 16-byte pieces in flight per thread

struct Token {
  int32_t b, i;   // sequence and index among its new tokens; b < 0: none
};

__device__ __forceinline__ Token find_token(const KvAppendArgs& a, int32_t t) {
  if (a.token_start == nullptr) return Token{t, 0};
  int32_t lo = 0, hi = a.B;   // token_start[lo] <= t < token_start[hi]
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (__ldg(a.token_start + mid) <= t) lo = mid; else hi = mid;
  }
  const int32_t first = __ldg(a.token_start + lo);
  if (t < first || t >= __ldg(a.token_start + lo + 1)) return Token{-1, 0};
  return Token{lo, t - first};
}

// Slots that sequence b may use, and its length after the call.
__device__ __forceinline__ int64_t capacity(const KvAppendArgs& a) {
  const int64_t c = (int64_t)a.kv.max_pages * a.kv.page_size;
  return a.slots > 0 && a.slots < c ? a.slots : c;
}

__device__ __forceinline__ void write_length(const KvAppendArgs& a, int32_t b) {
  const int64_t n = a.lens[b];
  int64_t add = 1;
  if (a.token_start != nullptr) {
    const int64_t s0 = a.token_start[b], s1 = a.token_start[b + 1];
    // rows past n_tokens do not exist
    add = (s1 < a.n_tokens ? s1 : a.n_tokens) - (s0 > 0 ? s0 : 0);
    if (add < 0) add = 0;
  }
  int64_t m = n + add;
  const int64_t room = capacity(a);
  if (m > room) m = room;
  a.lens_out[b] = (int32_t)(n < 0 ? n : m);
}

__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvAppendArgs a) {
  pdl_trigger();
  const int pieces = a.chunks * a.n_kv_heads;          // 16-byte pieces of a key (or value) of all heads
  const int64_t total = a.n_tokens * 2 * pieces;
  const int64_t room = capacity(a);
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  uint4 val[kPieces];
  char* dst[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int64_t i = first + j * kThreads;
    dst[j] = nullptr;
    if (i >= total) continue;
    const int32_t t = (int32_t)(i / (2 * pieces));
    int p = (int)(i - (int64_t)t * (2 * pieces));
    const bool is_v = p >= pieces;
    if (is_v) p -= pieces;
    const int h = p / a.chunks, c = p - h * a.chunks;
    const Token tk = find_token(a, t);
    if (tk.b < 0) continue;
    const int32_t n = __ldg(a.lens + tk.b);
    const int64_t slot = (int64_t)n + tk.i;
    const bool leader = !is_v && c == 0;
    if (n < 0 || slot >= room) {
      if (leader && h == 0) report(a.err, n < 0 ? kErrLength : kErrRoom, tk.b, n < 0 ? n : slot);
      continue;
    }
    if (leader) {
      const int64_t at = ((int64_t)tk.b * a.n_kv_heads + h) * a.slots + slot;
      if (a.weights) a.weights[at] = 0.f;
      if (a.slot_pos) a.slot_pos[at] = __ldg(a.pos + tk.b) + tk.i;
    }
    int32_t row;
    const int32_t page = kv_page(a.kv, tk.b, (int32_t)slot, &row, a.err);
    if (page < 0) continue;
    const char* src;
    if (is_v) {
      src = a.v_new + t * a.v_token + h * a.v_head + 16 * c;
      dst[j] = a.kv.v + page * a.kv.v_page + row * a.kv.v_slot + h * a.kv.v_head + 16 * c;
    } else {
      src = a.k_new + t * a.k_token + h * a.k_head + 16 * c;
      dst[j] = a.kv.k + page * a.kv.k_page + row * a.kv.k_slot + h * a.kv.k_head + 16 * c;
    }
    val[j] = *reinterpret_cast<const uint4*>(src);
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (dst[j] != nullptr) *reinterpret_cast<uint4*>(dst[j]) = val[j];
  if (a.lens_out != a.lens)
    for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < a.B; b += (int64_t)gridDim.x * kThreads)
      write_length(a, (int32_t)b);
}

__global__ void __launch_bounds__(kThreads) kv_append_lengths_kernel(KvAppendArgs a) {
  pdl_wait();   // the blocks that read the lengths are done
  const int32_t b = blockIdx.x * kThreads + threadIdx.x;
  if (b < a.B) write_length(a, b);
}

}  // namespace

cudaError_t launch_kv_append(const Launch& L, const KvAppendArgs& a) {
  const int64_t total = a.n_tokens * 2 * a.chunks * a.n_kv_heads;
  int64_t blocks = (total + kThreads * kPieces - 1) / (kThreads * kPieces);
  if (blocks == 0) blocks = 1;   // no new token: the lengths are still written
  L.begin(kKernelKvAppend);
  kv_append_kernel<<<(unsigned)blocks, kThreads, 0, L.stream>>>(a);
  cudaError_t e = L.end(kKernelKvAppend);
  if (e != cudaSuccess || a.lens_out != a.lens) return e;
  e = launch_kernel(kv_append_lengths_kernel, dim3((unsigned)((a.B + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                    L.stream, true, a);
  if (e != cudaSuccess) return e;
  return L.end(kKernelKvAppend);
}

}  // namespace csa
