// Appending tokens to a per-head key-value cache (csa_kv_append).
//
// A copy: every 16-byte piece of every new row is read once and written once to
// the page that its slot lies on.  Bound by HBM for prompts and by the launch
// and three dependent loads (length, page id, row) for a decode step.
//
// A CTA takes up to 8 consecutive tokens.  Its first threads look their slots
// up (sequence by binary search, length, page id), then warps copy rows, as many
// heads at a time as fit 32 lanes, 16 bytes a lane and four in flight.  With one
// token per sequence a length is read and written by the same CTA.  With
// several, lengths go out with the copies when they have an array of their
// own, and in place by a second launch, since any block may still read them.
#include "kernels.h"
#include "kv.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 8;    // of a CTA (packed prompts, 134 MB copied: 16 29.4 us, 8 26.3 us, 4 26.7 us, 2 34.2 us)
constexpr int kUnroll = 4;       // rows in flight per lane

struct Token {
  int32_t b, i;   // sequence and index among its new tokens; b < 0: none
};

__device__ __forceinline__ Token find_token(const KvAppendArgs& a, int32_t t) {
  if (a.token_start == nullptr) return Token{t, 0};
  int32_t lo = 0, hi = a.B;   // token_start[lo] <= t < token_start[hi]
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (a.token_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int32_t first = a.token_start[lo];
  if (t < first || t >= a.token_start[lo + 1]) return Token{-1, 0};
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

__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int per_cta) {
  __shared__ int64_t s_k[kMaxTokens], s_v[kMaxTokens];   // destination of a token's rows, head 0; -1: dropped
  __shared__ int64_t s_at[kMaxTokens];                   // of its weight and position, head 0; -1: none
  __shared__ int32_t s_pos[kMaxTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = (int64_t)blockIdx.x * per_cta;
  const int count = (int)(a.n_tokens - t0 < per_cta ? a.n_tokens - t0 : per_cta);
  if (tid < count) {
    const Token tk = find_token(a, (int32_t)(t0 + tid));
    int64_t k = -1, v = -1, at = -1;
    if (tk.b >= 0) {
      const int32_t n = a.lens[tk.b];
      const int64_t slot = (int64_t)n + tk.i;
      if (n < 0) {
        report(a.err, kErrLength, tk.b, n);
      } else if (slot >= capacity(a)) {
        report(a.err, kErrRoom, tk.b, slot);
      } else {
        int32_t row;
        const int64_t page = kv_page(a.kv, tk.b, (int32_t)slot, &row, a.err);
        if (page >= 0) {
          k = page * a.kv.k_page + row * a.kv.k_slot;
          v = page * a.kv.v_page + row * a.kv.v_slot;
        }
        at = (int64_t)tk.b * a.n_kv_heads * a.slots + slot;
        if (a.slot_pos) s_pos[tid] = a.pos[tk.b] + tk.i;
      }
    }
    s_k[tid] = k;
    s_v[tid] = v;
    s_at[tid] = at;
  }
  __syncthreads();
  if (a.token_start == nullptr && tid < count) write_length(a, (int32_t)(t0 + tid));
  // rows: (token, key or value, head), `fit` at a time per warp
  const int fit = 32 / a.chunks, sub = lane / a.chunks, piece = lane - sub * a.chunks;
  const int rows = count * 2 * a.n_kv_heads;
  if (sub < fit) {
    for (int r0 = warp * fit + sub; r0 < rows; r0 += kWarps * fit * kUnroll) {
      uint4 val[kUnroll];
      char* dst[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * kWarps * fit;
        dst[u] = nullptr;
        if (r >= rows) continue;
        const int t = r / (2 * a.n_kv_heads);
        int h = r - t * 2 * a.n_kv_heads;
        const bool is_v = h >= a.n_kv_heads;
        if (is_v) h -= a.n_kv_heads;
        const int64_t to = is_v ? s_v[t] : s_k[t];
        if (to < 0) continue;
        const char* const src = is_v ? a.v_new + (t0 + t) * a.v_token + h * a.v_head : a.k_new + (t0 + t) * a.k_token + h * a.k_head;
        dst[u] = (is_v ? a.kv.v + to + h * a.kv.v_head : a.kv.k + to + h * a.kv.k_head) + 16 * piece;
        val[u] = *reinterpret_cast<const uint4*>(src + 16 * piece);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = val[u];
    }
  }
  if (a.slots > 0)
    for (int i = tid; i < count * a.n_kv_heads; i += kThreads) {
      const int t = i / a.n_kv_heads, h = i - t * a.n_kv_heads;
      if (s_at[t] < 0) continue;
      const int64_t at = s_at[t] + h * a.slots;
      if (a.weights) a.weights[at] = 0.f;
      if (a.slot_pos) a.slot_pos[at] = s_pos[t];
    }
  if (a.token_start != nullptr && a.lens_out != a.lens)
    for (int64_t b = (int64_t)blockIdx.x * kThreads + tid; b < a.B; b += (int64_t)gridDim.x * kThreads)
      write_length(a, (int32_t)b);
}

__global__ void __launch_bounds__(kThreads) kv_append_lengths_kernel(const __grid_constant__ KvAppendArgs a) {
  const int32_t b = blockIdx.x * kThreads + threadIdx.x;
  if (b < a.B) write_length(a, b);
}

}  // namespace

cudaError_t launch_kv_append(const Launch& L, const KvAppendArgs& a) {
  int64_t per = a.n_tokens / (4 * 148);   // a few CTAs per SM before they take several tokens
  per = per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per;
  int64_t blocks = (a.n_tokens + per - 1) / per;
  if (blocks == 0) blocks = 1;   // no new token: the lengths are still written
  L.begin(kKernelKvAppend);
  kv_append_kernel<<<(unsigned)blocks, kThreads, 0, L.stream>>>(a, (int)per);
  cudaError_t e = L.end(kKernelKvAppend);
  if (e != cudaSuccess || a.token_start == nullptr || a.lens_out != a.lens) return e;
  L.begin(kKernelKvAppend);
  kv_append_lengths_kernel<<<(unsigned)((a.B + kThreads - 1) / kThreads), kThreads, 0, L.stream>>>(a);
  return L.end(kKernelKvAppend);
}

}  // namespace csa
