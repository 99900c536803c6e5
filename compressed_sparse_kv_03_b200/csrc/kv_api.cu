// C-ABI entry points of the per-head key-value caches: argument validation,
// workspace layout, dispatch (as api.cu for the compressed caches).
#include <cstdarg>
#include <cstdio>

#include "kernels.h"

namespace csa {

namespace {

csa_status_t fail(csa_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

csa_status_t cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return CSA_OK;
  return fail(CSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxSlots = int64_t(1) << 30;   // slots of a sequence
constexpr int32_t kMaxBatch = 65535;
constexpr int32_t kMaxGroup = 128;
constexpr int32_t kMaxBudget = 1 << 24;

csa_status_t check_ws(void* ws, size_t ws_bytes, size_t need, const char* name) {
  if (ws == nullptr || ws_bytes < need)
    return fail(CSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
  if (!aligned(ws, 256)) return fail(CSA_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", name);
  return CSA_OK;
}

csa_status_t check_kv(const csa_kv_cache_t* kv, const char* name) {
  if (kv == nullptr || kv->k == nullptr || kv->v == nullptr)
    return fail(CSA_ERR_INVALID_ARG, "%s: null key-value cache", name);
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16))
    return fail(CSA_ERR_INVALID_ARG, "%s: k and v must be 16-byte aligned", name);
  if (kv->dtype != CSA_KV_BF16 && kv->dtype != CSA_KV_FP16)
    return fail(CSA_ERR_INVALID_ARG, "%s: dtype %d is neither bf16 nor fp16", name, kv->dtype);
  if (kv->n_pages < 1 || kv->page_size < 1 || kv->n_kv_heads < 1 ||
      (kv->page_table != nullptr && kv->max_pages < 1))
    return fail(CSA_ERR_INVALID_ARG, "%s: n_pages, page_size, n_kv_heads and max_pages must be >= 1", name);
  if (kv->head_dim < 8 || kv->head_dim % 8 != 0)
    return fail(CSA_ERR_INVALID_ARG, "%s: head_dim must be a positive multiple of 8, got %d", name, kv->head_dim);
  if (kv->head_dim > 256) return fail(CSA_ERR_UNSUPPORTED, "%s: head_dim %d above 256", name, kv->head_dim);
  const int64_t st[6] = {kv->k_page_stride, kv->k_slot_stride, kv->k_head_stride,
                         kv->v_page_stride, kv->v_slot_stride, kv->v_head_stride};
  for (int64_t s : st)
    if (s < 0 || s % 8 != 0) return fail(CSA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 and >= 0", name);
  const int64_t pages = kv->page_table ? kv->max_pages : 1;
  if (pages * kv->page_size > kMaxSlots)
    return fail(CSA_ERR_UNSUPPORTED, "%s: more than 2^30 slots per sequence", name);
  if (kv->n_pages > 0x7fffffff || kv->n_kv_heads > 65535)
    return fail(CSA_ERR_UNSUPPORTED, "%s: n_pages or n_kv_heads too large", name);
  return CSA_OK;
}

// Whether [pages][slots][heads][d] under these strides gives every element a
// place of its own: by ascending stride, each dimension steps over all of the
// smaller ones.
bool disjoint(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t d) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[j] > s[j + 1]) {
        const int64_t ts = s[j], tn = n[j];
        s[j] = s[j + 1], n[j] = n[j + 1];
        s[j + 1] = ts, n[j + 1] = tn;
      }
  int64_t extent = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (s[i] < extent) return false;
    extent += (n[i] - 1) * s[i];
  }
  return true;
}

csa_status_t check_writable(const csa_kv_cache_t* kv, const char* name) {
  if (!disjoint(kv->n_pages, kv->k_page_stride, kv->page_size, kv->k_slot_stride, kv->n_kv_heads,
                kv->k_head_stride, kv->head_dim) ||
      !disjoint(kv->n_pages, kv->v_page_stride, kv->page_size, kv->v_slot_stride, kv->n_kv_heads,
                kv->v_head_stride, kv->head_dim))
    return fail(CSA_ERR_INVALID_ARG, "%s: the strides of a cache that is written must not overlap", name);
  return CSA_OK;
}

csa_status_t check_rows(const csa_kv_rows_t* r, const char* what, const char* name) {
  if (r == nullptr || r->data == nullptr) return fail(CSA_ERR_INVALID_ARG, "%s: %s is required", name, what);
  if (!aligned(r->data, 16) || r->token_stride < 0 || r->head_stride < 0 || r->token_stride % 8 != 0 ||
      r->head_stride % 8 != 0)
    return fail(CSA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with strides that are multiples of 8", name, what);
  return CSA_OK;
}

bool apart(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const intptr_t x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
  return x + a_bytes <= y || y + b_bytes <= x;
}

// Output arrays are the input's memory or wholly apart from it.
bool same_or_apart(const void* a, const void* b, int64_t bytes) {
  return a == b || apart(a, bytes, b, bytes);
}

KvRef to_ref(const csa_kv_cache_t* kv) {
  KvRef r;
  r.k = static_cast<char*>(kv->k);
  r.v = static_cast<char*>(kv->v);
  r.n_pages = kv->n_pages;
  r.k_page = kv->k_page_stride * 2;
  r.k_slot = kv->k_slot_stride * 2;
  r.k_head = kv->k_head_stride * 2;
  r.v_page = kv->v_page_stride * 2;
  r.v_slot = kv->v_slot_stride * 2;
  r.v_head = kv->v_head_stride * 2;
  r.table = kv->page_table;
  r.max_pages = kv->page_table ? kv->max_pages : 1;
  r.page_size = kv->page_size;
  r.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (kv->page_size == (1 << i)) r.page_shift = i;
  return r;
}

int64_t capacity(const csa_kv_cache_t* kv) {
  return (kv->page_table ? (int64_t)kv->max_pages : 1) * kv->page_size;
}

csa_status_t check_batch(int32_t B, const csa_kv_cache_t* kv, const char* name) {
  if (B < 0) return fail(CSA_ERR_INVALID_ARG, "%s: B must be >= 0", name);
  if (B > kMaxBatch) return fail(CSA_ERR_UNSUPPORTED, "%s: B above %d", name, kMaxBatch);
  if (kv != nullptr && kv->page_table == nullptr && B > kv->n_pages)
    return fail(CSA_ERR_INVALID_ARG, "%s: a cache without a page table needs a page per sequence", name);
  return CSA_OK;
}

// Attention workspace: header | piece (max, sum) | piece O | lse2 | scores.
struct AttnLayout {
  KvAttnPlan plan;
  int64_t score_stride;
  size_t ml_off, acc_off, lse_off, score_off, total;
};
AttnLayout attn_layout(const csa_kv_cache_t* kv, int32_t B, int32_t H, int64_t max_len, int32_t window, bool weights) {
  AttnLayout l;
  l.plan = kv_attn_plan(to_ref(kv), B, H, kv->n_kv_heads, kv->head_dim, max_len, window, batch_invariant());
  const size_t rows = (size_t)l.plan.pieces * l.plan.heads;
  l.ml_off = kWsHeader;
  l.acc_off = l.ml_off + align256(rows * 2 * sizeof(float));
  l.lse_off = l.acc_off + align256(rows * l.plan.dp * sizeof(float));
  l.score_off = l.lse_off + (weights ? align256((size_t)B * H * sizeof(float)) : 0);
  l.score_stride = (max_len + 31) / 32 * 32;
  l.total = l.score_off + (weights ? align256((size_t)B * H * l.score_stride * sizeof(float)) : 0);
  return l;
}

int64_t evict_list_len(int32_t budget, int64_t max_len) {
  const int64_t over = max_len - budget;
  return over <= 0 ? 0 : over < budget ? over : budget;
}

}  // namespace

}  // namespace csa

using namespace csa;

extern "C" {

csa_status_t csa_kv_append(const csa_kv_rows_t* k_new, const csa_kv_rows_t* v_new,
                           const csa_kv_cache_t* kv, const int32_t* token_start, int64_t n_tokens,
                           int32_t B, const int32_t* lens, int32_t* lens_out, const int32_t* pos,
                           float* weights, int32_t* slot_pos, int64_t slots, void* ws,
                           size_t ws_bytes, csa_stream_t stream) {
  const char* name = "csa_kv_append";
  csa_status_t st = check_batch(B, nullptr, name);
  if (st != CSA_OK) return st;
  if (n_tokens < 0) return fail(CSA_ERR_INVALID_ARG, "%s: n_tokens must be >= 0", name);
  if (token_start == nullptr && n_tokens != B)
    return fail(CSA_ERR_INVALID_ARG, "%s: without token_start there is one token per sequence (n_tokens == B)", name);
  if (B == 0) return CSA_OK;
  if ((st = check_kv(kv, name)) != CSA_OK) return st;
  if ((st = check_batch(B, kv, name)) != CSA_OK) return st;
  if ((st = check_writable(kv, name)) != CSA_OK) return st;
  if (kv->k == kv->v) return fail(CSA_ERR_INVALID_ARG, "%s: k and v must not be the same memory", name);
  if (n_tokens > 0 && ((st = check_rows(k_new, "k_new", name)) != CSA_OK ||
                       (st = check_rows(v_new, "v_new", name)) != CSA_OK))
    return st;
  if (lens == nullptr || lens_out == nullptr)
    return fail(CSA_ERR_INVALID_ARG, "%s: lens and lens_out are required", name);
  if (!same_or_apart(lens, lens_out, (int64_t)B * 4))
    return fail(CSA_ERR_INVALID_ARG, "%s: lens_out must be lens or apart from it", name);
  if (slot_pos != nullptr && pos == nullptr)
    return fail(CSA_ERR_INVALID_ARG, "%s: slot_pos needs pos", name);
  // Blocks write new lengths while others still read pos and token_start; lengths in
  // place are written by a launch of their own, except with one token per sequence,
  // where one block reads and writes all of a sequence's.
  const int64_t n4 = (int64_t)B * 4;
  if (token_start != nullptr && !apart(lens_out, n4, token_start, n4 + 4))
    return fail(CSA_ERR_INVALID_ARG, "%s: lens_out must be apart from token_start", name);
  if (slot_pos != nullptr && (token_start == nullptr ? !same_or_apart(pos, lens_out, n4)
                                                     : lens_out != lens && !apart(pos, n4, lens_out, n4)))
    return fail(CSA_ERR_INVALID_ARG, "%s: lens_out must be apart from pos", name);
  if ((weights != nullptr || slot_pos != nullptr) && slots < 1)
    return fail(CSA_ERR_INVALID_ARG, "%s: weights and slot_pos need slots >= 1", name);
  const int64_t pieces = (int64_t)kv->head_dim / 8 * kv->n_kv_heads * 2;
  if (n_tokens > 0x7fffffff || n_tokens * pieces / 1024 >= 0x7fffffff)
    return fail(CSA_ERR_UNSUPPORTED, "%s: too many tokens for one call", name);
  if ((st = check_ws(ws, ws_bytes, kWsHeader, name)) != CSA_OK) return st;
  KvAppendArgs a{};
  a.kv = to_ref(kv);
  if (n_tokens > 0) {
    a.k_new = static_cast<const char*>(k_new->data);
    a.v_new = static_cast<const char*>(v_new->data);
    a.k_token = k_new->token_stride * 2;
    a.k_head = k_new->head_stride * 2;
    a.v_token = v_new->token_stride * 2;
    a.v_head = v_new->head_stride * 2;
  }
  a.token_start = token_start;
  a.n_tokens = n_tokens;
  a.B = B;
  a.n_kv_heads = kv->n_kv_heads;
  a.chunks = kv->head_dim / 8;
  a.lens = lens;
  a.lens_out = lens_out;
  a.pos = pos;
  a.weights = weights;
  a.slot_pos = slot_pos;
  a.slots = weights != nullptr || slot_pos != nullptr ? slots : 0;
  a.err = static_cast<WsHeader*>(ws);
  Launch L{(cudaStream_t)stream};
  return cuda_status(launch_kv_append(L, a), "csa_kv_append launch");
}

size_t csa_kv_attn_decode_workspace_size(int32_t B, int32_t H, const csa_kv_cache_t* kv,
                                         int64_t max_len, int32_t with_weights) {
  if (B <= 0 || H <= 0 || kv == nullptr || kv->n_kv_heads < 1 || H % kv->n_kv_heads != 0 || kv->head_dim < 1 ||
      max_len < 0 || max_len > kMaxSlots)
    return kWsHeader;
  // a window only ever needs less
  return attn_layout(kv, B, H, max_len, 0, with_weights != 0).total;
}

csa_status_t csa_kv_attn_decode(const csa_kv_rows_t* q, const csa_kv_cache_t* kv,
                                const int32_t* lens, int32_t B, int32_t H, int64_t max_len,
                                int32_t window, float sm_scale, const float* sink, void* out,
                                float* lse, const float* weights, float* weights_out,
                                int64_t slots, void* ws, size_t ws_bytes, csa_stream_t stream) {
  const char* name = "csa_kv_attn_decode";
  csa_status_t st = check_batch(B, nullptr, name);
  if (st != CSA_OK) return st;
  if (B == 0) return CSA_OK;
  if ((st = check_kv(kv, name)) != CSA_OK) return st;
  if ((st = check_batch(B, kv, name)) != CSA_OK) return st;
  if ((st = check_rows(q, "q", name)) != CSA_OK) return st;
  if (lens == nullptr || out == nullptr) return fail(CSA_ERR_INVALID_ARG, "%s: lens and out are required", name);
  if (!aligned(out, 16)) return fail(CSA_ERR_INVALID_ARG, "%s: out must be 16-byte aligned", name);
  if (H < 1 || H % kv->n_kv_heads != 0)
    return fail(CSA_ERR_INVALID_ARG, "%s: H must be a multiple of n_kv_heads (got %d and %d)", name, H, kv->n_kv_heads);
  if (H / kv->n_kv_heads > kMaxGroup)
    return fail(CSA_ERR_UNSUPPORTED, "%s: more than %d query heads per KV head", name, kMaxGroup);
  if ((int64_t)B * H > (1 << 27)) return fail(CSA_ERR_UNSUPPORTED, "%s: too many sequences times heads", name);
  const char* const q0 = static_cast<const char*>(q->data);
  const char* const q1 = q0 + 2 * ((B - 1) * q->token_stride + (H - 1) * q->head_stride + kv->head_dim);
  const char* const o0 = static_cast<const char*>(out);
  if (q0 < o0 + (int64_t)B * H * kv->head_dim * 2 && o0 < q1)
    return fail(CSA_ERR_INVALID_ARG, "%s: out must not overlap q", name);
  if (max_len < 0 || max_len > capacity(kv))
    return fail(CSA_ERR_INVALID_ARG, "%s: max_len must be in [0, max_pages*page_size]", name);
  if (window < 0) return fail(CSA_ERR_INVALID_ARG, "%s: window must be >= 0", name);
  if (!(sm_scale == sm_scale)) return fail(CSA_ERR_INVALID_ARG, "%s: sm_scale is NaN", name);
  if (weights != nullptr && weights_out == nullptr)
    return fail(CSA_ERR_INVALID_ARG, "%s: weights needs weights_out", name);
  if (weights_out != nullptr) {
    if (slots < max_len || slots < 1)
      return fail(CSA_ERR_INVALID_ARG, "%s: weights_out needs slots >= max_len", name);
    if (window != 0) return fail(CSA_ERR_UNSUPPORTED, "%s: weights_out with a window", name);
    if (weights != nullptr && !same_or_apart(weights, weights_out, (int64_t)B * kv->n_kv_heads * slots * 4))
      return fail(CSA_ERR_INVALID_ARG, "%s: weights_out must be weights or apart from it", name);
  }
  const bool weigh = weights_out != nullptr;
  const AttnLayout l = attn_layout(kv, B, H, max_len, window, weigh);
  if ((st = check_ws(ws, ws_bytes, l.total, name)) != CSA_OK) return st;
  KvAttnArgs a{};
  a.kv = to_ref(kv);
  a.q = static_cast<const char*>(q->data);
  a.q_token = q->token_stride * 2;
  a.q_head = q->head_stride * 2;
  a.B = B;
  a.H = H;
  a.n_kv_heads = kv->n_kv_heads;
  a.d = kv->head_dim;
  a.dtype = kv->dtype;
  a.lens = lens;
  a.max_len = max_len;
  a.window = window;
  a.scale = sm_scale * kLog2e;
  a.sink = sink;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  a.weights = weights;
  a.weights_out = weights_out;
  a.slots = slots;
  char* const p = static_cast<char*>(ws);
  a.part_ml = reinterpret_cast<float*>(p + l.ml_off);
  a.part_acc = reinterpret_cast<float*>(p + l.acc_off);
  a.lse2 = weigh ? reinterpret_cast<float*>(p + l.lse_off) : nullptr;
  a.scores = weigh ? reinterpret_cast<float*>(p + l.score_off) : nullptr;
  a.score_stride = l.score_stride;
  a.runs = l.plan.runs;
  a.whole = l.plan.whole;
  a.atom = l.plan.atom;
  a.invariant = l.plan.invariant;
  a.max_atoms = l.plan.max_atoms;
  a.err = static_cast<WsHeader*>(ws);
  Launch L{(cudaStream_t)stream};
  return cuda_status(launch_kv_attn(L, a, l.plan), "csa_kv_attn_decode launch");
}

size_t csa_kv_evict_workspace_size(int32_t B, int32_t n_kv_heads, int32_t budget, int64_t max_len) {
  if (B <= 0 || n_kv_heads < 1 || budget < 1 || max_len < 0) return kWsHeader;
  // the slots of every move, and the number of moves
  const size_t units = (size_t)B * n_kv_heads;
  return kWsHeader + align256(units * 2 * evict_list_len(budget, max_len) * sizeof(int32_t)) + align256(units * sizeof(int32_t));
}

csa_status_t csa_kv_evict(const csa_kv_cache_t* kv, const int32_t* lens, int32_t* lens_out,
                          const float* weights, float* weights_out, const int32_t* slot_pos,
                          int32_t* slot_pos_out, int64_t slots, const int32_t* pos, int32_t B,
                          int32_t budget, int32_t recent, int32_t keep_first, int64_t max_len,
                          int32_t* src_out, void* ws, size_t ws_bytes, csa_stream_t stream) {
  const char* name = "csa_kv_evict";
  csa_status_t st = check_batch(B, nullptr, name);
  if (st != CSA_OK) return st;
  if (budget < 1 || recent < 1 || keep_first < 0 || (int64_t)recent + keep_first > budget)
    return fail(CSA_ERR_INVALID_ARG,
                "%s: need recent >= 1, keep_first >= 0 and recent + keep_first <= budget (got %d, %d, %d)", name,
                recent, keep_first, budget);
  if (budget > kMaxBudget) return fail(CSA_ERR_UNSUPPORTED, "%s: budget above 2^24", name);
  if (B == 0) return CSA_OK;
  if ((st = check_kv(kv, name)) != CSA_OK) return st;
  if ((st = check_batch(B, kv, name)) != CSA_OK) return st;
  if ((st = check_writable(kv, name)) != CSA_OK) return st;
  if (lens == nullptr || lens_out == nullptr || weights == nullptr || weights_out == nullptr ||
      slot_pos == nullptr || slot_pos_out == nullptr || pos == nullptr)
    return fail(CSA_ERR_INVALID_ARG, "%s: lens, weights, slot_pos (and their outputs) and pos are required", name);
  if (max_len < 0 || max_len > capacity(kv) || max_len > slots || slots < 1)
    return fail(CSA_ERR_INVALID_ARG, "%s: max_len must be in [0, max_pages*page_size] and at most slots", name);
  const int64_t bytes = (int64_t)B * kv->n_kv_heads * slots * 4;
  if (!same_or_apart(lens, lens_out, (int64_t)B * 4) || !same_or_apart(weights, weights_out, bytes) ||
      !same_or_apart(slot_pos, slot_pos_out, bytes))
    return fail(CSA_ERR_INVALID_ARG, "%s: an output must be its input or apart from it", name);
  if (lens_out != lens && !apart(lens_out, (int64_t)B * 4, pos, (int64_t)B * 4))   // other blocks still read it
    return fail(CSA_ERR_INVALID_ARG, "%s: lens_out must be lens or apart from pos", name);
  const bool shared = kv->k == kv->v;
  if (shared && (kv->k_page_stride != kv->v_page_stride || kv->k_slot_stride != kv->v_slot_stride ||
                 kv->k_head_stride != kv->v_head_stride))
    return fail(CSA_ERR_INVALID_ARG, "%s: k and v in the same memory need the same strides", name);
  if ((int64_t)B * kv->n_kv_heads > (1 << 27))
    return fail(CSA_ERR_UNSUPPORTED, "%s: too many sequences times KV heads", name);
  if ((st = check_ws(ws, ws_bytes, csa_kv_evict_workspace_size(B, kv->n_kv_heads, budget, max_len), name)) != CSA_OK)
    return st;
  KvEvictArgs a{};
  a.kv = to_ref(kv);
  a.B = B;
  a.n_kv_heads = kv->n_kv_heads;
  a.chunks = kv->head_dim / 8;
  a.shared = shared;
  a.lens = lens;
  a.lens_out = lens_out;
  a.weights = weights;
  a.weights_out = weights_out;
  a.slot_pos = slot_pos;
  a.slot_pos_out = slot_pos_out;
  a.slots = slots;
  a.pos = pos;
  a.budget = budget;
  a.recent = recent;
  a.keep_first = keep_first;
  a.max_len = max_len;
  a.src_out = src_out;
  a.list = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsHeader);
  a.list_len = evict_list_len(budget, max_len);
  a.moves = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsHeader +
                                       align256((size_t)B * kv->n_kv_heads * 2 * a.list_len * sizeof(int32_t)));
  a.err = static_cast<WsHeader*>(ws);
  Launch L{(cudaStream_t)stream};
  return cuda_status(launch_kv_evict(L, a), "csa_kv_evict launch");
}

}  // extern "C"
