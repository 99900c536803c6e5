// Per-head key-value caches (csa_kv_cache_t): device-side addressing shared by
// the append, attention and eviction kernels.
#pragma once

#include "common.cuh"

namespace csa {

// A cache with its strides in bytes.
struct KvRef {
  char* k;
  char* v;
  int64_t n_pages;
  int64_t k_page, k_slot, k_head;
  int64_t v_page, v_slot, v_head;
  const int32_t* table;   // null: sequence b is page b
  int32_t max_pages, page_size;
  int32_t page_shift;     // log2(page_size), or -1 when it is not a power of two
};

// Page of slot `s` of sequence `b` (s >= 0), and the slot's row in it; -1 when
// the page lies outside the pool (recorded).
__device__ __forceinline__ int32_t kv_page(const KvRef& c, int32_t b, int32_t s, int32_t* row,
                                           WsHeader* err) {
  int32_t page, pi;
  if (c.table == nullptr) {
    page = b;
    pi = s < c.page_size ? 0 : 1;
    *row = s;
  } else {
    pi = c.page_shift >= 0 ? s >> c.page_shift : s / c.page_size;
    *row = s - pi * c.page_size;
    page = pi < c.max_pages ? __ldg(c.table + (int64_t)b * c.max_pages + pi) : -1;
  }
  if (page < 0 || page >= c.n_pages || pi >= c.max_pages) {
    report(err, kErrPageId, b, page);
    return -1;
  }
  return page;
}

__device__ __forceinline__ int32_t kv_clamp_len(int32_t n, int64_t max_len, int32_t b, WsHeader* err) {
  if (n >= 0 && n <= max_len) return n;
  report(err, kErrLength, b, n);
  return n < 0 ? 0 : (int32_t)max_len;
}

}  // namespace csa
