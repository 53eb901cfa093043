// The paged key / value cache as the kernels see it (fa_cache.cu, fa_decode.cu)
// and the checks every entry point makes of its description.
#pragma once

#include <cstdint>

#include "fa.h"
#include "kernels.h"

namespace fa {

struct Cache {
  void* k;
  void* v;
  long long k_layer, v_layer;            // element strides of a layer
  long long k_page, k_head, k_row;       // of a page, a head and a row (d contiguous)
  long long v_page, v_head, v_row;
  int32_t* table;                        // [slots][max_pages]
  int32_t* lengths;                      // [slots]
  int32_t* refs;                         // [pages] or null
  int layers, pages, page_size, heads_kv, d;
  int slots, max_pages;
#ifdef FA_DEBUG_BOUNDS
  int* status;
  long long ext_k, ext_v;                // elements from k, v to the pool's end
#endif
};

// Element i of a list of n, and its store: what the kernels of the cache do to
// memory goes through these (or FA_IN_BOUNDS itself), so that checking builds
// skip and record an index beyond the list.
template <typename T>
__device__ __forceinline__ T get(const Cache& c, const T* list, long long i, long long n) {
  return FA_IN_BOUNDS(c.status, i, 1, n) ? list[i] : T{};
}
template <typename T>
__device__ __forceinline__ void put(const Cache& c, T* list, long long i, long long n, T x) {
  if (FA_IN_BOUNDS(c.status, i, 1, n)) list[i] = x;
}
// Cells of the table, slots' rows end to end.
__device__ __forceinline__ long long table_cells(const Cache& c) {
  return static_cast<long long>(c.slots) * c.max_pages;
}

inline bool cache_aligned(const void* p, uintptr_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// A stride that may be used with `count` entries: a multiple of 8 elements,
// and not zero where that would make entries share memory.
inline bool cache_stride_ok(int64_t s, int64_t count) {
  return s >= 0 && s % 8 == 0 && s < (int64_t{1} << 40) && (count <= 1 || s > 0);
}

inline fa_status_t cache_resolve(const fa_cache_t* a, bool needs_refs, Cache* c) {
  if (a == nullptr || a->layers < 1 || a->pages < 1 || a->page_size < 1 || a->heads_kv < 1 ||
      a->slots < 1 || a->max_pages < 1)
    return FA_ERR_INVALID_ARG;
  if (!cache_aligned(a->k, 16) || !cache_aligned(a->v, 16) || !cache_aligned(a->table, 4) ||
      !cache_aligned(a->lengths, 4) || (needs_refs && a->refs == nullptr) ||
      (reinterpret_cast<uintptr_t>(a->refs) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  const fa_strides_t* st[2] = {&a->ks, &a->vs};
  const int64_t layer[2] = {a->k_layer, a->v_layer};
  for (int t = 0; t < 2; ++t) {
    if (!cache_stride_ok(layer[t], a->layers) || !cache_stride_ok(st[t]->batch, a->pages) ||
        !cache_stride_ok(st[t]->head, a->heads_kv) || !cache_stride_ok(st[t]->row, a->page_size))
      return FA_ERR_INVALID_ARG;
  }
  const int d = a->head_dim;
  if (d != 32 && d != 64 && d != 96 && d != 128 && d != 192 && d != 256) return FA_ERR_UNSUPPORTED;
  // positions, row counts and the scans' partial sums are 32-bit
  if (a->max_pages > (1 << 20) ||
      static_cast<int64_t>(a->max_pages) * a->page_size > (int64_t{1} << 30) ||
      a->pages > (1 << 30) || a->slots > (1 << 30) || a->heads_kv > 65535 || a->layers > 65535)
    return FA_ERR_UNSUPPORTED;
  c->k = a->k;
  c->v = a->v;
  c->k_layer = a->k_layer;
  c->v_layer = a->v_layer;
  c->k_page = a->ks.batch;
  c->k_head = a->ks.head;
  c->k_row = a->ks.row;
  c->v_page = a->vs.batch;
  c->v_head = a->vs.head;
  c->v_row = a->vs.row;
  c->table = a->table;
  c->lengths = a->lengths;
  c->refs = a->refs;
  c->layers = a->layers;
  c->pages = a->pages;
  c->page_size = a->page_size;
  c->heads_kv = a->heads_kv;
  c->d = d;
  c->slots = a->slots;
  c->max_pages = a->max_pages;
#ifdef FA_DEBUG_BOUNDS
  c->status = device_status();
  auto extent = [&](int64_t layer_stride, const fa_strides_t& st) -> long long {
    return (a->layers - 1) * layer_stride + (a->pages - 1) * st.batch + (a->heads_kv - 1) * st.head +
           (a->page_size - 1) * st.row + d;
  };
  c->ext_k = extent(a->k_layer, a->ks);
  c->ext_v = extent(a->v_layer, a->vs);
#endif
  return FA_OK;
}

}  // namespace fa
