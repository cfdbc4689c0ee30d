// The paged KV cache as kernels see it, and the row-to-request map that the
// attention-side kernels share.
#pragma once

#include "sv_kernels.h"
#include "sv_ptx.cuh"

namespace sv {

constexpr int KV_MAX_DRAFT = 64;  // drafted rows per request: the bits of a tree mask

struct KvPtrs {
  uint8_t *k, *v;
  __half *ks, *kb, *vs, *vb;
};

struct KvCache {
  KvPtrs p;
  int n_pages, page_shift, heads, dim, bits;
};

// Requests' row ranges, by value in the launch parameters.
struct RowMap {
  int B;
  int offs[MAX_BATCH + 1];
};

// The request of a row below offs[B] (requests without rows are skipped over).
__device__ __forceinline__ int request_of(const RowMap& m, int row) {
  int lo = 0, hi = m.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (m.offs[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// Index of (page, head, place) in units of tokens: 64 bits, since a long cache
// passes 2^31 bytes.
__device__ __forceinline__ size_t kv_token(const KvCache& c, int page, int head, int place) {
  return (((size_t)page * c.heads + head) << c.page_shift) + place;
}

// Page of position `pos` of request b, or -1 for bad input (a position outside
// the table or a page outside the cache).
__device__ __forceinline__ long long kv_page_of(const KvCache& c, const int32_t* table, int table_pages, int b, long long pos) {
  if (pos < 0) return -1;
  const long long pi = pos >> c.page_shift;
  if (pi >= table_pages) return -1;
  const int page = table[(size_t)b * table_pages + pi];
  return page < 0 || page >= c.n_pages ? -1 : page;
}

// Host checks of a cache, and of the row map (fills `m`).
int check_cache(const sv_kv_cache* c, KvCache* out);
int check_rows_map(int B, const int32_t* row_offsets, int max_per_request, int max_total, RowMap* m);
int check_table(const KvCache& c, const int32_t* lens, const int32_t* block_table, int table_pages);

}  // namespace sv
