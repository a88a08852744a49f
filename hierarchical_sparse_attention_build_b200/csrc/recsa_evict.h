// Launch arguments of the eviction kernels.
#pragma once

#include <cstdint>

#include <vector_types.h>

#include "recsa_internal.h"

namespace recsa {

// One cache's rows as 16-byte pieces (16 a row).
struct EvictCache {
  uint4 *k, *v;
  const int32_t *pages;
  int64_t capacity;
  int32_t pages_per_seq, page_shift, num_pages;
};

struct EvictArgs {
  EvictCache from, to;
  const float *weights;
  float *to_weights;
  int32_t *kept;
  const int64_t *seq_len;
  int64_t capacity, to_capacity;  // slots of a weights row
  int32_t batch, hkv, length;
  int32_t keep, sinks, recent;
};

#ifdef __CUDACC__
__device__ __forceinline__ int evict_length(const EvictArgs &a, int b) {
  if (!a.seq_len) return a.length;
  const int64_t n = a.seq_len[b];
  return n < 0 ? 0 : n > a.length ? a.length : (int)n;
}
__device__ __forceinline__ bool evict_bad_length(const EvictArgs &a, int b) {
  return a.seq_len && (a.seq_len[b] < 0 || a.seq_len[b] > a.length);
}
// Row of slot t of (sequence, head), or -1 for a page outside the pool.
__device__ __forceinline__ int64_t evict_row(const EvictCache &c, int hkv, int b, int h, int t) {
  if (!c.pages) return ((int64_t)b * hkv + h) * c.capacity + t;
  const int pg = __ldg(c.pages + (int64_t)b * c.pages_per_seq + (t >> c.page_shift));
  if ((unsigned)pg >= (unsigned)c.num_pages) return -1;
  return (((int64_t)pg * hkv + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}
#endif

// Select, move (within one cache or to another), and set the receiving lengths (to_len may be NULL).
int launch_evict(const EvictArgs &a, bool in_place, int64_t *to_len, void *stream);

}  // namespace recsa
