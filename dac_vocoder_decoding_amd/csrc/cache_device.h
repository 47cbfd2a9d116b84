// cache_device.h -- device building blocks of the kernels that write and read
// the paged 8-bit cache.
#pragma once
#include "ops_device.h"

namespace voc {

// What one workgroup appends to: the page that is its sequence's j-th among
// those the new tokens touch; tokens [lo, hi) of it are new.
struct PageShare {
  int64_t slot;     // page * heads + head
  int64_t token;    // packed row of token lo
  int64_t first;    // position of the page's first token
  int lo, hi;       // hi <= lo: nothing to do
};
__device__ __forceinline__ PageShare page_share(const CacheView& c, int b, int j, int head) {
  PageShare s{0, 0, 0, 0, 0};
  const Seq q = load_seq(c, b);
  const int P = 1 << c.page_log;
  const int64_t column = (q.past >> c.page_log) + static_cast<int64_t>(j);
  if (column >= c.stride) return s;
  const int64_t first = column << c.page_log;  // position of the page's first token
  const int64_t end = static_cast<int64_t>(q.past) + q.count;
  const int page = c.table[b * c.stride + column];
  if (end <= first || page < 0 || page >= c.n_pages) return s;
  s.slot = static_cast<int64_t>(page) * c.heads + head;
  s.first = first;
  s.lo = q.past > first ? static_cast<int>(q.past - first) : 0;
  s.hi = end < first + P ? static_cast<int>(end - first) : P;
  s.token = q.start + (first + s.lo - q.past);
  return s;
}

// The scale that covers a page's older tokens (none: 0) and its new ones.
__device__ __forceinline__ float joint_scale(float old, uint32_t top) {
  const float own = scale_of_bits(top);
  return !(old == old) ? old : !(own == own) ? own : fmaxf(old, own);
}

// Four codes rounded again.
__device__ __forceinline__ uint32_t rescaled4(uint32_t c, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r |= (static_cast<uint32_t>(static_cast<int>(__builtin_rintf(static_cast<float>(static_cast<int8_t>(c >> (8 * k))) * ratio))) & 0xffu)
         << (8 * k);
  return r;
}

}  // namespace voc
