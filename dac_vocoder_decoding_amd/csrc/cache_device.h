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

// Eight codes in a row, codes8's own bits, of values that all lie within the
// page's scale (inv > 0: they are finite, and |v inv| rounds to 127 at the
// most): 1.5 2^23 added to the rounded product leaves its nearest integer, ties
// to even, in the sum's low bits.
__device__ __forceinline__ uint2 codes8_within(const float (&v)[8], float inv) {
#pragma clang fp contract(off)
  uint32_t t[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) t[k] = __float_as_uint(v[k] * inv + 12582912.f);
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
  };
  return inv > 0.f ? make_uint2(four(t[0], t[1], t[2], t[3]), four(t[4], t[5], t[6], t[7])) : make_uint2(0, 0);
}

}  // namespace voc
