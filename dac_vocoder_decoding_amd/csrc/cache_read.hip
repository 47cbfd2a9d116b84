// cache_read.hip -- the tokens of the paged 8-bit cache as rows again:
// code * scale of the page, rounded once.
#include "cache_device.h"

namespace voc {

template <int T, bool VEC>
__device__ __forceinline__ void put8(typename Elem<T>::type* p, const float (&v)[8]) {
  if constexpr (VEC) {
    store8<T>(p, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = static_cast<typename Elem<T>::type>(v[k]);
  }
}

__device__ __forceinline__ float code_at(uint32_t w, int k) {
  return static_cast<float>(static_cast<int8_t>(w >> (8 * k)));
}

// A thread reads a unit of 4 tokens x 8 values of one page and head: of keys
// eight codes of each token's row, of values (transposed inside a page) the
// four tokens of eight rows.  Units of a page follow one another over its
// heads, keys first: along a row of keys, along the tokens of values.
template <int T, bool VEC>
__global__ __launch_bounds__(256) void cache_read_kernel(const ReadArgs a, int blocks) {
  typedef typename Elem<T>::type E;
  const int log = a.c.page_log, P = 1 << log, D = a.D, D8 = D >> 3;
  const int j = blockIdx.x / blocks;
  const int64_t unit = static_cast<int64_t>(blockIdx.x % blocks) * 256 + threadIdx.x;
  const int per = (P >> 2) * D8;  // units of a head
  const int64_t all = static_cast<int64_t>(per) * a.c.heads;
  const bool value = a.k == nullptr || unit >= all;
  const int64_t at = a.k != nullptr && value ? unit - all : unit;
  if (at >= all || (value && a.v == nullptr)) return;
  const int head = static_cast<int>(at / per), r = static_cast<int>(at % per);
  const PageShare sh = page_share(a.c, blockIdx.y, j, head);
  const int t4 = value ? 4 * (r & ((P >> 2) - 1)) : r / D8 * 4, d8 = value ? 8 * (r >> (log - 2)) : r % D8 * 8;
  if (t4 + 4 <= sh.lo || t4 >= sh.hi) return;
  const int8_t* codes = (value ? a.c.v : a.c.k) + sh.slot * P * D;
  const float scale = (value ? a.c.vs : a.c.ks)[sh.slot];
  float v[4][8];
  if (!value) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(t4 + t) * D + d8);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[t][k] = code_at(k < 4 ? c.x : c.y, k & 3) * scale;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + static_cast<int64_t>(d8 + k) * P + t4);
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t][k] = code_at(c, t) * scale;
    }
  }
  E* out = value ? static_cast<E*>(a.v) + head * a.v_h : static_cast<E*>(a.k) + head * a.k_h;
  const int64_t st = value ? a.v_t : a.k_t;
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (t4 + t >= sh.lo && t4 + t < sh.hi) put8<T, VEC>(out + (sh.token + t4 + t - sh.lo) * st + d8, v[t]);
}

static int page_blocks(const ReadArgs& a) {
  const int64_t units = (int64_t(1) << a.c.page_log) / 4 * (a.D / 8) * a.c.heads * ((a.k != nullptr) + (a.v != nullptr));
  return static_cast<int>((units + 255) / 256);
}

int64_t read_workgroups(const ReadArgs& a) {
  return static_cast<int64_t>(page_blocks(a)) * (((a.c.max_new - 1) >> a.c.page_log) + 2);
}

template <int T>
static void go_read(const ReadArgs& a, hipStream_t s, Form& form) {
  constexpr int per16 = 16 / sizeof(typename Elem<T>::type);
  const bool vec = (reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) % 16 == 0 &&
                   (a.k_t | a.k_h | a.v_t | a.v_h) % per16 == 0;
  const int blocks = page_blocks(a);
  form = Form{"read", {1 << a.c.page_log, vec}};
  const dim3 grid(static_cast<unsigned>(read_workgroups(a)), a.batch);
  if (vec)
    cache_read_kernel<T, true><<<grid, 256, 0, s>>>(a, blocks);
  else
    cache_read_kernel<T, false><<<grid, 256, 0, s>>>(a, blocks);
}

hipError_t launch_read(int dtype, const ReadArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_read<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    go_read<EL_BF16>(a, s, form);
  else
    go_read<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
