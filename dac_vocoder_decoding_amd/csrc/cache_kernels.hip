// cache_kernels.hip -- appending keys and values to the paged 8-bit cache.
//
// Per page and cache head: s' = max(s_old, max|new| / 127); the new tokens'
// codes are rint(x / s'), the older codes are rounded again,
// rint(q s_old / s'), where s' grew.
#include "ops_device.h"

namespace voc {

// Workgroup (j, 2 * head + is_value, sequence): the j-th page that the
// sequence's new tokens touch.  Values are stored transposed inside a page.
template <int T>
__global__ __launch_bounds__(256) void append_kernel(const AppendArgs a) {
  typedef typename Elem<T>::type E;
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  const Seq q = load_seq(a.c, blockIdx.z);
  const int head = blockIdx.y >> 1;
  const bool value = blockIdx.y & 1;
  const int P = 1 << a.c.page_log, D = a.D;
  const int64_t column = (q.past >> a.c.page_log) + static_cast<int64_t>(blockIdx.x);
  if (column >= a.c.stride) return;
  const int64_t first = column << a.c.page_log;           // position of the page's first token
  const int64_t end = static_cast<int64_t>(q.past) + q.count;
  const int lo = q.past > first ? static_cast<int>(q.past - first) : 0;   // [lo, hi): new tokens
  const int hi = end < first + P ? static_cast<int>(end - first) : P;
  if (hi <= lo) return;
  const int page = a.c.table[blockIdx.z * a.c.stride + column];
  if (page < 0 || page >= a.c.n_pages) return;
  const int64_t slot = static_cast<int64_t>(page) * a.c.heads + head;
  const E* src = value ? static_cast<const E*>(a.v) + head * a.v_h : static_cast<const E*>(a.k) + head * a.k_h;
  const int64_t st = value ? a.v_t : a.k_t;
  src += (q.start + (first + lo - q.past)) * st;
  int8_t* codes = (value ? a.c.v : a.c.k) + slot * P * D;
  float* scales = value ? a.c.vs : a.c.ks;

  const int n = (hi - lo) * D;
  uint32_t top = 0;
  for (int i = tid; i < n; i += 256) {
    const int t = i / D, d = i - t * D;
    top = max(top, abs_bits(static_cast<float>(src[t * st + d])));
  }
  top = wave_max(top);
  if ((tid & 63) == 0) s_max[tid >> 6] = top;
  const float old = lo ? scales[slot] : 0.f;
  __syncthreads();
  top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const float own = scale_of_bits(top);
  const float scale = !(old == old) ? old : !(own == own) ? own : fmaxf(old, own);
  const float inv = inverse_of(scale);
  if (lo && scale != old) {
    const float ratio = inv > 0.f ? old * inv : 0.f;
    for (int i = tid; i < lo * D; i += 256) {
      const int t = i / D, d = i - t * D;
      int8_t* p = codes + (value ? d * P + t : i);
      *p = static_cast<int8_t>(__builtin_rintf(static_cast<float>(*p) * ratio));
    }
  }
  for (int i = tid; i < n; i += 256) {
    const int t = i / D, d = i - t * D;
    codes[value ? d * P + lo + t : lo * D + i] = static_cast<int8_t>(code_of(static_cast<float>(src[t * st + d]), inv));
  }
  if (tid == 0) scales[slot] = scale;
}

hipError_t launch_append(int dtype, const AppendArgs& a, hipStream_t s) {
  const int P = 1 << a.c.page_log;
  const dim3 grid((a.c.max_new + P - 1) / P + 1, 2 * a.c.heads, a.batch);
  if (dtype == EL_F32)
    append_kernel<EL_F32><<<grid, 256, 0, s>>>(a);
  else if (dtype == EL_BF16)
    append_kernel<EL_BF16><<<grid, 256, 0, s>>>(a);
  else
    append_kernel<EL_F16><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace voc
