// rows_kernels.hip -- rows of 8-bit codes with one scale each: the RMS norm
// with residual addition, and the plain row quantiser.
//
//   h = round(x + r);  y = h / sqrt(mean(h^2) + eps) * w;
//   s = max|y| / 127;  q = rint(y / s)
#include "ops_device.h"

namespace voc {

// One workgroup per row; NPT values of the row per thread stay in registers
// between the sum of squares, the maximum and the codes.
template <int T, int NPT>
__global__ __launch_bounds__(256) void rows_kernel(const RowsArgs a) {
  typedef typename Elem<T>::type E;
  __shared__ float s_sum[4];
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const E* x = static_cast<const E*>(a.x) + row * a.ldx;
  const E* r = a.r ? static_cast<const E*>(a.r) + row * a.ldr : nullptr;
  E* h = a.h ? static_cast<E*>(a.h) + row * a.ldh : nullptr;
  float v[NPT];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = tid + i * 256;
    v[i] = 0.f;
    if (c < a.C) {
      float f = static_cast<float>(x[c]);
      if (r) f = static_cast<float>(static_cast<E>(f + static_cast<float>(r[c])));
      if (h) h[c] = static_cast<E>(f);
      v[i] = f;
      sum += f * f;
    }
  }
  uint32_t top = 0;
  if (a.weight) {
    sum = wave_sum(sum);
    if ((tid & 63) == 0) s_sum[wave] = sum;
    __syncthreads();
    sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    const float rms = rsqrtf(sum / static_cast<float>(a.C) + a.eps);
    if (abs_bits(sum) >= kInfBits) top = kInfBits;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = tid + i * 256;
      if (c < a.C) v[i] = v[i] * rms * a.weight[c];
    }
  }
#pragma unroll
  for (int i = 0; i < NPT; ++i) top = max(top, abs_bits(v[i]));
  top = wave_max(top);
  if ((tid & 63) == 0) s_max[wave] = top;
  __syncthreads();
  top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const float scale = scale_of_bits(top), inv = inverse_of(scale);
  if (tid == 0) a.scale[row] = scale;
  int8_t* q = a.q + row * a.ldq;
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = tid + i * 256;
    if (c < a.C) q[c] = static_cast<int8_t>(code_of(v[i], inv));
  }
}

template <int T>
static void go_rows(const RowsArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.rows));
  if (a.C <= 1024)
    rows_kernel<T, 4><<<grid, 256, 0, s>>>(a);
  else if (a.C <= 4096)
    rows_kernel<T, 16><<<grid, 256, 0, s>>>(a);
  else
    rows_kernel<T, 64><<<grid, 256, 0, s>>>(a);
}

hipError_t launch_rows(int dtype, const RowsArgs& a, hipStream_t s) {
  if (dtype == EL_F32)
    go_rows<EL_F32>(a, s);
  else if (dtype == EL_BF16)
    go_rows<EL_BF16>(a, s);
  else
    go_rows<EL_F16>(a, s);
  return hipGetLastError();
}

}  // namespace voc
