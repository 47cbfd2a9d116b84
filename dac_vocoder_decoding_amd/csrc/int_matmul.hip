// int_matmul.hip -- the 8-bit integer product with row scales,
//   y[m][n] = act((sum_k a[m][k] b[n][k]) sa[m] sb[n] + bias[n]),
// on the gfx950 matrix cores (v_mfma_i32_16x16x64_i8: 32-bit integer sums,
// exact for K <= 131071).
//
// The matrix-core "A" operand is b (output features), "B" is a (tokens): a
// lane then holds four consecutive features of one token, which it stores
// together.
#include <string.h>

#include "ops_device.h"

namespace voc {

// 16 bytes of a row of K codes at k, zero past the row's end; any alignment.
__device__ __forceinline__ i32x4 load_codes(const int8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else if (k < K) {
    int8_t t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = k + i < K ? row[k + i] : int8_t(0);
    __builtin_memcpy(&v, t, 16);
  }
  return v;
}

__device__ __forceinline__ float activate(float v, int act) {
  return act ? 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)) : v;
}

// One wave per 16 tokens x 64 features, operands read straight from memory.
template <int T>
__global__ __launch_bounds__(256) void int_matmul_kernel(const IntMatmulArgs a) {
  typedef typename Elem<T>::type E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int n0 = (blockIdx.x * 4 + wave) * 64;
  const int m = blockIdx.y * 16 + lr;
  if (n0 >= a.N) return;
  i32x4 acc[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
  const int8_t* arow = a.a + static_cast<int64_t>(min(m, a.M - 1)) * a.lda;
  const int8_t* brow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) brow[j] = a.b + static_cast<int64_t>(min(n0 + j * 16 + lr, a.N - 1)) * a.ldb;
  for (int k = lg * 16; k < a.K + lg * 16; k += 64) {
    const i32x4 av = load_codes(arow, k, a.K);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_codes(brow[j], k, a.K), av, acc[j], 0, 0, 0);
  }
  if (m >= a.M) return;
  const float sa = a.sa[m];
  E* y = static_cast<E*>(a.y) + static_cast<int64_t>(m) * a.ldy;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + j * 16 + lg * 4 + i;
      if (n < a.N) {
        const float v = static_cast<float>(acc[j][i]) * sa * a.sb[n] + (a.bias ? a.bias[n] : 0.f);
        y[n] = static_cast<E>(activate(v, a.act));
      }
    }
}

hipError_t launch_int_matmul(int dtype, const IntMatmulArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 255) / 256, (a.M + 15) / 16);
  if (dtype == EL_F32)
    int_matmul_kernel<EL_F32><<<grid, 256, 0, s>>>(a);
  else if (dtype == EL_BF16)
    int_matmul_kernel<EL_BF16><<<grid, 256, 0, s>>>(a);
  else
    int_matmul_kernel<EL_F16><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace voc
