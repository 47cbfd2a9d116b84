// adapters.hip -- the 8-bit product with the low-rank adapter of each row
// beside the shared weights,
//   y[m][n] = act((sum_k a[m][k] b[n][k]) sa[m] sb[n] + bias[n]
//                 + sum_r up_i[n][r] u[m][r]),   i = adapter[m]
//   u[m][r] = scale[i] sa[m] sum_k down_i[r][k] a[m][k].
//
// Two launches: u (fp32, in the handle's workspace), then the product, whose
// epilogue adds the terms (int_matmul.h).  Codes are exact in fp16 and bf16, so
// that u is a sum of exact products in fp32.
#include "int_matmul.h"

namespace voc {

// 8 codes of a row of K at k, zero past its end.
__device__ __forceinline__ uint2 load_codes8(const int8_t* row, int k, int K) {
  uint2 c = {0, 0};
  if (k + 8 <= K) {
    __builtin_memcpy(&c, row + k, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) (i < 4 ? c.x : c.y) |= (static_cast<uint32_t>(row[k + i]) & 0xffu) << (8 * (i & 3));
  }
  return c;
}

// Eight weights of a row of K at k (16-byte aligned, ldd covers them).
template <bool BF16>
__device__ __forceinline__ void load_down(const uint16_t* p, float (&w)[8]) {
  if constexpr (BF16)
    load8<EL_BF16>(reinterpret_cast<const __bf16*>(p), w);
  else
    load8<EL_F16>(reinterpret_cast<const _Float16*>(p), w);
}

// A wave per token and four ranks.
template <bool BF16>
__global__ __launch_bounds__(256) void shrink_few_kernel(const AdaptArgs a) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.y, r0 = blockIdx.x * 16 + (threadIdx.x >> 6) * 4;
  const int id = a.g.adapter[m], K = a.g.K;
  if (id < 0 || id >= a.g.adapters) return;
  const int8_t* row = a.g.a + static_cast<int64_t>(m) * a.g.lda;
  const uint16_t* down = a.down + (static_cast<int64_t>(id) * a.g.rank + r0) * a.ldd;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = lane * 8; k < K; k += 512) {
    const uint2 c = load_codes8(row, k, K);
    float w[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_down<BF16>(down + i * a.ldd + k, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = static_cast<float>(static_cast<int8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3))));
      if (k + j < K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(x, w[i][j], sum[i]);
      }
    }
  }
  const float f = a.g.sa[m] * (a.scale ? a.scale[id] : 1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = wave_sum(sum[i]) * f;
  if (lane == 0) *reinterpret_cast<float4*>(a.u + static_cast<int64_t>(m) * a.g.rank + r0) = make_float4(sum[0], sum[1], sum[2], sum[3]);
}

hipError_t launch_int_matmul_adapters(int dtype, const AdaptArgs& a, hipStream_t s, Form& form) {
  if (a.g.up_bf16)
    shrink_few_kernel<true><<<dim3(a.g.rank / 16, a.g.M), 256, 0, s>>>(a);
  else
    shrink_few_kernel<false><<<dim3(a.g.rank / 16, a.g.M), 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dtype == EL_F32)
    go_int_matmul<EL_F32, true>(a.g, s, form);
  else if (dtype == EL_BF16)
    go_int_matmul<EL_BF16, true>(a.g, s, form);
  else
    go_int_matmul<EL_F16, true>(a.g, s, form);
  return hipGetLastError();
}

}  // namespace voc
