// rows_kernels.hip -- rows of 8-bit codes with one scale each: the RMS norm
// with residual addition, and the plain row quantiser.
//
//   h = round(x + r);  y = h / sqrt(mean(h^2) + eps) * w;
//   s = max|y| / 127;  q = rint(y / s)
#include "ops_device.h"

namespace voc {

// Group g (eight values) of a row of C: 16-byte loads and stores where the
// rows allow them (VEC), else whole groups at any alignment and the last,
// partial one value by value (what is missing reads as zero).
template <int T, bool VEC>
__device__ __forceinline__ void load_group(const typename Elem<T>::type* row, int g, int C, float (&v)[8]) {
  typedef typename Elem<T>::type E;
  if constexpr (VEC) {
    load8<T>(row + g * 8, v);
  } else {
    E e[8];
    if (g * 8 + 8 <= C) {
      __builtin_memcpy(e, row + g * 8, 8 * sizeof(E));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = g * 8 + k < C ? row[g * 8 + k] : static_cast<E>(0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(e[k]);
  }
}
template <int T, bool VEC>
__device__ __forceinline__ void store_group(typename Elem<T>::type* row, int g, int C, const float (&v)[8]) {
  typedef typename Elem<T>::type E;
  if constexpr (VEC) {
    store8<T>(row + g * 8, v);
  } else {
    E e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = static_cast<E>(v[k]);
    if (g * 8 + 8 <= C) {
      __builtin_memcpy(row + g * 8, e, 8 * sizeof(E));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (g * 8 + k < C) row[g * 8 + k] = e[k];
    }
  }
}

// NG groups of eight values per thread, all in registers, so that every row
// is read once.  WPR waves per row: one (four rows a workgroup, no barrier) up
// to 1024 values, four above (us, one wave / four: 20000 bf16 rows quantised,
// of 1024 13.0 / 17.2, of 2048 26.4 / 23.6; 32 rows of 2048 4.5 / 2.9).  A
// workgroup goes on with the row that is a grid further, so that its weights
// are read once.  The sums' order depends neither on the number of rows nor on
// their alignment (VEC).
// Bound by memory: the norm of 19292 x 4096 bf16 rows with a residual moves
// 553 MB in 100 us (5.5 TB/s; a plain copy of 1 GiB reaches 5.2).  Few rows
// are bound by latency, one round of loads and the sums: 32 x 1024 fp16 3.9 us.
template <int T, int NG, int WPR, bool VEC>
__global__ __launch_bounds__(256) void rows_kernel(const RowsArgs a) {
  typedef typename Elem<T>::type E;
  __shared__ float s_sum[2][4];
  __shared__ uint32_t s_max[2][4];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int at = WPR == 1 ? tid & 63 : tid;    // this thread's first group
  constexpr int STEP = WPR * 64;
  const int groups = (a.C + 7) >> 3;
  float w[NG][8];
  if (a.weight) {
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (at + i * STEP < groups) load_group<EL_F32, VEC>(a.weight, at + i * STEP, a.C, w[i]);
  }
  int turn = 0;
  for (int64_t row = WPR == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x; row < a.rows;
       row += WPR == 1 ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x, turn ^= 1) {
    const E* x = static_cast<const E*>(a.x) + row * a.ldx;
    float v[NG][8];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (at + i * STEP < groups) {
        load_group<T, VEC>(x, at + i * STEP, a.C, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
      }
    }
    if (a.r) {
      const E* r = static_cast<const E*>(a.r) + row * a.ldr;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (at + i * STEP < groups) {
          float f[8];
          load_group<T, VEC>(r, at + i * STEP, a.C, f);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = static_cast<float>(static_cast<E>(v[i][k] + f[k]));
        }
      }
    }
    if (a.h) {
      E* h = static_cast<E*>(a.h) + row * a.ldh;
#pragma unroll
      for (int i = 0; i < NG; ++i)
        if (at + i * STEP < groups) store_group<T, VEC>(h, at + i * STEP, a.C, v[i]);
    }
    uint32_t top = 0;
    if (a.weight) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += v[i][k] * v[i][k];
      sum = wave_sum(sum);
      if constexpr (WPR > 1) {
        if ((tid & 63) == 0) s_sum[turn][wave] = sum;
        __syncthreads();
        sum = (s_sum[turn][0] + s_sum[turn][1]) + (s_sum[turn][2] + s_sum[turn][3]);
      }
      const float rms = rsqrtf(sum / static_cast<float>(a.C) + a.eps);
      if (abs_bits(sum) >= kInfBits) top = kInfBits;
#pragma unroll
      for (int i = 0; i < NG; ++i)
        if (at + i * STEP < groups) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = v[i][k] * rms * w[i][k];
        }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, abs_bits(v[i][k]));
    top = wave_max(top);
    if constexpr (WPR > 1) {
      if ((tid & 63) == 0) s_max[turn][wave] = top;
      __syncthreads();
      top = max(max(s_max[turn][0], s_max[turn][1]), max(s_max[turn][2], s_max[turn][3]));
    }
    const float scale = scale_of_bits(top), inv = inverse_of(scale);
    if (at == 0) a.scale[row] = scale;
    int8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (at + i * STEP < groups) {
        const int c = (at + i * STEP) * 8;
        const uint2 u = codes8(v[i], inv);
        if (VEC) {
          *reinterpret_cast<uint2*>(q + c) = u;
        } else if (c + 8 <= a.C) {
          __builtin_memcpy(q + c, &u, 8);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.C) q[c + k] = static_cast<int8_t>((k < 4 ? u.x : u.y) >> (8 * (k & 3)));
        }
      }
  }
}

template <int T, int NG, int WPR, bool VEC>
static void launch_form(const RowsArgs& a, hipStream_t s, Form& form) {
  form = Form{"rows", {NG, WPR}};
  // Enough workgroups to fill every CU eight times over (1024 or 8192: within 10 %).
  const int64_t most = 2048, wgs = WPR == 1 ? (a.rows + 3) / 4 : a.rows;
  rows_kernel<T, NG, WPR, VEC><<<dim3(static_cast<unsigned>(wgs < most ? wgs : most)), 256, 0, s>>>(a);
}

template <int T, bool VEC>
static void pick_rows(const RowsArgs& a, hipStream_t s, Form& form) {
  if (a.C <= 512)
    launch_form<T, 1, 1, VEC>(a, s, form);
  else if (a.C <= 1024)
    launch_form<T, 2, 1, VEC>(a, s, form);
  else if (a.C <= 2048)
    launch_form<T, 1, 4, VEC>(a, s, form);
  else if (a.C <= 4096)
    launch_form<T, 2, 4, VEC>(a, s, form);
  else if (a.C <= 8192)
    launch_form<T, 4, 4, VEC>(a, s, form);
  else
    launch_form<T, 8, 4, VEC>(a, s, form);
}

template <int T>
static void go_rows(const RowsArgs& a, hipStream_t s, Form& form) {
  auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  constexpr int per16 = 16 / sizeof(typename Elem<T>::type);
  const bool vec = a.C % 8 == 0 && on16(a.x) && on16(a.r) && on16(a.h) && on16(a.weight) &&
                   reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && a.ldx % per16 == 0 && a.ldr % per16 == 0 &&
                   a.ldh % per16 == 0 && a.ldq % 8 == 0;
  if (vec)
    pick_rows<T, true>(a, s, form);
  else
    pick_rows<T, false>(a, s, form);
}

hipError_t launch_rows(int dtype, const RowsArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_rows<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    go_rows<EL_BF16>(a, s, form);
  else
    go_rows<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
