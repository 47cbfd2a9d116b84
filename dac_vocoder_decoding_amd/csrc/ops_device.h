// ops_device.h -- device building blocks shared by the 8-bit transformer
// operators: element types, the 8-bit row's scale, block reductions.
#pragma once
#include "ops.h"

namespace voc {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int T> struct Elem;
template <> struct Elem<EL_F32> { typedef float type; };
template <> struct Elem<EL_BF16> { typedef __bf16 type; };
template <> struct Elem<EL_F16> { typedef _Float16 type; };

// Eight consecutive elements (16-byte aligned) as floats, and back.
template <int T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* p, float (&v)[8]) {
  typedef typename Elem<T>::type E;
  union { uint4 u[sizeof(E) / 2]; E e[8]; } x;
#pragma unroll
  for (unsigned i = 0; i < sizeof(E) / 2; ++i) x.u[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(x.e[i]);
}
template <int T>
__device__ __forceinline__ void store8(typename Elem<T>::type* p, const float (&v)[8]) {
  typedef typename Elem<T>::type E;
  union { uint4 u[sizeof(E) / 2]; E e[8]; } x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x.e[i] = static_cast<E>(v[i]);
#pragma unroll
  for (unsigned i = 0; i < sizeof(E) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = x.u[i];
}

// The scale of a group whose largest magnitude has the bit pattern `bits`
// (magnitudes compare like their bits, with NaN above infinity above every
// finite value, so an integer maximum carries a NaN along).
constexpr uint32_t kInfBits = 0x7f800000u;
__device__ __forceinline__ float scale_of_bits(uint32_t bits) {
  if (bits >= kInfBits) return __uint_as_float(0x7fc00000u);
  const float m = __uint_as_float(bits);
  return m < 0x1p-100f ? 0.f : m * (1.0f / 127.0f);
}
// 1 / scale, or 0 where every code is 0 (scale 0 or NaN).
__device__ __forceinline__ float inverse_of(float scale) { return scale > 0.f ? 1.0f / scale : 0.f; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ int code_of(float v, float inv) {
  // inv is 0 where the group holds an infinity: 0 times it must not become a code.
  const float r = inv > 0.f ? __builtin_rintf(v * inv) : 0.f;
  return static_cast<int>(fminf(fmaxf(r, -127.f), 127.f));
}

// Eight codes in a row.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[h] |= (static_cast<uint32_t>(code_of(v[4 * h + i], inv)) & 0xffu) << (8 * i);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), m)));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Orders a wave's LDS accesses before this point against those after it, for
// exchanges between its own lanes: the hardware keeps a wave's LDS accesses in
// order, and the compiler, which sees one lane's addresses only, may not move
// them across.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace voc
