// cache_kernels.hip -- appending keys and values to the paged 8-bit cache.
//
// Per page and cache head: s' = max(s_old, max|new| / 127); the new tokens'
// codes are rint(x / s'), the older codes are rounded again,
// rint(q s_old / s'), where s' grew.
#include "cache_device.h"

namespace voc {

// Any alignment, and few new tokens.  Workgroup (j, 2 * head + is_value,
// sequence): the j-th page that the sequence's new tokens touch.  Values are
// stored transposed inside a page.  Bound by latency, a chain of three loads
// (the sequence, its page, the new row and the old scale): one token of 32 x 8
// heads x 128 d 5.2 us.
template <int T>
__global__ __launch_bounds__(256) void append_kernel(const AppendArgs a) {
  typedef typename Elem<T>::type E;
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  const int head = blockIdx.y >> 1;
  const bool value = blockIdx.y & 1;
  const int P = 1 << a.c.page_log, D = a.D;
  const PageShare sh = page_share(a.c, blockIdx.z, blockIdx.x, head);
  const int lo = sh.lo, hi = sh.hi;
  if (hi <= lo) return;
  const int64_t slot = sh.slot;
  const int64_t st = value ? a.v_t : a.k_t;
  const E* src = (value ? static_cast<const E*>(a.v) + head * a.v_h : static_cast<const E*>(a.k) + head * a.k_h) + sh.token * st;
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
  const float scale = joint_scale(old, top);
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

// Many new tokens, rows of 16-byte multiples.  The page's image is built in
// LDS and written whole, 16 bytes at a time: a value page is turned over
// there, four tokens of one d to a 32-bit word.  The new rows stay in
// registers between the maximum and the codes where a thread has up to two
// units (4 tokens x 8 values); larger pages read the rest a second time.
// Bound by memory and by each page's chain of loads: 8 prompts of up to 5168
// bf16 tokens of 8 x 128 d (217 MB) 58 us, 3.7 TB/s.  (Pages in the order of
// their heads: 63; stores around the L2: 59.)
// LDS: a key page [token][D], a value page [d][token] with rows of P + 4
// bytes (the writes of neighbouring d then fall on different banks).
template <int T, int D, int NT>
__global__ __launch_bounds__(NT) void append_page_kernel(const AppendArgs a) {
  typedef typename Elem<T>::type E;
  constexpr int KEEP = 2;
  constexpr int D8 = D >> 3;
  extern __shared__ __attribute__((aligned(16))) unsigned char s_page[];
  __shared__ uint32_t s_max[NT / 64];
  const int tid = threadIdx.x;
  const int head = blockIdx.y >> 1;
  const bool value = blockIdx.y & 1;
  const int P = 1 << a.c.page_log;
  const PageShare sh = page_share(a.c, blockIdx.z, blockIdx.x, head);
  const int lo = sh.lo, hi = sh.hi;
  if (hi <= lo) return;
  const int64_t st = value ? a.v_t : a.k_t;
  const E* src = (value ? static_cast<const E*>(a.v) + head * a.v_h : static_cast<const E*>(a.k) + head * a.k_h) +
                 (sh.token - lo) * st;  // row t of the page (t >= lo)
  int8_t* codes = (value ? a.c.v : a.c.k) + sh.slot * P * D;
  float* scales = value ? a.c.vs : a.c.ks;
  const float old = lo ? scales[sh.slot] : 0.f;

  const int units = (P >> 2) * D8;
  float keep[KEEP][4][8];
  uint32_t top = 0;
  auto load_unit = [&](int u, float (&v)[4][8]) {
    const int t4 = u / D8 * 4, d8 = u % D8 * 8;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t4 + t >= lo && t4 + t < hi) {
        load8<T>(src + (t4 + t) * st + d8, v[t]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[t][k] = 0.f;
      }
    }
  };
  auto raise = [&](const float (&v)[4][8]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, abs_bits(v[t][k]));
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (tid + i * NT < units) {
      load_unit(tid + i * NT, keep[i]);
      raise(keep[i]);
    }
  for (int u = tid + KEEP * NT; u < units; u += NT) {
    float v[4][8];
    load_unit(u, v);
    raise(v);
  }
  top = wave_max(top);
  if ((tid & 63) == 0) s_max[tid >> 6] = top;
  // The page as it is, where some of it stays.
  const int pitch = value ? P + 4 : D;  // bytes of a row of the image
  // Words of a row, as a shift (a key page is one long row: its image is the page).
  const int row_log = a.c.page_log - 2;
  if (lo > 0 || hi < P) {
    for (int w = tid; w < (P * D) >> 4; w += NT) {
      const uint4 c = reinterpret_cast<const uint4*>(codes)[w];
      uint32_t* p = reinterpret_cast<uint32_t*>(s_page + w * 16 + (value ? (w >> (row_log - 2)) * 4 : 0));
      p[0] = c.x;
      p[1] = c.y;
      p[2] = c.z;
      p[3] = c.w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) top = max(top, s_max[w]);
  const float scale = joint_scale(old, top), inv = inverse_of(scale);
  if (lo && scale != old) {
    const float ratio = inv > 0.f ? old * inv : 0.f;
    // Four codes at a time; what follows the older tokens in their last word is
    // either written below or holds no token.
    for (int w = tid; w < (P * D) >> 2; w += NT)
      if (value ? 4 * (w & ((P >> 2) - 1)) < lo : 4 * w < lo * D) {
        uint32_t* p = reinterpret_cast<uint32_t*>(s_page + w * 4 + (value ? (w >> row_log) * 4 : 0));
        *p = rescaled4(*p, ratio);
      }
    __syncthreads();
  }
  auto put = [&](int u, const float (&v)[4][8]) {
    const int t4 = u / D8 * 4, d8 = u % D8 * 8;
    if (t4 + 4 <= lo || t4 >= hi) return;
    uint2 c[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = codes8(v[t], inv);
    if (!value) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t4 + t >= lo && t4 + t < hi) *reinterpret_cast<uint2*>(s_page + (t4 + t) * pitch + d8) = c[t];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t w = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) w |= (((k < 4 ? c[t].x : c[t].y) >> (8 * (k & 3))) & 0xffu) << (8 * t);
        unsigned char* p = s_page + (d8 + k) * pitch + t4;
        if (t4 >= lo && t4 + 4 <= hi) {
          *reinterpret_cast<uint32_t*>(p) = w;
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (t4 + t >= lo && t4 + t < hi) p[t] = static_cast<unsigned char>(w >> (8 * t));
        }
      }
    }
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (tid + i * NT < units) put(tid + i * NT, keep[i]);
  for (int u = tid + KEEP * NT; u < units; u += NT) {
    float v[4][8];
    load_unit(u, v);
    put(u, v);
  }
  __syncthreads();
  for (int w = tid; w < (P * D) >> 4; w += NT) {
    uint4 v;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(s_page + w * 16 + (value ? (w >> (row_log - 2)) * 4 : 0));
    v.x = p[0];
    v.y = p[1];
    v.z = p[2];
    v.w = p[3];
    reinterpret_cast<uint4*>(codes)[w] = v;
  }
  if (tid == 0) scales[sh.slot] = scale;
}

// A thread for every unit of a page (4 tokens x 8 values), from one wave to
// four; one wave only where the pages are enough to fill the chip with them
// (us, two waves / as chosen: 8 prompts of 5168 x 8 heads x 64 d, pages of 32:
// 51.4 / 35.8; 2 prompts x 4 x 256, pages of 128: 44.0 / 27.0; 32 chunks of 25
// x 16 x 64, pages of 32: 10.1, one wave 15.4).
template <int T, int D>
static void go_pages(const AppendArgs& a, dim3 grid, hipStream_t s, Form& form) {
  const int P = 1 << a.c.page_log, units = P / 4 * (D / 8);
  const size_t lds = static_cast<size_t>(D) * (P + 4);
  const bool full = static_cast<int64_t>(grid.x) * grid.y * grid.z >= 4096;
  if constexpr (D <= 128)  // (larger heads have no page of 64 units, heads of 32 none of more than 128)
    if (units <= 64 && full) {
      form = Form{"append_page", {64, P}};
      append_page_kernel<T, D, 64><<<grid, 64, lds, s>>>(a);
      return;
    }
  if constexpr (D > 32)
    if (units > 128) {
      form = Form{"append_page", {256, P}};
      append_page_kernel<T, D, 256><<<grid, 256, lds, s>>>(a);
      return;
    }
  form = Form{"append_page", {128, P}};
  append_page_kernel<T, D, 128><<<grid, 128, lds, s>>>(a);
}

template <int T>
static void go_append(const AppendArgs& a, hipStream_t s, Form& form) {
  const int P = 1 << a.c.page_log;
  const dim3 grid((a.c.max_new + P - 1) / P + 1, 2 * a.c.heads, a.batch);
  constexpr int per16 = 16 / sizeof(typename Elem<T>::type);
  const bool vec = (reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) % 16 == 0 &&
                   (a.k_t | a.k_h | a.v_t | a.v_h) % per16 == 0;
  // A few tokens leave most of a page as it is, and only a scale that grew makes
  // the small kernel touch it (us, small / page kernel, 32 x 8 heads x 128 d,
  // pages of 64: 1 token 5.2 / 7.8, 8 tokens 9.1 / 9.0, 25 tokens 19.6 / 9.5;
  // 32 x 16 x 64, pages of 32: 5.5 / 7.0, 7.2 / 8.1, 10.7 / 8.2).
  if (!vec || a.c.max_new <= 8) {
    form = Form{"append", {256, P}};
    append_kernel<T><<<grid, 256, 0, s>>>(a);
    return;
  }
  switch (a.D / 32) {
    case 1: go_pages<T, 32>(a, grid, s, form); break;
    case 2: go_pages<T, 64>(a, grid, s, form); break;
    case 3: go_pages<T, 96>(a, grid, s, form); break;
    case 4: go_pages<T, 128>(a, grid, s, form); break;
    case 5: go_pages<T, 160>(a, grid, s, form); break;
    case 6: go_pages<T, 192>(a, grid, s, form); break;
    case 7: go_pages<T, 224>(a, grid, s, form); break;
    default: go_pages<T, 256>(a, grid, s, form); break;
  }
}

hipError_t launch_append(int dtype, const AppendArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_append<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    go_append<EL_BF16>(a, s, form);
  else
    go_append<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
