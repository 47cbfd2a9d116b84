// heads_kernels.hip -- the RMS norm of each head with the rotation by
// position, and the same with the keys quantised straight into the paged
// 8-bit cache beside the values.
//
//   y = x / sqrt(mean(x^2) + eps) * w           (over a head's D values)
//   (a, b) -> (a cos - b sin, b cos + a sin)    for each of F pairs of y,
//   angle = position * freq[pair]
//
// A head's values lie in units of eight, one a lane: four pairs where values
// rotate, eight values in a row behind them.  G lanes (a power of two) hold a
// head, so that its sum is a shuffle among them.
#include <type_traits>

#include "cache_device.h"

namespace voc {

// How a unit's pairs lie: 2i, 2i + 1 or i, i + F, both read in whole words;
// or either of them at any alignment and F, value by value.
enum Pairs { kAdjacent = 0, kHalves = 1, kAny = 2 };

// Four consecutive elements (aligned to their size).
template <int T>
__device__ __forceinline__ void load4(const typename Elem<T>::type* p, float* v, int step) {
  typename Elem<T>::type e[4];
  __builtin_memcpy(e, __builtin_assume_aligned(p, sizeof(e)), sizeof(e));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i * step] = static_cast<float>(e[i]);
}
template <int T>
__device__ __forceinline__ void store4(typename Elem<T>::type* p, const float* v, int step) {
  typename Elem<T>::type e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = static_cast<typename Elem<T>::type>(v[i * step]);
  __builtin_memcpy(__builtin_assume_aligned(p, sizeof(e)), e, sizeof(e));
}

// The place of a lane's unit in its head.
template <int MODE>
struct Unit {
  int at, hi;      // MODE < kAny: first value (kHalves: of the first and the second four)
  int unit, F, D;  // kAny
  bool adjacent, live, turns;
  __device__ __forceinline__ Unit(int u, int F, int D, bool adjacent)
      : unit(u), F(F), D(D), adjacent(MODE == kAdjacent || (MODE == kAny && adjacent)) {
    const int turning = (F + 3) >> 2;
    turns = u < turning;
    if constexpr (MODE == kHalves) {
      at = turns ? 4 * u : 8 * u;
      hi = turns ? F + 4 * u : 8 * u + 4;
    } else {
      at = 8 * u;
      hi = at + 4;
    }
    live = turns || 2 * F + 8 * (u - turning) < D;
  }
  // The value that sits at place k of the unit, or -1.
  __device__ __forceinline__ int value(int k) const {
    if (turns) {
      const int p = 4 * unit + (k >> 1);
      return p >= F ? -1 : adjacent ? 2 * p + (k & 1) : p + (k & 1) * F;
    }
    const int d = 2 * F + 8 * (unit - ((F + 3) >> 2)) + (adjacent ? k : (k >> 1) + 4 * (k & 1));
    return d < D ? d : -1;
  }
  // Places 2i and 2i + 1 are a pair; behind pairs of halves the first four
  // values have the even places.
  template <int T>
  __device__ __forceinline__ void load(const typename Elem<T>::type* head, float (&v)[8]) const {
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = value(k);
        v[k] = d >= 0 ? static_cast<float>(head[d]) : 0.f;
      }
    } else if (!live) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
    } else if constexpr (MODE == kAdjacent) {
      load8<T>(head + at, v);
    } else {
      load4<T>(head + at, v, 2);
      load4<T>(head + hi, v + 1, 2);
    }
  }
  template <int T>
  __device__ __forceinline__ void store(typename Elem<T>::type* head, const float (&v)[8]) const {
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = value(k);
        if (d >= 0) head[d] = static_cast<typename Elem<T>::type>(v[k]);
      }
    } else if (live) {
      if constexpr (MODE == kAdjacent) {
        store8<T>(head + at, v);
      } else {
        store4<T>(head + at, v, 2);
        store4<T>(head + hi, v + 1, 2);
      }
    }
  }
  // The unit's codes into a row of D codes.
  __device__ __forceinline__ void store_codes(int8_t* row, const float (&v)[8], float inv) const {
    if constexpr (MODE == kAdjacent) {
      if (live) *reinterpret_cast<uint2*>(row + at) = codes8(v, inv);
    } else if constexpr (MODE == kHalves) {
      if (!live) return;
      const float o[8] = {v[0], v[2], v[4], v[6], v[1], v[3], v[5], v[7]};
      const uint2 c = codes8(o, inv);
      *reinterpret_cast<uint32_t*>(row + at) = c.x;
      *reinterpret_cast<uint32_t*>(row + hi) = c.y;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = value(k);
        if (d >= 0) row[d] = static_cast<int8_t>(code_of(v[k], inv));
      }
    }
  }
};

// cos and sin of `turns` (revolutions): the fraction of a quarter turn in 64
// bits, where a far position's angle keeps its places (at 2^20 radians fp32
// holds steps of 1/16), the rest in fp32.  The polynomials are minimax fits of
// sin(pi t / 2) and cos(pi t / 2) over |t| <= 1/2 (errors 3e-12 and 5e-11).
__device__ __forceinline__ void cos_sin(double turns, float& c, float& s) {
  const double r = (turns - __builtin_rint(turns)) * 4.0;
  const double q = __builtin_rint(r);
  const float t = static_cast<float>(r - q), z = t * t;
  float a = fmaf(z, 0.000158206531f, -0.00468126638f);
  a = fmaf(z, a, 0.0796925798f);
  a = fmaf(z, a, -0.645964086f);
  const float sn = fmaf(t, 1.57079637f, t * z * a);
  float b = fmaf(z, 0.000903629872f, -0.0208600704f);
  b = fmaf(z, b, 0.253669202f);
  b = fmaf(z, b, -1.23370051f);
  const float cn = fmaf(z, b, 1.f);
  const int quarter = static_cast<int>(q) & 3;
  const float x = quarter & 1 ? sn : cn, y = quarter & 1 ? cn : sn;
  c = quarter == 1 || quarter == 2 ? -x : x;
  s = quarter >= 2 ? -y : y;
}

template <int MODE>
__device__ __forceinline__ void angles(const HeadShape& h, const Unit<MODE>& u, int position, float (&c)[4], float (&s)[4]) {
  constexpr double kTurn = 0.15915494309189535;  // 1 / (2 pi)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 4 * u.unit + i;
    c[i] = 1.f;
    s[i] = 0.f;
    if (p < h.pairs) cos_sin(static_cast<double>(position) * (static_cast<double>(h.freq[p]) * kTurn), c[i], s[i]);
  }
}

// One head in place: the norm (with weights), then the rotation.  A head whose
// sum of squares is not finite becomes NaN.
template <int G, int MODE>
__device__ __forceinline__ void turn(const HeadShape& h, const Unit<MODE>& u, bool norm, const float (&w)[8],
                                     const float (&c)[4], const float (&s)[4], float (&v)[8]) {
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);  // (the same steps whatever the alignment)
#pragma unroll
    for (int m = G / 2; m; m >>= 1) sum += __shfl_xor(sum, m);
    float rms = rsqrtf(sum / static_cast<float>(h.D) + h.eps);
    if (abs_bits(sum) >= kInfBits) rms = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * rms * w[k];
  }
  if (u.turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = fmaf(a, c[i], -(b * s[i]));
      v[2 * i + 1] = fmaf(b, c[i], a * s[i]);
    }
  }
}

template <int MODE>
__device__ __forceinline__ void load_weight(const Unit<MODE>& u, const float* w, float (&v)[8]) {
  if (w) {
    u.template load<EL_F32>(w, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 1.f;
  }
}

// A wave turns the heads of one token from its own share of them, 64 / G at a
// time, queries first.
template <int T, int MODE, int G>
__device__ __forceinline__ void turn_token(const HeadShape& h, const HeadSet& q, const HeadSet& k, int64_t row,
                                           int position, int part, int parts) {
  typedef typename Elem<T>::type E;
  constexpr int GW = 64 / G;
  const int lane = threadIdx.x & 63;
  const Unit<MODE> u(lane % G, h.pairs, h.D, h.adjacent);
  float c[4], s[4], wq[8], wk[8];
  load_weight(u, q.w, wq);
  load_weight(u, k.w, wk);
  angles(h, u, position, c, s);
  const int heads = q.heads + k.heads;
  for (int h0 = part * GW; h0 < heads; h0 += parts * GW) {
    const int head = h0 + lane / G;
    const bool key = head >= q.heads;
    if (head >= heads) continue;  // (a whole group of lanes: the shuffles stay inside one)
    const HeadSet& set = key ? k : q;
    const int at = key ? head - q.heads : head;
    float v[8], w[8];
    u.template load<T>(static_cast<const E*>(set.x) + row * set.x_t + at * set.x_h, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = key ? wk[i] : wq[i];
    turn<G>(h, u, set.w != nullptr, w, c, s, v);
    u.template store<T>(static_cast<E*>(set.y) + row * set.y_t + at * set.y_h, v);
  }
}

template <int T, int MODE, int G>
__global__ __launch_bounds__(256) void norm_rotate_kernel(const NormRotateArgs a, int parts) {
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t row = wave / parts;
  if (row >= a.tokens) return;
  turn_token<T, MODE, G>(a.h, a.q, a.k, row, a.position ? a.position[row] : 0, static_cast<int>(wave % parts), parts);
}

// Workgroup roles along x: the pages that a sequence's new tokens touch times
// its cache heads, keys and then values; behind them the queries.
template <int T, int MODE, int G>
__global__ __launch_bounds__(256) void step_few_kernel(const StepArgs a, int pages, int parts) {
  typedef typename Elem<T>::type E;
  constexpr int TC = 256 / G;  // tokens at a time
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  const int cached = pages * 2 * a.c.heads;
  if (static_cast<int>(blockIdx.x) >= cached) {
    const Seq s = load_seq(a.c, b);
    const int wave = (blockIdx.x - cached) * 4 + (tid >> 6), i = wave / parts;
    if (i < s.count) turn_token<T, MODE, G>(a.h, a.q, HeadSet{}, s.start + i, s.past + i, wave % parts, parts);
    return;
  }
  const int j = blockIdx.x / (2 * a.c.heads), y = blockIdx.x % (2 * a.c.heads), head = y >> 1;
  const bool value = y & 1;
  const PageShare sh = page_share(a.c, b, j, head);
  const int lo = sh.lo, hi = sh.hi;
  if (hi <= lo) return;
  const int P = 1 << a.c.page_log, D = a.h.D;
  int8_t* codes = (value ? a.c.v : a.c.k) + sh.slot * P * D;
  float* scales = value ? a.c.vs : a.c.ks;
  const float old = lo ? scales[sh.slot] : 0.f;
  const Unit<MODE> u(tid % G, value ? 0 : a.h.pairs, D, a.h.adjacent);
  float w[8];
  load_weight(u, value ? nullptr : a.k.w, w);
  const E* src = (value ? static_cast<const E*>(a.v) + head * a.v_h : static_cast<const E*>(a.k.x) + head * a.k.x_h) +
                 (sh.token - lo) * (value ? a.v_t : a.k.x_t);
  const int64_t st = value ? a.v_t : a.k.x_t;
  float v[8];
  auto load = [&](int t) {
    u.template load<T>(src + t * st, v);
    if (!value) {
      float c[4], s[4];
      angles(a.h, u, static_cast<int>(sh.first) + t, c, s);
      turn<G>(a.h, u, a.k.w != nullptr, w, c, s, v);
    }
  };
  uint32_t top = 0;
  for (int t = lo + tid / G; t < hi; t += TC) {
    load(t);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, abs_bits(v[k]));
  }
  top = wave_max(top);
  if ((tid & 63) == 0) s_max[tid >> 6] = top;
  __syncthreads();
  top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const float scale = joint_scale(old, top), inv = inverse_of(scale);
  if (lo && scale != old) {
    const float ratio = inv > 0.f ? old * inv : 0.f;
    for (int i = tid; i < lo * D; i += 256) {
      const int t = i / D, d = i - t * D;
      int8_t* p = codes + (value ? d * P + t : i);
      *p = static_cast<int8_t>(__builtin_rintf(static_cast<float>(*p) * ratio));
    }
  }
  for (int t = lo + tid / G; t < hi; t += TC) {
    if (hi - lo > TC) load(t);  // (else its values are still here)
    if (!value) {
      u.store_codes(codes + static_cast<int64_t>(t) * D, v, inv);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = u.value(k);
        if (d >= 0) codes[static_cast<int64_t>(d) * P + t] = static_cast<int8_t>(code_of(v[k], inv));
      }
    }
  }
  if (tid == 0) scales[sh.slot] = scale;
}

// Lanes that hold a head.
static int head_lanes(int D, int pairs) {
  const int units = (pairs + 3) / 4 + (D - 2 * pairs + 7) / 8;
  int g = 4;
  while (g < units) g *= 2;
  return g;
}

template <class F>
static void by_lanes(int g, F&& f) {
  if (g == 4)
    f(std::integral_constant<int, 4>{});
  else if (g == 8)
    f(std::integral_constant<int, 8>{});
  else if (g == 16)
    f(std::integral_constant<int, 16>{});
  else if (g == 32)
    f(std::integral_constant<int, 32>{});
  else
    f(std::integral_constant<int, 64>{});
}
template <class F>
static void by_pairs(int mode, F&& f) {
  if (mode == kAdjacent)
    f(std::integral_constant<int, kAdjacent>{});
  else if (mode == kHalves)
    f(std::integral_constant<int, kHalves>{});
  else
    f(std::integral_constant<int, kAny>{});
}
template <class F>
static void by_type(int dtype, F&& f) {
  if (dtype == EL_F32)
    f(std::integral_constant<int, EL_F32>{});
  else if (dtype == EL_BF16)
    f(std::integral_constant<int, EL_BF16>{});
  else
    f(std::integral_constant<int, EL_F16>{});
}

static bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
static bool whole_words(const HeadSet& s, int dtype) {
  const int per16 = 16 / elem_size(dtype);
  return on16(s.x) && on16(s.y) && on16(s.w) && (s.x_t | s.x_h | s.y_t | s.y_h) % per16 == 0;
}
static int pairs_mode(const HeadShape& h, bool whole) {
  return !whole || h.D % 8 || h.pairs % 4 ? kAny : h.adjacent || !h.pairs ? kAdjacent : kHalves;
}

// Waves that share a token's heads: each has at least one round of them, and
// all of them together fill the chip four times over.
static int token_parts(int heads, int g, int64_t tokens) {
  const int rounds = (heads * g + 63) / 64;
  const int64_t want = (4096 + tokens - 1) / tokens;
  return static_cast<int>(want < rounds ? want : rounds);
}

hipError_t launch_norm_rotate(int dtype, const NormRotateArgs& a, hipStream_t s, Form& form) {
  const int g = head_lanes(a.h.D, a.h.pairs), mode = pairs_mode(a.h, whole_words(a.q, dtype) && whole_words(a.k, dtype));
  const int parts = token_parts(a.q.heads + a.k.heads, g, a.tokens);
  form = Form{"heads", {g, mode}};
  const unsigned grid = static_cast<unsigned>((a.tokens * parts + 3) / 4);
  by_type(dtype, [&](auto t) {
    by_pairs(mode, [&](auto m) {
      by_lanes(g, [&](auto l) {
        norm_rotate_kernel<decltype(t)::value, decltype(m)::value, decltype(l)::value><<<grid, 256, 0, s>>>(a, parts);
      });
    });
  });
  return hipGetLastError();
}

static int step_pages(const StepArgs& a) { return ((a.c.max_new - 1) >> a.c.page_log) + 2; }

int64_t step_workgroups(const StepArgs& a) {
  const int parts = token_parts(a.q.heads, head_lanes(a.h.D, a.h.pairs), a.c.tokens);
  return static_cast<int64_t>(step_pages(a)) * 2 * a.c.heads + (static_cast<int64_t>(a.c.max_new) * parts + 3) / 4;
}

hipError_t launch_step(int dtype, const StepArgs& a, hipStream_t s, Form& form) {
  const int g = head_lanes(a.h.D, a.h.pairs), per16 = 16 / elem_size(dtype);
  const bool whole = whole_words(a.q, dtype) && whole_words(a.k, dtype) && on16(a.v) && (a.v_t | a.v_h) % per16 == 0;
  const int mode = pairs_mode(a.h, whole);
  const int pages = step_pages(a), parts = token_parts(a.q.heads, g, a.c.tokens);
  form = Form{"step", {g, mode}};
  const dim3 grid(static_cast<unsigned>(step_workgroups(a)), a.batch);
  by_type(dtype, [&](auto t) {
    by_pairs(mode, [&](auto m) {
      by_lanes(g, [&](auto l) {
        step_few_kernel<decltype(t)::value, decltype(m)::value, decltype(l)::value><<<grid, 256, 0, s>>>(a, pages, parts);
      });
    });
  });
  return hipGetLastError();
}

}  // namespace voc
