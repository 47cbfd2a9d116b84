// cache_read.hip -- the tokens of the paged 8-bit cache as rows again:
// code * scale of the page, rounded once.
#include "cache_device.h"

namespace voc {

template <int T, bool VEC>
__device__ __forceinline__ void put8(typename Elem<T>::type* p, const float (&v)[8], bool stream) {
  if constexpr (VEC) {
    if (stream) {
      stream8<T>(p, v);
      asm volatile("");  // (else the compiler makes one plain store of both)
    } else {
      store8<T>(p, v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = static_cast<typename Elem<T>::type>(v[k]);
  }
}

// Code k of a word times its scale as an fp32 product of its own: the compiler
// would otherwise make one instruction of it and the rounding to fp16, in some
// places, whose result differs where the product is halfway between two.
__device__ __forceinline__ float value_at(uint32_t w, int k, float scale) {
  float v = static_cast<float>(static_cast<int8_t>(w >> (8 * k))) * scale;
  asm("" : "+v"(v));
  return v;
}

// A workgroup reads BYTES of codes of one page, keys or values, over its heads.
// Keys: a thread takes eight codes of a row at a time.  Values are transposed
// inside a page, so that they are turned over in LDS: these are rows of P tokens
// for consecutive d (and heads), a thread takes four tokens of eight of them,
// and its neighbours the next eight, which makes whole rows of stores.  (Turned
// over in registers, 16 bytes of a row a lane: 2 x 65536 tokens of 8 x 128 d in
// bf16 165 us.)
template <int T, bool VEC, int BYTES>
__global__ __launch_bounds__(256) void cache_read_kernel(const ReadArgs a, int blocks, uint32_t by_dim) {
  typedef typename Elem<T>::type E;
  __shared__ __attribute__((aligned(16))) unsigned char s_codes[BYTES + BYTES / 32];
  const int log = a.c.page_log, P = 1 << log, D = a.D, tid = threadIdx.x;
  const int kinds = (a.k != nullptr) + (a.v != nullptr);
  const int per = blocks / kinds;  // workgroups of the page's keys, or values
  const int j = blockIdx.x / blocks, in_page = blockIdx.x % blocks;
  const bool value = a.k == nullptr || in_page >= per;
  const int part = a.k != nullptr && value ? in_page - per : in_page;
  const PageShare sh = page_share(a.c, blockIdx.y, j, 0);
  const int lo = sh.lo, hi = sh.hi;
  if (hi <= lo) return;
  const int64_t page = sh.slot * P * D;  // (of head 0: the page's first code)
  const int bytes = a.c.heads * P * D, from = part * BYTES, to = min(bytes, from + BYTES);
  if (!value) {
    const int8_t* codes = a.c.k + page + from;
    constexpr int N = BYTES / 2048;
    uint2 c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = (i * 256 + tid) * 8;
      c[i] = from + x < to ? *reinterpret_cast<const uint2*>(codes + x) : make_uint2(0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = from + (i * 256 + tid) * 8;
      if (at >= to) break;
      const int row = __umulhi(at >> 3, by_dim), d = at - row * D, head = row >> log, t = row & (P - 1);
      if (t < lo || t >= hi) continue;
      const float scale = a.c.ks[sh.slot + head];
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = value_at(k < 4 ? c[i].x : c[i].y, k & 3, scale);
      put8<T, VEC>(static_cast<E*>(a.k) + (sh.token + t - lo) * a.k_t + head * a.k_h + d, v, a.stream);
    }
    return;
  }
  // Byte x of these rows lies at x + 4 (x / 8 P): rows that are eight apart, of
  // neighbouring lanes, then fall on different banks.
  const int8_t* codes = a.c.v + page + from;
  uint4 c[BYTES / 4096];
#pragma unroll
  for (int i = 0; i < BYTES / 4096; ++i) {
    const int x = (i * 256 + tid) * 16;
    if (from + x < to) c[i] = *reinterpret_cast<const uint4*>(codes + x);
  }
#pragma unroll
  for (int i = 0; i < BYTES / 4096; ++i) {
    const int x = (i * 256 + tid) * 16;
    if (from + x >= to) break;
    uint32_t* q = reinterpret_cast<uint32_t*>(s_codes + x + (x >> (log + 3)) * 4);
    q[0] = c[i].x;
    q[1] = c[i].y;
    q[2] = c[i].z;
    q[3] = c[i].w;
  }
  __syncthreads();
  constexpr int LOG = BYTES == 8192 ? 10 : 12;
  const int eights_log = LOG - log;  // groups of eight rows: BYTES / 8 P
  const int row0 = from >> log;      // (head, d)
#pragma unroll
  for (int i = 0; i < BYTES / 8192; ++i) {
    const int unit = i * 256 + tid;
    const int g = unit & ((1 << eights_log) - 1), t4 = (unit >> eights_log) * 4;
    const int row = row0 + 8 * g;
    if (row * P >= to || t4 + 4 <= lo || t4 >= hi) continue;
    const int head = __umulhi(row >> 3, by_dim), d = row - head * D;
    const float scale = a.c.vs[sh.slot + head];
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const uint32_t*>(s_codes + (8 * g + k) * P + g * 4 + t4);
    E* out = static_cast<E*>(a.v) + head * a.v_h + d;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t4 + t < lo || t4 + t >= hi) continue;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = value_at(w[k], t, scale);
      put8<T, VEC>(out + (sh.token + t4 + t - lo) * a.v_t, v, a.stream);
    }
  }
}

// Codes of a workgroup: 32 KB, where a page has them and that leaves eight
// workgroups a CU, so that more loads are in flight behind the chain sequence,
// page, scale (2 x 65536 tokens of 8 x 128 d in bf16: 8 KB 161 us, 32 KB 141).
static int read_bytes(const ReadArgs& a) {
  const int64_t row = static_cast<int64_t>(a.c.heads) * a.D;
  return row << a.c.page_log >= 32768 && 2 * (row * a.c.tokens >> 15) >= 2048 ? 32768 : 8192;
}
// Workgroups of a page.
static int page_blocks(const ReadArgs& a) {
  const int64_t bytes = (static_cast<int64_t>(a.c.heads) << a.c.page_log) * a.D, of = read_bytes(a);
  return static_cast<int>((bytes + of - 1) / of) * ((a.k != nullptr) + (a.v != nullptr));
}

int64_t read_workgroups(const ReadArgs& a) {
  return static_cast<int64_t>(page_blocks(a)) * (((a.c.max_new - 1) >> a.c.page_log) + 2);
}

template <int T, bool VEC>
static void go_read(const ReadArgs& a, hipStream_t s, Form& form) {
  const int blocks = page_blocks(a), bytes = read_bytes(a);
  // x / (D / 8) = x by_dim / 2^32 for x < 2^27 (a page has fewer eights: 2^22).
  const uint32_t D8 = a.D / 8, by_dim = static_cast<uint32_t>(((uint64_t(1) << 32) + D8 - 1) / D8);
  form = Form{VEC ? "read" : "read_any", {bytes, 1 << a.c.page_log}};
  const dim3 grid(static_cast<unsigned>(read_workgroups(a)), a.batch);
  if (bytes == 32768)
    cache_read_kernel<T, VEC, 32768><<<grid, 256, 0, s>>>(a, blocks, by_dim);
  else
    cache_read_kernel<T, VEC, 8192><<<grid, 256, 0, s>>>(a, blocks, by_dim);
}

template <int T>
static void pick_read(const ReadArgs& a, hipStream_t s, Form& form) {
  constexpr int per16 = 16 / sizeof(typename Elem<T>::type);
  const bool vec = (reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) % 16 == 0 &&
                   (a.k_t | a.k_h | a.v_t | a.v_h) % per16 == 0;
  if (vec)
    go_read<T, true>(a, s, form);
  else
    go_read<T, false>(a, s, form);
}

hipError_t launch_read(int dtype, const ReadArgs& args, hipStream_t s, Form& form) {
  ReadArgs a = args;
  a.stream = 2 * static_cast<int64_t>(a.c.tokens) * a.c.heads * a.D * elem_size(dtype) > kStreamBytes;
  if (dtype == EL_F32)
    pick_read<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    pick_read<EL_BF16>(a, s, form);
  else
    pick_read<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
