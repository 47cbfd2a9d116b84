// attention.hip -- attention of new queries over the paged 8-bit cache.
//
//   s_j = softmax_scale ks[page(j)] q . kcode_j     (visible j)
//   o   = sum_j 2^(s_j - m) vs[page(j)] vcode_j / sum_j 2^(s_j - m)
//
// with s in units of log2, m the running maximum of the row.  One pass over
// the keys: the maximum, the sum and the output are carried along and
// rescaled when the maximum grows.
//
// Matrix-core layout.  A wave works on 16 query rows (the new tokens of one
// sequence times the query heads of one cache head) and 64 keys at a time.
// It forms S^T = K Q^T in four 16x16 blocks with v_mfma_f32_16x16x32_f16:
// row m of block t is key 16 (m / 4) + 4 t + m % 4, so that lane l = 16 g + r
// ends up with the 16 consecutive keys 16 g .. 16 g + 15 of query row r --
// exactly the reduction slots its lane supplies to O^T = V^T P^T, which
// therefore needs no exchange between lanes.  In both products a lane's
// operand is 16 consecutive codes of the reduction (of d in a key row, of
// the keys in a transposed value page), one 16-byte load.  Pages hold
// multiples of 16 tokens, so a group of 16 keys has one page and one scale.
//
// Codes become fp16 exactly: the byte, its sign bit flipped, as the low
// mantissa byte of 1024 + u, minus 1152.
#include "ops_device.h"

namespace voc {

// Eight codes -> eight fp16 values.
__device__ __forceinline__ f16x8 codes_to_f16(uint32_t a, uint32_t b) {
  const f16x2 bias = {static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  union { f16x2 h[4]; f16x8 v; } u;
  u.h[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) - bias;
  u.h[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) - bias;
  u.h[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) - bias;
  u.h[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) - bias;
  return u.v;
}

// The probabilities enter the matrix cores as p * (page scale / largest page
// scale so far) * kLift: at most kLift, and far above fp16's subnormals.
constexpr float kLift = 4096.f;

constexpr int kTileRows = 16, kBlockKeys = 64;

// The share of one workgroup: rows r0 .. r0 + nrows - 1 of (sequence, cache
// head), keys of [lo, hi) in blocks of 64 from kb0.
struct Share {
  int r0, nrows, total, kb0, lo, hi;
};
__device__ __forceinline__ Share share_of(const AttendArgs& a, const Seq& s, int tile, int tile_rows) {
  Share h;
  const int rows = s.count * a.group;
  h.r0 = tile * tile_rows;
  h.nrows = min(tile_rows, rows - h.r0);
  const int64_t cap = a.c.stride << a.c.page_log;
  h.total = static_cast<int>(min(static_cast<int64_t>(s.past) + s.count, cap));
  h.lo = 0;
  h.hi = h.total;
  if (h.nrows > 0) {
    const int i_lo = h.r0 / a.group, i_hi = (h.r0 + h.nrows - 1) / a.group;
    if (a.window) h.lo = max(0, s.past + i_lo - a.window + 1);
    if (a.causal) h.hi = min(h.total, s.past + i_hi + 1);
  }
  h.kb0 = h.lo & ~(kBlockKeys - 1);
  return h;
}

// Workgroup: 16 rows, one part of the keys; its four waves take every fourth
// block of 64 keys and are joined in order at the end.  parts > 1: the
// results go to the workspace (unnormalised, with their maxima and sums) for
// join_kernel.
template <int T, int DC>
__global__ __launch_bounds__(256) void attend_kernel(const AttendArgs a, int tiles, int parts) {
  typedef typename Elem<T>::type E;
  constexpr int D = DC * 32, NC = DC / 2, REM = DC & 1;
  constexpr bool TWO = T == EL_F32;
  constexpr int NT = TWO ? 2 : 1;
  constexpr int PITCH = D + 4;
  __shared__ float s_o[kTileRows * PITCH];
  __shared__ float s_m[4][kTileRows], s_l[4][kTileRows];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  int id = blockIdx.x;
  const int part = id % parts;
  id /= parts;
  const int tile = id % tiles;
  const int head = id / tiles % a.c.heads, b = id / tiles / a.c.heads;
  const Seq sq = load_seq(a.c, b);
  const Share sh = share_of(a, sq, tile, kTileRows);
  if (sh.nrows <= 0) return;

  // This lane's query row.
  const int row = sh.r0 + min(lr, sh.nrows - 1);
  const int qi = row / a.group, qh = head * a.group + row % a.group;
  const int pos = sq.past + qi;
  const int row_hi = a.causal ? min(pos + 1, sh.total) : sh.total;
  const int row_lo = a.window ? max(0, pos - a.window + 1) : 0;
  const E* qp = static_cast<const E*>(a.q) + (sq.start + qi) * a.q_t + qh * a.q_h;
  f16x8 qf[NT][DC];
  float cq;
  {
    float v[DC][8];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      const int d = c < 2 * NC ? 64 * (c / 2) + 16 * lg + 8 * (c & 1) : 64 * NC + 8 * lg;
      load8<T>(qp + d, v[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[c][i]));
    }
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
    // The row times a power of two that brings its largest value to [2^14, 2^15).
    const uint32_t e = max(top >> 23, 15u);
    const float up = __uint_as_float((268u - e) << 23), down = __uint_as_float((e - 14u) << 23);
    cq = a.scale * down;
#pragma unroll
    for (int c = 0; c < DC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = v[c][i] * up;
        const _Float16 hi = static_cast<_Float16>(f);
        qf[0][c][i] = hi;
        if constexpr (TWO) qf[1][c][i] = static_cast<_Float16>(f - static_cast<float>(hi));
      }
  }

  f32x4 acc[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f, vref = 0.f;

  const int nblk = sh.hi > sh.lo ? (sh.hi - sh.kb0 + kBlockKeys - 1) / kBlockKeys : 0;
  const int per = (nblk + parts - 1) / parts;
  const int blk_end = min(nblk, (part + 1) * per);
  const int P = 1 << a.c.page_log;
  const int32_t* table = a.c.table + b * a.c.stride;
  // Every row of the tile sees all keys of [full_lo, full_hi).
  const int i_lo = sh.r0 / a.group, i_hi = (sh.r0 + sh.nrows - 1) / a.group;
  const int full_lo = a.window ? max(0, sq.past + i_hi - a.window + 1) : 0;
  const int full_hi = a.causal ? min(sq.past + i_lo + 1, sh.total) : sh.total;

  for (int blk = part * per + wave; blk < blk_end; blk += 4) {
    const int kb = sh.kb0 + blk * kBlockKeys;
    // Pages of the 16-key groups lr / 4 (keys) and lg (values, scales).
    const int gk = kb + 16 * (lr >> 2), gv = kb + 16 * lg;
    int pk = -1, pv = -1;
    if (gk < sh.hi) pk = table[gk >> a.c.page_log];
    if (gv < sh.hi) pv = table[gv >> a.c.page_log];
    const bool ok_k = pk >= 0 && pk < a.c.n_pages, ok_v = pv >= 0 && pv < a.c.n_pages;
    const int64_t slot_k = (ok_k ? static_cast<int64_t>(pk) : 0) * a.c.heads + head;
    const int64_t slot_v = (ok_v ? static_cast<int64_t>(pv) : 0) * a.c.heads + head;
    const int8_t* kp = a.c.k + (slot_k * P + (gk & (P - 1)) + (lr & 3)) * D;
    const int8_t* vp = a.c.v + (slot_v * D + lr) * P + (gv & (P - 1));
    const float ks = ok_v ? a.c.ks[slot_v] : 0.f;
    const float vs = ok_v ? a.c.vs[slot_v] : 0.f;

    f32x4 st[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 u = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 64 * c + 16 * lg);
        const f16x8 k0 = codes_to_f16(u.x, u.y), k1 = codes_to_f16(u.z, u.w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * c], st[t], 0, 0, 0);
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][2 * c + 1], st[t], 0, 0, 0);
        }
      }
      if constexpr (REM) {
        const uint2 u = *reinterpret_cast<const uint2*>(kp + 4 * t * D + 64 * NC + 8 * lg);
        const f16x8 k0 = codes_to_f16(u.x, u.y);
#pragma unroll
        for (int n = 0; n < NT; ++n) st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * NC], st[t], 0, 0, 0);
      }
    }

    const float sc = ks * cq;
    float s[16], top = -INFINITY;
    uint32_t seen = 0xffffu;
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = st[j >> 2][j & 3] * sc;
    if (!(kb >= full_lo && kb + kBlockKeys <= full_hi && __all(ok_v))) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int key = gv + j;
        const bool in = ok_v && key >= row_lo && key < row_hi;
        if (!in) seen &= ~(1u << j);
        s[j] = in ? s[j] : -INFINITY;
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, s[j]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m_new = fmaxf(m, top), m_use = m_new == -INFINITY ? 0.f : m_new;
    float vtop = fmaxf(vs, __shfl_xor(vs, 16));
    vtop = fmaxf(vtop, __shfl_xor(vtop, 32));
    const float vref_new = fmaxf(vref, vtop);
    const float vinv = vref_new > 0.f ? kLift / vref_new : 0.f;
    const float alpha = __builtin_amdgcn_exp2f(m - m_use);
    const float beta = vref_new > 0.f ? alpha * (vref / vref_new) : alpha;
    const float vf = vs * vinv;
    l *= alpha;
    f16x8 pf[NT][2];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float p = __builtin_amdgcn_exp2f(s[j] - m_use);
      l += p;
      const float w = (seen >> j) & 1u ? p * vf : 0.f;
      const _Float16 hi = static_cast<_Float16>(w);
      pf[0][j >> 3][j & 7] = hi;
      if constexpr (TWO) pf[1][j >> 3][j & 7] = static_cast<_Float16>(w - static_cast<float>(hi));
    }
    m = m_new;
    vref = vref_new;
    if (!__all(beta == 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i] *= beta;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(vp + static_cast<int64_t>(16 * i) * P);
      const f16x8 v0 = codes_to_f16(u.x, u.y), v1 = codes_to_f16(u.z, u.w);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[n][0], acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[n][1], acc[i], 0, 0, 0);
      }
    }
  }

  // Join the four waves.  (m is -inf where a wave saw no key; a NaN sum stays
  // NaN whatever its factor.)
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lg == 0) {
    s_m[wave][lr] = m;
    s_l[wave][lr] = l;
  }
  __syncthreads();
  const float mj = fmaxf(fmaxf(s_m[0][lr], s_m[1][lr]), fmaxf(s_m[2][lr], s_m[3][lr]));
  const float m_use = mj == -INFINITY ? 0.f : mj;
  const float f = __builtin_amdgcn_exp2f(m - m_use) * (vref / kLift);
  for (int w = 0; w < 4; ++w) {
    if (w == wave && lr < sh.nrows) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        float* p = s_o + lr * PITCH + 16 * i + 4 * lg;
        const f32x4 v = acc[i] * f;
        *reinterpret_cast<f32x4*>(p) = w ? *reinterpret_cast<f32x4*>(p) + v : v;
      }
    }
    __syncthreads();
  }
  for (int k = tid; k < sh.nrows * D; k += 256) {
    const int r = k / D, d = k - r * D;
    float mm = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
    const float mu = mm == -INFINITY ? 0.f : mm;
    float lt = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) lt += s_l[w][r] * __builtin_amdgcn_exp2f(s_m[w][r] - mu);
    const float v = s_o[r * PITCH + d];
    if (parts == 1) {
      const int rr = sh.r0 + r;
      E* o = static_cast<E*>(a.o) + (sq.start + rr / a.group) * a.o_t + (head * a.group + rr % a.group) * a.o_h;
      o[d] = static_cast<E>(lt == 0.f ? 0.f : v / lt);
    } else {
      float* ws = static_cast<float*>(a.ws) + static_cast<int64_t>(blockIdx.x) * kTileRows * (D + 2);
      ws[r * D + d] = v;
      if (d == 0) {
        ws[kTileRows * D + r] = mm;
        ws[kTileRows * D + kTileRows + r] = lt;
      }
    }
  }
}

// Joins the parts of each tile of 16 rows, in order.
template <int T>
__global__ __launch_bounds__(256) void join_kernel(const AttendArgs a, int tiles, int parts) {
  typedef typename Elem<T>::type E;
  const int D = a.D;
  const int id = blockIdx.x;
  const int tile = id % tiles, head = id / tiles % a.c.heads, b = id / tiles / a.c.heads;
  const Seq sq = load_seq(a.c, b);
  const int r0 = tile * kTileRows, nrows = min(kTileRows, sq.count * a.group - r0);
  const int64_t size = kTileRows * (D + 2);
  const float* ws = static_cast<const float*>(a.ws) + static_cast<int64_t>(id) * parts * size;
  for (int k = threadIdx.x; k < nrows * D; k += 256) {
    const int r = k / D, d = k - r * D;
    float m = -INFINITY;
    for (int p = 0; p < parts; ++p) m = fmaxf(m, ws[p * size + kTileRows * D + r]);
    m = m == -INFINITY ? 0.f : m;
    float l = 0.f, v = 0.f;
    for (int p = 0; p < parts; ++p) {
      const float f = __builtin_amdgcn_exp2f(ws[p * size + kTileRows * D + r] - m);
      l += f * ws[p * size + kTileRows * D + kTileRows + r];
      v += f * ws[p * size + r * D + d];
    }
    const int rr = r0 + r;
    E* o = static_cast<E*>(a.o) + (sq.start + rr / a.group) * a.o_t + (head * a.group + rr % a.group) * a.o_h;
    o[d] = static_cast<E>(l == 0.f ? 0.f : v / l);
  }
}

template <int T>
static void go_attend(const AttendArgs& a, hipStream_t s) {
  const int tiles = static_cast<int>((static_cast<int64_t>(a.c.max_new) * a.group + kTileRows - 1) / kTileRows);
  const int64_t wgs = static_cast<int64_t>(a.batch) * a.c.heads * tiles;
  const int64_t part_bytes = static_cast<int64_t>(kTileRows) * (a.D + 2) * 4;
  int64_t parts = 1024 / wgs;
  parts = parts < (a.max_total + 255) / 256 ? parts : (a.max_total + 255) / 256;
  const int64_t room = static_cast<int64_t>(a.ws_bytes) / (part_bytes * wgs);
  parts = parts < room ? parts : room;
  if (parts < 1) parts = 1;
  const dim3 grid(static_cast<unsigned>(wgs * parts));
  const int np = static_cast<int>(parts);
  switch (a.D / 32) {
    case 1: attend_kernel<T, 1><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 2: attend_kernel<T, 2><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 3: attend_kernel<T, 3><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 4: attend_kernel<T, 4><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 5: attend_kernel<T, 5><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 6: attend_kernel<T, 6><<<grid, 256, 0, s>>>(a, tiles, np); break;
    case 7: attend_kernel<T, 7><<<grid, 256, 0, s>>>(a, tiles, np); break;
    default: attend_kernel<T, 8><<<grid, 256, 0, s>>>(a, tiles, np); break;
  }
  if (np > 1) join_kernel<T><<<dim3(static_cast<unsigned>(wgs)), 256, 0, s>>>(a, tiles, np);
}

hipError_t launch_attend(int dtype, const AttendArgs& a, hipStream_t s) {
  if (dtype == EL_F32)
    go_attend<EL_F32>(a, s);
  else if (dtype == EL_BF16)
    go_attend<EL_BF16>(a, s);
  else
    go_attend<EL_F16>(a, s);
  return hipGetLastError();
}

}  // namespace voc
