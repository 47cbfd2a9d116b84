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
#include "gemm_common.h"
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

// The probabilities enter the matrix cores with their value scales, as
// p * vs * lift with p = 2^(s - m) and lift a power of two that brings the
// row's largest p * vs to [2^10, 2^11): what weighs most in the output then
// uses all of an fp16 number, whatever the scales (up to 2^100 apart) of pages
// that weigh little.
// fp16 reaches 2^-25 below (half its last step), so a key's term is off by at
// most 2^-35 of the row's largest besides its own rounding.  m follows a score
// that passes it by more than kSlack (a factor of 8), lift a product past
// kHigh, which fp16 still holds.  A product that high needs vs * lift past
// kLook, so that a block of keys usually costs two comparisons (two prompts of
// 5168, 32 / 8 heads x 128 d: 438 us; 457 with the product in the test).
constexpr float kSlack = 3.f, kHigh = 32768.f, kLook = 4096.f;

constexpr int kBlockKeys = 64;

// The share of one workgroup: rows r0 .. r0 + nrows - 1 of (sequence, cache
// head), keys of [lo, hi) in blocks of 64 from kb0.
struct Share {
  int r0, nrows, total, kb0, lo, hi, blk0, blk1;
};
__device__ __forceinline__ Share share_of(const AttendArgs& a, const Seq& s, int tile, int tile_rows, int part, int parts) {
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
  h.kb0 = h.lo & ~15;
  const int nblk = h.hi > h.lo ? (h.hi - h.kb0 + kBlockKeys - 1) / kBlockKeys : 0;
  const int per = (nblk + parts - 1) / parts;
  h.blk0 = min(nblk, part * per);
  h.blk1 = min(nblk, h.blk0 + per);
  return h;
}

// The keys [lo, hi) that query row r of a share sees.
struct Sight {
  int lo, hi;
};
__device__ __forceinline__ Sight sight_of(const AttendArgs& a, const Seq& s, int total, int row) {
  const int pos = s.past + row / a.group;
  return Sight{a.window ? max(0, pos - a.window + 1) : 0, a.causal ? min(pos + 1, total) : total};
}

// One query row as matrix-core operands: the row times a power of two that
// brings its largest value to [2^14, 2^15), in NT fp16 terms.  Returns the
// factor of its scores.  DOF(c): this lane's first d of fragment c.
template <int T, int DC, int NT, typename FD>
__device__ __forceinline__ float load_query(const typename Elem<T>::type* qp, float scale, f16x8 (&qf)[NT][DC], FD dof) {
  float v[DC][8];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < DC; ++c) {
    load8<T>(qp + dof(c), v[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[c][i]));
  }
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
  const uint32_t e = max(top >> 23, 15u);
  // A negative softmax scale goes into the query: the factor stays positive.
  const float up = copysignf(__uint_as_float((268u - e) << 23), scale), down = __uint_as_float((e - 14u) << 23);
#pragma unroll
  for (int c = 0; c < DC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = v[c][i] * up;
      const _Float16 hi = static_cast<_Float16>(f);
      qf[0][c][i] = hi;
      if constexpr (NT > 1) qf[1][c][i] = static_cast<_Float16>(f - static_cast<float>(hi));
    }
  return fabsf(scale) * down;
}

// What a wave carries along for 16 query rows (a lane: row lr, the sum over
// its own keys only).  ref is the largest p * vs when lift was last set.
struct RowState {
  float m = -INFINITY, l = 0.f, ref = 0.f, lift = 1.f;
};

// Scores stay products st * sc up to the exponential, which takes their exact
// difference from m, a rounded one: 2^-25 of a score, which is small beside
// kSlack up to scores of 2^20 (of 2^30 it makes zeros and infinities).  The
// sums are below 2^22 D, so that a block whose factors pass this limit goes
// through hide(), which rounds them.
__device__ __forceinline__ bool small_scores(float sc, int D) { return sc <= 0x1p-2f / static_cast<float>(D); }

// Hides what a row does not see: this lane's keys key0 .. key0 + 15 count
// where `in` and inside the row's sight.  Scores become final (their factor
// sc 1) with -inf in hidden places, and the scale of values of which the row
// sees none becomes 0, so that a hidden page's NaN scale stays out.
__device__ __forceinline__ void hide(f32x4 (&st)[4], float& sc, float& vs, bool in, int key0, const Sight& see) {
  bool any = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const bool s = in && key0 + j >= see.lo && key0 + j < see.hi;
    any |= s;
    st[j >> 2][j & 3] = s ? st[j >> 2][j & 3] * sc : -INFINITY;
  }
  sc = 1.f;
  vs = any ? vs : 0.f;
}

// Rescales what was summed when the scores of 16 more keys (this lane's, of
// one page group: st times sc, value scale vs) make m or lift move.  Returns
// vs * lift.
template <int NA>
__device__ __forceinline__ float follow_maximum(const f32x4 (&st)[4], float sc, float vs, RowState& r, f32x4 (&acc)[NA]) {
  float top = st[0][0];
#pragma unroll
  for (int j = 1; j < 16; ++j) top = fmaxf(top, st[j >> 2][j & 3]);
  top *= sc;
  float vf = vs * r.lift;
  if (__any(top > r.m + kSlack || vf > kLook)) {
    // (Where m is -inf the first test decides: the second has an infinity or a
    // NaN on its left.)
    if (__any(top > r.m + kSlack || __builtin_amdgcn_exp2f(top - r.m) * vf > kHigh)) {
      float t = fmaxf(top, __shfl_xor(top, 16));
      t = fmaxf(t, __shfl_xor(t, 32));
      const float m = t > r.m + kSlack ? t : r.m;
      const float alpha = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(r.m - m);
      float w = __builtin_amdgcn_exp2f(top - (m == -INFINITY ? 0.f : m)) * vs;
      w = fmaxf(w, __shfl_xor(w, 16));
      w = fmaxf(w, __shfl_xor(w, 32));
      // At least 2^-112: lift and its inverse stay normal numbers.
      const float ref = fmaxf(fmaxf(r.ref * alpha, w), 0x1p-112f);
      const float lift = __uint_as_float((264u - (__float_as_uint(ref) >> 23)) << 23);
      // alpha * lift / r.lift (their quotient alone may pass fp32's range).
      const float beta = __builtin_amdgcn_ldexpf(
          alpha, static_cast<int>(__float_as_uint(lift) >> 23) - static_cast<int>(__float_as_uint(r.lift) >> 23));
      r.m = m;
      r.ref = ref;
      r.lift = lift;
      r.l *= alpha;
#pragma unroll
      for (int i = 0; i < NA; ++i) acc[i] *= beta;
    }
    // Past 2^126 p is below 2^-111; an infinity would make NaN of p = 0.  (A
    // NaN scale stays.)
    vf = vs * r.lift;
    vf = vf > 0x1p126f ? 0x1p126f : vf;
  }
  return vf;
}

// The probabilities of those keys as operands of the second product, in NP fp16
// terms.  Two hold about 22 bits; one rounds each to 11, which against 64 bits
// costs (RMS of the output's, one term / two / the output's own rounding alone)
// fp16 2.85e-4 / 2.07e-4 / 2.07e-4, bf16 1.67e-3 / 1.66e-3 / 1.66e-3; of the
// outputs 38 % / 0.1 % (fp16) and 9 % / 0.02 % are not the nearest value.  Hence
// two where rows are few, which wait for memory (us, one / two, bf16: 4 x 65536 keys
// of 8 x 128 d 89.5 / 90.4, 32 x 2000 30.6 / 31.2, 32 x 25 rows of window 72
// 10.3 / 10.5), and for fp32; one for 16 bits where rows are many (2 prompts of
// 5168 440 / 567, 32 of 250 x 16 x 64 30.4 / 33.9, 2 x 2000 x 16 x 256 112 / 132).
template <int NP>
__device__ __forceinline__ void probabilities(const f32x4 (&st)[4], float sc, float vf, RowState& r, f16x8 (&pf)[NP][2]) {
  // A row that has seen nothing yet has only -inf here: any finite m will do.
  const float neg = r.m == -INFINITY ? 0.f : -r.m;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float p = __builtin_amdgcn_exp2f(fmaf(st[j >> 2][j & 3], sc, neg));
    sum[j & 3] += p;
    float w = p * vf;
    // Both terms start from the rounded product: the compiler would otherwise
    // take the first from the exact one (a fused multiply and conversion) for
    // one of its two uses, and near a tie the second term would belong to
    // another first one (seen: 2^-10 of a probability).
    if constexpr (NP > 1) asm volatile("" : "+v"(w));
    const _Float16 hi = static_cast<_Float16>(w);
    pf[0][j >> 3][j & 7] = hi;
    if constexpr (NP > 1) pf[1][j >> 3][j & 7] = static_cast<_Float16>(w - static_cast<float>(hi));
  }
  r.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Few query rows.  Workgroup: 16 rows, one part of the keys; its four waves
// take every fourth block of 64 keys, operands straight from memory, and are
// joined in order at the end.  parts > 1: the results go to the workspace
// (unnormalised, with their maxima and sums) for join_kernel.  (A join by the
// workgroup that ends last saves a launch and costs what the launch does: its
// reads and writes have to go past eight L2s.  1 x 8000 keys of 8 x 128 d:
// 14.3 us for 7.9 + 5.2; with a write-back of the L2 19.2.)
// Every key and value is read once, from memory to registers, so a long cache
// is bound by memory: one token of 4 x 32 / 8 heads x 128 d over 65536 tokens,
// 409 MB, 76 us (5.4 TB/s) and 5 for the join.  Short ones are bound by latency
// (sequence, page, codes, joins): 32 x 16 x 64 over 250 tokens 8.4 us; 25 rows
// each over a window of 72 10.9.
constexpr int kFewRows = 16;
constexpr int few_waves(int t, int dc) { return t == EL_F32 ? (dc <= 2 ? 3 : dc <= 4 ? 2 : 1) : dc <= 2 ? 4 : dc <= 4 ? 3 : dc <= 6 ? 2 : 1; }

template <int T, int DC>
__global__ __launch_bounds__(256, few_waves(T, DC)) void attend_few_kernel(const AttendArgs a, int tiles, int parts) {
  typedef typename Elem<T>::type E;
  constexpr int D = DC * 32, NC = DC / 2, REM = DC & 1;
  constexpr int NT = T == EL_F32 ? 2 : 1, NP = 2;
  constexpr int PITCH = D + 4;
  __shared__ float s_o[kFewRows * PITCH];
  __shared__ float s_m[4][kFewRows], s_l[4][kFewRows];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  int id = blockIdx.x;
  const int part = id % parts;
  id /= parts;
  const int tile = id % tiles;
  const int head = id / tiles % a.c.heads, b = id / tiles / a.c.heads;
  const Seq sq = load_seq(a.c, b);
  const Share sh = share_of(a, sq, tile, kFewRows, part, parts);
  if (sh.nrows <= 0) return;

  // This lane's query row (past the last one: the last one again).  A lane's
  // operands are 16 consecutive d of 64, then 8 of the last 32.
  const int row = sh.r0 + min(lr, sh.nrows - 1);
  const Sight see = sight_of(a, sq, sh.total, row);
  f16x8 qf[NT][DC];
  const float cq = load_query<T, DC, NT>(
      static_cast<const E*>(a.q) + (sq.start + row / a.group) * a.q_t + (head * a.group + row % a.group) * a.q_h, a.scale,
      qf, [&](int c) { return c < 2 * NC ? 64 * (c / 2) + 16 * lg + 8 * (c & 1) : 64 * NC + 8 * lg; });

  f32x4 acc[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  RowState rs;

  const int P = 1 << a.c.page_log;
  const int32_t* table = a.c.table + b * a.c.stride;
  // Every row of the tile sees all keys of [full_lo, full_hi).
  const int full_lo = sight_of(a, sq, sh.total, sh.r0 + sh.nrows - 1).lo;
  const int full_hi = sight_of(a, sq, sh.total, sh.r0).hi;

  for (int blk = sh.blk0 + wave; blk < sh.blk1; blk += 4) {
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
    // The whole block's loads first: keys, scales, then the values that are
    // needed last.
    uint4 kc[4][NC ? NC : 1];
    uint2 kr[4];
    uint4 vc[D / 16];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int c = 0; c < NC; ++c) kc[t][c] = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 64 * c + 16 * lg);
      if constexpr (REM) kr[t] = *reinterpret_cast<const uint2*>(kp + 4 * t * D + 64 * NC + 8 * lg);
    }
    const float ks = ok_v ? a.c.ks[slot_v] : 0.f;
    const float vs = ok_v ? a.c.vs[slot_v] : 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) vc[i] = *reinterpret_cast<const uint4*>(vp + static_cast<int64_t>(16 * i) * P);

    f32x4 st[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const f16x8 k0 = codes_to_f16(kc[t][c].x, kc[t][c].y), k1 = codes_to_f16(kc[t][c].z, kc[t][c].w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * c], st[t], 0, 0, 0);
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][2 * c + 1], st[t], 0, 0, 0);
        }
      }
      if constexpr (REM) {
        const f16x8 k0 = codes_to_f16(kr[t].x, kr[t].y);
#pragma unroll
        for (int n = 0; n < NT; ++n) st[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * NC], st[t], 0, 0, 0);
      }
    }
    f16x8 pf[NP][2];
    float sc = ks * cq, vsc = vs;
    if (!(kb >= full_lo && kb + kBlockKeys <= full_hi && __all(ok_v && small_scores(sc, D)))) hide(st, sc, vsc, ok_v, gv, see);
    const float vf = follow_maximum(st, sc, vsc, rs, acc);
    probabilities<NP>(st, sc, vf, rs, pf);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const f16x8 v0 = codes_to_f16(vc[i].x, vc[i].y), v1 = codes_to_f16(vc[i].z, vc[i].w);
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[n][0], acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[n][1], acc[i], 0, 0, 0);
      }
    }
  }

  // Join the four waves.  (m is -inf where a wave saw no key; a NaN sum stays
  // NaN whatever its factor.)
  float l = rs.l;
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lg == 0) {
    s_m[wave][lr] = rs.m;
    s_l[wave][lr] = l;
  }
  __syncthreads();
  const float mj = fmaxf(fmaxf(s_m[0][lr], s_m[1][lr]), fmaxf(s_m[2][lr], s_m[3][lr]));
  const float m_use = mj == -INFINITY ? 0.f : mj;
  const float f = __builtin_amdgcn_exp2f(rs.m - m_use) * (1.f / rs.lift);
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
    const float mm = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
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
      float* ws = static_cast<float*>(a.ws) + static_cast<int64_t>(blockIdx.x) * kFewRows * (D + 2);
      ws[r * D + d] = v;
      if (d == 0) {
        ws[kFewRows * D + r] = mm;
        ws[kFewRows * D + kFewRows + r] = lt;
      }
    }
  }
}

// Keeps DEPTH operand fragments (one LDS read each) on their way ahead of the
// matrix-core instructions that use them, PER to a fragment, N fragments in
// all.  (Left alone, the compiler waits for every read right after it.)
template <int N, int DEPTH, int PER>
__device__ __forceinline__ void read_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, DEPTH, 0);
#pragma unroll
  for (int q = 0; q < N; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    if (q + DEPTH < N) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
}

// Many query rows.  Workgroup: 8 waves of RT tiles of 16 rows (one above 128 d
// and for fp32 queries: four waves of two tiles keep a SIMD to one wave, us, as
// chosen / that: 2 x 2000 x 16 heads of 256 d, bf16 118 / 207, of 128 d, fp32
// 111 / 144; eight waves of two tiles spill there).  Blocks of 64 keys and values are brought to LDS as
// fp16 once for all waves, two buffers in turn: while one is worked on, the
// next block's codes are on their way into registers and are converted at
// the end of the step.  Page numbers run two blocks ahead, scales one
// (threads 0 .. 3, one to a group of 16 keys), so that no step waits for a
// chain of loads.
// LDS holds the operands fragment by fragment, 1 KB each, in the order in
// which the lanes read them; key fragment (t, c): keys 16 g + 4 t + i at row
// 4 g + i, d 32 c .., value fragment (i, h): d 16 i .., keys 16 g + 8 h ...
// A wave's copies take 64 bytes of each of 16 rows, which spreads its writes
// over all banks.
// Two prompts of 5168, 32 / 8 heads x 128 d, causal (386 G operations): 455 us,
// 0.85 P operations a second (539 in a profiled run); a large fp16 library
// product reaches 1.32.  The matrix cores are busy 38 % of the cycles
// and the vector units about half (146 instructions for 1024 scores of a wave,
// conversion included): a SIMD's two waves seldom do the one while the other
// does the other.  fp32 queries, with two terms in both products, take 832.
// Not kept, of an earlier form: scores a block ahead of the products 710 (630
// then), two groups of waves a phase apart 523 to 677 (499), wave priorities
// 553 to 581, the value scale inside the exponent 553 (550), 64 rows a wave
// 1269 (spills).
constexpr int kManyWaves = 8;
constexpr int many_rt(int t, int dc) { return t == EL_F32 || dc > 4 ? 1 : 2; }

template <int T, int DC>
__global__ __launch_bounds__(64 * kManyWaves) void attend_many_kernel(const AttendArgs a, int tiles, int parts) {
  typedef typename Elem<T>::type E;
  constexpr int D = DC * 32;
  constexpr int NT = T == EL_F32 ? 2 : 1, NP = NT;
  constexpr int RT = many_rt(T, DC), NW = kManyWaves, ROWS = NW * 16 * RT;
  constexpr int TILE = kBlockKeys * D * 2;                         // bytes of a key or value tile
  constexpr int CK = ((D + 63) / 64 + NW / 4 - 1) / (NW / 4);      // 16-code units of a key tile per thread
  constexpr int CV = (D / 16 + NW - 1) / NW;                       // and of a value tile
  __shared__ __attribute__((aligned(16))) unsigned char s_k[2 * TILE], s_v[2 * TILE];
  __shared__ int64_t s_koff[4][4], s_voff[4][4];  // byte offsets of a block's groups; -1: no tokens
  __shared__ float s_ks[4][4], s_vs[4][4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  // An XCD takes a contiguous range: whole (head, sequence) pairs share their
  // keys and values in its L2, and sequences of different lengths meet on
  // every XCD.  The longest causal rows come first.
  int id = xcd_remap(blockIdx.x, gridDim.x);
  const int part = id % parts;
  id /= parts;
  const int tile = tiles - 1 - id % tiles;
  const int b = id / tiles % a.batch, head = id / tiles / a.batch;
  const Seq sq = load_seq(a.c, b);
  const Share sh = share_of(a, sq, tile, ROWS, part, parts);
  if (sh.nrows <= 0) return;

  f16x8 qf[RT][NT][DC];
  float cq[RT];
  Sight see[RT];
  RowState rs[RT];
  f32x4 acc[RT][D / 16];
  const int w0 = wave * 16 * RT;                                   // the wave's first row
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = sh.r0 + min(w0 + 16 * r + lr, sh.nrows - 1);
    see[r] = sight_of(a, sq, sh.total, row);
    cq[r] = load_query<T, DC, NT>(
        static_cast<const E*>(a.q) + (sq.start + row / a.group) * a.q_t + (head * a.group + row % a.group) * a.q_h,
        a.scale, qf[r], [&](int c) { return 32 * c + 8 * lg; });
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int P = 1 << a.c.page_log;
  const int32_t* table = a.c.table + b * a.c.stride;
  const int nblk = sh.blk1 - sh.blk0;
  const int kb0 = sh.kb0 + sh.blk0 * kBlockKeys;
  // Blocks [na, nb) are seen by some row of the wave; every row of it sees
  // all keys of [last.lo, first.hi).
  const Sight first = sight_of(a, sq, sh.total, sh.r0 + min(w0, sh.nrows - 1));
  const Sight last = sight_of(a, sq, sh.total, sh.r0 + min(w0 + 16 * RT - 1, sh.nrows - 1));
  const int na = max(0, first.lo - kb0) / kBlockKeys;
  const int nb = w0 < sh.nrows ? min(nblk, (max(0, last.hi - kb0) + kBlockKeys - 1) / kBlockKeys) : 0;

  // Threads 0 .. 3: page number, then offsets and scales, of group tid of block n.
  auto page_of = [&](int n) {
    const int key = kb0 + n * kBlockKeys + 16 * tid;
    return n < nblk && key < sh.hi ? table[key >> a.c.page_log] : -1;
  };
  auto place = [&](int n, int page) {
    const bool ok = page >= 0 && page < a.c.n_pages;
    const int64_t slot = ok ? static_cast<int64_t>(page) * a.c.heads + head : 0;
    const int64_t at = (slot * D) << a.c.page_log;
    const int token = (kb0 + n * kBlockKeys + 16 * tid) & (P - 1);
    s_koff[n & 3][tid] = ok ? at + token * D : -1;
    s_voff[n & 3][tid] = ok ? at + token : -1;
    return ok ? slot : int64_t(-1);
  };
  // This thread's units: keys 16 g + 4 (wave % 4) + i (g = lane / 4 % 4, i = lane % 4)
  // and d 64 dq + 16 (lane / 16), dq = wave / 4 + NW / 4 u; values d 16 (wave + NW u) + lane % 16,
  // keys 16 (lane / 16).
  const int kg = (lane >> 2) & 3, dq0 = wave >> 2;
  const int kin = (4 * (wave & 3) + (lane & 3)) * D + 64 * dq0 + 16 * lg;
  const int vin = (16 * wave + lr) << a.c.page_log;
  uint4 ck[CK], cv[CV];
  auto has_k = [&](int u) { return D % (16 * NW) == 0 || 64 * (dq0 + NW / 4 * u) + 16 * lg < D; };
  auto has_v = [&](int u) { return D % (16 * NW) == 0 || 16 * (wave + NW * u) < D; };
  auto fetch_k = [&](int n) {
    const int8_t* p = a.c.k + max(s_koff[n & 3][kg], int64_t(0)) + kin;
#pragma unroll
    for (int u = 0; u < CK; ++u)
      if (has_k(u)) ck[u] = *reinterpret_cast<const uint4*>(p + 16 * NW * u);
  };
  auto fetch_v = [&](int n) {
    const int8_t* p = a.c.v + max(s_voff[n & 3][lg], int64_t(0)) + vin;
#pragma unroll
    for (int u = 0; u < CV; ++u)
      if (has_v(u)) cv[u] = *reinterpret_cast<const uint4*>(p + (static_cast<int64_t>(16 * NW * u) << a.c.page_log));
  };
  auto store_k = [&](int n) {
    unsigned char* p = s_k + (n & 1) * TILE + ((wave & 3) * DC + 2 * dq0 + (lg >> 1)) * 1024 + (lg & 1) * 512 + lr * 16;
#pragma unroll
    for (int u = 0; u < CK; ++u)
      if (has_k(u)) {
        *reinterpret_cast<f16x8*>(p + 512 * NW * u) = codes_to_f16(ck[u].x, ck[u].y);
        *reinterpret_cast<f16x8*>(p + 512 * NW * u + 256) = codes_to_f16(ck[u].z, ck[u].w);
      }
  };
  auto store_v = [&](int n) {
    unsigned char* p = s_v + (n & 1) * TILE + wave * 2048 + lane * 16;
#pragma unroll
    for (int u = 0; u < CV; ++u)
      if (has_v(u)) {
        *reinterpret_cast<f16x8*>(p + 2048 * NW * u) = codes_to_f16(cv[u].x, cv[u].y);
        *reinterpret_cast<f16x8*>(p + 2048 * NW * u + 1024) = codes_to_f16(cv[u].z, cv[u].w);
      }
  };
  auto scores = [&](int n, f32x4 (&st)[RT][4]) {
    const unsigned char* kt = s_k + (n & 1) * TILE + lane * 16;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) st[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (Products into the same accumulator are kept apart, here and below.)
#pragma unroll
    for (int c = 0; c < DC; ++c) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f16x8 k = *reinterpret_cast<const f16x8*>(kt + (t * DC + c) * 1024);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int x = 0; x < NT; ++x) st[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qf[r][x][c], st[r][t], 0, 0, 0);
      }
    }
  };

  int page3 = -1;                    // page number of block n + 3
  float ks1 = 0.f, vs1 = 0.f;        // scales of block n + 1
  int64_t slot2 = -1;                // slot of block n + 2
  if (tid < 4) {
    const int64_t s0 = place(0, page_of(0)), s1 = place(1, page_of(1));
    slot2 = place(2, page_of(2));
    page3 = page_of(3);
    s_ks[0][tid] = s0 >= 0 ? a.c.ks[s0] : 0.f;
    s_vs[0][tid] = s0 >= 0 ? a.c.vs[s0] : 0.f;
    ks1 = s1 >= 0 ? a.c.ks[s1] : 0.f;
    vs1 = s1 >= 0 ? a.c.vs[s1] : 0.f;
  }
  __syncthreads();
  if (nblk > 0) {
    fetch_k(0);
    fetch_v(0);
    store_k(0);
    store_v(0);
  }
  __syncthreads();

  for (int n = 0; n < nblk; ++n) {
    if (n + 1 < nblk) {
      fetch_k(n + 1);
      fetch_v(n + 1);
    }
    if (tid < 4) {
      s_ks[(n + 1) & 3][tid] = ks1;
      s_vs[(n + 1) & 3][tid] = vs1;
      ks1 = slot2 >= 0 ? a.c.ks[slot2] : 0.f;
      vs1 = slot2 >= 0 ? a.c.vs[slot2] : 0.f;
      slot2 = place(n + 3, page3);
      page3 = page_of(n + 4);
    }
    if (n >= na && n < nb) {
      const int kb = kb0 + n * kBlockKeys;
      f32x4 st[RT][4];
      scores(n, st);
      read_ahead<4 * DC, 4, RT * NT>();
      const bool in = s_koff[n & 3][lg] >= 0;
      const float ks = s_ks[n & 3][lg], vs = s_vs[n & 3][lg];
      float sc[RT], vsc[RT];
      bool plain = in;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        sc[r] = ks * cq[r];
        vsc[r] = vs;
        plain = plain && small_scores(sc[r], D);
      }
      if (!(kb >= last.lo && kb + kBlockKeys <= first.hi && __all(plain))) {
#pragma unroll
        for (int r = 0; r < RT; ++r) hide(st[r], sc[r], vsc[r], in, kb + 16 * lg, see[r]);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) vsc[r] = follow_maximum(st[r], sc[r], vsc[r], rs[r], acc[r]);
      f16x8 pf[RT][NP][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) probabilities<NP>(st[r], sc[r], vsc[r], rs[r], pf[r]);
      const unsigned char* vt = s_v + (n & 1) * TILE + lane * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const f16x8 v = *reinterpret_cast<const f16x8*>(vt + (2 * i + h) * 1024);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int x = 0; x < NP; ++x) acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pf[r][x][h], acc[r][i], 0, 0, 0);
        }
      read_ahead<D / 8, 4, RT * NP>();
    }
    if (n + 1 < nblk) {
      store_k(n + 1);
      store_v(n + 1);
    }
    __syncthreads();
  }

#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float l = rs[r].l;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const int k = w0 + 16 * r + lr;
    if (k >= sh.nrows) continue;
    const float lift = 1.f / rs[r].lift;
    if (parts == 1) {
      const int rr = sh.r0 + k;
      E* o = static_cast<E*>(a.o) + (sq.start + rr / a.group) * a.o_t + (head * a.group + rr % a.group) * a.o_h;
      const float f = l == 0.f ? 0.f : lift / l;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        E e[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = static_cast<E>(l == 0.f ? 0.f : acc[r][i][q] * f);
        __builtin_memcpy(__builtin_assume_aligned(o + 16 * i + 4 * lg, 4 * sizeof(E)), e, 4 * sizeof(E));
      }
    } else {
      // The workgroup's place in the workspace goes by its share, not its number.
      const int64_t at = ((static_cast<int64_t>(b) * a.c.heads + head) * tiles + tile) * parts + part;
      float* ws = static_cast<float*>(a.ws) + at * ROWS * (D + 2);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f32x4*>(ws + k * D + 16 * i + 4 * lg) = acc[r][i] * lift;
      if (lg == 0) {
        ws[ROWS * D + k] = rs[r].m;
        ws[ROWS * D + ROWS + k] = l;
      }
    }
  }
}

// Joins the parts of the tiles.  Workgroup: one row (of the first `live` rows
// of a tile).  The factors of all parts first, then four d a thread, the parts
// split over the threads that are left; every order of summation follows from
// the sizes alone.  Bound by the latency of three dependent steps: 256 parts of
// 16 rows x 64 d take 5.6 us (16.5 when a row's threads go over all the parts),
// 24 parts of 32 x 4 rows x 128 d 5.3.
constexpr int kMaxParts = 256, kJoinThreads = 256;

template <int T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const AttendArgs a, int tiles, int tile_rows, int live,
                                                            int parts) {
  typedef typename Elem<T>::type E;
  __shared__ float s_f[kMaxParts], s_m[4], s_l[4];
  __shared__ __attribute__((aligned(16))) float s_part[4 * kJoinThreads];
  const int D = a.D, tid = threadIdx.x;
  const int k = static_cast<int>(blockIdx.x) % live, id = static_cast<int>(blockIdx.x) / live;
  const int tile = id % tiles, head = id / tiles % a.c.heads, b = id / tiles / a.c.heads;
  const Seq sq = load_seq(a.c, b);
  const int row = tile * tile_rows + k;
  if (row >= sq.count * a.group) return;
  const int64_t size = static_cast<int64_t>(tile_rows) * (D + 2);
  const float* ws = static_cast<const float*>(a.ws) + static_cast<int64_t>(id) * parts * size;
  // Thread p: the maximum and the sum of part p.
  float mp = -INFINITY, l = 0.f;
  if (tid < parts) {
    mp = ws[tid * size + tile_rows * D + k];
    l = ws[tid * size + tile_rows * D + tile_rows + k];
  }
  float m = mp;
#pragma unroll
  for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
  if ((tid & 63) == 0) s_m[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  m = m == -INFINITY ? 0.f : m;
  const float f = __builtin_amdgcn_exp2f(mp - m);
  s_f[tid] = f;
  l *= f;
#pragma unroll
  for (int x = 32; x; x >>= 1) l += __shfl_xor(l, x);
  if ((tid & 63) == 0) s_l[tid >> 6] = l;
  __syncthreads();
  const int d4 = D >> 2, slices = kJoinThreads / d4, slice = tid / d4, d = 4 * (tid - slice * d4);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (slice < slices) {
    const float* p = ws + static_cast<int64_t>(k) * D + d;
#pragma unroll 8
    for (int j = slice; j < parts; j += slices) v += *reinterpret_cast<const f32x4*>(p + j * size) * s_f[j];
    *reinterpret_cast<f32x4*>(s_part + 4 * tid) = v;
  }
  __syncthreads();
  if (slice) return;
  for (int j = 1; j < min(slices, parts); ++j) v += *reinterpret_cast<const f32x4*>(s_part + 4 * (tid + j * d4));
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  E* o = static_cast<E*>(a.o) + (sq.start + row / a.group) * a.o_t + (head * a.group + row % a.group) * a.o_h + d;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<E>(l == 0.f ? 0.f : v[i] / l);
}

// The same for 16 rows a workgroup, 16 threads a row: for tiles whose rows are
// all there and in up to four parts (us, against a workgroup a row: 2 parts of
// 512 x 16 rows of 64 d 4.6 / 14.0, 2 parts of 128 x 256 rows of 128 d 29 /
// 42; 32 parts 52 / 36, 4 parts of one row of 256 d 6.1 / 4.0).
template <int T>
__global__ __launch_bounds__(256) void join_many_kernel(const AttendArgs a, int tiles, int tile_rows, int parts) {
  typedef typename Elem<T>::type E;
  const int D = a.D, tid = threadIdx.x;
  const int slices = tile_rows / 16;
  const int k = static_cast<int>(blockIdx.x) % slices * 16 + (tid >> 4), id = static_cast<int>(blockIdx.x) / slices;
  const int tile = id % tiles, head = id / tiles % a.c.heads, b = id / tiles / a.c.heads;
  const Seq sq = load_seq(a.c, b);
  const int row = tile * tile_rows + k;
  if (row >= sq.count * a.group) return;
  const int64_t size = static_cast<int64_t>(tile_rows) * (D + 2);
  const float* ws = static_cast<const float*>(a.ws) + static_cast<int64_t>(id) * parts * size;
  const float* wm = ws + tile_rows * D + k;
  float m = -INFINITY;
  for (int p = 0; p < parts; ++p) m = fmaxf(m, wm[p * size]);
  m = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int p = 0; p < parts; ++p) l += __builtin_amdgcn_exp2f(wm[p * size] - m) * wm[p * size + tile_rows];
  E* o = static_cast<E*>(a.o) + (sq.start + row / a.group) * a.o_t + (head * a.group + row % a.group) * a.o_h;
  for (int d = (tid & 15) * 4; d < D; d += 64) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < parts; ++p)
      v += *reinterpret_cast<const f32x4*>(ws + p * size + static_cast<int64_t>(k) * D + d) *
           __builtin_amdgcn_exp2f(wm[p * size] - m);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[d + i] = static_cast<E>(l == 0.f ? 0.f : v[i] / l);
  }
}

template <int T, int DC>
static void go_attend(const AttendArgs& a, hipStream_t s, Form& form) {
  const int64_t rows = static_cast<int64_t>(a.c.max_new) * a.group, pairs = static_cast<int64_t>(a.batch) * a.c.heads;
  int64_t keys = a.max_total;
  if (a.window && keys > static_cast<int64_t>(a.window) + a.c.max_new) keys = static_cast<int64_t>(a.window) + a.c.max_new;
  // The kernel for many rows pays where its tiles are filled and the chip is:
  // from about 80 rows (128 up to 64 d) a sequence and cache head, with a tile
  // for every CU (us, few / many: 32 prompts of 250 x 16 x 64 61 / 33, of 90 x
  // 16 x 256 143 / 29) or enough units of 16 rows x 64 keys over all tiles
  // (100 rows of 128 d, 20000 units 44 / 33; 256 rows, 16000 units 39 / 36; 100
  // rows, 2500 units 21 / 25; 2000 rows of 64 d, 32000 units 44 / 51), which a
  // window thins out where tiles are few (48 tiles, 1500 rows, window 700 25 /
  // 49; 171 tiles, window 4 19 / 13).
  const int64_t seen = a.causal && !a.window ? keys - a.c.max_new / 2 : keys;
  const int64_t units = pairs * ((rows + 15) / 16) * ((seen + kBlockKeys - 1) / kBlockKeys);
  constexpr int kManyRows = 16 * kManyWaves * many_rt(T, DC);
  const int64_t many_wgs = pairs * ((rows + kManyRows - 1) / kManyRows);
  const bool sliding = a.causal && a.window;
  const bool many = rows > (DC <= 2 ? 128 : 80) &&
                    (many_wgs >= 256 || (units >= (DC <= 2 ? 40000 : 16000) && !(sliding && many_wgs < 128)));
  const int tile_rows = many ? kManyRows : kFewRows;
  const int64_t tiles = (rows + tile_rows - 1) / tile_rows, wgs = pairs * tiles;
  // Parts of the keys where the rows alone do not fill the chip, each at
  // least one round of the workgroup's waves long, as the workspace allows: as
  // many workgroups as the chip holds (us, half as many / these / twice: 4 x
  // 65536 keys of 8 x 128 d 90 / 84 / 87, 32 x 2000 29 / 25 / 30, 16 x 16000
  // of 2 x 256 74 / 49 / 55).
  const int64_t span = static_cast<int64_t>(a.window) + (tile_rows + a.group - 1) / a.group;  // of a sliding tile
  const int64_t most = ((sliding && span < keys ? span : keys) + 255) / 256, room = static_cast<int64_t>(a.ws_bytes) / (tile_rows * (a.D + 2) * 4 * wgs);
  int64_t parts = 256 * (many ? 1 : few_waves(T, DC)) / wgs;
  // Causal tiles differ in length: where each has a CU of its own, two parts
  // let the short ones' CUs help (us, one / two: 136 tiles of 192 d 78 / 55, 160
  // of 128 d 168 / 106, 256 of 192 d 78 / 67; not 324 of 128 d 233 / 245).
  if (many && a.causal && !a.window && wgs <= 256 && keys >= 1024 && parts < 2) parts = 2;
  parts = parts < kMaxParts ? parts : kMaxParts;
  parts = parts < most ? parts : most;
  parts = parts < room ? parts : room;
  if (parts < 1) parts = 1;
  const int nt = static_cast<int>(tiles), np = static_cast<int>(parts);
  const dim3 grid(static_cast<unsigned>(wgs * parts));
  const int live = static_cast<int>(rows < tile_rows ? rows : tile_rows);
  form = Form{many ? "attend_many" : "attend_few", {tile_rows, np}};
  if (many)
    attend_many_kernel<T, DC><<<grid, 64 * kManyWaves, 0, s>>>(a, nt, np);
  else
    attend_few_kernel<T, DC><<<grid, 256, 0, s>>>(a, nt, np);
  if (np > 1 && np <= 4 && live >= 16)
    join_many_kernel<T><<<dim3(static_cast<unsigned>(wgs * (tile_rows / 16))), 256, 0, s>>>(a, nt, tile_rows, np);
  else if (np > 1)
    join_kernel<T><<<dim3(static_cast<unsigned>(wgs * live)), kJoinThreads, 0, s>>>(a, nt, tile_rows, live, np);
}

template <int T>
static void go_dim(const AttendArgs& a, hipStream_t s, Form& form) {
  switch (a.D / 32) {
    case 1: go_attend<T, 1>(a, s, form); break;
    case 2: go_attend<T, 2>(a, s, form); break;
    case 3: go_attend<T, 3>(a, s, form); break;
    case 4: go_attend<T, 4>(a, s, form); break;
    case 5: go_attend<T, 5>(a, s, form); break;
    case 6: go_attend<T, 6>(a, s, form); break;
    case 7: go_attend<T, 7>(a, s, form); break;
    default: go_attend<T, 8>(a, s, form); break;
  }
}

hipError_t launch_attend(int dtype, const AttendArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_dim<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    go_dim<EL_BF16>(a, s, form);
  else
    go_dim<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
