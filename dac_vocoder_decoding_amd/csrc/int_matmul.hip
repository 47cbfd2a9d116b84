// int_matmul.hip -- the 8-bit integer product with row scales,
//   y[m][n] = act((sum_k a[m][k] b[n][k]) sa[m] sb[n] + bias[n]),
// on the gfx950 matrix cores (v_mfma_i32_16x16x64_i8: 32-bit integer sums,
// exact for K <= 131071).
//
// The matrix-core "A" operand is b (output features), "B" is a (tokens): a
// lane then holds four consecutive features of one token, which it stores
// together.  Integer sums are exact, so every variant gives the same bits.
#include <string.h>

#include "gemm_common.h"
#include "ops_device.h"

namespace voc {

// Rows of any alignment can be read in the aligned 32-bit words that hold
// their bytes (each of them has a byte of the row, so none lies outside the
// caller's pages) and shifted into place.  That pays where the loads are all
// there is, for few tokens (us, as they lie / shifted: 105 x 1527 x 3563 28.0 /
// 16.3, 64 x 7680 x 1709 25.3 / 14.8); where they wait for LDS tiles it does
// not (6011 x 869 x 2789 54 / 64).
__device__ __forceinline__ i32x4 shifted(const uint32_t (&w)[5], uint32_t sh) {
  i32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = static_cast<int>(__builtin_amdgcn_alignbyte(w[i + 1], w[i], sh));
  return v;
}

// 16 codes at p.
template <bool SHIFT>
__device__ __forceinline__ i32x4 load_whole(const int8_t* p) {
  i32x4 v;
  if constexpr (!SHIFT) {
    __builtin_memcpy(&v, p, 16);
    return v;
  }
  const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p - sh);
  uint32_t w[5];
  __builtin_memcpy(w, q, 16);
  w[4] = q[sh ? 4 : 3];
  return shifted(w, sh);
}

// 16 codes of a row of K at k, zero past the row's end.
template <bool SHIFT>
__device__ __forceinline__ i32x4 load_codes(const int8_t* row, int k, int K) {
  const int8_t* p = row + k;
  const int n = K - k;
  if (!SHIFT && n >= 16) return load_whole<false>(p);  // (one path for all lanes is faster where words are read)
  const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p - sh);
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = n > 0 && 4 * i < n + static_cast<int>(sh) && (i < 4 || sh) ? q[i] : 0;
  i32x4 v = shifted(w, sh);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n < 4 * i + 4) v[i] &= n <= 4 * i ? 0 : (1 << (8 * (n - 4 * i))) - 1;
  return v;
}

// GELU: v (1 - erfc(z) / 2) for v >= 0, v erfc(z) / 2 below, z = |v| / sqrt(2),
// with Hastings' form erfc(z) = exp(-z^2) t (c0 + c1 t + ...), t = 1 / (1 + 0.4 z).
// The coefficients are a minimax fit over z in [0, 6] (error 2.8e-8); in fp32
// this alone is within 3.9 |v| 2^-24 of GELU, most of it near zero, where erfc is
// 1 less a small number.  fp32 outputs therefore take v / 2 (1 + v R(v^2))
// up to |v| = sqrt(2), R a minimax polynomial of erf(v / sqrt(2)) / v (relative
// error 3.1e-8): within 1.7 |v| 2^-24 everywhere (0.5 v (1 + erf) in fp32: 2.0),
// and for v of spread 0.1 the RMS error is 2.6e-8 of the RMS in place of 1.1e-7.
// 16-bit outputs, whose rounding hides that, keep erfc alone (us, 4606 x 6848 x
// 576: fp32 62, with erfc alone 54, without GELU 44; bf16 43).
template <int T>
__device__ __forceinline__ float activate(float v, int act) {
  if (!act) return v;
  const float v2 = v * v;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.282842712f, fabsf(v), 1.f));
  float p = fmaf(-0.100135252f, t, 0.354596674f);  // (c0 .. c5, halved)
  p = fmaf(p, t, -0.185491294f);
  p = fmaf(p, t, 0.234167159f);
  p = fmaf(p, t, 0.0808997527f);
  p = fmaf(p, t, 0.11596296f);
  const float half = p * t * __builtin_amdgcn_exp2f(v2 * -0.72134752f);
  const float large = v * (v >= 0.f ? 1.f - half : half);
  if constexpr (T != EL_F32) return large;
  const float h = 0.5f * v;
  float r = fmaf(8.67737242e-07f, v2, -1.77001948e-05f);
  r = fmaf(r, v2, 0.000229293859f);
  r = fmaf(r, v2, -0.00237356406f);
  r = fmaf(r, v2, 0.0199467484f);
  r = fmaf(r, v2, -0.132980719f);
  r = fmaf(r, v2, 0.797884583f);
  return fabsf(v) < 1.41421356f ? fmaf(h * v, r, h) : large;
}

// Four consecutive features n .. n + 3 of token m (n a multiple of 4).
template <int T>
__device__ __forceinline__ void store4(const IntMatmulArgs& a, bool vec, int m, int n, float sa, const i32x4& acc) {
  typedef typename Elem<T>::type E;
  E* y = static_cast<E*>(a.y) + static_cast<int64_t>(m) * a.ldy + n;
  E e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = min(n + i, a.N - 1);
    const float v = static_cast<float>(acc[i]) * sa * a.sb[c] + (a.bias ? a.bias[c] : 0.f);
    e[i] = static_cast<E>(activate<T>(v, a.act));
  }
  if (vec && n + 4 <= a.N) {
    __builtin_memcpy(__builtin_assume_aligned(y, 4 * sizeof(E)), e, 4 * sizeof(E));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) y[i] = e[i];
  }
}

// ------------------------------------------------------------- few tokens
// One workgroup per 16 features: its eight waves split K and read the weights
// once, straight into registers; the integer partial sums meet in LDS.
// MB blocks of 16 tokens.  Nothing is shared between workgroups but the
// tokens, so LDS tiles would only add a wait; bound by the latency of the
// loads (four steps of them in flight): 32 x 4096 x 1024, 4.2 MB of weights,
// 4.9 us.
template <int T, int MB, bool SHIFT>
__global__ __launch_bounds__(512) void int_matmul_few_kernel(const IntMatmulArgs a, int vec) {
  __shared__ i32x4 s_acc[8][MB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * MB * 16;
  const int steps = (a.K + 63) / 64, per = (steps + 7) / 8;
  const int k1 = min(a.K + 63, (wave + 1) * per * 64) & ~63;
  const int8_t* brow = a.b + static_cast<int64_t>(min(n0 + lr, a.N - 1)) * a.ldb;
  const int8_t* arow[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) arow[j] = a.a + static_cast<int64_t>(min(m0 + j * 16 + lr, a.M - 1)) * a.lda;
  i32x4 acc[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) acc[j] = i32x4{0, 0, 0, 0};
  // Four steps' loads are issued together; only the step that holds K's end
  // needs the masked load.
  for (int k0 = wave * per * 64; k0 < k1; k0 += 256) {
    i32x4 w[4], x[4][MB];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 64 + lg * 16;
      if (k0 + u * 64 >= k1) continue;
      if (k0 + u * 64 + 64 <= a.K) {
        w[u] = load_whole<SHIFT>(brow + k);
#pragma unroll
        for (int j = 0; j < MB; ++j) x[u][j] = load_whole<SHIFT>(arow[j] + k);
      } else {
        w[u] = load_codes<SHIFT>(brow, k, a.K);
#pragma unroll
        for (int j = 0; j < MB; ++j) x[u][j] = load_codes<SHIFT>(arow[j], k, a.K);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (k0 + u * 64 >= k1) continue;
#pragma unroll
      for (int j = 0; j < MB; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u], x[u][j], acc[j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < MB; ++j) s_acc[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave >= MB) return;  // wave j finishes token block j
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < 8; ++w) v += s_acc[w][wave][lane];
  const int m = m0 + wave * 16 + lr, n = n0 + 4 * lg;
  if (m < a.M && n < a.N) store4<T>(a, vec, m, n, a.sa[m], v);
}

// ------------------------------------------------------------- tiles
// BF features x BT tokens per workgroup, WF x WT waves.  K passes in stages
// of 128 codes (whole cache lines) through a ring of NS stages in LDS.  A
// stage holds rows of 128 bytes, features first; the 16-byte unit u of row r
// sits at unit u ^ (r / 2 % 8) of its row, which spreads the fragment reads
// (16 rows, 4 units) over all banks.
// DMA: global -> LDS copies through buffer resources, NS - 1 stages in
// flight, out-of-range rows and codes read as zero (16-byte aligned rows, K
// a multiple of 16).  Otherwise the rows go through registers, two stages
// ahead, with their tails masked (any alignment).
// Bound by the matrix cores: 8000 x 8192 x 4096 in 256 x 256 tiles takes 230 us
// (2.3 P operations a second; 280 in a profiled run, the matrix cores busy 55 %
// of the cycles at 1.9 GHz; the library's product 244).  Four waves of
// 128 x 128, one a SIMD, in place of eight: 414 to 460; 128 x 128 tiles with a
// four-stage ring: 425.
constexpr int kStageK = 128;

template <int T, int BF, int BT, int WF, int WT, int NS, bool DMA>
__global__ __launch_bounds__(WF * WT * 64) void int_matmul_tile_kernel(const IntMatmulArgs a, int tf, int tt, int vec) {
  typedef typename Elem<T>::type E;
  constexpr int NW = WF * WT;
  constexpr int FF = BF / WF / 16, FT = BT / WT / 16;
  constexpr int FB = BF / 8, TB = FB + BT / 8;  // 1 KB blocks of 8 rows in a stage
  constexpr int LW = TB / NW;
  constexpr int STAGE = TB * 1024;
  static_assert(TB % NW == 0 && NW % 2 == 0 && (NS - 2) * LW <= 63, "whole blocks per wave");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[NS * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int wf = wave % WF, wt = wave / WF;

  // Each XCD takes a contiguous range of tiles, in bands of 8 token tiles, so
  // that the tiles it runs together share feature and token rows in its L2.
  const int L = xcd_remap(blockIdx.x, tf * tt);
  const int band = L / (8 * tf), left = tt - band * 8;
  const int bh = left < 8 ? left : 8;
  const int in_band = L - band * 8 * tf;
  const int n0 = (in_band / bh) * BF, m0 = (band * 8 + in_band % bh) * BT;
  const int nstages = (a.K + kStageK - 1) / kStageK;

  i32x4 acc[FF][FT];
#pragma unroll
  for (int i = 0; i < FF; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // This lane's part of a block copy: row 8 b + lane / 8, the unit that sits
  // at position lane % 8 there (b has the parity of the wave).
  const int crow = lane >> 3;
  const int cunit = ((lane & 7) ^ ((crow >> 1) + 4 * (wave & 1))) * 16;
  // Its fragment rows within 16 rows, for both halves of a stage.
  const int frow = (lr >> 3) * 1024 + (lr & 7) * 128;
  const int fu[2] = {frow + ((lg ^ (lr >> 1)) * 16), frow + (((lg + 4) ^ (lr >> 1)) * 16)};
  auto stage_mma = [&](const unsigned char* s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned char* pf = s + fu[h] + wf * FF * 2048;
      const unsigned char* pt = s + fu[h] + FB * 1024 + wt * FT * 2048;
      i32x4 xf[FF], xt[FT];
#pragma unroll
      for (int j = 0; j < FT; ++j) xt[j] = *reinterpret_cast<const i32x4*>(pt + j * 2048);
#pragma unroll
      for (int i = 0; i < FF; ++i) xf[i] = *reinterpret_cast<const i32x4*>(pf + i * 2048);
#pragma unroll
      for (int i = 0; i < FF; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xf[i], xt[j], acc[i][j], 0, 0, 0);
    }
    // The second half's fragments are read between the first half's products.
    if constexpr (FF * FT >= FF + FT) {
      __builtin_amdgcn_sched_group_barrier(0x100, FT + FF, 0);
#pragma unroll
      for (int q = 0; q < FF + FT; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, FF * FT / (FF + FT), 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    }
  };

  if constexpr (DMA) {
    const uint32_t lds = lds_addr(smem);
    // The host keeps 256 rows below 2^31 bytes.
    const int nf = min(a.N - n0, BF), nt = min(a.M - m0, BT);
    const i4 fs = buf_rsrc(a.b + static_cast<int64_t>(n0) * a.ldb, static_cast<uint32_t>((nf - 1) * a.ldb + a.K));
    const i4 ts = buf_rsrc(a.a + static_cast<int64_t>(m0) * a.lda, static_cast<uint32_t>((nt - 1) * a.lda + a.K));
    uint32_t off[LW];
#pragma unroll
    for (int u = 0; u < LW; ++u) {
      const int b = wave + NW * u;
      const int row = (b < FB ? b : b - FB) * 8 + crow;
      off[u] = row < (b < FB ? nf : nt) ? static_cast<uint32_t>(row) * static_cast<uint32_t>(b < FB ? a.ldb : a.lda) + cunit
                                        : 0x80000000u;
    }
    auto issue = [&](int c, int slot) {
      const int k = c * kStageK;
      const bool past = k + cunit >= a.K;
#pragma unroll
      for (int u = 0; u < LW; ++u) {
        const int b = wave + NW * u;
        dma16(b < FB ? fs : ts, past ? 0x80000000u : off[u] + k, lds + slot * STAGE + b * 1024);
      }
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      if (s < nstages) issue(s, s);
    int slot = 0;
    for (int c = 0; c < nstages; ++c) {
      if (c + NS - 1 <= nstages)
        wait_vm<(NS - 2) * LW>();
      else
        wait_vm<0>();
      lds_barrier();  // stage c is in LDS; every wave has read stage c - 1
      if (c + NS - 1 < nstages) issue(c + NS - 1, slot == 0 ? NS - 1 : slot - 1);
      stage_mma(smem + slot * STAGE);
      slot = slot + 1 == NS ? 0 : slot + 1;
    }
  } else {
    const int8_t* row[LW];
#pragma unroll
    for (int u = 0; u < LW; ++u) {
      const int b = wave + NW * u;
      row[u] = b < FB ? a.b + static_cast<int64_t>(min(n0 + b * 8 + crow, a.N - 1)) * a.ldb
                      : a.a + static_cast<int64_t>(min(m0 + (b - FB) * 8 + crow, a.M - 1)) * a.lda;
    }
    constexpr int AHEAD = 2;
    i32x4 g[AHEAD][LW];
#pragma unroll
    for (int p = 0; p < AHEAD; ++p)
#pragma unroll
      for (int u = 0; u < LW; ++u) g[p][u] = load_codes<false>(row[u], p * kStageK + cunit, a.K);
    for (int c0 = 0; c0 < nstages; c0 += AHEAD) {
#pragma unroll
      for (int p = 0; p < AHEAD; ++p) {
        const int c = c0 + p;
        if (c >= nstages) break;
        unsigned char* s = smem + (c & 1) * STAGE;
#pragma unroll
        for (int u = 0; u < LW; ++u) *reinterpret_cast<i32x4*>(s + (wave + NW * u) * 1024 + lane * 16) = g[p][u];
        __syncthreads();
        if ((c + AHEAD + 1) * kStageK <= a.K) {  // uniform: the whole stage lies inside the rows
#pragma unroll
          for (int u = 0; u < LW; ++u) g[p][u] = load_whole<false>(row[u] + (c + AHEAD) * kStageK + cunit);
        } else if (c + AHEAD < nstages) {
#pragma unroll
          for (int u = 0; u < LW; ++u) g[p][u] = load_codes<false>(row[u], (c + AHEAD) * kStageK + cunit, a.K);
        }
        stage_mma(s);
      }
    }
  }

  // Epilogue: each wave turns its tile over in its own part of LDS, so that
  // whole rows of features go out in 16-byte pieces.
  constexpr int ES = sizeof(E);
  constexpr int RC = FF * 16 * ES / 16;               // 16-byte pieces of a token's row
  constexpr int ROOM = NS * STAGE / NW / (RC * 16);   // token rows that fit
  constexpr int CT = ROOM >= FT * 16 ? FT : ROOM / 16;  // blocks of 16 tokens at a time
  static_assert(CT >= 1 && FT % CT == 0 && (RC & (RC - 1)) == 0, "the epilogue's part of LDS");
  __syncthreads();
  unsigned char* part = smem + wave * (NS * STAGE / NW);
  const int nw = n0 + wf * FF * 16, mw = m0 + wt * FT * 16;
  f4 sb[FF], bi[FF];
#pragma unroll
  for (int i = 0; i < FF; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = min(nw + i * 16 + 4 * lg + e, a.N - 1);
      sb[i][e] = a.sb[n];
      bi[i][e] = a.bias ? a.bias[n] : 0.f;
    }
#pragma unroll
  for (int j0 = 0; j0 < FT; j0 += CT) {
#pragma unroll
    for (int jj = 0; jj < CT; ++jj) {
      const float sa = a.sa[min(mw + (j0 + jj) * 16 + lr, a.M - 1)];
      unsigned char* pr = part + (jj * 16 + lr) * RC * 16;
#pragma unroll
      for (int i = 0; i < FF; ++i) {
        E e[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = static_cast<E>(activate<T>(static_cast<float>(acc[i][j0 + jj][q]) * sa * sb[i][q] + bi[i][q], a.act));
        const int byte = (i * 16 + 4 * lg) * ES;
        __builtin_memcpy(__builtin_assume_aligned(pr + (((byte >> 4) ^ (lr & (RC - 1))) << 4) + (byte & 15), 4 * ES), e, 4 * ES);
      }
    }
    wave_lds_sync();
    // Whole pieces are stored past the L2, which keeps its place for operands
    // (us, through it / past it: 8000 x 8192 x 4096 258 / 230, 8000 x 4096 x 1024
    // 58 / 51, 2000 x 8192 x 512 24.5 / 18.8).
    if (vec) {
#pragma unroll
      for (int q = 0; q < CT * 16 * RC / 64; ++q) {
        const int p = q * 64 + lane, t = p / RC, c = p % RC;
        const int m = mw + j0 * 16 + t, n = nw + c * (16 / ES);
        const i32x4 v = *reinterpret_cast<const i32x4*>(part + t * RC * 16 + ((c ^ (t & 15 & (RC - 1))) << 4));
        if (m < a.M && n < a.N) {
          E* y = static_cast<E*>(a.y) + static_cast<int64_t>(m) * a.ldy + n;
          if (n + 16 / ES <= a.N) {
            __builtin_nontemporal_store(v, reinterpret_cast<i32x4*>(y));
          } else {
            const E* e = reinterpret_cast<const E*>(&v);
#pragma unroll
            for (int k = 0; k < 16 / ES; ++k)
              if (n + k < a.N) y[k] = e[k];
          }
        }
      }
    } else {
      // Rows of any alignment: a wave's stores cover consecutive features (16
      // bytes a lane, stored value by value: 3693 x 4201 x 192 58 us for 26).
      constexpr int NF = FF * 16;
#pragma unroll 4
      for (int q = 0; q < CT * 16 * NF / 64; ++q) {
        const int p = q * 64 + lane, t = p / NF, f = p % NF;
        const int m = mw + j0 * 16 + t, n = nw + f, byte = f * ES;
        const E v = *reinterpret_cast<const E*>(part + t * RC * 16 + (((byte >> 4) ^ (t & (RC - 1) & 15)) << 4) + (byte & 15));
        if (m < a.M && n < a.N) static_cast<E*>(a.y)[static_cast<int64_t>(m) * a.ldy + n] = v;
      }
    }
    if (j0 + CT < FT) wave_lds_sync();
  }
}

template <int T, bool SHIFT>
static void go_few(const IntMatmulArgs& a, hipStream_t s, Form& form) {
  const int vec = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % (4 * elem_size(T)) == 0;
  const unsigned gx = (a.N + 15) / 16;
  auto rows = [&](int mb) { return static_cast<unsigned>((a.M + 16 * mb - 1) / (16 * mb)); };
  // As many tokens a workgroup as leave about one to each CU (us, 64 x 1024 x
  // 4096 with 4 / 2 / 1 blocks of 16: 11.3 / 7.7 / 7.3, 64 x 2048 x 4096 11.7 /
  // 8.1, 32 x 4096 x 1024 4.2 with 2, 4.6 with 1; 64 x 3500 x 2048, whose rows
  // come here where they are not 16-byte aligned, 7.3 / 8.4).
  const int blocks = a.M > 32 && gx * rows(4) >= 192 ? 4 : a.M > 16 && gx * rows(2) >= 192 ? 2 : 1;
  form = Form{SHIFT ? "product_few_shifted" : "product_few", {16, 16 * blocks}};
  if (blocks == 4)
    int_matmul_few_kernel<T, 4, SHIFT><<<dim3(gx, rows(4)), 512, 0, s>>>(a, vec);
  else if (blocks == 2)
    int_matmul_few_kernel<T, 2, SHIFT><<<dim3(gx, rows(2)), 512, 0, s>>>(a, vec);
  else
    int_matmul_few_kernel<T, 1, SHIFT><<<dim3(gx, rows(1)), 512, 0, s>>>(a, vec);
}

template <int T, int BF, int BT, int WF, int WT, int NS, bool DMA>
static void go_tile(const IntMatmulArgs& a, hipStream_t s, Form& form) {
  const int tf = (a.N + BF - 1) / BF, tt = (a.M + BT - 1) / BT;
  const int vec = a.ldy * elem_size(T) % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
  form = Form{DMA ? "product_tile" : "product_tile_rows", {BF, BT}};
  int_matmul_tile_kernel<T, BF, BT, WF, WT, NS, DMA>
      <<<dim3(static_cast<unsigned>(tf) * tt), WF * WT * 64, 0, s>>>(a, tf, tt, vec);
}

// Which kernel (us):
//  * up to 16 tokens, or so few outputs that 64x64 tiles would leave most of the
//    chip idle: the K-splitting kernel (K-splitting / tiles: 16x8192x4096 10.6 /
//    12.0; 128x1024x4096, 2^17 outputs, 7.8 / 11.5; 192x1024x4096 13.2 / 11.5;
//    64x8192x4096 21 / 12.3); for unaligned rows, which reach tiles through
//    registers, to twice that (64x4096x4096 16.0 / 22.2);
//  * the largest tile that still gives the 256 CUs enough workgroups:
//    256x256 from 192 tiles (8000x8192x2048: 137 against 150 for 128x128;
//    8000x1024x4096, 128 tiles: 50 against 33), 128x128 from 384 (two
//    workgroups a CU; 2000x4096x1024 13.6 against 17.8), 128x64 from 384
//    (1000x4096x1024: 9.6 against 11.5 and 12.9), else 64x64
//    (500x1024x4096: 12.4 against 15.8) with eight waves (with four half a us
//    more);
//  * rows that are not 16-byte aligned go through registers in 64x64 tiles
//    (689x1000x1501: 11.1; four waves 12.5, 128x64 17.4).
template <int T>
static void go_int_matmul(const IntMatmulArgs& a, hipStream_t s, Form& form) {
  auto tiles = [&](int f, int t) { return static_cast<int64_t>((a.N + f - 1) / f) * ((a.M + t - 1) / t); };
  const bool dma = a.K % 16 == 0 && a.lda % 16 == 0 && a.ldb % 16 == 0 && a.lda < (1 << 22) && a.ldb < (1 << 22) &&
                   (reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.b)) % 16 == 0;
  if (a.M <= 16 || static_cast<int64_t>(a.M) * a.N <= (dma ? 1 << 17 : 1 << 18)) {
    if ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.b) | a.lda | a.ldb) % 4 == 0)
      go_few<T, false>(a, s, form);
    else
      go_few<T, true>(a, s, form);
  } else if (!dma) {
    go_tile<T, 64, 64, 4, 2, 2, false>(a, s, form);
  } else if (tiles(256, 256) >= 192) {
    go_tile<T, 256, 256, 2, 4, 2, true>(a, s, form);
  } else if (tiles(128, 128) >= 384) {
    go_tile<T, 128, 128, 2, 2, 2, true>(a, s, form);
  } else if (tiles(128, 64) >= 384) {
    go_tile<T, 128, 64, 2, 2, 3, true>(a, s, form);
  } else {
    go_tile<T, 64, 64, 4, 2, 4, true>(a, s, form);
  }
}

hipError_t launch_int_matmul(int dtype, const IntMatmulArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_int_matmul<EL_F32>(a, s, form);
  else if (dtype == EL_BF16)
    go_int_matmul<EL_BF16>(a, s, form);
  else
    go_int_matmul<EL_F16>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
