// ops.h -- device-side arguments and launch interfaces of the 8-bit
// transformer operators (not part of the public ABI; the meaning of every
// operator is in vocoder.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace voc {

enum ElemType { EL_F32 = 0, EL_BF16 = 1, EL_F16 = 2 };  // = voc_dtype
inline int elem_size(int t) { return t == EL_F32 ? 4 : 2; }

// The kernel that a launch chose (vocoder.h: voc_dbg_last_kernel).
struct Form {
  const char* kernel = "";
  int shape[2] = {0, 0};
};

// Rows of 8-bit codes with one scale each (weight == null: no norm).
struct RowsArgs {
  const void* x;
  const void* r;        // residual, or null
  void* h;              // x + r, or null
  const float* weight;  // null: quantise x (+ r) as it is
  float eps;
  int8_t* q;
  float* scale;
  int64_t rows, ldx, ldr, ldh, ldq;
  int C;
};
constexpr int kRowsMaxC = 16384;
hipError_t launch_rows(int dtype, const RowsArgs& a, hipStream_t s, Form& form);

struct IntMatmulArgs {
  const int8_t* a;
  const int8_t* b;
  const float* sa;
  const float* sb;
  const float* bias;  // or null
  void* y;
  int64_t lda, ldb, ldy;
  int M, N, K;
  int act;            // VOC_ACT_*
};
hipError_t launch_int_matmul(int dtype, const IntMatmulArgs& a, hipStream_t s, Form& form);

// The cache and the sequences of one step, as every kernel reads them.
struct CacheView {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  const int32_t* starts;
  const int32_t* past;
  const int32_t* table;
  int64_t stride;     // pages per sequence in table
  int64_t n_pages;
  int page_log;       // log2(page_tokens)
  int heads;          // cache heads
  int tokens;         // packed rows
  int max_new;
};

// One sequence of a step, brought into bounds: tokens held before, new
// tokens, its first packed row (vocoder.h says what counts as empty).
struct Seq {
  int past, count, start;
};
__device__ __forceinline__ Seq load_seq(const CacheView& c, int b) {
  const int64_t cap = c.stride << c.page_log;  // the host keeps it below 2^31
  const int s0 = c.starts[b], s1 = c.starts[b + 1];
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= c.tokens && s1 - s0 <= c.max_new;
  const int p = c.past[b];
  Seq q;
  q.past = p < 0 ? 0 : p > cap ? static_cast<int>(cap) : p;
  q.count = ok ? s1 - s0 : 0;
  q.start = ok ? s0 : 0;
  return q;
}

struct AppendArgs {
  CacheView c;
  const void* k;
  const void* v;
  int64_t k_t, k_h, v_t, v_h;  // element strides of the new keys and values
  int D, batch;
};
hipError_t launch_append(int dtype, const AppendArgs& a, hipStream_t s, Form& form);

struct AttendArgs {
  CacheView c;
  const void* q;
  void* o;
  int64_t q_t, q_h, o_t, o_h;
  int D, batch, group;     // query heads per cache head
  float scale;             // softmax scale times log2(e)
  int causal;
  int window;              // 0: none
  int max_total;
  void* ws;
  size_t ws_bytes;
};
hipError_t launch_attend(int dtype, const AttendArgs& a, hipStream_t s, Form& form);

}  // namespace voc
