// ops_host.hip -- host side of the 8-bit transformer operators: the C entry
// points declared in vocoder.h, their argument checks, the handle and its
// workspace.  Nothing here throws: messages are formatted into fixed buffers.
#include "../../include/vocoder.h"
#include "ops.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#define VOC_API extern "C" __attribute__((visibility("default")))

using namespace voc;

struct voc_ops {
  int device = 0;
  void* ws = nullptr;
  Form form;  // of the last launch
  char err[256] = "";
};

namespace {

thread_local char g_ops_create_error[256] = "";

__attribute__((format(printf, 3, 4)))
voc_status fail(voc_ops* o, voc_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(o ? o->err : g_ops_create_error, 256, fmt, ap);
  va_end(ap);
  return st;
}

voc_status hip_fail(voc_ops* o, hipError_t e, const char* what) {
  return fail(o, e == hipErrorOutOfMemory ? VOC_OOM : VOC_DEVICE_ERROR, "%s: %s", what, hipGetErrorString(e));
}

// Makes the handle's device current for a launch and puts the caller's back.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    err_ = hipGetDevice(&before_);
    if (err_ == hipSuccess && before_ != device) {
      err_ = hipSetDevice(device);
      moved_ = err_ == hipSuccess;
    }
  }
  ~OnDevice() {
    if (moved_) (void)hipSetDevice(before_);
  }
  hipError_t error() const { return err_; }

 private:
  int before_ = 0;
  bool moved_ = false;
  hipError_t err_ = hipSuccess;
};

template <class F>
voc_status on_device(voc_ops* o, const char* what, F&& fn) {
  OnDevice d(o->device);
  hipError_t e = d.error();
  if (e == hipSuccess) e = fn();
  return e == hipSuccess ? VOC_OK : hip_fail(o, e, what);
}

bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool dtype_ok(int t) { return t == VOC_F32 || t == VOC_BF16 || t == VOC_F16; }

constexpr int64_t kMaxInt = 0x7fffffff;
// Bound of every stride (elements): offsets of any row then stay within 63 bits.
constexpr int64_t kMaxStride = int64_t(1) << 40;
bool stride_ok(int64_t s, int64_t least) { return s >= least && s <= kMaxStride; }

voc_status check_rows(voc_ops* o, int dtype, int64_t rows, int64_t C, const void* x, int64_t ldx, const int8_t* q,
                      int64_t ldq, const float* scale) {
  if (!dtype_ok(dtype)) return fail(o, VOC_INVALID_PARAMS, "unknown dtype %d", dtype);
  if (rows < 0 || rows > kMaxInt) return fail(o, VOC_INVALID_PARAMS, "rows out of range");
  if (C < 1 || C > kRowsMaxC) return fail(o, VOC_INVALID_PARAMS, "C must be 1 .. %d", kRowsMaxC);
  if (rows == 0) return VOC_OK;
  if (!x || !q || !scale) return fail(o, VOC_INVALID_PARAMS, "NULL pointer");
  if (!stride_ok(ldx, C) || !stride_ok(ldq, C)) return fail(o, VOC_INVALID_PARAMS, "row strides must be at least C");
  if (!aligned(x, elem_size(dtype)) || !aligned(scale, 4))
    return fail(o, VOC_INVALID_PARAMS, "pointers must be aligned to their elements");
  return VOC_OK;
}

// Checks the cache and the batch and fills the kernels' view of them.
voc_status check_cache(voc_ops* o, const voc_kv_cache* c, const voc_kv_batch* b, CacheView* v) {
  if (!c || !b) return fail(o, VOC_INVALID_PARAMS, "NULL pointer");
  int log = 4;
  while (log < 8 && (1 << log) != c->page_tokens) ++log;
  if (log == 8) return fail(o, VOC_INVALID_PARAMS, "page_tokens must be 16, 32, 64 or 128");
  if (c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32)
    return fail(o, VOC_INVALID_PARAMS, "head_dim must be a multiple of 32 up to 256");
  if (c->kv_heads < 1 || c->kv_heads > 1024) return fail(o, VOC_INVALID_PARAMS, "kv_heads out of range");
  if (c->n_pages < 1 || c->n_pages > kMaxInt) return fail(o, VOC_INVALID_PARAMS, "n_pages out of range");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(o, VOC_INVALID_PARAMS, "NULL cache pointer");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(o, VOC_INVALID_PARAMS, "the cache's codes must be 16-byte aligned, its scales 4-byte aligned");
  if (b->batch < 0 || b->batch > 65535) return fail(o, VOC_INVALID_PARAMS, "batch must be 0 .. 65535");
  if (b->tokens < 0 || b->tokens > kMaxInt || b->max_new < 0 || b->max_new > (1 << 24))
    return fail(o, VOC_INVALID_PARAMS, "tokens or max_new out of range");
  if (b->table_stride < 1 || b->table_stride > (kMaxInt - (1 << 25)) >> log)
    return fail(o, VOC_INVALID_PARAMS, "table_stride out of range");
  if (b->max_total < 0 || b->max_total > kMaxInt) return fail(o, VOC_INVALID_PARAMS, "max_total out of range");
  if (b->batch && (!b->starts || !b->past || !b->page_table)) return fail(o, VOC_INVALID_PARAMS, "NULL batch pointer");
  if (!aligned(b->starts, 4) || !aligned(b->past, 4) || !aligned(b->page_table, 4))
    return fail(o, VOC_INVALID_PARAMS, "the batch's arrays must be 4-byte aligned");
  v->k = c->k;
  v->v = c->v;
  v->ks = c->k_scale;
  v->vs = c->v_scale;
  v->starts = b->starts;
  v->past = b->past;
  v->table = b->page_table;
  v->stride = b->table_stride;
  v->n_pages = c->n_pages;
  v->page_log = log;
  v->heads = c->kv_heads;
  v->tokens = static_cast<int>(b->tokens);
  v->max_new = static_cast<int>(b->max_new);
  return VOC_OK;
}

}  // namespace

VOC_API voc_status voc_ops_create(int hip_device, voc_ops** out) {
  if (!out) return fail(nullptr, VOC_INVALID_PARAMS, "out is NULL");
  *out = nullptr;
  int n = 0;
  hipError_t e = hipGetDeviceCount(&n);
  if (e != hipSuccess) return hip_fail(nullptr, e, "hipGetDeviceCount");
  if (hip_device < 0 || hip_device >= n) return fail(nullptr, VOC_INVALID_PARAMS, "no HIP device %d", hip_device);
  voc_ops* o = new (std::nothrow) voc_ops;
  if (!o) return fail(nullptr, VOC_OOM, "out of host memory");
  o->device = hip_device;
  {
    OnDevice d(hip_device);
    e = d.error();
    if (e == hipSuccess) e = hipMalloc(&o->ws, VOC_OPS_WORKSPACE_BYTES);
  }
  if (e != hipSuccess) {
    delete o;
    return hip_fail(nullptr, e, "workspace");
  }
  *out = o;
  return VOC_OK;
}

VOC_API const char* voc_ops_last_error(const voc_ops* ops) { return ops ? ops->err : g_ops_create_error; }

VOC_API const char* voc_dbg_last_kernel(const voc_ops* ops, int shape[2]) {
  const Form none, &f = ops ? ops->form : none;
  if (shape) {
    shape[0] = f.shape[0];
    shape[1] = f.shape[1];
  }
  return f.kernel;
}

VOC_API void voc_ops_destroy(voc_ops* ops) {
  if (!ops) return;
  {
    OnDevice d(ops->device);
    (void)hipFree(ops->ws);
  }
  delete ops;
}

VOC_API voc_status vocoder_rms_norm(voc_ops* o, int dtype, int64_t rows, int64_t C, const void* x, int64_t ldx,
                                    const void* residual, int64_t ldr, void* h_out, int64_t ldh, const float* weight,
                                    float eps, int8_t* q, int64_t ldq, float* scale, void* hip_stream) {
  if (!o) return VOC_INVALID_PARAMS;
  o->err[0] = 0;
  voc_status st = check_rows(o, dtype, rows, C, x, ldx, q, ldq, scale);
  if (st != VOC_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(o, VOC_INVALID_PARAMS, "eps must be finite and not negative");
  if (rows == 0) return VOC_OK;
  if (!weight) return fail(o, VOC_INVALID_PARAMS, "weight is NULL");
  if ((residual && !stride_ok(ldr, C)) || (h_out && !stride_ok(ldh, C)))
    return fail(o, VOC_INVALID_PARAMS, "row strides must be at least C");
  if (!aligned(residual, elem_size(dtype)) || !aligned(h_out, elem_size(dtype)) || !aligned(weight, 4))
    return fail(o, VOC_INVALID_PARAMS, "pointers must be aligned to their elements");
  const RowsArgs a{x, residual, h_out, weight, eps, q, scale, rows, ldx, ldr, ldh, ldq, static_cast<int>(C)};
  return on_device(o, "rms_norm", [&] { return launch_rows(dtype, a, static_cast<hipStream_t>(hip_stream), o->form); });
}

VOC_API voc_status vocoder_quantize_rows(voc_ops* o, int dtype, int64_t rows, int64_t C, const void* x, int64_t ldx,
                                         int8_t* q, int64_t ldq, float* scale, void* hip_stream) {
  if (!o) return VOC_INVALID_PARAMS;
  o->err[0] = 0;
  voc_status st = check_rows(o, dtype, rows, C, x, ldx, q, ldq, scale);
  if (st != VOC_OK || rows == 0) return st;
  const RowsArgs a{x, nullptr, nullptr, nullptr, 0.f, q, scale, rows, ldx, 0, 0, ldq, static_cast<int>(C)};
  return on_device(o, "quantize_rows", [&] { return launch_rows(dtype, a, static_cast<hipStream_t>(hip_stream), o->form); });
}

VOC_API voc_status vocoder_matmul_int(voc_ops* o, int out_dtype, int64_t M, int64_t N, int64_t K, const int8_t* a,
                                      int64_t lda, const float* a_scale, const int8_t* b, int64_t ldb,
                                      const float* b_scale, const float* bias, int act, void* y, int64_t ldy,
                                      void* hip_stream) {
  if (!o) return VOC_INVALID_PARAMS;
  o->err[0] = 0;
  if (!dtype_ok(out_dtype)) return fail(o, VOC_INVALID_PARAMS, "unknown dtype %d", out_dtype);
  if (act != VOC_ACT_NONE && act != VOC_ACT_GELU) return fail(o, VOC_INVALID_PARAMS, "unknown act %d", act);
  if (M < 0 || M > (1 << 24) || N < 0 || N > (1 << 24)) return fail(o, VOC_INVALID_PARAMS, "M or N out of range");
  if (K < 1 || K > 131071) return fail(o, VOC_INVALID_PARAMS, "K must be 1 .. 131071");
  if (M == 0 || N == 0) return VOC_OK;
  // A launch holds fewer than 2^32 threads (the smallest tiles: 64 x 64 in 512).
  if (((M + 63) / 64) * ((N + 63) / 64) >= 1 << 23) return fail(o, VOC_INVALID_PARAMS, "too many outputs for one call");
  if (!a || !a_scale || !b || !b_scale || !y) return fail(o, VOC_INVALID_PARAMS, "NULL pointer");
  if (!stride_ok(lda, K) || !stride_ok(ldb, K) || !stride_ok(ldy, N))
    return fail(o, VOC_INVALID_PARAMS, "row strides must be at least the row's length");
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(bias, 4) || !aligned(y, elem_size(out_dtype)))
    return fail(o, VOC_INVALID_PARAMS, "pointers must be aligned to their elements");
  const IntMatmulArgs g{a, b, a_scale, b_scale, bias, y, lda, ldb, ldy, static_cast<int>(M), static_cast<int>(N),
                        static_cast<int>(K), act};
  return on_device(o, "matmul_int", [&] { return launch_int_matmul(out_dtype, g, static_cast<hipStream_t>(hip_stream), o->form); });
}

VOC_API voc_status vocoder_cache_append(voc_ops* o, const voc_kv_cache* cache, const voc_kv_batch* batch, int dtype,
                                        const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                        int64_t v_token_stride, int64_t v_head_stride, void* hip_stream) {
  if (!o) return VOC_INVALID_PARAMS;
  o->err[0] = 0;
  AppendArgs a{};
  voc_status st = check_cache(o, cache, batch, &a.c);
  if (st != VOC_OK) return st;
  if (!dtype_ok(dtype)) return fail(o, VOC_INVALID_PARAMS, "unknown dtype %d", dtype);
  if (batch->batch == 0 || batch->tokens == 0 || batch->max_new == 0) return VOC_OK;
  if (!k || !v) return fail(o, VOC_INVALID_PARAMS, "NULL pointer");
  if (!aligned(k, elem_size(dtype)) || !aligned(v, elem_size(dtype)))
    return fail(o, VOC_INVALID_PARAMS, "pointers must be aligned to their elements");
  if (!stride_ok(k_token_stride, 0) || !stride_ok(k_head_stride, 0) || !stride_ok(v_token_stride, 0) ||
      !stride_ok(v_head_stride, 0))
    return fail(o, VOC_INVALID_PARAMS, "strides out of range");
  a.k = k;
  a.v = v;
  a.k_t = k_token_stride;
  a.k_h = k_head_stride;
  a.v_t = v_token_stride;
  a.v_h = v_head_stride;
  a.D = cache->head_dim;
  a.batch = static_cast<int>(batch->batch);
  return on_device(o, "cache_append", [&] { return launch_append(dtype, a, static_cast<hipStream_t>(hip_stream), o->form); });
}

VOC_API voc_status vocoder_cache_attention(voc_ops* o, const voc_kv_cache* cache, const voc_kv_batch* batch, int dtype,
                                           int heads, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                           float softmax_scale, int causal, int64_t window, void* out,
                                           int64_t o_token_stride, int64_t o_head_stride, void* hip_stream) {
  if (!o) return VOC_INVALID_PARAMS;
  o->err[0] = 0;
  AttendArgs a{};
  voc_status st = check_cache(o, cache, batch, &a.c);
  if (st != VOC_OK) return st;
  if (!dtype_ok(dtype)) return fail(o, VOC_INVALID_PARAMS, "unknown dtype %d", dtype);
  if (heads < cache->kv_heads || heads % cache->kv_heads || heads / cache->kv_heads > 256)
    return fail(o, VOC_INVALID_PARAMS, "heads must be 1 .. 256 times kv_heads");
  if (!std::isfinite(softmax_scale)) return fail(o, VOC_INVALID_PARAMS, "softmax_scale must be finite");
  if (causal != 0 && causal != 1) return fail(o, VOC_INVALID_PARAMS, "causal must be 0 or 1");
  if (window < 0) return fail(o, VOC_INVALID_PARAMS, "window must not be negative");
  if (batch->batch == 0 || batch->tokens == 0 || batch->max_new == 0) return VOC_OK;
  if (!q || !out) return fail(o, VOC_INVALID_PARAMS, "NULL pointer");
  const int es = elem_size(dtype);
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(o, VOC_INVALID_PARAMS, "q and o must be 16-byte aligned");
  for (const int64_t s : {q_token_stride, q_head_stride, o_token_stride, o_head_stride})
    if (!stride_ok(s, 0) || s * es % 16)
      return fail(o, VOC_INVALID_PARAMS, "strides of q and o must be multiples of 16 bytes");
  a.q = q;
  a.o = out;
  a.q_t = q_token_stride;
  a.q_h = q_head_stride;
  a.o_t = o_token_stride;
  a.o_h = o_head_stride;
  a.D = cache->head_dim;
  a.batch = static_cast<int>(batch->batch);
  a.group = heads / cache->kv_heads;
  a.scale = softmax_scale * 1.4426950408889634f;
  a.causal = causal;
  // A window at least as long as any sequence hides nothing.
  a.window = window > (batch->table_stride << a.c.page_log) ? 0 : static_cast<int>(window);
  a.max_total = static_cast<int>(batch->max_total);
  a.ws = o->ws;
  a.ws_bytes = VOC_OPS_WORKSPACE_BYTES;
  // A launch holds fewer than 2^32 threads (16 query rows in 256).
  if (static_cast<int64_t>(a.batch) * heads * ((batch->max_new + 15) / 16 + 1) >= 1 << 24)
    return fail(o, VOC_INVALID_PARAMS, "too many query rows for one call");
  return on_device(o, "cache_attention", [&] { return launch_attend(dtype, a, static_cast<hipStream_t>(hip_stream), o->form); });
}
