// C ABI of the serving operators (declared in include/int8lin.h).  As in
// int8lin_abi.hip: every argument is checked on the host before any HIP call,
// then the kernels go onto the caller's stream; nothing is allocated, nothing
// synchronizes and no exception leaves an entry point.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "../../include/int8lin.h"
#include "launch.h"
#include "serve.h"

#define I8L_API extern "C" __attribute__((visibility("default")))

namespace {

i8l_status fail(i8l_status s, const char* fn, const char* fmt, ...) {
  size_t n = 0;
  char* buf = i8l::error_buffer(&n);
  const int k = snprintf(buf, n, "%s: ", fn);
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf + k, n - (size_t)k, fmt, ap);
  va_end(ap);
  return s;
}

i8l_status ok() {
  size_t n = 0;
  i8l::error_buffer(&n)[0] = 0;
  return I8L_OK;
}

i8l_status hip_status(const char* fn, hipError_t e) {
  return e == hipSuccess ? ok() : fail(I8L_ERR_HIP, fn, "%s", hipGetErrorString(e));
}

i8l_status check_ptr(const char* fn, const char* name, const void* p, size_t align) {
  if (!p) return fail(I8L_ERR_INVALID_ARG, fn, "%s is NULL", name);
  if ((uintptr_t)p % align)
    return fail(I8L_ERR_INVALID_ARG, fn, "%s must be %d-byte aligned", name, (int)align);
  return I8L_OK;
}

#define CHECK(x)                        \
  do {                                  \
    const i8l_status s_ = (x);          \
    if (s_ != I8L_OK) return s_;        \
  } while (0)
#define CHECK_PTR(p, align) CHECK(check_ptr(fn, #p, (p), (align)))

i8l_status check_dtype(const char* fn, int dtype) {
  if (dtype != I8L_FP16 && dtype != I8L_BF16)
    return fail(I8L_ERR_INVALID_ARG, fn, "dtype %d is neither I8L_FP16 nor I8L_BF16", dtype);
  return I8L_OK;
}

// The layer's shape rules (int8_linear's).
i8l_status check_shape(const char* fn, int64_t M, int64_t K, int64_t N) {
  i8l_workspace_layout L;
  const i8l_status s = i8l_linear_workspace(M, K, N, &L);
  if (s != I8L_OK) {   // the same message under this entry's name
    char text[256];
    snprintf(text, sizeof(text), "%s", i8l_last_error());
    const char* at = text;
    for (const char* c = text; *c; ++c)
      if (c[0] == ':' && c[1] == ' ') {
        at = c + 2;
        break;
      }
    return fail(s, fn, "%s", at);
  }
  return I8L_OK;
}

// No outlier column: the count and the first indices that the product kernels
// read, all 0.  One copy per GPU in the library's image.
static __device__ __align__(64) int32_t no_outliers[16];
constexpr int kMaxDevices = 64;
std::atomic<uintptr_t> g_zero_addr[kMaxDevices];

i8l_status zero_words(const char* fn, const int32_t** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(I8L_ERR_HIP, fn, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices)
    return fail(I8L_ERR_INVALID_ARG, fn, "device %d outside the %d the library tracks", dev,
                kMaxDevices);
  uintptr_t a = g_zero_addr[dev].load(std::memory_order_acquire);
  if (a == 0) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(no_outliers));
    if (e != hipSuccess || p == nullptr)
      return fail(I8L_ERR_HIP, fn, "hipGetSymbolAddress on device %d: %s", dev,
                  hipGetErrorString(e));
    a = reinterpret_cast<uintptr_t>(p);
    g_zero_addr[dev].store(a, std::memory_order_release);   // the same value on every race
  }
  *out = reinterpret_cast<const int32_t*>(a);
  return I8L_OK;
}

}  // namespace

I8L_API i8l_status int8_rmsnorm_quant(const uint16_t* X, const uint16_t* residual,
                                      const uint16_t* weight, int64_t M, int64_t K, float eps,
                                      int dtype, int8_t* Xq, float* sx, uint16_t* h,
                                      void* stream) {
  const char* fn = "int8_rmsnorm_quant";
  CHECK(check_shape(fn, M, K, 0));
  CHECK(check_dtype(fn, dtype));
  if (!(eps >= 0.0f) || isinf(eps))
    return fail(I8L_ERR_INVALID_ARG, fn, "eps must be finite and >= 0");
  if (M == 0) return ok();
  CHECK_PTR(X, 16);
  if (residual) CHECK_PTR(residual, 16);
  if (weight) CHECK_PTR(weight, 16);
  if (h) CHECK_PTR(h, 16);
  CHECK_PTR(Xq, 16);
  CHECK_PTR(sx, 4);
  (void)hipGetLastError();
  return hip_status(fn, i8l::launch_rmsnorm_quant(X, residual, weight, (int)M, (int)K, eps,
                                                  dtype == I8L_BF16, Xq, sx, h,
                                                  static_cast<hipStream_t>(stream)));
}

I8L_API size_t i8l_codes_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_shape("i8l_codes_workspace_bytes", M, K, N) != I8L_OK) return 0;
  return M > 0 && N > 0 ? i8l::codes_plan((int)M, (int)N, (int)K).workspace : 0;
}

I8L_API i8l_status int8_linear_codes(const int8_t* Xq, const float* sx, int64_t M, int64_t K,
                                     const int8_t* Wq, const float* sw, int64_t N,
                                     const uint16_t* bias, uint16_t* Y, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const char* fn = "int8_linear_codes";
  CHECK(check_shape(fn, M, K, N));
  if (M == 0 || N == 0) return ok();
  CHECK_PTR(Xq, 16);
  CHECK_PTR(sx, 4);
  CHECK_PTR(Wq, 16);
  CHECK_PTR(sw, 4);
  CHECK_PTR(Y, 16);
  if (bias) CHECK_PTR(bias, 2);
  const i8l::CodesPlan p = i8l::codes_plan((int)M, (int)N, (int)K);
  if (workspace) {
    CHECK_PTR(workspace, 16);
    if (workspace_bytes < p.workspace)
      return fail(I8L_ERR_WORKSPACE, fn, "workspace has %zu bytes, %zu required", workspace_bytes,
                  p.workspace);
  }
  const int32_t* zeros = nullptr;
  if (p.kind != i8l::CodesPlan::kRows && p.kind != i8l::CodesPlan::kTiles)
    CHECK(zero_words(fn, &zeros));   // the layer's own kernels read an outlier count
  (void)hipGetLastError();
  const i8l::CodesArgs a{Xq, sx, Wq, sw, bias, Y,
                         p.workspace ? static_cast<int32_t*>(workspace) : nullptr,
                         (int)M, (int)N, (int)K, 1};
  return hip_status(fn, i8l::launch_codes(a, p, zeros, static_cast<hipStream_t>(stream)));
}

// ---- The cache and attention over it ------------------------------------------------

namespace {

i8l_status check_cache(const char* fn, const i8l_kv_cache* c, i8l::Cache* out) {
  if (!c) return fail(I8L_ERR_INVALID_ARG, fn, "cache is NULL");
  CHECK(check_dtype(fn, c->dtype));
  if (c->heads < 1 || c->heads > 4096)
    return fail(I8L_ERR_INVALID_ARG, fn, "heads=%d must be in 1 .. 4096", c->heads);
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
    return fail(I8L_ERR_INVALID_ARG, fn, "head_dim=%d must be a multiple of 16 in 16 .. 256",
                c->head_dim);
  int ps = 0;
  for (int s = 4; s <= 7; ++s)
    if (c->page_size == 1 << s) ps = s;
  if (!ps)
    return fail(I8L_ERR_INVALID_ARG, fn, "page_size=%d must be 16, 32, 64 or 128", c->page_size);
  if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->n_slots < 1 || c->n_slots > INT32_MAX)
    return fail(I8L_ERR_INVALID_ARG, fn, "n_pages=%lld and n_slots=%lld must be in 1 .. 2^31 - 1",
                (long long)c->n_pages, (long long)c->n_slots);
  CHECK(check_ptr(fn, "k_codes", c->k_codes, 16));
  CHECK(check_ptr(fn, "v_codes", c->v_codes, 16));
  CHECK(check_ptr(fn, "k_scale", c->k_scale, 4));
  CHECK(check_ptr(fn, "v_scale", c->v_scale, 4));
  CHECK(check_ptr(fn, "k_tail", c->k_tail, 16));
  CHECK(check_ptr(fn, "v_tail", c->v_tail, 16));
  *out = i8l::Cache{c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_tail, c->v_tail,
                    (int)c->n_pages, (int)c->n_slots, c->heads, c->head_dim, ps,
                    c->dtype == I8L_BF16};
  return I8L_OK;
}

i8l_status check_seqs(const char* fn, const i8l_sequences* s, int ps, bool need_cu,
                      i8l::Sequences* out) {
  if (!s) return fail(I8L_ERR_INVALID_ARG, fn, "seqs is NULL");
  if (s->n < 0 || s->n > 65535)
    return fail(I8L_ERR_INVALID_ARG, fn, "n=%d must be in 0 .. 65535", s->n);
  if (s->max_pages < 0 || ((int64_t)s->max_pages << ps) >= (1 << 30))
    return fail(I8L_ERR_INVALID_ARG, fn, "max_pages=%d: max_pages * page_size must be in 0 .. 2^30",
                s->max_pages);
  *out = i8l::Sequences{s->page_table, s->lengths, s->cu, s->slots, s->n, s->max_pages};
  if (s->n == 0 || s->max_pages == 0) return I8L_OK;
  CHECK(check_ptr(fn, "page_table", s->page_table, 4));
  CHECK(check_ptr(fn, "lengths", s->lengths, 4));
  if (need_cu || s->cu) CHECK(check_ptr(fn, "cu", s->cu, 4));
  if (s->slots) CHECK(check_ptr(fn, "slots", s->slots, 4));
  return I8L_OK;
}

// Strides and extent of a [rows][heads][head_dim] tensor of 16-bit elements.
i8l_status check_rows(const char* fn, const char* name, const void* p, int64_t token_stride,
                      int64_t head_stride) {
  CHECK(check_ptr(fn, name, p, 16));
  if (token_stride < 0 || head_stride < 0 || token_stride % 8 || head_stride % 8 ||
      token_stride > (1ll << 40) || head_stride > (1ll << 40))
    return fail(I8L_ERR_INVALID_ARG, fn,
                "%s: strides %lld, %lld must be multiples of 8 elements in 0 .. 2^40", name,
                (long long)token_stride, (long long)head_stride);
  return I8L_OK;
}

i8l_status check_count(const char* fn, const char* name, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi)
    return fail(I8L_ERR_INVALID_ARG, fn, "%s=%lld must be in %lld .. %lld", name, (long long)v,
                (long long)lo, (long long)hi);
  return I8L_OK;
}

// Workgroups of a launch: one for each page, head, and keys or values, of up to 256
// threads; the threads along an axis are counted in 32 bits.
i8l_status check_pages(const char* fn, const i8l::Cache& c, int64_t tokens) {
  if (((tokens >> c.ps) + 2) * 2 * c.H >= 1 << 24)
    return fail(I8L_ERR_INVALID_ARG, fn, "%lld tokens of %d heads are too many for one call",
                (long long)tokens, c.H);
  return I8L_OK;
}

constexpr int64_t kMaxRows = 1ll << 31;
constexpr int64_t kMaxTokens = 1 << 30;

i8l_status check_attention(const char* fn, const i8l::Cache& c, int64_t q_heads, int64_t max_q,
                           int64_t max_len, int64_t window) {
  CHECK(check_count(fn, "q_heads", q_heads, 1, 65536));
  if (q_heads % c.H)
    return fail(I8L_ERR_INVALID_ARG, fn, "q_heads=%lld must be a multiple of the cache's %d heads",
                (long long)q_heads, c.H);
  CHECK(check_count(fn, "max_q", max_q, 1, kMaxTokens));
  CHECK(check_count(fn, "max_len", max_len, 0, kMaxTokens));
  CHECK(check_count(fn, "window", window, 0, INT32_MAX));
  // rows of a kv head and workgroups of a launch stay within 31 bits
  CHECK(check_count(fn, "q_heads * max_q", q_heads * max_q, 1, kMaxTokens));
  return I8L_OK;
}

}  // namespace

I8L_API i8l_status int8_cache_write(const i8l_kv_cache* cache, const i8l_sequences* seqs,
                                    const uint16_t* k, int64_t k_token_stride,
                                    int64_t k_head_stride, const uint16_t* v,
                                    int64_t v_token_stride, int64_t v_head_stride, int64_t rows,
                                    int64_t max_new, void* stream) {
  const char* fn = "int8_cache_write";
  i8l::Cache c;
  i8l::Sequences s;
  CHECK(check_cache(fn, cache, &c));
  CHECK(check_seqs(fn, seqs, c.ps, false, &s));
  CHECK(check_count(fn, "rows", rows, 0, kMaxRows));
  CHECK(check_count(fn, "max_new", max_new, 0, kMaxTokens));
  if (rows == 0 || max_new == 0 || s.B == 0 || s.max_pages == 0) return ok();
  // no sequence gets more rows than the call has, nor more tokens than its pages hold
  max_new = std::min(std::min(max_new, rows), (int64_t)s.max_pages << c.ps);
  CHECK(check_pages(fn, c, max_new));
  CHECK(check_rows(fn, "k", k, k_token_stride, k_head_stride));
  CHECK(check_rows(fn, "v", v, v_token_stride, v_head_stride));
  (void)hipGetLastError();
  return hip_status(fn, i8l::launch_cache_write(c, s, k, v, k_token_stride, k_head_stride,
                                                v_token_stride, v_head_stride, rows, (int)max_new,
                                                static_cast<hipStream_t>(stream)));
}

I8L_API i8l_status int8_cache_read(const i8l_kv_cache* cache, const i8l_sequences* seqs,
                                   uint16_t* k, uint16_t* v, int64_t rows, int64_t max_len,
                                   void* stream) {
  const char* fn = "int8_cache_read";
  i8l::Cache c;
  i8l::Sequences s;
  CHECK(check_cache(fn, cache, &c));
  CHECK(check_seqs(fn, seqs, c.ps, true, &s));
  CHECK(check_count(fn, "rows", rows, 0, kMaxRows));
  CHECK(check_count(fn, "max_len", max_len, 0, kMaxTokens));
  if (rows == 0 || max_len == 0 || s.B == 0 || s.max_pages == 0) return ok();
  max_len = std::min(std::min(max_len, rows), (int64_t)s.max_pages << c.ps);
  CHECK(check_pages(fn, c, max_len));
  CHECK_PTR(k, 16);
  CHECK_PTR(v, 16);
  (void)hipGetLastError();
  return hip_status(fn, i8l::launch_cache_read(c, s, k, v, rows, (int)max_len,
                                               static_cast<hipStream_t>(stream)));
}

I8L_API size_t i8l_attention_workspace_bytes(const i8l_kv_cache* cache, int64_t n,
                                             int64_t q_heads, int64_t max_q, int64_t max_len,
                                             int64_t window) {
  const char* fn = "i8l_attention_workspace_bytes";
  i8l::Cache c;
  if (check_cache(fn, cache, &c) != I8L_OK || check_count(fn, "n", n, 0, 65535) != I8L_OK ||
      check_attention(fn, c, q_heads, max_q, max_len, window) != I8L_OK)
    return 0;
  if (n == 0) return 0;
  window = std::min(window, kMaxTokens);
  return sizeof(float) * i8l::attention_partials((int)n, c.H, (int)(q_heads / c.H), c.D,
                                                 (int)max_q, (int)max_len, (int)window);
}

I8L_API i8l_status int8_cache_attention(const i8l_kv_cache* cache, const i8l_sequences* seqs,
                                        const uint16_t* q, int64_t q_token_stride,
                                        int64_t q_head_stride, int64_t q_heads, int64_t rows,
                                        int64_t max_q, int64_t max_len, float scale,
                                        int64_t window, const float* alibi, uint16_t* out,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "int8_cache_attention";
  i8l::Cache c;
  i8l::Sequences s;
  CHECK(check_cache(fn, cache, &c));
  CHECK(check_seqs(fn, seqs, c.ps, false, &s));
  CHECK(check_attention(fn, c, q_heads, max_q, max_len, window));
  CHECK(check_count(fn, "rows", rows, 0, kMaxRows));
  if (!isfinite(scale)) return fail(I8L_ERR_INVALID_ARG, fn, "scale must be finite");
  if (rows == 0 || s.B == 0) return ok();
  if (s.max_pages == 0)   // the kernels read the arrays of every sequence
    return fail(I8L_ERR_INVALID_ARG, fn, "max_pages=0 with %d sequences", s.B);
  CHECK(check_rows(fn, "q", q, q_token_stride, q_head_stride));
  CHECK_PTR(out, 16);
  if (alibi) CHECK_PTR(alibi, 4);
  window = std::min(window, kMaxTokens);   // (no position is as far; sums of the two stay in 32 bits)
  const size_t need = sizeof(float) * i8l::attention_partials(s.B, c.H, (int)(q_heads / c.H), c.D,
                                                              (int)max_q, (int)max_len,
                                                              (int)window);
  if (need) {
    CHECK_PTR(workspace, 16);
    if (workspace_bytes < need)
      return fail(I8L_ERR_WORKSPACE, fn, "workspace has %zu bytes, %zu required", workspace_bytes,
                  need);
  }
  (void)hipGetLastError();
  i8l::AttnArgs a{c, s, q, q_token_stride, q_head_stride, out, rows, (int)(q_heads / c.H),
                  (int)max_q, (int)max_len, (int)window, scale, alibi,
                  static_cast<float*>(workspace), 1, 0};
  return hip_status(fn, i8l::launch_attention(a, static_cast<hipStream_t>(stream)));
}
