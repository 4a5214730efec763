// The 8-bit key/value cache: quantizing pages as they are written, and reading
// a cache back.
//
// A page holds P tokens of every kv head; keys and values have one scale each
// per page and head:
//   scale = fl32(absmax / 127) over the page's P * D values,
//   code = clamp(round_half_away(x * fl32(127 / absmax)), -127, 127),
//   value = code * scale.
// A page's codes are made once, when its last token arrives; until then its
// tokens are kept in 16 bits in the sequence's tail slot.  So no value is ever
// rounded twice, and what the cache holds depends on the tokens alone, not on
// how many calls brought them.  A page that holds a NaN or an infinity gets the
// scale NaN (every value of it then reads as NaN).
//
// Keys are stored [token][D], values [D][token]: each is contiguous along the
// dimension that attention sums over.
//
// Bound by HBM: 2 bytes in and 1 byte out per element written, 1 in and 2 out
// per element read back.
#include "half.h"
#include "serve.h"

namespace i8l {

constexpr int kCwThreads = 256;
constexpr int kMaxP = 128, kMaxD = 256;

struct CacheRows {
  const uint16_t* x[2];   // keys, values
  int64_t ts[2], hs[2];
  int64_t rows;
};

// A sequence's part of a call, from device data that is clamped to what the
// tensors hold: rows c0 .. c0 + n - 1 are its last n tokens.
struct Span {
  int64_t c0;
  int n, len;
};
__device__ __forceinline__ Span seq_span(const Sequences& s, int b, int ps, int64_t rows) {
  Span r;
  const int64_t most = (int64_t)s.max_pages << ps;
  r.len = (int)min((int64_t)max(s.lengths[b], 0), most);
  int64_t c0 = s.cu ? s.cu[b] : b, c1 = s.cu ? s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), rows);
  c1 = min(max(c1, c0), rows);
  if (c1 - c0 > r.len) c0 = c1 - r.len;   // more rows than tokens: the last ones
  r.c0 = c0;
  r.n = (int)(c1 - c0);
  return r;
}

// One page of one head: task j of a sequence is the j-th page that its new
// tokens touch.  Task 0 also stores the tokens that stay in the tail (after it
// has read the tokens that were there), so no two workgroups touch one tail.
// V: values (else keys).
template <bool BF, bool V>
__device__ __forceinline__ void write_page(const Cache& c, const Sequences& s, const CacheRows& x,
                                           int b, int h, int task, uint8_t* lds, float* red) {
  const int ps = c.ps, P = 1 << ps, D = c.D, D8 = D >> 3, t = threadIdx.x;
  const Span sp = seq_span(s, b, ps, x.rows);
  if (sp.n == 0) return;
  const int p0 = sp.len - sp.n, g0 = p0 >> ps, gl = (sp.len - 1) >> ps;
  const int g = g0 + task;
  if (g > gl) return;
  const int full = sp.len >> ps;   // complete pages
  const int slot = s.slots ? s.slots[b] : b;
  const bool slot_ok = slot >= 0 && slot < c.n_slots;
  uint16_t* tail = (V ? c.vt : c.kt) + ((size_t)(slot_ok ? slot : 0) * c.H + h) * P * D;
  const uint16_t* rows = x.x[V] + h * x.hs[V];
  // 8 elements (d8 * 8 ..) of the page's token p
  auto load = [&](int p, int d8) -> v4u {
    const int pos = (g << ps) + p;
    if (pos >= p0)
      return *reinterpret_cast<const v4u*>(rows + (sp.c0 + pos - p0) * x.ts[V] + d8 * 8);
    v4u r = {0, 0, 0, 0};
    if (!slot_ok) return r;
    if (!V) return *reinterpret_cast<const v4u*>(tail + p * D + d8 * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      r[e >> 1] |= (uint32_t)tail[(d8 * 8 + e) * P + p] << (16 * (e & 1));
    return r;
  };
  if (g < full) {
    const int page = s.table[(size_t)b * s.max_pages + g];
    const bool page_ok = page >= 0 && page < c.n_pages;
    float top = 0.0f;
    bool bad = false;
    for (int q = t; q < P * D8; q += kCwThreads) {
      const v4u r = load(q / D8, q % D8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = to_f32<BF>((uint16_t)(r[e >> 1] >> (16 * (e & 1))));
        bad |= !(__builtin_fabsf(f) < __builtin_inff());
        top = __builtin_fmaxf(top, __builtin_fabsf(f));
      }
    }
    if (bad) top = __builtin_inff();
    top = wave_max(top);
    if ((t & 63) == 0) red[t >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCwThreads / 64; ++i) top = __builtin_fmaxf(top, red[i]);
    const bool finite = top < __builtin_inff();
    const float inv = finite ? quant_scale(top) : 0.0f;
    int8_t* out = (V ? c.vc : c.kc) + ((size_t)(page_ok ? page : 0) * c.H + h) * P * D;
    for (int q = t; q < P * D8; q += kCwThreads) {
      const int p = q / D8, d8 = q % D8;
      const v4u r = load(p, d8);
      int k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = to_f32<BF>((uint16_t)(r[e >> 1] >> (16 * (e & 1))));
        k[e] = finite ? quant_code(f, inv) : 0;
      }
      if (!V) {
        uint2 o;
        o.x = pack4_i8(k[0], k[1], k[2], k[3]);
        o.y = pack4_i8(k[4], k[5], k[6], k[7]);
        if (page_ok) *reinterpret_cast<uint2*>(out + p * D + d8 * 8) = o;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[(d8 * 8 + e) * P + p] = (uint8_t)k[e];
      }
    }
    if (V) {
      __syncthreads();
      if (page_ok)
        for (int q = t; q < P * D / 16; q += kCwThreads)
          *reinterpret_cast<v4u*>(out + q * 16) = *reinterpret_cast<const v4u*>(lds + q * 16);
    }
    if (t == 0 && page_ok)
      (V ? c.vs : c.ks)[(size_t)page * c.H + h] = finite ? top / 127.0f : __builtin_nanf("");
  }
  if (task == 0 && gl >= full && slot_ok) {   // the last page stays incomplete
    __syncthreads();   // the old tail has been read
    const int lo = max(p0, full << ps);
    for (int q = t; q < (sp.len - lo) * D8; q += kCwThreads) {
      const int pos = lo + q / D8, d8 = q % D8, p = pos & (P - 1);
      const v4u r = *reinterpret_cast<const v4u*>(rows + (sp.c0 + pos - p0) * x.ts[V] + d8 * 8);
      if (!V) {
        *reinterpret_cast<v4u*>(tail + p * D + d8 * 8) = r;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          tail[(d8 * 8 + e) * P + p] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <bool BF>
__global__ __launch_bounds__(kCwThreads) void cache_write_kernel(Cache c, Sequences s,
                                                                 CacheRows x) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kMaxP * kMaxD];
  __shared__ float red[kCwThreads / 64];
  const int task = blockIdx.x, h = blockIdx.y >> 1, b = blockIdx.z;
  if (blockIdx.y & 1) write_page<BF, true>(c, s, x, b, h, task, lds, red);
  else write_page<BF, false>(c, s, x, b, h, task, lds, red);
}

hipError_t launch_cache_write(const Cache& c, const Sequences& s, const uint16_t* k,
                              const uint16_t* v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                              int64_t v_hs, int64_t rows, int max_new, hipStream_t stream) {
  const CacheRows x{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}, rows};
  // max_new tokens touch at most this many pages (the first may hold others before them)
  const int tasks = (max_new + (1 << c.ps) - 2) / (1 << c.ps) + 1;
  const dim3 grid(tasks, 2 * c.H, s.B), block(kCwThreads);
  if (c.bf16) hipLaunchKernelGGL(cache_write_kernel<true>, grid, block, 0, stream, c, s, x);
  else hipLaunchKernelGGL(cache_write_kernel<false>, grid, block, 0, stream, c, s, x);
  return hipGetLastError();
}

// One page of one head back to 16 bits: keys and values [rows][H][D].
template <bool BF>
__global__ __launch_bounds__(kCwThreads) void cache_read_kernel(Cache c, Sequences s,
                                                                uint16_t* __restrict__ k,
                                                                uint16_t* __restrict__ v,
                                                                int64_t rows) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[kMaxP * kMaxD];
  const int g = blockIdx.x, h = blockIdx.y >> 1, b = blockIdx.z, t = threadIdx.x;
  const bool V = blockIdx.y & 1;
  const int ps = c.ps, P = 1 << ps, D = c.D, D8 = D >> 3;
  // the sequence's rows are all of its tokens
  const int64_t most = (int64_t)s.max_pages << ps;
  const int len = (int)min((int64_t)max(s.lengths[b], 0), most);
  const int64_t c0 = max((int64_t)s.cu[b], (int64_t)0);
  const int p0 = g << ps;
  if (p0 >= len) return;
  const int n = (int)min((int64_t)min(P, len - p0), rows - (c0 + p0));
  const bool full = p0 + P <= len;
  uint16_t* out = (V ? v : k) + (c0 + p0) * c.H * D + (int64_t)h * D;
  const int64_t step = (int64_t)c.H * D;
  float scale = 0.0f;
  size_t base = 0;
  bool ok;
  if (full) {
    const int page = s.table[(size_t)b * s.max_pages + g];
    ok = page >= 0 && page < c.n_pages;
    base = ((size_t)(ok ? page : 0) * c.H + h) * P * D;
    if (ok) scale = (V ? c.vs : c.ks)[(size_t)page * c.H + h];
  } else {
    const int slot = s.slots ? s.slots[b] : b;
    ok = slot >= 0 && slot < c.n_slots;
    base = ((size_t)(ok ? slot : 0) * c.H + h) * P * D;
  }
  // 8 stored elements at q * 8 as 16-bit values
  auto stored = [&](int q) -> v4u {
    if (!ok) return v4u{0, 0, 0, 0};
    if (!full) return *reinterpret_cast<const v4u*>((V ? c.vt : c.kt) + base + q * 8);
    const uint2 w = *reinterpret_cast<const uint2*>((V ? c.vc : c.kc) + base + q * 8);
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
      r[i] = pack2<BF>((float)(int8_t)(uint8_t)x * scale, (float)(int8_t)(uint8_t)(x >> 8) * scale);
    }
    return r;
  };
  if (!V) {
    for (int q = t; q < n * D8; q += kCwThreads)
      *reinterpret_cast<v4u*>(out + (q / D8) * step + (q % D8) * 8) = stored(q);
    return;
  }
  for (int q = t; q < P * D8; q += kCwThreads) {   // [D][P] in memory: transposed through LDS
    const v4u r = stored(q);
    const int d = q * 8 >> ps, p = q * 8 & (P - 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) lds[(p + e) * D + d] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
  for (int q = t; q < n * D8; q += kCwThreads)
    *reinterpret_cast<v4u*>(out + (q / D8) * step + (q % D8) * 8) =
        *reinterpret_cast<const v4u*>(lds + q * 8);
}

hipError_t launch_cache_read(const Cache& c, const Sequences& s, uint16_t* k, uint16_t* v,
                             int64_t rows, int max_len, hipStream_t stream) {
  const int pages = (max_len + (1 << c.ps) - 1) >> c.ps;
  const dim3 grid(pages, 2 * c.H, s.B), block(kCwThreads);
  if (c.bf16) hipLaunchKernelGGL(cache_read_kernel<true>, grid, block, 0, stream, c, s, k, v, rows);
  else hipLaunchKernelGGL(cache_read_kernel<false>, grid, block, 0, stream, c, s, k, v, rows);
  return hipGetLastError();
}

}  // namespace i8l
