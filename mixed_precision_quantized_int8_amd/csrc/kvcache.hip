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
// scale NaN (every value of it then reads as NaN); one of bf16 values that are all
// below 2^-93 counts as zeros, which keeps 127 * 2^16 / absmax and attention's
// 1 / scale inside fp32.
//
// Keys are stored [token][D], values [D][token]: each is contiguous along the
// dimension that attention sums over.
//
// Bound by HBM: 2 bytes in and 1 byte out per element written, 1 in and 2 out
// per element read back.  24.8 thousand tokens of four sequences, 32 heads of 128,
// bf16: 610 MB written in 135 us (4.5 TB/s), read back in 109 us (5.6 TB/s; a large
// copy reaches 5.15).  One token each of 16 sequences, 8 heads: 5.8 us, latency.
#include "half.h"
#include "serve.h"

namespace i8l {

constexpr int kMaxP = 128, kMaxD = 256;

struct CacheRows {
  const uint16_t* x[2];   // keys, values
  int64_t ts[2], hs[2];
  int64_t rows;
};

// A sequence's part of a call, from device data that is clamped to what the
// tensors hold: row c0 + i is token p0 + i, up to token len - 1, the last that the
// page table has a place for (the rows after it are skipped).
struct Span {
  int64_t c0;
  int p0, len;
};
__device__ __forceinline__ Span seq_span(const Sequences& s, int b, int ps, int64_t rows) {
  Span r;
  const int most = s.max_pages << ps, len = max(s.lengths[b], 0);
  int64_t c0 = s.cu ? s.cu[b] : b, c1 = s.cu ? s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), rows);
  c1 = min(max(c1, c0), rows);
  if (c1 - c0 > len) c0 = c1 - len;   // more rows than tokens: the last ones
  r.c0 = c0;
  r.p0 = len - (int)(c1 - c0);
  r.len = min(len, most);
  return r;
}

// A page of one head is cut into units of 4 tokens x 8 dimensions, a thread each:
// four 16-byte pieces of token rows on the one side, on the other 4 x 8 codes that
// are dwords of 8 codes a token (keys) or of 4 tokens a dimension (values), so that
// the two layouts differ by a transposition of 4 x 4 bytes in registers.  The
// values' dwords pass through LDS, where a page is a run of 16-byte pieces with the
// number of each exchanged by its dimension group: the threads of a wave, which hold
// different groups of the same tokens, then write to different banks.
//
// BS threads, NU units each: 64 x 1 up to 256 x 4 (P * D / 32 units).
__device__ __forceinline__ uint32_t page_piece(uint32_t c, int ps) {   // 16-byte piece number
  return c ^ ((c >> (ps - 4) >> 3) & 7);                               // c >> (ps - 4): dimension
}

// clamp(round_half_away(x * inv), -127, 127) for |x| <= absmax as a byte in bits
// 16 .. 23: with w = trunc(x * inv * 2^16), exact, (w + 2^15 - (w < 0)) >> 16; the
// product of |x| <= absmax with fl32(127 / absmax) stays below 127.5, so nothing is
// left to clamp.  (inv65: inv * 2^16.)
__device__ __forceinline__ uint32_t code_bits(float x, float inv65) {
  const int w = (int)(x * inv65);
  return (uint32_t)(w + 0x8000 + (w >> 31));
}

// 4 x 4 bytes: r[e] holds bytes (token 0 .. 3) of column e from t[token] of columns.
__device__ __forceinline__ void transpose4(const uint32_t (&t)[4], uint32_t (&r)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(t[1], t[0], 0x05010400u);   // t0.0 t1.0 t0.1 t1.1
  const uint32_t b = __builtin_amdgcn_perm(t[3], t[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(t[1], t[0], 0x07030602u);
  const uint32_t d = __builtin_amdgcn_perm(t[3], t[2], 0x07030602u);
  r[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
  r[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  r[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
  r[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// One page of one head: task j of a sequence is the j-th page that its new
// tokens touch.  Task 0 also stores the tokens that stay in the tail (after it
// has read the tokens that were there), so no two workgroups touch one tail.
// V: values (else keys).
template <bool BF, bool V, int BS, int NU>
__device__ __forceinline__ void write_page(const Cache& c, const Sequences& s, const CacheRows& x,
                                           int b, int h, int task, uint8_t* lds, uint32_t* red) {
  const int ps = c.ps, P = 1 << ps, D = c.D, D8 = D >> 3, t = threadIdx.x;
  const Span sp = seq_span(s, b, ps, x.rows);
  const int p0 = sp.p0;
  if (p0 >= sp.len) return;
  const int g0 = p0 >> ps, gl = (sp.len - 1) >> ps;
  const int g = g0 + task;
  if (g > gl) return;
  const int full = sp.len >> ps;   // complete pages
  const int slot = s.slots ? s.slots[b] : b;
  const bool slot_ok = slot >= 0 && slot < c.n_slots;
  uint16_t* tail = (V ? c.vt : c.kt) + ((size_t)(slot_ok ? slot : 0) * c.H + h) * P * D;
  const uint16_t* rows = x.x[V] + h * x.hs[V];
  if (g < full) {
    const int page = s.table[(size_t)b * s.max_pages + g];
    const bool page_ok = page >= 0 && page < c.n_pages;
    const int units = (P >> 2) * D8;
    v4u r[NU][4];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int q = t + u * BS, d8 = q % D8, t4 = q / D8 * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[u][e] = v4u{0, 0, 0, 0};
        const int pos = (g << ps) + t4 + e;
        if (q < units) {
          if (pos >= p0)
            r[u][e] = *reinterpret_cast<const v4u*>(rows + (sp.c0 + pos - p0) * x.ts[V] + d8 * 8);
          else if (slot_ok && !V)
            r[u][e] = *reinterpret_cast<const v4u*>(tail + (t4 + e) * D + d8 * 8);
          else if (slot_ok)
#pragma unroll
            for (int w = 0; w < 8; ++w)
              r[u][e][w >> 1] |= (uint32_t)tail[(d8 * 8 + w) * P + t4 + e] << (16 * (w & 1));
        }
      }
    }
    // magnitudes of both types are in the order of their bits, infinities and NaNs last
    u16x2 mag = {0, 0};
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          mag = __builtin_elementwise_max(mag, __builtin_bit_cast(u16x2, r[u][e][w] & 0x7fff7fffu));
    uint32_t bits = wave_max_u32(mag[0] > mag[1] ? mag[0] : mag[1]);
    if constexpr (BS > 64) {
      if ((t & 63) == 0) red[t >> 6] = bits;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < BS / 64; ++i) bits = max(bits, red[i]);
    }
    const bool finite = bits < (BF ? 0x7f80u : 0x7c00u);
    const float absmax = to_f32<BF>((uint16_t)bits);
    const float top = absmax < kLeastMax ? 0.0f : absmax;
    const float inv65 = (finite ? quant_scale(top) : 0.0f) * 65536.0f;
    int8_t* out = (V ? c.vc : c.kc) + ((size_t)(page_ok ? page : 0) * c.H + h) * P * D;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int q = t + u * BS, d8 = q % D8, t4 = q / D8 * 4;
      if (q >= units) continue;
      uint32_t k[2][4];   // [dimensions 0 .. 3, 4 .. 7][token]
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t z[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int d = 4 * w + y;
            const float f = to_f32<BF>((uint16_t)(r[u][e][d >> 1] >> (16 * (d & 1))));
            z[y] = code_bits(finite ? f : 0.0f, inv65);
          }
          const uint32_t lo = __builtin_amdgcn_perm(z[1], z[0], 0x0c0c0602u);
          const uint32_t hi = __builtin_amdgcn_perm(z[3], z[2], 0x06020c0cu);
          k[w][e] = lo | hi;
        }
      if (!V) {
        if (page_ok)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint2*>(out + (t4 + e) * D + d8 * 8) = make_uint2(k[0][e], k[1][e]);
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t y[4];
          transpose4(k[w], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t at = (uint32_t)(d8 * 8 + 4 * w + e) * P + t4;
            *reinterpret_cast<uint32_t*>(lds + page_piece(at >> 4, ps) * 16 + (at & 15)) = y[e];
          }
        }
      }
    }
    if (V) {
      __syncthreads();
      if (page_ok)
        for (int q = t; q < P * D / 16; q += BS)
          *reinterpret_cast<v4u*>(out + q * 16) =
              *reinterpret_cast<const v4u*>(lds + page_piece(q, ps) * 16);
    }
    if (t == 0 && page_ok)
      (V ? c.vs : c.ks)[(size_t)page * c.H + h] = finite ? top / 127.0f : __builtin_nanf("");
  }
  if (task == 0 && gl >= full && slot_ok) {   // the last page stays incomplete
    __syncthreads();   // the old tail has been read
    const int lo = max(p0, full << ps);
    for (int q = t; q < (sp.len - lo) * D8; q += BS) {
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

template <bool BF, int BS, int NU>
__global__ __launch_bounds__(BS) void cache_write_kernel(Cache c, Sequences s, CacheRows x) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[BS * NU * 32];   // a page of values
  __shared__ uint32_t red[BS / 64];
  // heads first: neighbours in a launch read neighbours in memory
  const uint32_t hk = blockIdx.x % (2 * c.H);
  const int task = blockIdx.x / (2 * c.H), h = hk >> 1, b = blockIdx.z;
  if (hk & 1) write_page<BF, true, BS, NU>(c, s, x, b, h, task, lds, red);
  else write_page<BF, false, BS, NU>(c, s, x, b, h, task, lds, red);
}

// One page of one head back to 16 bits: keys and values [rows][H][D].
template <bool BF, int BS, int NU>
__global__ __launch_bounds__(BS) void cache_read_kernel(Cache c, Sequences s,
                                                        uint16_t* __restrict__ k,
                                                        uint16_t* __restrict__ v, int64_t rows) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[BS * NU * 32];
  const uint32_t hk = blockIdx.x % (2 * c.H);
  const int g = blockIdx.x / (2 * c.H), h = hk >> 1, b = blockIdx.z, t = threadIdx.x;
  const bool V = hk & 1;
  const int ps = c.ps, P = 1 << ps, D = c.D, D8 = D >> 3, p0 = g << ps;
  // the sequence's rows are all of its tokens
  const int64_t most = (int64_t)s.max_pages << ps;
  const int len = (int)min((int64_t)max(s.lengths[b], 0), most);
  if (p0 >= len) return;
  const int64_t c0 = max((int64_t)s.cu[b], (int64_t)0) + p0;
  const int n = (int)max(min((int64_t)min(P, len - p0), rows - c0), (int64_t)0);
  uint16_t* out = (V ? v : k) + c0 * c.H * D + (int64_t)h * D;
  const int64_t step = (int64_t)c.H * D;
  if (p0 + P > len) {   // the tail, as it is
    const int slot = s.slots ? s.slots[b] : b;
    const bool ok = slot >= 0 && slot < c.n_slots;
    const uint16_t* tail = (V ? c.vt : c.kt) + ((size_t)(ok ? slot : 0) * c.H + h) * P * D;
    for (int q = t; q < n * D8; q += BS) {
      const int p = q / D8, d8 = q % D8;
      v4u r = {0, 0, 0, 0};
      if (ok && !V) r = *reinterpret_cast<const v4u*>(tail + p * D + d8 * 8);
      else if (ok)
#pragma unroll
        for (int w = 0; w < 8; ++w)
          r[w >> 1] |= (uint32_t)tail[(d8 * 8 + w) * P + p] << (16 * (w & 1));
      *reinterpret_cast<v4u*>(out + p * step + d8 * 8) = r;
    }
    return;
  }
  const int page = s.table[(size_t)b * s.max_pages + g];
  const bool ok = page >= 0 && page < c.n_pages;   // (none: zeros)
  const int8_t* in = (V ? c.vc : c.kc) + ((size_t)(ok ? page : 0) * c.H + h) * P * D;
  const float scale = ok ? (V ? c.vs : c.ks)[(size_t)page * c.H + h] : 0.0f;
  auto put = [&](int p, int d8, uint32_t lo, uint32_t hi) {   // 8 codes of one token
    if (p >= n) return;
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = (i < 2 ? lo : hi) >> (16 * (i & 1));
      const float f0 = ok ? (float)(int8_t)(uint8_t)x * scale : 0.0f;
      const float f1 = ok ? (float)(int8_t)(uint8_t)(x >> 8) * scale : 0.0f;
      r[i] = pack2<BF>(f0, f1);
    }
    *reinterpret_cast<v4u*>(out + p * step + d8 * 8) = r;
  };
  const int units = (P >> 2) * D8;
  if (!V) {
    uint2 w[NU][4];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // 8 codes of a token each, the page in order
        const int q = min(t + (4 * u + e) * BS, 4 * units - 1);
        w[u][e] = *reinterpret_cast<const uint2*>(in + q * 8);
      }
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = t + (4 * u + e) * BS;
        if (q < 4 * units) put(q / D8, q % D8, w[u][e].x, w[u][e].y);
      }
    return;
  }
  v4u w[2 * NU];
#pragma unroll
  for (int u = 0; u < 2 * NU; ++u)
    w[u] = *reinterpret_cast<const v4u*>(in + min(t + u * BS, 2 * units - 1) * 16);
#pragma unroll
  for (int u = 0; u < 2 * NU; ++u)
    if (t + u * BS < 2 * units)
      *reinterpret_cast<v4u*>(lds + page_piece(t + u * BS, ps) * 16) = w[u];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int q = t + u * BS, d8 = q % D8, t4 = q / D8 * 4;
    if (q >= units) continue;
    uint32_t k[2][4];   // [dimensions 0 .. 3, 4 .. 7][token]
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t at = (uint32_t)(d8 * 8 + 4 * y + e) * P + t4;
        z[e] = *reinterpret_cast<const uint32_t*>(lds + page_piece(at >> 4, ps) * 16 + (at & 15));
      }
      transpose4(z, k[y]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) put(t4 + e, d8, k[0][e], k[1][e]);
  }
}

namespace {
// Threads and units a thread for pages of P * D / 32 units.
template <bool BF, int BS, int NU>
void launch_write(const Cache& c, const Sequences& s, const CacheRows& x, dim3 grid,
                  hipStream_t stream) {
  hipLaunchKernelGGL((cache_write_kernel<BF, BS, NU>), grid, dim3(BS), 0, stream, c, s, x);
}
template <bool BF, int BS, int NU>
void launch_read(const Cache& c, const Sequences& s, uint16_t* k, uint16_t* v, int64_t rows,
                 dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((cache_read_kernel<BF, BS, NU>), grid, dim3(BS), 0, stream, c, s, k, v, rows);
}
#define I8L_CACHE_SIZES(F, ...)                                         \
  do {                                                                  \
    const int units = (c.D << c.ps) / 32;                               \
    if (units <= 64) F(64, 1, __VA_ARGS__);                             \
    else if (units <= 128) F(128, 1, __VA_ARGS__);                      \
    else if (units <= 256) F(256, 1, __VA_ARGS__);                      \
    else if (units <= 512) F(256, 2, __VA_ARGS__);                      \
    else F(256, 4, __VA_ARGS__);                                        \
  } while (0)
}  // namespace

static_assert(kMaxP * kMaxD / 32 <= 256 * 4, "the largest page");

hipError_t launch_cache_write(const Cache& c, const Sequences& s, const uint16_t* k,
                              const uint16_t* v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                              int64_t v_hs, int64_t rows, int max_new, hipStream_t stream) {
  const CacheRows x{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}, rows};
  // max_new tokens touch at most this many pages (the first may hold others before them)
  const int tasks = (max_new + (1 << c.ps) - 2) / (1 << c.ps) + 1;
  const dim3 grid(tasks * 2 * c.H, 1, s.B);
#define I8L_W(BS, NU, BF) launch_write<BF, BS, NU>(c, s, x, grid, stream)
  if (c.bf16) I8L_CACHE_SIZES(I8L_W, true);
  else I8L_CACHE_SIZES(I8L_W, false);
#undef I8L_W
  return hipGetLastError();
}

hipError_t launch_cache_read(const Cache& c, const Sequences& s, uint16_t* k, uint16_t* v,
                             int64_t rows, int max_len, hipStream_t stream) {
  const int pages = (max_len + (1 << c.ps) - 1) >> c.ps;
  const dim3 grid(pages * 2 * c.H, 1, s.B);
#define I8L_R(BS, NU, BF) launch_read<BF, BS, NU>(c, s, k, v, rows, grid, stream)
  if (c.bf16) I8L_CACHE_SIZES(I8L_R, true);
  else I8L_CACHE_SIZES(I8L_R, false);
#undef I8L_R
  return hipGetLastError();
}

}  // namespace i8l
