// Pages of the 8-bit key/value cache as they are written (internal header of
// kvcache.hip, which explains the layout and the codes, and append.hip).
#pragma once

#include "half.h"
#include "serve.h"

namespace i8l {

constexpr int kMaxP = 128, kMaxD = 256;

struct CacheRows {
  const uint16_t* x[2];   // keys, values
  int64_t ts[2], hs[2];
  int64_t rows;
  // only where a template says PICK: row r of the call is row index[r] of the tensors
  // (NULL: r; entries are clamped to its `src` rows), and a sequence has its first
  // counts[b] rows (NULL: all)
  const int32_t* index;
  const int32_t* counts;
  int64_t src;
};
template <bool PICK>
__device__ __forceinline__ int64_t row_of(const CacheRows& x, int64_t r) {
  if constexpr (PICK)
    if (x.index) return min(max((int64_t)x.index[r], (int64_t)0), x.src - 1);
  return r;
}

// A sequence's part of a call, from device data that is clamped to what the
// tensors hold: row c0 + i is token p0 + i, up to token len - 1, the last that the
// page table has a place for (the rows after it are skipped).
struct Span {
  int64_t c0;
  int p0, len;
};
template <bool PICK>
__device__ __forceinline__ Span seq_span(const Sequences& s, int b, int ps, const CacheRows& x) {
  Span r;
  const int most = s.max_pages << ps, len = max(s.lengths[b], 0);
  int64_t c0 = s.cu ? s.cu[b] : b, c1 = s.cu ? s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), x.rows);
  c1 = min(max(c1, c0), x.rows);
  if constexpr (PICK)
    if (x.counts) c1 = min(c1, c0 + max(x.counts[b], 0));
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
template <bool BF, bool V, int BS, int NU, bool PICK>
__device__ __forceinline__ void write_page(const Cache& c, const Sequences& s, const CacheRows& x,
                                           int b, int h, int task, uint8_t* lds, uint32_t* red) {
  const int ps = c.ps, P = 1 << ps, D = c.D, D8 = D >> 3, t = threadIdx.x;
  const Span sp = seq_span<PICK>(s, b, ps, x);
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
            r[u][e] = *reinterpret_cast<const v4u*>(
                rows + row_of<PICK>(x, sp.c0 + pos - p0) * x.ts[V] + d8 * 8);
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
      const v4u r = *reinterpret_cast<const v4u*>(
          rows + row_of<PICK>(x, sp.c0 + pos - p0) * x.ts[V] + d8 * 8);
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

// Threads and units a thread for pages of `units` units.
#define I8L_CACHE_SIZES(units, F, ...)            \
  do {                                            \
    const int units_ = units;                     \
    if (units_ <= 64) F(64, 1, __VA_ARGS__);      \
    else if (units_ <= 128) F(128, 1, __VA_ARGS__); \
    else if (units_ <= 256) F(256, 1, __VA_ARGS__); \
    else if (units_ <= 512) F(256, 2, __VA_ARGS__); \
    else F(256, 4, __VA_ARGS__);                  \
  } while (0)

static_assert(kMaxP * kMaxD / 32 <= 256 * 4, "the largest page");

}  // namespace i8l
