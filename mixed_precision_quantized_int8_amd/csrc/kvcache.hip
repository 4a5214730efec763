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
#include "pages.h"

namespace i8l {

template <bool BF, int BS, int NU>
__global__ __launch_bounds__(BS) void cache_write_kernel(Cache c, Sequences s, CacheRows x) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[BS * NU * 32];   // a page of values
  __shared__ uint32_t red[BS / 64];
  // heads first: neighbours in a launch read neighbours in memory
  const uint32_t hk = blockIdx.x % (2 * c.H);
  const int task = blockIdx.x / (2 * c.H), h = hk >> 1, b = blockIdx.z;
  if (hk & 1) write_page<BF, true, BS, NU, false>(c, s, x, b, h, task, lds, red);
  else write_page<BF, false, BS, NU, false>(c, s, x, b, h, task, lds, red);
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
}  // namespace

hipError_t launch_cache_write(const Cache& c, const Sequences& s, const uint16_t* k,
                              const uint16_t* v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                              int64_t v_hs, int64_t rows, int max_new, hipStream_t stream) {
  const CacheRows x{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}, rows, nullptr, nullptr, 0};
  // max_new tokens touch at most this many pages (the first may hold others before them)
  const int tasks = (max_new + (1 << c.ps) - 2) / (1 << c.ps) + 1;
  const dim3 grid(tasks * 2 * c.H, 1, s.B);
#define I8L_W(BS, NU, BF) launch_write<BF, BS, NU>(c, s, x, grid, stream)
  if (c.bf16) I8L_CACHE_SIZES((c.D << c.ps) / 32, I8L_W, true);
  else I8L_CACHE_SIZES((c.D << c.ps) / 32, I8L_W, false);
#undef I8L_W
  return hipGetLastError();
}

hipError_t launch_cache_read(const Cache& c, const Sequences& s, uint16_t* k, uint16_t* v,
                             int64_t rows, int max_len, hipStream_t stream) {
  const int pages = (max_len + (1 << c.ps) - 1) >> c.ps;
  const dim3 grid(pages * 2 * c.H, 1, s.B);
#define I8L_R(BS, NU, BF) launch_read<BF, BS, NU>(c, s, k, v, rows, grid, stream)
  if (c.bf16) I8L_CACHE_SIZES((c.D << c.ps) / 32, I8L_R, true);
  else I8L_CACHE_SIZES((c.D << c.ps) / 32, I8L_R, false);
#undef I8L_R
  return hipGetLastError();
}

}  // namespace i8l
