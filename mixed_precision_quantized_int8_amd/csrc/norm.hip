// Residual addition, root-mean-square norm and int8 row codes in one pass.
//
//   h = round16(x + r),   g_k = h_k w_k,   a = max_k |g_k|,
//   code_k = clamp(round_half_away(g_k * fl32(127 / a)), -127, 127),
//   sx = a / sqrt(mean_k h_k^2 + eps),      value_k = code_k * sx / 127.
//
// The norm's factor 1 / rms is the same for the whole row, so it cancels out
// of the codes and only enters the scale: the codes are decided on g, the
// exact fp32 product of two 16-bit values, and do not depend on the order of
// the sum of squares.  One read of the row then serves the sum and the maximum.
// The maximum is taken over the bits of |g|, whose order puts infinities and NaNs
// last, so that either shows in sx.  A row whose a is below 2^-93 counts as zeros
// (127 / a stays finite).  Rows of bf16 whose squares leave fp32's range are read
// again and summed scaled by 2^-80 or 2^80: 88 us instead of 77 for 4096 x 14336 of them,
// back to back.
//
// Bound by HBM: 2 + 2 bytes in, 2 + 1 bytes out per element.  4096 x 14336 fp16 with
// a residual: 70 us among the kernels of its case, 5.9 TB/s (a large copy reaches 5.15;
// part of the rows is still in the last-level cache), 77 us back to back over five
// inputs; below a few hundred rows by latency: 1 x 4096 2.7 us, 1 x 14336 4.4 us.
#include "half.h"
#include "serve.h"

namespace i8l {

constexpr int kNormChunk = 8;   // elements per 16-byte load

// h of one chunk: x + r, rounded to the 16-bit type.
template <bool BF>
__device__ __forceinline__ v4u add_chunk(v4u x, v4u r) {
#pragma unroll
  for (int d = 0; d < 4; ++d)
    x[d] = pack2<BF>(to_f32<BF>((uint16_t)x[d]) + to_f32<BF>((uint16_t)r[d]),
                     to_f32<BF>((uint16_t)(x[d] >> 16)) + to_f32<BF>((uint16_t)(r[d] >> 16)));
  return x;
}
template <bool BF>
__device__ __forceinline__ float half_of(const v4u& x, int e) {
  return to_f32<BF>((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
}
template <bool BF>
__device__ __forceinline__ void chunk_stats(const v4u& h, const v4u& w, float* sum,
                                            uint32_t* top) {
#pragma unroll
  for (int e = 0; e < kNormChunk; ++e) {
    const float hv = half_of<BF>(h, e);
    *sum = __builtin_fmaf(hv, hv, *sum);
    *top = max(*top, __builtin_bit_cast(uint32_t, hv * half_of<BF>(w, e)) & 0x7fffffffu);
  }
}
template <bool BF>
__device__ __forceinline__ uint2 chunk_codes(const v4u& h, const v4u& w, float inv) {
  int q[kNormChunk];
#pragma unroll
  for (int e = 0; e < kNormChunk; ++e)
    q[e] = quant_code(half_of<BF>(h, e) * half_of<BF>(w, e), inv);
  return make_uint2(pack4_i8(q[0], q[1], q[2], q[3]), pack4_i8(q[4], q[5], q[6], q[7]));
}

// The row's sum and maximum, from every thread's.
template <int BS>
__device__ __forceinline__ void row_totals(float* s_sum, uint32_t* s_top, float* sum,
                                           uint32_t* bits) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    *sum += __shfl_xor(*sum, off, 64);
    *bits = max(*bits, (uint32_t)__shfl_xor((int)*bits, off, 64));
  }
  if constexpr (BS > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s_sum[wave] = *sum;
      s_top[wave] = *bits;
    }
    __syncthreads();
    *sum = 0.0f;
#pragma unroll
    for (int i = 0; i < BS / 64; ++i) {
      *sum += s_sum[i];
      *bits = max(*bits, s_top[i]);
    }
  }
}

// A workgroup of BS threads per row; a thread holds NCH chunks of it, chunk
// t + i * BS (K <= BS * NCH * 8), or none (NCH 0: any K; the second pass reads the
// row again, from h where that is stored, since h may be X or R).
template <int BS, int NCH, bool BF>
__global__ __launch_bounds__(BS, NCH > 4 ? 4 : 8) void rmsnorm_quant_kernel(
    const uint16_t* X, const uint16_t* R, const uint16_t* __restrict__ W, int K, float eps,
    int8_t* __restrict__ Xq, float* __restrict__ sx, uint16_t* H) {
  constexpr bool kHold = NCH > 0;
  constexpr bool kHoldW = kHold && NCH <= 4;   // wider rows read W again (from L2)
  const int t = threadIdx.x, nch = K / kNormChunk;
  const size_t base = (size_t)blockIdx.x * K;
  const v4u ones = BF ? v4u{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}
                      : v4u{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
  auto at = [&](const uint16_t* p, int c) { return *reinterpret_cast<const v4u*>(p + c * kNormChunk); };
  auto load = [&](const uint16_t* p, int i) -> v4u {   // chunk i of this thread, zero past the row
    const int c = t + i * BS;
    return c < nch ? at(p, c) : v4u{0, 0, 0, 0};
  };

  v4u h[kHold ? NCH : 1], w[kHoldW ? NCH : 1];
  float sum = 0.0f;
  uint32_t bits = 0;
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) h[i] = load(X + base, i);
    if constexpr (kHoldW) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) w[i] = W ? load(W, i) : ones;
    }
    if (R) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) h[i] = add_chunk<BF>(h[i], load(R + base, i));
    }
    if (H) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = t + i * BS;
        if (c < nch) *reinterpret_cast<v4u*>(H + base + c * kNormChunk) = h[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      chunk_stats<BF>(h[i], kHoldW ? w[kHoldW ? i : 0] : W ? load(W, i) : ones, &sum, &bits);
  } else {
    for (int c = t; c < nch; c += BS) {
      v4u x = at(X + base, c);
      if (R) x = add_chunk<BF>(x, at(R + base, c));
      if (H) *reinterpret_cast<v4u*>(H + base + c * kNormChunk) = x;
      chunk_stats<BF>(x, W ? at(W, c) : ones, &sum, &bits);
    }
  }
  __shared__ float s_sum[BS / 64];
  __shared__ uint32_t s_top[BS / 64];
  row_totals<BS>(s_sum, s_top, &sum, &bits);
  const float a = __builtin_bit_cast(float, bits), top = a < kLeastMax ? 0.0f : a;
  const float inv = quant_scale(top);
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * BS;
      if (c < nch)
        *reinterpret_cast<uint2*>(Xq + base + c * kNormChunk) =
            chunk_codes<BF>(h[i], kHoldW ? w[kHoldW ? i : 0] : W ? at(W, c) : ones, inv);
    }
  } else {
    for (int c = t; c < nch; c += BS) {
      v4u x = at((H ? H : X) + base, c);
      if (!H && R) x = add_chunk<BF>(x, at(R + base, c));
      *reinterpret_cast<uint2*>(Xq + base + c * kNormChunk) =
          chunk_codes<BF>(x, W ? at(W, c) : ones, inv);
    }
  }
  if constexpr (BF) {
    // Squares of bf16 can leave fp32's range: then the row again (rare), scaled by a power of
    // two.  Within it, what fp32 loses of a square (2^-150) does not show in mean + eps.
    const bool small = sum < 0x1p-92f && eps < 0x1p-110f, large = !(sum < 0x1p100f);
    if (top != 0.0f && (small || large)) {   // the same for all of the workgroup
      const float by = large ? 0x1p-80f : 0x1p80f;
      sum = 0.0f;
      for (int c = t; c < nch; c += BS) {   // (each thread the chunks it had before)
        v4u x = at((H ? H : X) + base, c);
        if (!H && R) x = add_chunk<BF>(x, at(R + base, c));
#pragma unroll
        for (int e = 0; e < kNormChunk; ++e) {
          const float v = half_of<BF>(x, e) * by;   // (exact)
          sum = __builtin_fmaf(v, v, sum);
        }
      }
      __syncthreads();   // the first totals have been read
      row_totals<BS>(s_sum, s_top, &sum, &bits);
      if (t == 0)
        sx[blockIdx.x] = (float)((double)top / __builtin_sqrt((double)sum * (large ? 0x1p160 : 0x1p-160) / K + eps));
      return;
    }
  }
  // a NaN, or an infinity in h, makes the scale NaN; a row of zeros has 0 for any eps
  if (t == 0)
    sx[blockIdx.x] = top == 0.0f ? 0.0f : top / __builtin_sqrtf(sum / (float)K + eps);
}

template <int BS, int NCH>
static void launch_norm(const uint16_t* X, const uint16_t* R, const uint16_t* W, int M, int K,
                        float eps, bool bf16, int8_t* Xq, float* sx, uint16_t* H,
                        hipStream_t stream) {
  if (bf16)
    hipLaunchKernelGGL((rmsnorm_quant_kernel<BS, NCH, true>), dim3(M), dim3(BS), 0, stream, X, R, W,
                       K, eps, Xq, sx, H);
  else
    hipLaunchKernelGGL((rmsnorm_quant_kernel<BS, NCH, false>), dim3(M), dim3(BS), 0, stream, X, R,
                       W, K, eps, Xq, sx, H);
}

// Few chunks a thread: one row of 4096 takes 2.7 us with 512 threads, 3.1 with 256 and
// 6.9 with 64, 4096 rows 25.3, 25.7 and 32.1; two chunks of 8192 elements 3.4 against
// 4.1 us with four.  Up to 16384 elements four chunks cost nothing (4096 x 14336: 77 us
// back to back either way) and 16384 x 4096 87 against 91 us.
hipError_t launch_rmsnorm_quant(const uint16_t* X, const uint16_t* R, const uint16_t* W, int M,
                                int K, float eps, bool bf16, int8_t* Xq, float* sx, uint16_t* H,
                                hipStream_t stream) {
  const int nch = K / kNormChunk;
#define I8L_NORM(BS, NCH) launch_norm<BS, NCH>(X, R, W, M, K, eps, bf16, Xq, sx, H, stream)
  if (nch <= 64) I8L_NORM(64, 1);
  else if (nch <= 128) I8L_NORM(128, 1);
  else if (nch <= 256) I8L_NORM(256, 1);
  else if (nch <= 512) I8L_NORM(512, 1);
  else if (nch <= 1024) I8L_NORM(512, 2);
  else if (nch <= 2048) I8L_NORM(512, 4);
  else if (nch <= 4096) I8L_NORM(1024, 4);
  else if (nch <= 8192) I8L_NORM(1024, 8);
  else I8L_NORM(1024, 0);   // past the registers of 16 waves
#undef I8L_NORM
  return hipGetLastError();
}

}  // namespace i8l
