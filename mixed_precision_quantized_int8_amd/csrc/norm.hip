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
//
// Bound by HBM: 2 + 2 bytes in, 2 + 1 bytes out per element.
#include "half.h"
#include "serve.h"

namespace i8l {

constexpr int kNormChunk = 8;   // elements per 16-byte load

// TPR threads per row, BS / TPR rows per workgroup; a thread holds NCH chunks of
// its row, chunk t + i * TPR.  K % 16 == 0, K <= TPR * NCH * 8.
template <int BS, int TPR, int NCH, bool BF>
__global__ __launch_bounds__(BS) void rmsnorm_quant_kernel(
    const uint16_t* X, const uint16_t* R, const uint16_t* __restrict__ W, int M, int K, float eps,
    int8_t* __restrict__ Xq, float* __restrict__ sx, uint16_t* H) {   // H may be X or R
  constexpr int RPB = BS / TPR;
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * RPB + threadIdx.x / TPR;
  const bool in = row < M;
  const int nch = K / kNormChunk;
  const size_t base = (size_t)(in ? row : 0) * K;

  // chunk i of this thread in a tensor of rows at `p`, zero past the row
  auto load = [&](const uint16_t* p, int i) -> v4u {
    const int c = t + i * TPR;
    return in && c < nch ? *reinterpret_cast<const v4u*>(p + c * kNormChunk) : v4u{0, 0, 0, 0};
  };
  // wide rows read W again (from L2) rather than hold it: h alone is 4 NCH registers
  constexpr bool kHoldW = NCH <= 4;
  const v4u ones = BF ? v4u{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}
                      : v4u{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
  v4u h[NCH], w[kHoldW ? NCH : 1];
  float sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) h[i] = load(X + base, i);
  if constexpr (kHoldW) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) w[i] = W ? load(W, i) : ones;
  }
  if (R) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const v4u r = load(R + base, i);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        h[i][d] = pack2<BF>(to_f32<BF>((uint16_t)h[i][d]) + to_f32<BF>((uint16_t)r[d]),
                            to_f32<BF>((uint16_t)(h[i][d] >> 16)) +
                                to_f32<BF>((uint16_t)(r[d] >> 16)));
    }
  }
  if (H) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * TPR;
      if (in && c < nch) *reinterpret_cast<v4u*>(H + base + c * kNormChunk) = h[i];
    }
  }
  auto half = [](const v4u& x, int e) -> float {
    return to_f32<BF>((uint16_t)(x[e >> 1] >> (16 * (e & 1))));
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const v4u wi = kHoldW ? w[kHoldW ? i : 0] : W ? load(W, i) : ones;
#pragma unroll
    for (int e = 0; e < kNormChunk; ++e) {
      const float hv = half(h[i], e);
      sum = __builtin_fmaf(hv, hv, sum);
      top = __builtin_fmaxf(top, __builtin_fabsf(hv * half(wi, e)));
    }
  }
  // the row's sum and maximum
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    sum += __shfl_xor(sum, off, 64);
    top = __builtin_fmaxf(top, __shfl_xor(top, off, 64));
  }
  if constexpr (TPR > 64) {
    static_assert(RPB == 1, "rows wider than a wave take the whole workgroup");
    __shared__ float s_sum[BS / 64], s_top[BS / 64];
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s_sum[wave] = sum;
      s_top[wave] = top;
    }
    __syncthreads();
    sum = 0.0f;
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < BS / 64; ++i) {
      sum += s_sum[i];
      top = __builtin_fmaxf(top, s_top[i]);
    }
  }
  const float inv = quant_scale(top);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = t + i * TPR;
    if (in && c < nch) {
      const v4u wi = kHoldW ? w[kHoldW ? i : 0] : W ? load(W, i) : ones;
      int q[kNormChunk];
#pragma unroll
      for (int e = 0; e < kNormChunk; ++e) q[e] = quant_code(half(h[i], e) * half(wi, e), inv);
      uint2 o;
      o.x = pack4_i8(q[0], q[1], q[2], q[3]);
      o.y = pack4_i8(q[4], q[5], q[6], q[7]);
      *reinterpret_cast<uint2*>(Xq + base + c * kNormChunk) = o;
    }
  }
  // a non-finite value anywhere in the row makes the scale NaN
  if (in && t == 0) sx[row] = top / __builtin_sqrtf(sum / (float)K + eps);
}

template <int BS, int TPR, int NCH>
static void launch_norm(const uint16_t* X, const uint16_t* R, const uint16_t* W, int M, int K,
                        float eps, bool bf16, int8_t* Xq, float* sx, uint16_t* H,
                        hipStream_t stream) {
  const dim3 grid((M + BS / TPR - 1) / (BS / TPR)), block(BS);
  if (bf16)
    hipLaunchKernelGGL((rmsnorm_quant_kernel<BS, TPR, NCH, true>), grid, block, 0, stream, X, R, W,
                       M, K, eps, Xq, sx, H);
  else
    hipLaunchKernelGGL((rmsnorm_quant_kernel<BS, TPR, NCH, false>), grid, block, 0, stream, X, R,
                       W, M, K, eps, Xq, sx, H);
}

hipError_t launch_rmsnorm_quant(const uint16_t* X, const uint16_t* R, const uint16_t* W, int M,
                                int K, float eps, bool bf16, int8_t* Xq, float* sx, uint16_t* H,
                                hipStream_t stream) {
  const int nch = K / kNormChunk;
#define I8L_NORM(BS, TPR, NCH) launch_norm<BS, TPR, NCH>(X, R, W, M, K, eps, bf16, Xq, sx, H, stream)
  if (nch <= 64) I8L_NORM(256, 64, 1);
  else if (nch <= 128) I8L_NORM(256, 64, 2);
  else if (nch <= 256) I8L_NORM(256, 256, 1);
  else if (nch <= 512) I8L_NORM(256, 256, 2);
  else if (nch <= 1024) I8L_NORM(256, 256, 4);
  else if (nch <= 2048) I8L_NORM(512, 512, 4);
  else if (nch <= 4096) I8L_NORM(1024, 1024, 4);
  else if (nch <= 8192) I8L_NORM(1024, 1024, 8);
  else I8L_NORM(1024, 1024, 17);   // K <= 133136 (the layer's largest): 16642 chunks
#undef I8L_NORM
  return hipGetLastError();
}

}  // namespace i8l
