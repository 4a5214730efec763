// The two 16-bit element types of the serving operators (internal header).
#pragma once

#include "common.h"

namespace i8l {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// A page or row whose largest magnitude is below this counts as zeros (fp16 values
// are 2^-24 and above).
constexpr float kLeastMax = 0x1p-93f;

// fp16 (BF false) or bf16 (BF true) bits to fp32 and back, rounding to nearest
// even, overflow to infinity.
template <bool BF>
__device__ __forceinline__ float to_f32(uint16_t b) {
  if constexpr (BF) return __builtin_bit_cast(float, (uint32_t)b << 16);
  return h2f(b);
}
template <bool BF>
__device__ __forceinline__ uint16_t from_f32(float f) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, (__bf16)f);
  return f2h(f);
}
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // one v_cvt_pk
  typedef float v2f __attribute__((ext_vector_type(2)));
  if constexpr (BF) return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2b));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2h));
}

// Infinities and NaNs among two packed values: the top bit of each such half (the
// exponent's ones carry into it), those halves cleared, and one value alone (0 if finite).
template <bool BF>
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
  return ((x & 0x7fff7fffu) + (BF ? 0x00800080u : 0x04000400u)) & 0x80008000u;
}
__device__ __forceinline__ uint32_t clear_halves(uint32_t x, uint32_t odd) {
  return x & ~(odd | (odd - (odd >> 15)));
}
template <bool BF>
__device__ __forceinline__ float odd_value(uint16_t b) {
  return odd_halves<BF>(b) ? to_f32<BF>(b) : 0.0f;
}

// D = A . B + C over 32 contraction elements, 16 x 16 (A row / B column =
// lane & 15, elements 8 * (lane >> 4) .. +7; D column = lane & 15, rows
// 4 * (lane >> 4) .. +3).
template <bool BF>
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// The same over 16 contraction elements, 32 x 32 (A row / B column = lane & 31,
// elements 8 * (lane >> 5) .. +7; D column = lane & 31, register r the row
// 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)).
typedef float v16f32 __attribute__((ext_vector_type(16)));
template <bool BF>
__device__ __forceinline__ v16f32 mfma32(v4u a, v4u b, v16f32 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// The value of the lane 32 places away, with this lane's own.
__device__ __forceinline__ void halves(float v, float* lo, float* hi) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const v2u r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  *lo = __builtin_bit_cast(float, (uint32_t)r[0]);
  *hi = __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Two dwords of int8 codes (8 values) to eight 16-bit floats, exactly.
//   fp16: code + 128 as the low byte of 1024 + u (bits 0x6400 | u), less 1152;
//   bf16: through fp32, whose upper half holds an integer up to 128 in full.
template <bool BF>
__device__ __forceinline__ v4u codes8(uint32_t lo, uint32_t hi) {
  v4u r;
  if constexpr (BF) {
    const uint32_t x[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f0 = (float)(int8_t)(uint8_t)(x[i] >> (16 * e));
        const float f1 = (float)(int8_t)(uint8_t)(x[i] >> (16 * e + 8));
        r[2 * i + e] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f1),
                                             __builtin_bit_cast(uint32_t, f0), 0x07060302u);
      }
  } else {
    const v2h off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    const uint32_t x[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __builtin_amdgcn_perm(0x64646464u, x[i], 0x04010400u);
      const uint32_t b = __builtin_amdgcn_perm(0x64646464u, x[i], 0x04030402u);
      r[2 * i] = __builtin_bit_cast(uint32_t, (v2h)(__builtin_bit_cast(v2h, a) + off));
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, (v2h)(__builtin_bit_cast(v2h, b) + off));
    }
  }
  return r;
}

}  // namespace i8l
