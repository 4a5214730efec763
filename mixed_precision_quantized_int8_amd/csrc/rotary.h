// Norm and rotary rotation of one head in registers (internal header): shared by
// the row kernels (rotate.hip) and the cache's (append.hip), which therefore give the
// same bits.
//
//   n_d = x_d / sqrt(mean x^2 + eps) * w_d     (without a weight: x_d),
//   pair (a, b) of frequency i, t = position * freqs[i], f a common factor:
//   y_a = f (n_a cos t - n_b sin t),  y_b = f (n_a sin t + n_b cos t),
// pairs (i, i + R / 2) or, interleaved, (2 i, 2 i + 1); elements from R = 2 * pairs on
// stay.  All of it in fp32, rounded once at the end.
//
// A thread holds 16 elements of a head as two runs of 8, lanes_of(D) neighbouring
// lanes a head.  The runs are chosen so that both elements of a pair are in one
// thread: run j and its partner at R / 2 for halves, 16 neighbours for interleaved
// pairs.  Halves that do not start at a multiple of 8 (R / 2 = 10, say) have their
// partners in other lanes: those pass through LDS.
#pragma once

#include "half.h"
#include "serve.h"

namespace i8l {

enum TurnLayout { kTurnHalves, kTurnPairs, kTurnOdd };   // kTurnOdd: halves through LDS

inline TurnLayout turn_layout(const Turn& r) {
  return r.interleaved ? kTurnPairs : r.pairs % 8 == 0 ? kTurnHalves : kTurnOdd;
}
// Where the runs of lane j (of its head) begin; at D or past it there is no run.
struct Runs {
  int at[2];
};
template <int LAYOUT>
__device__ __forceinline__ Runs runs_of(const Turn& r, int j) {
  const int h = r.pairs;
  if (LAYOUT == kTurnHalves) {
    if (8 * j < h) return Runs{{8 * j, 8 * j + h}};
    // (the rest in order: 2 h + 16 (j - h / 8))
    return Runs{{16 * j, 16 * j + 8}};
  }
  return Runs{{16 * j, 16 * j + 8}};
}

// cos and sin (times the factor) of one pair's angle.  position * freq is formed in 64
// bits, since at position 10^6 a 32-bit product is off by 0.06 radians, and reduced to
// a quarter turn there; then Taylor's series over |x| <= pi / 4 (the first terms left
// out, x^11 / 11! and x^10 / 10!, are below 2^-25).
__device__ __forceinline__ void angle(int pos, float freq, float f, float* c, float* s) {
  double t = (double)pos * (double)freq * 0.15915494309189533577;   // turns
  t -= __builtin_rint(t);
  const float u = (float)t;                          // -1/2 .. 1/2
  const float q = __builtin_rintf(4.0f * u);
  const float x = (float)(t - 0.25 * (double)q) * 6.28318530717958647693f;
  const float z = x * x;
  const float sx = x + x * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
  const float cx = 1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320))));
  const int n = (int)q;                              // quarter turns, -2 .. 2
  const bool odd = n & 1;
  const float cc = odd ? sx : cx, ss = odd ? cx : sx;
  *c = f * ((n + 1) & 2 ? -cc : cc);
  *s = f * (n & 2 ? -ss : ss);
}

// The 8 (kTurnOdd: 16) angles of a thread; an element past the pairs has angle 0 and
// factor 1.  `back`: the other way.
template <int LAYOUT>
struct Angles {
  static constexpr int N = LAYOUT == kTurnOdd ? 16 : 8;
  float c[N], s[N];
  __device__ __forceinline__ void of(const Turn& r, int j, int pos, bool back) {
    const int h = r.pairs;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      int i = 8 * j + e;
      bool on = i < h;
      bool second = false;
      if (LAYOUT == kTurnOdd) {
        const int d = 16 * j + e;
        on = d < 2 * h;
        second = d >= h;
        i = second ? d - h : d;
      }
      c[e] = 1.0f;
      s[e] = 0.0f;
      if (on) angle(pos, r.freqs[i], r.factor, &c[e], &s[e]);
      if (back) s[e] = -s[e];
      if (LAYOUT == kTurnOdd && !second) s[e] = -s[e];   // y_a = a c + b (-s), y_b = b c + a s
    }
  }
};

// x turned in place: x[8 r + e] is element e of run r.  kTurnOdd: `row` is this wave's
// kTurnRow floats of LDS.
constexpr int kTurnRow = 64 * 17;   // (a lane's 16 elements, and one that shifts the banks)
template <int LAYOUT>
__device__ __forceinline__ void turn(float (&x)[16], const Angles<LAYOUT>& a, const Turn& r, int j,
                                     float* row, int lane) {
  if constexpr (LAYOUT == kTurnHalves) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = x[e], q = x[8 + e];
      if (8 * j < r.pairs) {
        x[e] = p * a.c[e] - q * a.s[e];
        x[8 + e] = p * a.s[e] + q * a.c[e];
      }
    }
  } else if constexpr (LAYOUT == kTurnPairs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = x[2 * e], q = x[2 * e + 1];
      x[2 * e] = p * a.c[e] - q * a.s[e];
      x[2 * e + 1] = p * a.s[e] + q * a.c[e];
    }
  } else {
    // (a wave's LDS accesses are done in order; no other wave uses this part)
    float* mine = row + lane * 17;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int e = 0; e < 16; ++e) mine[e] = x[e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float* head = mine - 17 * j;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = 16 * j + e;
      const int other = d < r.pairs ? d + r.pairs : d < 2 * r.pairs ? d - r.pairs : d;
      x[e] = x[e] * a.c[e] + head[other + (other >> 4)] * a.s[e];
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool BF>
__device__ __forceinline__ void unpack(const v4u (&p)[2], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = to_f32<BF>((uint16_t)p[i >> 2][i & 3]);
    x[2 * i + 1] = to_f32<BF>((uint16_t)(p[i >> 2][i & 3] >> 16));
  }
}
template <bool BF>
__device__ __forceinline__ void pack(const float (&x)[16], v4u (&p)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = pack2<BF>(x[2 * i], x[2 * i + 1]);
}

__device__ __forceinline__ float head_sum(float v, int lanes) {   // over a head's lanes
  for (int off = 1; off < lanes; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// 1 / rms of a head is pre * r: pre is 1 unless squares of bf16 leave fp32's range
// (then a power of two that brings them back).  A head of zeros gets 0 for any eps.
// Every lane of the wave takes part.
struct Rms {
  float pre, r;
};
template <bool BF>
__device__ __forceinline__ Rms rms_of(const float (&x)[16], int D, int lanes, float eps) {
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
  sum = head_sum(sum, lanes);
  float pre = 1.0f;
  if constexpr (BF) {
    const bool small = sum < 0x1p-92f && eps < 0x1p-110f, large = !(sum < 0x1p100f);
    if (__any(small || large)) {
      pre = large ? 0x1p-80f : small ? 0x1p80f : 1.0f;
      sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = x[e] * pre;   // (exact, or below what counts)
        sum = __builtin_fmaf(v, v, sum);
      }
      sum = head_sum(sum, lanes);
    }
  }
  const float mean = sum / (float)D + eps * pre * pre;
  return Rms{pre, mean == 0.0f ? 0.0f : 1.0f / __builtin_sqrtf(mean)};
}

template <bool BF>
__device__ __forceinline__ void normed(float (&x)[16], const v4u (&w)[2], const Rms& m) {
  float wf[16];
  unpack<BF>(w, wf);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x[e] * m.pre * m.r * wf[e];
}

// The heads of one token: a wave takes 64 / lanes_of(D) of them at a time, IT times
// (`group` counts these), so that the angles are formed once for all.  `back`: the
// gradient without a norm, dy turned the other way.
template <bool BF, int LAYOUT, int IT, bool BACK>
__device__ __forceinline__ void turn_heads(const HeadArgs& a, int64_t tok, int pos, int group,
                                           int lanes, float* row, int lane) {
  const int j = lane & (lanes - 1), per = 64 / lanes;
  const int head0 = group * per * IT + lane / lanes;
  const int n0 = a.side[0].n, all = n0 + a.side[1].n, D = a.D;
  const Runs at = runs_of<LAYOUT>(a.turn, j);
  v4u p[IT][2], w[IT][2];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int hh = head0 + i * per;
    const bool k = hh >= n0;
    const auto& sd = a.side[k];
    const uint16_t* x = BACK ? sd.dy + tok * sd.dy_ts + (hh - (k ? n0 : 0)) * sd.dy_hs
                             : sd.x + tok * sd.x_ts + (hh - (k ? n0 : 0)) * sd.x_hs;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      p[i][r] = w[i][r] = v4u{0, 0, 0, 0};
      if (hh < all && at.at[r] < D) {
        p[i][r] = *reinterpret_cast<const v4u*>(x + at.at[r]);
        if (!BACK && sd.w) w[i][r] = *reinterpret_cast<const v4u*>(sd.w + at.at[r]);
      }
    }
  }
  Angles<LAYOUT> angles;
  angles.of(a.turn, j, pos, BACK);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int hh = head0 + i * per;
    const bool k = hh >= n0;
    const auto& sd = a.side[k];
    float x[16];
    unpack<BF>(p[i], x);
    if (!BACK && (a.side[0].w || a.side[1].w)) {
      const Rms m = rms_of<BF>(x, D, lanes, a.eps);
      if (sd.w) normed<BF>(x, w[i], m);
    }
    turn<LAYOUT>(x, angles, a.turn, j, row, lane);
    pack<BF>(x, p[i]);
    uint16_t* y = sd.y + tok * sd.y_ts + (hh - (k ? n0 : 0)) * sd.y_hs;
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (hh < all && at.at[r] < D) *reinterpret_cast<v4u*>(y + at.at[r]) = p[i][r];
  }
}

}  // namespace i8l
