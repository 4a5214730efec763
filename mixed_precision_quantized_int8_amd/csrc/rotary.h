// Norm and rotary rotation of one head in registers (internal header): shared by
// the row kernels (rotate.hip) and the cache's (append.hip), which therefore give the
// same bits (sums of products are explicit fused operations, not the compiler's choice).
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

// cos and sin (times the factor) of one pair's angle, position * freq reduced to half a
// turn: a 32-bit product alone is off by 0.06 radians at position 10^6.  Up to 2^20 turns
// the product is formed in two parts, each exact or below 2^-25 of a turn (the part past
// the first 24 bits of freq / 2 pi, what the product's rounding left); past that in 64
// bits, which takes three times as long.  The hardware's sine and cosine of turns are
// within 1.3e-7 over half a turn (measured).
__device__ __forceinline__ float near_turns(int pos, float freq, bool* far) {
#pragma clang fp contract(off)   // (the same bits wherever it is inlined)
  constexpr float kTurn = 0.15915494f;                              // 1 / 2 pi
  constexpr float kRest = (float)(0.15915494309189533577 - (double)kTurn);
  const float p = (float)pos, h = freq * kTurn, t = p * h;
  const float l = __builtin_fmaf(freq, kRest, __builtin_fmaf(freq, kTurn, -h));
  *far = !(__builtin_fabsf(t) < 0x1p20f && __builtin_fabsf(p) < 0x1p24f);
  return (t - __builtin_rintf(t)) + __builtin_fmaf(p, l, __builtin_fmaf(p, h, -t));
}
__device__ __forceinline__ float far_turns(int pos, float freq) {
#pragma clang fp contract(off)
  const double t = (double)pos * (double)freq * 0.15915494309189533577;
  return (float)(t - __builtin_rint(t));
}
__device__ __forceinline__ float2 turned_by(float u, float f) {
  return make_float2(f * __builtin_amdgcn_cosf(u), f * __builtin_amdgcn_sinf(u));
}
__device__ __forceinline__ float2 angle(int pos, float freq, float f) {
  bool far;
  float u = near_turns(pos, freq, &far);
  if (far) u = far_turns(pos, freq);
  return turned_by(u, f);
}

// The 8 (kTurnOdd: 16) angles of a thread, from get(i, e), pair i's cos and sin for place
// e; a place past the pairs has pair 0's (no branch, so that what get loads is on its way
// together), which turn() does not use, or for kTurnOdd what keeps its element there: 1 and
// -0.  `back`: the other way.
template <int LAYOUT>
struct Angles {
  static constexpr int N = LAYOUT == kTurnOdd ? 16 : 8;
  float c[N], s[N];
  // pair of place e, -1: none
  static __device__ __forceinline__ int pair(const Turn& r, int j, int e) {
    const int h = r.pairs;
    if (LAYOUT == kTurnHalves) return 8 * j < h ? 8 * j + e : -1;
    if (LAYOUT == kTurnPairs) return 8 * j + e < h ? 8 * j + e : -1;
    const int d = 16 * j + e;
    return d < h ? d : d < 2 * h ? d - h : -1;
  }
  template <class Get>
  __device__ __forceinline__ void of(const Turn& r, int j, bool back, Get get) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int i = pair(r, j, e);
      float2 a = make_float2(1.0f, 0.0f);
      if (r.pairs) a = get(max(i, 0), e);   // uniform
      const bool on = LAYOUT != kTurnOdd || i >= 0;
      c[e] = on ? a.x : 1.0f;
      s[e] = !on ? -0.0f : back ? -a.y : a.y;
      if (LAYOUT == kTurnOdd && 16 * j + e < r.pairs) s[e] = -s[e];   // y_a = a c + b (-s), y_b = b c + a s
    }
  }
};

// The angles of a thread at one position, freq[e] that of place e.
template <int LAYOUT>
__device__ __forceinline__ void angles_at(Angles<LAYOUT>& a, const Turn& r, int j, int pos,
                                          const float (&freq)[Angles<LAYOUT>::N]) {
  constexpr int N = Angles<LAYOUT>::N;
  float u[N];
  bool far[N], some = false;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    u[e] = near_turns(pos, freq[e], &far[e]);
    some |= far[e];
  }
  if (__any(some))
#pragma unroll
    for (int e = 0; e < N; ++e) u[e] = far[e] ? far_turns(pos, freq[e]) : u[e];
  a.of(r, j, false, [&](int, int e) { return turned_by(u[e], r.factor); });
}

// The same for kTurnOdd, where both lanes of a pair need its angle: a head's lanes form
// each of them once and pass them through `row`, the wave's part of LDS.
constexpr int kTurnRow = 64 * 17;   // floats a wave: 64 / lanes * pairs angles, or a lane's 16
                                    // elements and a 0, which also shifts the banks
__device__ __forceinline__ void odd_angles_at(Angles<kTurnOdd>& a, const Turn& r, int lanes, int j, int pos,
                                              float* row, int lane) {
  float2* head = reinterpret_cast<float2*>(row) + lane / lanes * r.pairs;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int q = j; q < r.pairs; q += lanes) head[q] = angle(pos, r.freqs[q], r.factor);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  a.of(r, j, false, [&](int i, int) { return head[i]; });
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// x turned in place: x[8 r + e] is element e of run r.  What has no pair is kept, not turned
// by 0: with an infinite neighbour it would become a NaN.  kTurnOdd: `row` is this wave's
// kTurnRow floats of LDS; what has no pair meets a 0 there, and x 1 + 0 (-0) is x, zeros and
// infinities too (selects at the end instead: 8192 tokens with a quarter of 80 turned 44 us,
// so 41).
template <int LAYOUT>
__device__ __forceinline__ void turn(float (&x)[16], const Angles<LAYOUT>& a, const Turn& r, int j,
                                     float* row, int lane) {
  if constexpr (LAYOUT == kTurnHalves) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = x[e], q = x[8 + e];
      if (8 * j < r.pairs) {
        x[e] = __builtin_fmaf(p, a.c[e], -(q * a.s[e]));
        x[8 + e] = __builtin_fmaf(p, a.s[e], q * a.c[e]);
      }
    }
  } else if constexpr (LAYOUT == kTurnPairs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = x[2 * e], q = x[2 * e + 1];
      const bool on = 8 * j + e < r.pairs;
      x[2 * e] = on ? __builtin_fmaf(p, a.c[e], -(q * a.s[e])) : p;
      x[2 * e + 1] = on ? __builtin_fmaf(p, a.s[e], q * a.c[e]) : q;
    }
  } else {
    // (a wave's LDS accesses are done in order; no other wave uses this part)
    float* mine = row + lane * 17;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int e = 0; e < 16; ++e) mine[e] = x[e];
    mine[16] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float* head = mine - 17 * j;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = 16 * j + e;
      const int other = d < r.pairs ? d + r.pairs : d - r.pairs;
      const int at = d < 2 * r.pairs ? other + (other >> 4) : 17 * j + 16;
      x[e] = __builtin_fmaf(x[e], a.c[e], head[at] * a.s[e]);
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

// The sum over a head's lanes (up to 16 neighbours), in all of them.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf,
                                                               0xf, true));
}
__device__ __forceinline__ float head_sum(float v, int lanes) {
  if (lanes > 1) v += dpp<0xb1>(v);     // neighbours
  if (lanes > 2) v += dpp<0x4e>(v);     // pairs
  if (lanes > 4) v += dpp<0x141>(v);    // fours, mirrored within 8: all of a four hold the same
  if (lanes > 8) v += dpp<0x140>(v);    // eights, mirrored within 16
  return v;
}

// 1 / rms of a head is pre * r: pre is 1 unless squares of bf16 leave fp32's range
// (then a power of two that brings them back).  A head of zeros gets 0 for any eps.
// Every lane of the wave takes part.  inv: 1 / D.
struct Rms {
  float pre, r;
};
template <bool BF>
__device__ __forceinline__ Rms rms_of(const float (&x)[16], float inv, int lanes, float eps) {
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
  const float mean = __builtin_fmaf(sum, inv, eps * pre * pre);
  return Rms{pre, mean < 0x1p-126f ? 0.0f : __builtin_amdgcn_rsqf(mean)};
}
// x / rms; a NaN stays one.
__device__ __forceinline__ void over_rms(float (&x)[16], const Rms& m) {
  if (__any(m.pre != 1.0f)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= m.pre;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] *= m.r;
}

// The heads of some tokens, by a workgroup of NW waves: tok0 .. tok0 + n_tok - 1 at
// positions pos(0) .. pos(n_tok - 1), the groups of heads from g0 on, ng of them: a group
// is 64 / lanes_of(D) heads of one side, the first side's groups first (SIDES 1: there is
// no other).  The angles are formed once, into s_cs (n_tok * pairs), and a wave takes a
// token's group at a time, with the next one's elements on their way.  BACK: the gradient
// without a norm, dy turned the other way.
constexpr int kTurnTokens = 4;   // at most n_tok
constexpr int kMaxPairs = 128;
__host__ __device__ inline int head_groups(const HeadArgs& a, int k) {
  const int per = 64 / lanes_of(a.D);
  return (a.side[k].n + per - 1) / per;
}
template <bool BF, int LAYOUT, int NW, int SIDES, bool BACK, class Pos>
__device__ __forceinline__ void turn_heads(const HeadArgs& a, int64_t tok0, int n_tok, Pos pos, int g0,
                                           int ng, int lanes, float2* s_cs, float* row) {
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int j = lane & (lanes - 1), sub = lane / lanes, per = 64 / lanes;
  const int D = a.D, pairs = a.turn.pairs, groups0 = SIDES > 1 ? head_groups(a, 0) : 0;
  const Runs at = runs_of<LAYOUT>(a.turn, j);
  const float inv = 1.0f / (float)D;
  v4u w[SIDES][2];   // this lane's weights
#pragma unroll
  for (int k = 0; k < SIDES; ++k)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      w[k][r] = v4u{0, 0, 0, 0};
      if (!BACK && a.side[k].w && at.at[r] < D)
        w[k][r] = *reinterpret_cast<const v4u*>(a.side[k].w + at.at[r]);
    }
  // (side and first head of a group are the same for the wave: they stay in scalar registers)
  auto side_of = [&](int g) { return SIDES > 1 && g0 + g >= groups0 ? 1 : 0; };
  auto head_of = [&](int g) { return (g0 + g - (side_of(g) ? groups0 : 0)) * per + sub; };
  auto load = [&](int i, int g, v4u (&p)[2]) {
    const auto& sd = a.side[side_of(g)];
    const int h = head_of(g);
    const uint16_t* x = BACK ? sd.dy + (tok0 + i) * sd.dy_ts + h * sd.dy_hs
                             : sd.x + (tok0 + i) * sd.x_ts + h * sd.x_hs;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      p[r] = v4u{0, 0, 0, 0};
      if (h < sd.n && at.at[r] < D) p[r] = *reinterpret_cast<const v4u*>(x + at.at[r]);
    }
  };
  // this wave's token and group: the wave'th of them in order, then every NW'th
  int i = 0, g = wave;
  auto settle = [&](int& i, int& g) {
    for (; g >= ng; g -= ng) ++i;
  };
  settle(i, g);
  v4u p[2], next[2];
  if (i < n_tok) load(i, g, p);
  for (int q = t; q < n_tok * pairs; q += 64 * NW) {
    const int i = q / pairs;
    s_cs[q] = angle(pos(i), a.turn.freqs[q - i * pairs], a.turn.factor);
  }
  __syncthreads();
  while (i < n_tok) {
    int i1 = i, g1 = g + NW;
    settle(i1, g1);
    if (i1 < n_tok) load(i1, g1, next);
    const int k = side_of(g);
    const auto& sd = a.side[k];
    Angles<LAYOUT> angles;
    angles.of(a.turn, j, BACK, [&](int q, int) { return s_cs[i * pairs + q]; });
    float x[16];
    unpack<BF>(p, x);
    if (!BACK && sd.w) {   // uniform
      const Rms m = rms_of<BF>(x, inv, lanes, a.eps);
      float wf[16];
      const v4u wk[2] = {w[SIDES - 1][0], w[SIDES - 1][1]};
      unpack<BF>(SIDES > 1 && k == 0 ? w[0] : wk, wf);
      over_rms(x, m);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= wf[e];
    }
    turn<LAYOUT>(x, angles, a.turn, j, row, lane);
    pack<BF>(x, p);
    const int h = head_of(g);
    uint16_t* y = sd.y + (tok0 + i) * sd.y_ts + h * sd.y_hs;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (h < sd.n && at.at[r] < D) *reinterpret_cast<v4u*>(y + at.at[r]) = p[r];
      p[r] = next[r];
    }
    i = i1;
    g = g1;
  }
}

}  // namespace i8l
