// Norms of query and key heads with the rotary rotation in the same pass, and their
// gradient (the formulas are in rotary.h).
//
// Backward, with r = 1 / rms and g = the gradient of y turned by minus its angle:
//   dw_d = sum over tokens and heads of g_d x_d r,
//   dx = r (g w - x r^2 mean_d(g_d w_d x_d));   without a norm dx = g.
// What the forward pass computed (r, the angles) is computed again: it costs less than
// reading it.
//
// Bound by HBM: 2 bytes in and 2 out per element, the gradient 4 in and 2 out.  8192 tokens,
// 40 heads of 128, bf16, norms on queries and keys: 168 MB in 33 us, 5.1 TB/s (a large copy
// reaches 5.2); the gradient 252 MB in 54 us and 5 for the sums of the weights' gradients, 4.3
// TB/s.  One token 3.4 us, latency.
#include "rotary.h"

namespace i8l {

constexpr int kRotThreads = 256, kRotWaves = kRotThreads / 64;

template <bool BF, int LAYOUT, int SIDES, bool BACK>
__global__ __launch_bounds__(kRotThreads) void rotate_heads_kernel(HeadArgs a, int lanes, int n_tok,
                                                                   int groups, int per_wg) {
  __shared__ float2 s_cs[kTurnTokens * kMaxPairs];
  __shared__ float s_turn[LAYOUT == kTurnOdd ? kRotWaves * kTurnRow : 1];
  const int64_t tok0 = (int64_t)blockIdx.x * n_tok;
  const int g0 = blockIdx.y * per_wg;
  const int32_t* pos = a.positions + tok0;
  turn_heads<BF, LAYOUT, kRotWaves, SIDES, BACK>(
      a, tok0, (int)min((int64_t)n_tok, a.rows - tok0), [&](int i) { return pos[i]; }, g0,
      min(per_wg, groups - g0), lanes, s_cs,
      s_turn + (LAYOUT == kTurnOdd ? (threadIdx.x >> 6) * kTurnRow : 0));
}

// The gradient of one side (blockIdx.y): a workgroup takes n_tok tokens at a time, a wave
// a token's group of heads; each lane keeps the sums of its 16 elements of dw, which meet
// in the workgroup's row of `part`.
template <bool BF, int LAYOUT>
__global__ __launch_bounds__(kRotThreads) void rotate_grad_kernel(HeadArgs a, int lanes, int n_tok) {
  __shared__ float2 s_cs[kTurnTokens * kMaxPairs];
  __shared__ float s_turn[LAYOUT == kTurnOdd ? kRotWaves * kTurnRow : 1];
  __shared__ float s_dw[kRotWaves][16 * 16];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int j = lane & (lanes - 1), sub = lane / lanes, per = 64 / lanes, D = a.D, pairs = a.turn.pairs;
  const auto& sd = a.side[blockIdx.y];
  const Runs at = runs_of<LAYOUT>(a.turn, j);
  const float inv = 1.0f / (float)D;
  const int groups = (sd.n + per - 1) / per;
  float* row = s_turn + (LAYOUT == kTurnOdd ? wave * kTurnRow : 0);
  v4u w[2];
  float dw[16];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    w[r] = v4u{0, 0, 0, 0};
    if (sd.w && at.at[r] < D) w[r] = *reinterpret_cast<const v4u*>(sd.w + at.at[r]);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.0f;
  for (int64_t tok0 = (int64_t)blockIdx.x * n_tok; tok0 < a.rows; tok0 += (int64_t)gridDim.x * n_tok) {
    const int n = (int)min((int64_t)n_tok, a.rows - tok0);
    int i = 0, g = wave;   // a wave's token and group, as in turn_heads
    auto settle = [&](int& i, int& g) {
      for (; g >= groups; g -= groups) ++i;
    };
    settle(i, g);
    auto load = [&](int i, int g, v4u (&p)[2], v4u (&q)[2]) {
      const int64_t hh = g * per + sub;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        p[r] = q[r] = v4u{0, 0, 0, 0};
        if (hh < sd.n && at.at[r] < D) {
          p[r] = *reinterpret_cast<const v4u*>(sd.dy + (tok0 + i) * sd.dy_ts + hh * sd.dy_hs + at.at[r]);
          if (sd.w) q[r] = *reinterpret_cast<const v4u*>(sd.x + (tok0 + i) * sd.x_ts + hh * sd.x_hs + at.at[r]);
        }
      }
    };
    v4u p[2], q[2], p1[2], q1[2];
    if (i < n) load(i, g, p, q);
    for (int c = t; c < n * pairs; c += kRotThreads) {
      const int tok = c / pairs;
      s_cs[c] = angle(a.positions[tok0 + tok], a.turn.freqs[c - tok * pairs], a.turn.factor);
    }
    __syncthreads();
    while (i < n) {
      int i1 = i, g1 = g + kRotWaves;
      settle(i1, g1);
      if (i1 < n) load(i1, g1, p1, q1);
      const int64_t hh = g * per + sub;
      Angles<LAYOUT> angles;
      angles.of(a.turn, j, true, [&](int q, int) { return s_cs[i * pairs + q]; });
      float y[16];
      unpack<BF>(p, y);
      turn<LAYOUT>(y, angles, a.turn, j, row, lane);
      if (sd.w) {   // uniform
        float x[16], wf[16];
        unpack<BF>(q, x);
        unpack<BF>(w, wf);
        const Rms m = rms_of<BF>(x, inv, lanes, a.eps);
        over_rms(x, m);
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          dw[e] = __builtin_fmaf(y[e], x[e], dw[e]);
          y[e] *= wf[e];
          dot = __builtin_fmaf(y[e], x[e], dot);
        }
        dot = head_sum(dot, lanes) * inv;
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = __builtin_fmaf(-x[e], dot, y[e]) * m.r;
        if (__any(m.pre != 1.0f)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] *= m.pre;
        }
      }
      pack<BF>(y, p);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (hh < sd.n && at.at[r] < D)
          *reinterpret_cast<v4u*>(sd.y + (tok0 + i) * sd.y_ts + hh * sd.y_hs + at.at[r]) = p[r];
        p[r] = p1[r];
        q[r] = q1[r];
      }
      i = i1;
      g = g1;
    }
    __syncthreads();   // the angles have been read
  }
  if (!sd.w) return;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    for (int off = lanes; off < 64; off <<= 1) dw[e] += __shfl_xor(dw[e], off, 64);
  if (lane < lanes)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at.at[r] < D) s_dw[wave][at.at[r] + e] = dw[8 * r + e];
  __syncthreads();
  for (int d = t; d < D; d += kRotThreads) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kRotWaves; ++i) v += s_dw[i][d];
    a.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = v;
  }
}

// dw of one side (blockIdx.y) from the `n` rows of its partial sums, 16 elements a
// workgroup (D is a multiple of 16), in a fixed order.
template <bool BF>
__global__ __launch_bounds__(1024) void rotate_dw_kernel(HeadArgs a, int n) {
  __shared__ float s[64][17];
  const auto& sd = a.side[blockIdx.y];
  if (!sd.w) return;
  const int c = threadIdx.x & 15, row = threadIdx.x >> 4, d = blockIdx.x * 16 + c;
  const float* p = a.part + (size_t)blockIdx.y * n * a.D + d;
  float v = 0.0f;
#pragma unroll 4
  for (int i = row; i < n; i += 64) v += p[(size_t)i * a.D];
  s[row][c] = v;
  __syncthreads();
  if (row == 0) {
#pragma unroll
    for (int i = 1; i < 64; ++i) v += s[i][c];
    sd.dw[d] = from_f32<BF>(v);
  }
}

namespace {

// Four tokens a workgroup where there are workgroups enough, each wave's next heads then
// being on their way (40 heads of 128: 4096 tokens 16.3 us against 18.3 with one token, 1024
// tokens 9.9 against 9.3, 64 tokens 7.2 against 3.8).  With one, all of its heads a workgroup or,
// where that is few waves, a group of heads a wave (512 tokens 5.4 us against 5.6, one token
// 3.5 against 4.3, 2048 tokens 13.8 against 11.7).
template <bool BF, int LAYOUT, bool BACK>
void launch_rows(const HeadArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.D), groups = head_groups(a, 0) + head_groups(a, 1);
  const int n_tok = a.rows >= 2048 ? kTurnTokens : 1;
  const int per_wg = n_tok == 1 && groups > kRotWaves && (int64_t)a.rows * groups < 8192 ? kRotWaves : groups;
  const dim3 grid((a.rows + n_tok - 1) / n_tok, (groups + per_wg - 1) / per_wg);
  if (a.side[1].n)
    hipLaunchKernelGGL((rotate_heads_kernel<BF, LAYOUT, 2, BACK>), grid, dim3(kRotThreads), 0, stream, a,
                       lanes, n_tok, groups, per_wg);
  else
    hipLaunchKernelGGL((rotate_heads_kernel<BF, LAYOUT, 1, BACK>), grid, dim3(kRotThreads), 0, stream, a,
                       lanes, n_tok, groups, per_wg);
}

template <bool BF, int LAYOUT>
void launch_forward(const HeadArgs& a, hipStream_t stream) {
  launch_rows<BF, LAYOUT, false>(a, stream);
}

// (333 tokens 13.3 us with one a workgroup against 15.8 with four, 1024 tokens 24.7 against 17.6)
int grad_tokens(int rows) { return rows >= 768 ? kTurnTokens : 1; }
// At most four workgroups a compute unit and side: their rows of partial sums are read again.
int grad_blocks(int rows) {
  const int n = grad_tokens(rows), blocks = (int)(((int64_t)rows + n - 1) / n);
  return blocks < 1 ? 1 : blocks > 1024 ? 1024 : blocks;
}

template <bool BF, int LAYOUT>
void launch_grad(const HeadArgs& a, hipStream_t stream) {
  if (!a.side[0].w && !a.side[1].w) {   // a turn the other way
    launch_rows<BF, LAYOUT, true>(a, stream);
    return;
  }
  const int sides = a.side[1].n ? 2 : 1, blocks = grad_blocks(a.rows);
  hipLaunchKernelGGL((rotate_grad_kernel<BF, LAYOUT>), dim3(blocks, sides), dim3(kRotThreads), 0, stream, a,
                     lanes_of(a.D), grad_tokens(a.rows));
  hipLaunchKernelGGL((rotate_dw_kernel<BF>), dim3(a.D / 16, sides), dim3(1024), 0, stream, a, blocks);
}

}  // namespace

#define I8L_TURN(F)                                                     \
  do {                                                                  \
    const TurnLayout layout = turn_layout(a.turn);                      \
    if (a.bf16) {                                                       \
      if (layout == kTurnHalves) F<true, kTurnHalves>(a, stream);       \
      else if (layout == kTurnPairs) F<true, kTurnPairs>(a, stream);    \
      else F<true, kTurnOdd>(a, stream);                                \
    } else {                                                            \
      if (layout == kTurnHalves) F<false, kTurnHalves>(a, stream);      \
      else if (layout == kTurnPairs) F<false, kTurnPairs>(a, stream);   \
      else F<false, kTurnOdd>(a, stream);                               \
    }                                                                   \
  } while (0)

hipError_t launch_rotate_heads(const HeadArgs& a, hipStream_t stream) {
  I8L_TURN(launch_forward);
  return hipGetLastError();
}

size_t head_partials(int rows, int D) { return 2 * (size_t)grad_blocks(rows) * D; }

hipError_t launch_rotate_heads_backward(const HeadArgs& a, hipStream_t stream) {
  I8L_TURN(launch_grad);
  return hipGetLastError();
}

}  // namespace i8l
