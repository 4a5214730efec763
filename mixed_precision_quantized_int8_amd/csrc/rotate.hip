// Norms of query and key heads with the rotary rotation in the same pass, and their
// gradient (the formulas are in rotary.h).
//
// Backward, with r = 1 / rms and g = the gradient of y turned by minus its angle:
//   dw_d = sum over tokens and heads of g_d x_d r,
//   dx = r (g w - x r^2 mean_d(g_d w_d x_d));   without a norm dx = g.
// What the forward pass computed (r, the angles) is computed again: it costs less than
// reading it.
#include "rotary.h"

namespace i8l {

constexpr int kRotThreads = 256, kRotWaves = kRotThreads / 64;

template <bool BF, int LAYOUT, int IT, bool BACK>
__global__ __launch_bounds__(kRotThreads) void rotate_heads_kernel(HeadArgs a, int lanes, int groups) {
  __shared__ float s_turn[LAYOUT == kTurnOdd ? kRotWaves * kTurnRow : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task = (int64_t)blockIdx.x * kRotWaves + wave;
  const int tok = (int)(task / groups);
  if (tok >= a.rows) return;
  turn_heads<BF, LAYOUT, IT, BACK>(a, tok, a.positions[tok], (int)(task % groups), lanes,
                                   s_turn + (LAYOUT == kTurnOdd ? wave * kTurnRow : 0), lane);
}

// The gradient of one side (blockIdx.y): its waves go through the side's tokens and
// heads; each lane keeps the sums of its 16 elements of dw, which meet in the
// workgroup's row of `part`.
template <bool BF, int LAYOUT>
__global__ __launch_bounds__(kRotThreads) void rotate_grad_kernel(HeadArgs a, int lanes) {
  __shared__ float s_turn[LAYOUT == kTurnOdd ? kRotWaves * kTurnRow : 1];
  __shared__ float s_dw[kRotWaves][16 * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto& sd = a.side[blockIdx.y];
  const int per = 64 / lanes, j = lane & (lanes - 1), D = a.D;
  const int groups = (sd.n + per - 1) / per;
  const Runs at = runs_of<LAYOUT>(a.turn, j);
  float wf[16], dw[16];
  {
    v4u w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      w[r] = v4u{0, 0, 0, 0};
      if (sd.w && at.at[r] < D) w[r] = *reinterpret_cast<const v4u*>(sd.w + at.at[r]);
    }
    unpack<BF>(w, wf);
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.0f;
  }
  const int64_t tasks = (int64_t)a.rows * groups, step = (int64_t)gridDim.x * kRotWaves;
  for (int64_t task = (int64_t)blockIdx.x * kRotWaves + wave; task < tasks; task += step) {
    const int tok = (int)(task / groups), hh = (int)(task % groups) * per + lane / lanes;
    v4u p[2], q[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      p[r] = q[r] = v4u{0, 0, 0, 0};
      if (hh < sd.n && at.at[r] < D) {
        p[r] = *reinterpret_cast<const v4u*>(sd.dy + tok * sd.dy_ts + hh * sd.dy_hs + at.at[r]);
        if (sd.w) q[r] = *reinterpret_cast<const v4u*>(sd.x + tok * sd.x_ts + hh * sd.x_hs + at.at[r]);
      }
    }
    Angles<LAYOUT> angles;
    angles.of(a.turn, j, a.positions[tok], true);
    float g[16];
    unpack<BF>(p, g);
    turn<LAYOUT>(g, angles, a.turn, j, s_turn + (LAYOUT == kTurnOdd ? wave * kTurnRow : 0), lane);
    if (sd.w) {   // uniform
      float x[16];
      unpack<BF>(q, x);
      const Rms m = rms_of<BF>(x, D, lanes, a.eps);
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = x[e] * m.pre * m.r;      // normed
        dw[e] = __builtin_fmaf(g[e], x[e], dw[e]);
        g[e] *= wf[e];
        dot = __builtin_fmaf(g[e], x[e], dot);
      }
      dot = head_sum(dot, lanes) / (float)D;
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] = (g[e] - x[e] * dot) * m.r * m.pre;
    }
    pack<BF>(g, p);
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (hh < sd.n && at.at[r] < D)
        *reinterpret_cast<v4u*>(sd.y + tok * sd.y_ts + hh * sd.y_hs + at.at[r]) = p[r];
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
  for (int d = threadIdx.x; d < D; d += kRotThreads) {
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

// Groups of heads that a wave takes one after another (kIt) and waves a token.
template <bool BF, int LAYOUT, bool BACK>
void launch_rows(const HeadArgs& a, hipStream_t stream) {
  const int lanes = lanes_of(a.D), per = 64 / lanes;
  const int groups = (a.side[0].n + a.side[1].n + per - 1) / per;
  // Up to four groups a wave where there are waves enough without.
  int it = (int64_t)a.rows * groups >= 16384 ? 4 : 1;
  const int waves = (groups + it - 1) / it;
  it = (groups + waves - 1) / waves;
  const int64_t blocks = ((int64_t)a.rows * waves + kRotWaves - 1) / kRotWaves;
#define I8L_ROT(IT)                                                                         \
  hipLaunchKernelGGL((rotate_heads_kernel<BF, LAYOUT, IT, BACK>), dim3((uint32_t)blocks),   \
                     dim3(kRotThreads), 0, stream, a, lanes, waves)
  if (it == 1) I8L_ROT(1);
  else if (it == 2) I8L_ROT(2);
  else if (it == 3) I8L_ROT(3);
  else I8L_ROT(4);
#undef I8L_ROT
}

int grad_blocks(int rows, int heads, int D) {
  const int per = 64 / lanes_of(D);
  const int64_t tasks = (int64_t)rows * ((heads + per - 1) / per);
  const int64_t blocks = (tasks + 2 * kRotWaves - 1) / (2 * kRotWaves);
  return (int)(blocks < 1 ? 1 : blocks > 1024 ? 1024 : blocks);
}

template <bool BF, int LAYOUT>
void launch_grad(const HeadArgs& a, hipStream_t stream) {
  if (!a.side[0].w && !a.side[1].w) {   // a turn the other way
    launch_rows<BF, LAYOUT, true>(a, stream);
    return;
  }
  const int sides = a.side[1].n ? 2 : 1;
  const int blocks = grad_blocks(a.rows, a.side[0].n, a.D);
  hipLaunchKernelGGL((rotate_grad_kernel<BF, LAYOUT>), dim3(blocks, sides), dim3(kRotThreads), 0,
                     stream, a, lanes_of(a.D));
  hipLaunchKernelGGL((rotate_dw_kernel<BF>), dim3(a.D / 16, sides), dim3(1024), 0, stream, a, blocks);
}

}  // namespace

#define I8L_TURN(F, ...)                                                       \
  do {                                                                         \
    const TurnLayout layout = turn_layout(a.turn);                             \
    if (a.bf16) {                                                              \
      if (layout == kTurnHalves) F<true, kTurnHalves __VA_ARGS__>(a, stream);  \
      else if (layout == kTurnPairs) F<true, kTurnPairs __VA_ARGS__>(a, stream); \
      else F<true, kTurnOdd __VA_ARGS__>(a, stream);                           \
    } else {                                                                   \
      if (layout == kTurnHalves) F<false, kTurnHalves __VA_ARGS__>(a, stream); \
      else if (layout == kTurnPairs) F<false, kTurnPairs __VA_ARGS__>(a, stream); \
      else F<false, kTurnOdd __VA_ARGS__>(a, stream);                          \
    }                                                                          \
  } while (0)

hipError_t launch_rotate_heads(const HeadArgs& a, hipStream_t stream) {
  I8L_TURN(launch_rows, , false);
  return hipGetLastError();
}

size_t head_partials(int rows, int heads, int D) {
  return 2 * (size_t)grad_blocks(rows, heads, D) * D;
}

hipError_t launch_rotate_heads_backward(const HeadArgs& a, hipStream_t stream) {
  I8L_TURN(launch_grad);
  return hipGetLastError();
}

}  // namespace i8l
