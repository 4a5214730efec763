// Product of row codes with a quantized weight where the output is small: the
// shapes that leave the streaming kernel or the 256 x 256 tiles of gemm.hip with
// too few workgroups for 256 compute units.
//
//   Y = fp16(acc * sx[i] * sw[n] / 127^2 + bias[n]),  acc = sum_k Xq[i][k] Wq[n][k]
// in int32, exact, so that neither the tile nor a split along k changes a bit.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "serve.h"

namespace i8l {

typedef int v16i_c __attribute__((ext_vector_type(16)));

__device__ __attribute__((aligned(64))) int8_t g_codes_zero[64];

__device__ __forceinline__ uint16_t codes_out(int acc, float sx, float sw, float bias) {
  return f2h((float)acc * (sx * (sw * (1.0f / 16129.0f))) + bias);
}

// ---- up to 64 rows -----------------------------------------------------------------
// 16 features a workgroup (decode_stream_kernel takes 64), eight waves that split k
// in steps of 64; a wave has up to eight steps' weights on their way at once.  MG:
// groups of 16 rows.
constexpr int kCrThreads = 512, kCrWaves = 8, kCrUnroll = 8;

template <int MG>
__global__ __launch_bounds__(kCrThreads) void codes_row_kernel(CodesArgs a) {
  __shared__ v4i s_acc[kCrWaves][MG][64];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int l16 = lane & 15, kl = (lane >> 4) * 16;
  const int M = a.M, N = a.N, K = a.K, n0 = blockIdx.x * 16;
  const int steps = (K + 63) >> 6;
  const int s0 = wave * steps / kCrWaves, s1 = (wave + 1) * steps / kCrWaves;
  const int8_t* w_row = a.Wq + (size_t)min(n0 + l16, N - 1) * K + kl;

  v4i acc[MG];
#pragma unroll
  for (int g = 0; g < MG; ++g) acc[g] = v4i{0, 0, 0, 0};
  for (int s = s0; s < s1; s += kCrUnroll) {
    v4i fb[kCrUnroll], fa[MG][kCrUnroll];
#pragma unroll
    for (int u = 0; u < kCrUnroll; ++u) {
      const int k = (s + u) * 64;
      const bool in = s + u < s1 && k + kl < K;
      fb[u] = *reinterpret_cast<const v4i*>(in ? w_row + k : g_codes_zero);
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const int row = 16 * g + l16;
        fa[g][u] = *reinterpret_cast<const v4i*>(
            in && row < M ? a.Xq + (size_t)row * K + k + kl : g_codes_zero);
      }
    }
#pragma unroll
    for (int u = 0; u < kCrUnroll; ++u)
#pragma unroll
      for (int g = 0; g < MG; ++g)
        acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[g][u], fb[u], acc[g], 0, 0, 0);
  }
#pragma unroll
  for (int g = 0; g < MG; ++g) s_acc[wave][g][lane] = acc[g];
  __syncthreads();
  // group g, lane: rows 16 g + 4 (lane / 16) + r of feature n0 + lane % 16
  for (int q = t; q < MG * 64; q += kCrThreads) {
    const int g = q >> 6, ln = q & 63, n = n0 + (ln & 15);
    v4i sum = s_acc[0][g][ln];
#pragma unroll
    for (int w = 1; w < kCrWaves; ++w) {
      const v4i p = s_acc[w][g][ln];
      sum[0] += p[0]; sum[1] += p[1]; sum[2] += p[2]; sum[3] += p[3];
    }
    if (n < N) {
      const float sw = a.sw[n], bias = a.bias ? h2f(a.bias[n]) : 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * g + 4 * (ln >> 4) + r;
        if (m < M) a.Y[(size_t)m * N + n] = codes_out(sum[r], a.sx[m], sw, bias);
      }
    }
  }
}

// ---- more rows: 128 x 64 or 128 x 128 tiles, split along k ----------------------------
// Eight waves, NB blocks of 32 x 32 each (v_mfma_i32_32x32x32_i8); steps of 128 bytes of
// k through a ring of four LDS slots, filled by direct loads three steps ahead.  With
// more than one split the int32 sums go to part [split][M][N] and codes_join_kernel
// adds them: 4 bytes times the number of splits per output, against the 64 MB that
// 256 x 256 tiles need to fill the chip.  Bound by latency while k is short (257 x 1040
// x 300 8.4 us, nine steps), then by the wait for loads of rows that several tiles share, with
// the eight waves in step (4096 x 14336 x 256: 32 us, 235 MB through L2, 7 TB/s; of the
// busy cycles the matrix cores take 24 %, LDS 18 %, and 36 % of the waves' are waits).
constexpr int kCtM = 128, kCtK = 128, kCtRing = 4, kCtThreads = 512;
constexpr int kCtA = kCtM * kCtK;

__device__ __forceinline__ int ct_swz(int row) { return ((row >> 1) & 3) | (((row >> 4) & 1) << 2); }

template <int NB>
__global__ __launch_bounds__(kCtThreads, 1) void codes_tile_kernel(CodesArgs a) {
  constexpr int kCtN = 64 * NB, kCtB = kCtN * kCtK;
  __shared__ __attribute__((aligned(1024))) int8_t smem[kCtRing * (kCtA + kCtB)];
  int8_t* const sA = smem;
  int8_t* const sB = smem + kCtRing * kCtA;
  const int M = a.M, N = a.N, K = a.K;
  const int tiles_n = (N + kCtN - 1) / kCtN, tiles = tiles_n * ((M + kCtM - 1) / kCtM);
  // Workgroup b runs on XCD b % 8.  Narrow products give each XCD a run of
  // neighbouring tiles, whose rows of codes its L2 then reads once (4096 x 14336 x 256
  // in tiles of 64: 42 -> 36 us); wide ones, tile by tile, a share of the weight (1024 x
  // 4096 x 1024: 16.5 against 18.9).
  const int items = tiles * a.n_split;
  const int item = tiles_n * kCtN > 512 ? (int)blockIdx.x : blockIdx.x % 8 * ((items + 7) / 8) + blockIdx.x / 8;
  if (item >= items) return;
  const int tile = item % tiles, split = item / tiles;
  const int m0 = tile / tiles_n * kCtM, n0 = tile % tiles_n * kCtN;
  const int nk = (K + kCtK - 1) / kCtK;
  const int s0 = (int)((int64_t)split * nk / a.n_split), s1 = (int)((int64_t)(split + 1) * nk / a.n_split);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int l32 = lane & 31, lh = lane >> 5;
  const int wm = (wave & 3) * 32, wn = (wave >> 2) * 32 * NB;

  // loads of a step: A rows 16 wave .. +15 (two of 8), B rows 8 NB wave .. +8 NB - 1,
  // 16 bytes a lane; rows past the end repeat the last
  const int8_t *ga[2], *gb[NB];
  int ka[2], kb[NB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (wave * 2 + i) * 8 + (lane >> 3);
    ka[i] = ((lane & 7) ^ ct_swz(row)) * 16;
    ga[i] = a.Xq + (size_t)min(m0 + row, M - 1) * K;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = (wave * NB + i) * 8 + (lane >> 3);
    kb[i] = ((lane & 7) ^ ct_swz(row)) * 16;
    gb[i] = a.Wq + (size_t)min(n0 + row, N - 1) * K;
  }
#define I8L_CT_LDS(p) ((__attribute__((address_space(3))) void*)(p))
  auto load_step = [&](int s) {   // past the end: the last step again, into a free slot
    const int slot = s % kCtRing, k = min(s, s1 - 1) * kCtK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int8_t* g = k + ka[i] < K ? ga[i] + k + ka[i] : g_codes_zero;
      __builtin_amdgcn_global_load_lds((const void*)g,
                                       I8L_CT_LDS(&sA[slot * kCtA + (wave * 2 + i) * 1024]), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int8_t* g = k + kb[i] < K ? gb[i] + k + kb[i] : g_codes_zero;
      __builtin_amdgcn_global_load_lds((const void*)g,
                                       I8L_CT_LDS(&sB[slot * kCtB + (wave * NB + i) * 1024]), 16, 0, 0);
    }
  };
  // the epilogue's scales, of this lane's rows m0 + wm + 8 (r / 4) + 4 lh + r % 4 and
  // features, on their way before the first step
  float sx[16], sw[NB], bias[NB];
  if (a.n_split == 1) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      sx[r] = a.sx[min(m0 + wm + 8 * (r >> 2) + 4 * lh + (r & 3), M - 1)];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = min(n0 + wn + 32 * j + l32, N - 1);
      sw[j] = a.sw[n];
      bias[j] = a.bias ? h2f(a.bias[n]) : 0.0f;
    }
  }
  v16i_c acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = v16i_c{};
  load_step(s0);
  load_step(s0 + 1);
  load_step(s0 + 2);
  const int ra = wm + l32, rw = wn + l32;
  for (int s = s0; s < s1; ++s) {
    // vmcnt: step s has landed, the 2 (2 + NB) loads of steps s + 1 and s + 2 may fly;
    // lgkmcnt(0): step s - 1 has been read from the slot that step s + 3 goes to
    __builtin_amdgcn_s_waitcnt((4 + 2 * NB) | (0x7 << 4));
    asm volatile("s_barrier" ::: "memory");   // for every wave; step s - 1 is consumed
    load_step(s + 3);
    const int slot = s % kCtRing;
    v4i fa[4], fb[4][NB];   // all of the step's operands on their way before the first product
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = 2 * q + lh;
      fa[q] = *reinterpret_cast<const v4i*>(&sA[slot * kCtA + ra * kCtK + ((c ^ ct_swz(ra)) << 4)]);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int row = rw + 32 * j;
        fb[q][j] = *reinterpret_cast<const v4i*>(&sB[slot * kCtB + row * kCtK + ((c ^ ct_swz(row)) << 4)]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[q], fb[q][j], acc[j], 0, 0, 0);
  }
  // (the loads still on their way go to LDS, which must outlive them)
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));   // vmcnt(0)
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int n = n0 + wn + 32 * j + l32;
    if (n >= N) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = m0 + wm + 8 * (r >> 2) + 4 * lh + (r & 3);
      if (m >= M) continue;
      if (a.n_split > 1) a.part[((size_t)split * M + m) * N + n] = acc[j][r];
      else a.Y[(size_t)m * N + n] = codes_out(acc[j][r], sx[r], sw[j], bias[j]);
    }
  }
}

__global__ __launch_bounds__(256) void codes_join_kernel(CodesArgs a) {
  const size_t total = (size_t)a.M * a.N, at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= total) return;
  if (a.N % 4 == 0) {   // uniform: four neighbours of one row
    v4i sum = {0, 0, 0, 0};
    for (int s = 0; s < a.n_split; ++s) {
      const v4i p = *reinterpret_cast<const v4i*>(a.part + (size_t)s * total + at);
      sum[0] += p[0]; sum[1] += p[1]; sum[2] += p[2]; sum[3] += p[3];
    }
    const int m = (int)(at / a.N), n = (int)(at % a.N);
    const float sx = a.sx[m];
    uint16_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = codes_out(sum[e], sx, a.sw[n + e], a.bias ? h2f(a.bias[n + e]) : 0.0f);
    uint2 o;
    o.x = y[0] | ((uint32_t)y[1] << 16);
    o.y = y[2] | ((uint32_t)y[3] << 16);
    *reinterpret_cast<uint2*>(a.Y + at) = o;
    return;
  }
  for (size_t i = at; i < std::min(at + 4, total); ++i) {
    int sum = 0;
    for (int s = 0; s < a.n_split; ++s) sum += a.part[(size_t)s * total + i];
    const int m = (int)(i / a.N), n = (int)(i % a.N);
    a.Y[i] = codes_out(sum, a.sx[m], a.sw[n], a.bias ? h2f(a.bias[n]) : 0.0f);
  }
}

CodesPlan codes_plan(int M, int N, int K) {
  CodesPlan p{CodesPlan::kGemm, 1, 0, 0};
  if (M <= kStreamMaxM) {
    // 16 features a workgroup until 64 of them fill the chip as well: 1 x 4096 x 8192
    // 8.3 against 10.8 us, x 16384 14.1 against 13.0; 64 x 4096 x 4096 12.6 against
    // 17.9, x 8192 21.5 against 18.4 (each wave reads all of the rows' codes).
    p.kind = (int64_t)N * (M <= 16 ? 1 : 2) <= 8192 ? CodesPlan::kRows : CodesPlan::kStream;
    return p;
  }
  // 128 x 64 tiles while 256 x 256 ones would leave three quarters of the chip idle,
  // or half of it over a short k: 256 x 4096 x 4096 18.8 against 24.2 us (skinny
  // tiles), x 16384 39.4 against 30.1; 1024 x 4096 x 2048 20.4 against 42.4 (256 x 256),
  // x 4096 29.3 against 46.7, 1024 x 14336 x 4096 no gain.
  const int64_t wide = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
  if (wide < 64 || (M > kSkinnyMaxM && wide < 128 && K <= 8192)) {
    p.kind = CodesPlan::kTiles;
    // 128 features a tile where 64 would need more workgroups than compute units (1024 x
    // 4096 x 4096 37.4 -> 29.3 us), or over a long k that is split anyway (4096 x 14336 x
    // 256 37.0 -> 34.2, 300 x 14336 x 2048 31.9 -> 27.2); else they start later and leave
    // units idle (256 x 4096 x 1024 14.1 against 15.8, x 14336 x 1024 16.6 against 21.1).
    // About the bound of 96: with 24 to 78 tiles of 64 they win or are level (300 x 8208 x
    // 1664 19.2 against 21.5, x 14336 24.9 against 26.5, x 28672 40.9 against 41.0; 64 at a
    // k of 28672 are the exception, 34 against 32 - 33), with 96 those of 128 (300 x
    // 8208 x 2048 22.1 against 21.5, x 14336 30.9 against 26.7, x 28672 53.5 against 40.9).
    const int64_t rows = (M + kCtM - 1) / kCtM, narrow = rows * ((N + 63) / 64);
    p.tile_n = narrow > 256 || (narrow >= 96 && K > 8192) ? 128 : 64;
    const int64_t tiles = rows * ((N + p.tile_n - 1) / p.tile_n);
    // a workgroup a compute unit; at least four steps of k a split, and none where k is
    // so short that the join would take longer (16 steps)
    const int nk = (K + kCtK - 1) / kCtK;
    const int64_t most = nk < 16 ? 1 : nk / 4;
    p.n_split = (int)std::max<int64_t>(std::min<int64_t>(256 / tiles, most), 1);
    if (p.n_split > 1) p.workspace = (size_t)p.n_split * M * N * sizeof(int32_t);
    return p;
  }
  if (M <= kSkinnyMaxM) {
    p.kind = CodesPlan::kSkinny;
    return p;
  }
  const GemmSplit g = gemm_split_plan(M, N, K, kGemmMaxSlices);
  p.n_split = g.split_tiles * g.S;   // partial tiles of 256 x 256
  p.workspace = (size_t)p.n_split * 256 * 256 * sizeof(int32_t);
  return p;
}

hipError_t launch_codes(CodesArgs a, const CodesPlan& p, const int32_t* zeros, hipStream_t stream) {
  if (p.kind == CodesPlan::kStream)
    return launch_stream_codes(a.Xq, a.sx, a.M, a.K, a.Wq, a.sw, a.N, a.bias, a.Y, zeros, stream);
  if (p.kind == CodesPlan::kRows) {
    const dim3 grid((a.N + 15) / 16), block(kCrThreads);
    if (a.M <= 16) hipLaunchKernelGGL(codes_row_kernel<1>, grid, block, 0, stream, a);
    else if (a.M <= 32) hipLaunchKernelGGL(codes_row_kernel<2>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(codes_row_kernel<4>, grid, block, 0, stream, a);
    return hipGetLastError();
  }
  if (p.kind == CodesPlan::kTiles) {
    a.n_split = a.part ? p.n_split : 1;
    const int tiles = ((a.M + kCtM - 1) / kCtM) * ((a.N + p.tile_n - 1) / p.tile_n);
    const dim3 grid((tiles * a.n_split + 7) / 8 * 8), block(kCtThreads);
    if (p.tile_n == 64) hipLaunchKernelGGL(codes_tile_kernel<1>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(codes_tile_kernel<2>, grid, block, 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_split == 1) return e;
    const size_t quads = ((size_t)a.M * a.N + 3) / 4;
    hipLaunchKernelGGL(codes_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  // the layer's tiles, with no outlier column (X_O and idx are read for those alone)
  GemmArgs g{a.Xq, a.Wq, a.M, a.N, a.K, a.sx, a.sw, zeros, zeros, nullptr, nullptr, a.Y, nullptr,
             a.bias, nullptr, nullptr, nullptr, a.part, a.part ? p.n_split : 0, 0, 1};
  return p.kind == CodesPlan::kSkinny ? launch_gemm_skinny(g, stream) : launch_gemm(g, stream);
}

}  // namespace i8l
