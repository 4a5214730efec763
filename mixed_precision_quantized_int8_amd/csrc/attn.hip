// Attention over the 8-bit key/value cache: single queries and short runs of
// them against long contexts.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - slope (i - j))
// over the keys j <= i (and i - j < window) of the sequence, k_j = ks c^k_j and
// v_j = vs c^v_j with one ks and vs per page and head.
//
// The value scale of a key's page joins its exponent: with
//   s'_j = s_j + ln vs_j,   m = max_j s'_j,   w_j = exp(s'_j - m) <= 1,
//   o = sum_j w_j c^v_j / sum_j w_j / vs_j,
// so the product on the matrix cores runs on the codes themselves, and the
// rounding of w_j to 16 bits is relative to the largest contribution.  Codes
// are exact in fp16 and bf16; m and the sums are fp32.
#include <algorithm>

#include "half.h"
#include "serve.h"

namespace i8l {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kAdThreads = 256;           // 4 waves
constexpr int kAdTile = 64;               // keys per wave and step
constexpr int kAdWaves = kAdThreads / 64;
// A page of zeros has no value scale of its own: any one will do for its codes.
// The smallest a page of fp16 values can have (2^-24 / 127 and above) keeps it
// from setting the maximum m.
constexpr float kZeroScale = 0x1p-31f;
constexpr float kLeastScale = 0x1p-100f;

struct Rows {          // a sequence's part of the call
  int64_t c0;          // first row in q and out
  int n, len;          // queries, tokens held
};
__device__ __forceinline__ Rows rows_of(const AttnArgs& a, int b) {
  Rows r;
  const int64_t most = (int64_t)a.s.max_pages << a.c.ps;
  r.len = (int)min((int64_t)max(a.s.lengths[b], 0), most);
  int64_t c0 = a.s.cu ? a.s.cu[b] : b, c1 = a.s.cu ? a.s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), a.rows);
  c1 = min(max(c1, c0), a.rows);
  r.c0 = c0;
  r.n = (int)min(c1 - c0, (int64_t)a.max_q);
  return r;
}

__device__ __forceinline__ float xmax16(float v) {   // over the four 16-lane groups
  v = __builtin_fmaxf(v, __shfl_xor(v, 16, 64));
  return __builtin_fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float xsum16(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// 16 rows (queries of one kv head: token-major, the G heads of a token together)
// against a range of keys.  S^T = K . Q^T and O^T = V^T . P^T on 16x16x32
// matrix instructions; lane l holds query l & 15, and of a tile of 64 keys the
// sixteen 16 g .. 16 g + 15 of group g = l >> 4: row i of score block j is key
// 16 (i / 4) + 4 j + i % 4, so that a lane's sixteen scores are neighbours, lie
// in one page (P >= 16), and are, in order, the lane's operand for the second
// product, whose V^T operand is then 16 contiguous bytes of the [D][P] page.
//
// DP: head dimension padded to a multiple of 64 (64, 128, 256).
template <bool BF, int DP, bool ALIBI>
__global__ __launch_bounds__(kAdThreads, DP > 128 ? 1 : 2) void attn_decode_kernel(AttnArgs a) {
  constexpr int NC = DP / 64, ND = DP / 16;
  __shared__ float s_o[kAdWaves][16][DP + 4];
  __shared__ float s_m[kAdWaves][16], s_l[kAdWaves][16];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i16 = lane & 15, grp = lane >> 4;
  const int H = a.c.H, D = a.c.D, ps = a.c.ps, P = 1 << ps, G = a.G;
  const int split = blockIdx.y, h = blockIdx.x % H, r0 = blockIdx.x / H * 16, b = blockIdx.z;
  const Rows sq = rows_of(a, b);
  const int n_rows = sq.n * G;   // rows of this kv head
  if (r0 >= n_rows) return;

  // this lane's query
  const int r = r0 + i16;
  const bool live = r < n_rows;
  const int rr = live ? r : n_rows - 1;
  const int qi = rr / G, qg = rr % G;
  const int pos = sq.len - sq.n + qi;              // its position; keys <= pos
  const int hi = min(pos + 1, sq.len);
  const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
  // the tile's range (rows are in the order of their positions)
  const int q_last = (min(r0 + 16, n_rows) - 1) / G;
  const int all_hi = min(sq.len - sq.n + q_last + 1, sq.len);
  const int lo_first = a.window > 0 ? max(0, sq.len - sq.n + r0 / G + 1 - a.window) : 0;
  const int hi_first = min(sq.len - sq.n + r0 / G + 1, sq.len);       // seen by every row
  const int lo_last = a.window > 0 ? max(0, sq.len - sq.n + q_last + 1 - a.window) : 0;
  // keys of this split: whole pages of any size (128 divides begin and chunk)
  const int first = lo_first & ~127;
  const int begin = first + split * a.chunk;
  const int end = split == a.n_split - 1 ? all_hi : min(begin + a.chunk, all_hi);
  const int coded = sq.len >> ps << ps;            // tokens in complete pages

  // query operands: elements 64 c + 16 grp + 8 s .. +7 of chunk c, step s
  v4u qf[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int d = 64 * c + 16 * grp + 8 * s;
      qf[c][s] = v4u{0, 0, 0, 0};
      if (live && d < D)
        qf[c][s] = *reinterpret_cast<const v4u*>(a.q + (sq.c0 + qi) * a.q_ts +
                                                 (h * G + qg) * a.q_hs + d);
    }
  const float slope = ALIBI ? a.alibi[h * G + qg] * kLog2e : 0.0f;
  const float sc = a.scale * kLog2e;

  float m = -__builtin_inff(), l = 0.0f;   // l: this lane's keys only
  v4f o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int32_t* table = a.s.table + (size_t)b * a.s.max_pages;
  const size_t page_sz = (size_t)P * D;
  auto page_at = [&](int tok) -> int {   // -1: none
    const int g = tok >> ps;
    const int p = g < a.s.max_pages ? table[g] : -1;
    return p >= 0 && p < a.c.n_pages ? p : -1;
  };

  // scores of one tile (scaled, in log2 units, base included) to weights, the
  // running maximum and sum; then O
  auto soften = [&](v4f (&s)[4], float mul, float base, float inv_vs, int t0, bool all, int from,
                    int to, bool ok) {
    // from, to: the tile's valid keys for this lane's query and kind of page
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = __builtin_fmaf(s[j][e], mul, base);
        if (ALIBI) x = __builtin_fmaf(slope, (float)(4 * j + e), x);
        if (!all) {
          const int k = t0 + 16 * grp + 4 * j + e;
          x = ok && k >= from && k < to ? x : -__builtin_inff();
        }
        s[j][e] = x;
        // a NaN score must reach the result: maxNum would drop it here, the sum keeps it
        top = __builtin_fmaxf(top, x);
      }
    top = xmax16(top);
    const float mn = __builtin_fmaxf(m, top);
    const float ms = mn == -__builtin_inff() ? 0.0f : mn;
    if (__any(mn != m)) {
      const float f = __builtin_amdgcn_exp2f(m - ms);
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] *= f;
    }
    m = mn;
    float add = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = __builtin_amdgcn_exp2f(s[j][e] - ms);
        add += s[j][e];
      }
    if (add != 0.0f) l = __builtin_fmaf(add, inv_vs, l);   // (no 0 * NaN of a masked page)
  };
  auto weights = [&](const v4f (&s)[4], int st) -> v4u {   // contraction step st
    v4u p;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      p[2 * u] = pack2<BF>(s[2 * st + u][0], s[2 * st + u][1]);
      p[2 * u + 1] = pack2<BF>(s[2 * st + u][2], s[2 * st + u][3]);
    }
    return p;
  };

  auto coded_tile = [&](int t0) {
    const int tk = t0 + 16 * (i16 >> 2), tv = t0 + 16 * grp;   // this lane's keys as K row, as P
    const int pk = tk < coded ? page_at(tk) : -1, pv = tv < coded ? page_at(tv) : -1;
    const size_t fk = (size_t)max(pk, 0) * H + h, fv = (size_t)max(pv, 0) * H + h;
    const int8_t* kp = a.c.kc + fk * page_sz + (size_t)((tk & (P - 1)) + (i16 & 3)) * D + 16 * grp;
    const int8_t* vp = a.c.vc + fv * page_sz + (size_t)i16 * P + (tv & (P - 1));
    v4u kb[4][NC], vb[ND];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        kb[j][c] = v4u{0, 0, 0, 0};
        if (64 * c + 16 * grp < D)
          kb[j][c] = *reinterpret_cast<const v4u*>(kp + 4 * j * D + 64 * c);
      }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      vb[d] = v4u{0, 0, 0, 0};
      if (16 * d < D) vb[d] = *reinterpret_cast<const v4u*>(vp + (size_t)16 * d * P);
    }
    const float ks = a.c.ks[fv], vs0 = a.c.vs[fv];
    const float vs = vs0 == 0.0f ? kZeroScale : vs0 < kLeastScale ? kLeastScale : vs0;
    v4f s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int st = 0; st < 2; ++st)
          s[j] = mfma16<BF>(codes8<BF>(kb[j][c][2 * st], kb[j][c][2 * st + 1]), qf[c][st], s[j]);
    }
    const bool all = t0 >= lo_last && t0 + kAdTile <= min(hi_first, coded) && !__any(pv < 0);
    float base = __builtin_amdgcn_logf(vs);
    if (ALIBI) base = __builtin_fmaf(slope, (float)(tv - pos), base);
    soften(s, sc * ks, base, 1.0f / vs, t0, all, lo, min(hi, coded), pv >= 0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const v4u p = weights(s, st);
#pragma unroll
      for (int d = 0; d < ND; ++d)
        o[d] = mfma16<BF>(codes8<BF>(vb[d][2 * st], vb[d][2 * st + 1]), p, o[d]);
    }
  };

  // keys of the incomplete page, 16 bits each; values past the length are
  // whatever the slot held before and are cleared
  auto tail_tile = [&](int t0) {
    const int slot = a.s.slots ? a.s.slots[b] : b;
    const bool ok = slot >= 0 && slot < a.c.n_slots;
    const size_t f = ((size_t)(ok ? slot : 0) * H + h) * page_sz;
    const int tk = t0 + 16 * (i16 >> 2), tv = t0 + 16 * grp;
    const bool in_k = tk >= coded && tk < coded + P, in_v = tv >= coded && tv < coded + P;
    v4f s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      const uint16_t* kp = a.c.kt + f + (size_t)(in_k ? tk - coded + 4 * j + (i16 & 3) : 0) * D;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const int d = 64 * c + 16 * grp + 8 * st;
          v4u k = {0, 0, 0, 0};
          if (d < D) k = *reinterpret_cast<const v4u*>(kp + d);
          s[j] = mfma16<BF>(k, qf[c][st], s[j]);
        }
    }
    float base = 0.0f;
    if (ALIBI) base = slope * (float)(tv - pos);
    soften(s, sc, base, 1.0f, t0, false, max(lo, coded), hi, ok);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const v4u p = weights(s, st);
      const int k0 = tv + 8 * st, nv = in_v ? sq.len - k0 : 0;   // valid keys of these eight
      const uint16_t* vp = a.c.vt + f + (size_t)i16 * P + (in_v ? k0 - coded : 0);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        v4u v = {0, 0, 0, 0};
        if (16 * d < D) v = *reinterpret_cast<const v4u*>(vp + (size_t)16 * d * P);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] &= (2 * u < nv ? 0xffffu : 0u) | (2 * u + 1 < nv ? 0xffff0000u : 0u);
        o[d] = mfma16<BF>(v, p, o[d]);
      }
    }
  };

  for (int t0 = begin + wave * kAdTile; t0 < end; t0 += kAdWaves * kAdTile) {
    if (t0 + kAdTile <= lo_first) continue;
    if (t0 < coded) coded_tile(t0);
    if (t0 + kAdTile > coded) tail_tile(t0);
  }

  // the four waves' results together
  l = xsum16(l);
  if (grp == 0) {
    s_m[wave][i16] = m;
    s_l[wave][i16] = l;
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[wave][i16][16 * d + 4 * grp + e] = o[d][e];
  __syncthreads();
  const int rows = min(16, n_rows - r0);
  for (int q = t; q < rows * (D / 4); q += kAdThreads) {
    const int row = q / (D / 4), d = q % (D / 4) * 4;
    float mm = s_m[0][row];
#pragma unroll
    for (int w = 1; w < kAdWaves; ++w) mm = __builtin_fmaxf(mm, s_m[w][row]);
    const float ms = mm == -__builtin_inff() ? 0.0f : mm;
    float ll = 0.0f;
    v4f oo = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kAdWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][row] - ms);
      ll = __builtin_fmaf(s_l[w][row], f, ll);
#pragma unroll
      for (int e = 0; e < 4; ++e) oo[e] = __builtin_fmaf(s_o[w][row][d + e], f, oo[e]);
    }
    const int R = r0 + row, i = R / G, g = R % G;
    if (a.n_split == 1) {
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;   // no key at all: 0
      uint2 w;
      w.x = pack2<BF>(oo[0] * inv, oo[1] * inv);
      w.y = pack2<BF>(oo[2] * inv, oo[3] * inv);
      *reinterpret_cast<uint2*>(a.out + ((sq.c0 + i) * H * G + h * G + g) * (int64_t)D + d) = w;
    } else {
      const size_t at = (((size_t)b * H + h) * ((size_t)G * a.max_q) + R) * a.n_split + split;
      const size_t n_part = (size_t)a.s.B * H * G * a.max_q * a.n_split;
      *reinterpret_cast<v4f*>(a.part + 2 * n_part + at * D + d) = oo;
      if (d == 0) {
        a.part[2 * at] = mm;
        a.part[2 * at + 1] = ll;
      }
    }
  }
}

// The splits of one row together: one wave per row.
template <bool BF>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63, h = blockIdx.y, b = blockIdx.z;
  const int R = blockIdx.x * 4 + (threadIdx.x >> 6);
  const Rows sq = rows_of(a, b);
  if (R >= sq.n * a.G) return;
  const int H = a.c.H, D = a.c.D;
  const size_t at = (((size_t)b * H + h) * ((size_t)a.G * a.max_q) + R) * a.n_split;
  const size_t n_part = (size_t)a.s.B * H * a.G * a.max_q * a.n_split;
  const float* ml = a.part + 2 * at;
  const float* po = a.part + 2 * n_part + at * D;
  float m = -__builtin_inff();
  for (int s = lane; s < a.n_split; s += 64) m = __builtin_fmaxf(m, ml[2 * s]);
  m = wave_max(m);
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f;
  const int i = R / a.G, g = R % a.G;
  uint16_t* out = a.out + ((sq.c0 + i) * H * a.G + h * a.G + g) * (int64_t)D;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // elements lane + 64 u
  for (int s = 0; s < a.n_split; ++s) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - ms);
    l = __builtin_fmaf(ml[2 * s + 1], f, l);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (lane + 64 * u < D) acc[u] = __builtin_fmaf(po[(size_t)s * D + lane + 64 * u], f, acc[u]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (lane + 64 * u < D) out[lane + 64 * u] = from_f32<BF>(acc[u] * inv);
}

namespace {

// Keys per workgroup and the number of them.
void plan(int B, int H, int G, int max_q, int max_len, int window, int* chunk, int* n_split) {
  int range = max_len;
  if (window > 0) range = (int)std::min((int64_t)max_len, (int64_t)window + max_q + 128);
  const int64_t tiles = (int64_t)B * H * (((int64_t)G * max_q + 15) / 16);
  // at least 256 keys a workgroup (a tile per wave); about four workgroups a compute unit
  const int64_t want = 1024 / tiles > 1 ? 1024 / tiles : 1;
  int64_t c = (range + want - 1) / want;
  c = (c + 255) / 256 * 256;
  if (c < 256) c = 256;
  *chunk = (int)c;
  *n_split = (int)((range + c - 1) / c);
  if (*n_split < 1) *n_split = 1;
}

template <bool BF>
hipError_t launch_typed(const AttnArgs& a, hipStream_t stream) {
  const int D = a.c.D;
  const dim3 grid(a.c.H * ((a.G * a.max_q + 15) / 16), a.n_split, a.s.B), block(kAdThreads);
#define I8L_AD(DP)                                                                               \
  do {                                                                                           \
    if (a.alibi)                                                                                 \
      hipLaunchKernelGGL((attn_decode_kernel<BF, DP, true>), grid, block, 0, stream, a);         \
    else                                                                                         \
      hipLaunchKernelGGL((attn_decode_kernel<BF, DP, false>), grid, block, 0, stream, a);        \
  } while (0)
  if (D <= 64) I8L_AD(64);
  else if (D <= 128) I8L_AD(128);
  else I8L_AD(256);
#undef I8L_AD
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_split == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<BF>), dim3((a.G * a.max_q + 3) / 4, a.c.H, a.s.B),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t attention_partials(int B, int H, int G, int D, int max_q, int max_len, int window) {
  int chunk, n;
  plan(B, H, G, max_q, max_len, window, &chunk, &n);
  return n == 1 ? 0 : (size_t)B * H * G * max_q * n * (size_t)(D + 2);
}

hipError_t launch_attention(AttnArgs a, hipStream_t stream) {
  plan(a.s.B, a.c.H, a.G, a.max_q, a.max_len, a.window, &a.chunk, &a.n_split);
  return a.c.bf16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace i8l
