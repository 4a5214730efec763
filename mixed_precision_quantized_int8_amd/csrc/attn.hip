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
#include <type_traits>

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

// ---- runs of queries ----------------------------------------------------------
// NW waves of 32 rows each against tiles of 64 keys that the workgroup shares:
// the codes of a tile are converted to 16 bits once, on their way into LDS
// (double buffered; the next tile's codes are in flight meanwhile), and every
// wave multiplies them with its own rows on 32x32x16 matrix instructions,
// S^T = K . Q^T and O^T = V^T . P^T.  Lane l holds query l & 31; score row i of
// a block of 32 is key i with bits 2 and 3 exchanged, so that a lane's scores
// are runs of eight keys, the order in which the second product takes them.
// The running maximum moves only when a score passes it by 8 (in log2): the
// weights then stay below 2^8 and most tiles leave O alone.
constexpr int kApTile = 64;
constexpr float kApSlack = 8.0f;

template <bool BF, int DP, int NW, bool ALIBI>
__global__ __launch_bounds__(64 * NW, 2) void attn_run_kernel(AttnArgs a) {
  constexpr int NT = 64 * NW;
  constexpr int NK = DP / 16;               // contraction steps of Q . K
  constexpr int ND = DP / 32;               // 32-row blocks of O^T
  constexpr int CH = 4 * DP;                // 16-code chunks of a tile of keys, and of values
  constexpr int CPT = 2 * CH / NT;          // chunks per thread
  constexpr int KMASK = DP / 8 - 1 < 15 ? DP / 8 - 1 : 15;
  static_assert(CPT >= 1 && 2 * CH % NT == 0, "whole chunks per thread");
  // A tile of keys [key][d] and one of values [d][key] in 16 bits, in 16-byte
  // pieces exchanged within each row (by key & KMASK, by (d >> 1) & 7) so that the
  // lanes of a fragment read fall on different banks; two buffers of each.
  constexpr int kKeys = kApTile * DP * 2, kBuf = 2 * kKeys;   // bytes
  __shared__ __attribute__((aligned(1024))) uint8_t s_kv[2 * kBuf];
  // per 16 keys: score factor, log2 of the value scale, 1 / it
  __shared__ __attribute__((aligned(16))) float s_mul[2][4], s_base[2][4], s_inv[2][4];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int l32 = lane & 31, hf = lane >> 5;
  const int H = a.c.H, D = a.c.D, ps = a.c.ps, P = 1 << ps, G = a.G;
  const int b = blockIdx.z, split = blockIdx.y, h = blockIdx.x % H;
  const Rows sq = rows_of(a, b);
  const int n_rows = sq.n * G;
  // the last rows see the most keys: they go first
  const int tiles = (int)gridDim.x / H;
  const int r_wg = (tiles - 1 - (int)blockIdx.x / H) * 32 * NW;
  if (r_wg >= n_rows) return;
  const int first_pos = sq.len - sq.n;      // position of query 0

  // this lane's query; rows past the end repeat the last
  const int r_wave = r_wg + 32 * wave;
  const bool live = r_wave + l32 < n_rows;
  const int rr = min(r_wave + l32, n_rows - 1);
  const int qi = rr / G, qg = rr % G;
  const int pos = first_pos + qi;
  const int hi = min(pos + 1, sq.len);
  const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
  auto low = [&](int row) -> int {   // first key that a row sees
    const int p = first_pos + row / G;
    return a.window > 0 ? max(0, p + 1 - a.window) : 0;
  };
  auto high = [&](int row) -> int { return min(first_pos + row / G + 1, sq.len); };
  const int wv0 = min(r_wave, n_rows - 1), wv1 = min(r_wave + 31, n_rows - 1);
  const int wv_lo1 = low(wv1), wv_hi0 = high(wv0);   // what every row of the wave sees
  const int wg_lo = low(r_wg), wg_hi = high(min(r_wg + 32 * NW, n_rows) - 1);

  const int coded = sq.len >> ps << ps;
  const int first = wg_lo & ~127;
  const int begin = first + split * a.chunk;
  const int end = split == a.n_split - 1 ? wg_hi : min(begin + a.chunk, wg_hi);
  const int c_begin = max(begin, wg_lo & ~(kApTile - 1));
  const int c_end = min(end, coded);
  const int n_coded = c_end > c_begin ? (c_end - c_begin + kApTile - 1) / kApTile : 0;
  const int n_tail = end > coded && coded >= begin ? (end - coded + kApTile - 1) / kApTile : 0;
  const int n_tiles = n_coded + n_tail;

  v4u qf[NK];
#pragma unroll
  for (int s = 0; s < NK; ++s) {
    const int d = 16 * s + 8 * hf;
    qf[s] = v4u{0, 0, 0, 0};
    if (live && d < D)
      qf[s] = *reinterpret_cast<const v4u*>(a.q + (sq.c0 + qi) * a.q_ts + (h * G + qg) * a.q_hs + d);
  }
  const float sc = a.scale * kLog2e;
  const float slope = ALIBI ? a.alibi[h * G + qg] * kLog2e : 0.0f;

  // ---- staging -----------------------------------------------------------------
  const int32_t* table = a.s.table + (size_t)b * a.s.max_pages;
  const size_t page_sz = (size_t)P * D;
  // as the table has it (looked at when it is used, a step later); -1: none
  auto page_at = [&](int tok) -> int { return tok < coded ? table[tok >> ps] : -1; };
  auto exists = [&](int page) { return (uint32_t)page < (uint32_t)a.c.n_pages; };
  // chunk u of this thread: keys (rows of D codes) first, then values (rows of P);
  // its place within a page and its group of 16 keys do not change from tile to
  // tile (tiles start at multiples of 64, and P <= 128: only bit 6 of t0 moves it)
  auto is_k = [&](int u) { return t + u * NT < CH; };
  const int8_t* at0[CPT];   // the chunk in page 0
  int sub[CPT];             // its keys' offset in the tile, a multiple of 16
  bool use[CPT];
#pragma unroll
  for (int u = 0; u < CPT; ++u) {
    const int c = t + u * NT;
    const int key = is_k(u) ? c / (DP / 16) : ((c - CH) & 3) * 16;
    const int d = is_k(u) ? c % (DP / 16) * 16 : (c - CH) >> 2;
    sub[u] = key & ~15;
    use[u] = d < D;
    at0[u] = (is_k(u) ? a.c.kc : a.c.vc) + h * page_sz +
             (is_k(u) ? (key & (P - 1)) * D + d : d * P + (key & (P - 1)));
  }
  const uint32_t page_step = (uint32_t)(H * page_sz);   // at most 4096 * 128 * 256
  int pg[CPT];          // pages of the chunks to load next
  v4u raw[CPT];         // codes in flight
  int pm = -1;          // threads 0 .. 3: the page of 16-key group t
  float ks = 0.0f, vs = 0.0f;
  bool meta_ok = false;
  // a thread's value chunks run one tile behind its key chunks (see the loop):
  // step j takes keys of tile j and values of tile j - 1
  auto tile_of = [&](int u, int j) { return is_k(u) ? j : j - 1; };
  auto load_pages = [&](int j) {
#pragma unroll
    for (int u = 0; u < CPT; ++u) {
      const int i = tile_of(u, j);
      pg[u] = i >= 0 && i < n_coded ? page_at(c_begin + i * kApTile + sub[u]) : -1;
    }
    pm = j < n_coded && t < 4 ? page_at(c_begin + j * kApTile + 16 * t) : -1;
  };
  auto load_codes = [&](int j) {   // after load_pages(j)
#pragma unroll
    for (int u = 0; u < CPT; ++u) {
      const int in_page = (c_begin + tile_of(u, j) * kApTile) & (P - 1) & kApTile;
      raw[u] = v4u{0, 0, 0, 0};
      if (exists(pg[u]) && use[u])
        raw[u] = *reinterpret_cast<const v4u*>(at0[u] + (uint64_t)(uint32_t)pg[u] * page_step +
                                               (is_k(u) ? in_page * D : in_page));
    }
    meta_ok = exists(pm);
    if (meta_ok) {
      ks = a.c.ks[(size_t)pm * H + h];
      vs = a.c.vs[(size_t)pm * H + h];
    }
  };
  // byte offset of this thread's first piece of chunk u in its buffer; the second
  // piece is its neighbour (16 bytes, exchanged: ^ 16)
  auto place = [&](int u) -> uint32_t {
    const int c = t + u * NT;
    if (is_k(u)) {
      const int key = c / (DP / 16), p = c % (DP / 16) * 2;
      return (uint32_t)(key * DP * 2 + ((p ^ (key & KMASK)) << 4));
    }
    const int d = (c - CH) >> 2, p = ((c - CH) & 3) * 2;
    return (uint32_t)(kKeys + d * kApTile * 2 + ((p ^ ((d >> 1) & 7)) << 4));
  };
  auto put = [&](int i, int u, v4u x, v4u y) {
    const uint32_t at = (uint32_t)(i & 1) * kBuf + place(u);
    *reinterpret_cast<v4u*>(s_kv + at) = x;
    *reinterpret_cast<v4u*>(s_kv + (at ^ 16)) = y;
  };
  auto key0 = [&](int i) { return i < n_coded ? c_begin + i * kApTile : coded + (i - n_coded) * kApTile; };
  // step j into LDS: keys and scales of tile j, values of tile j - 1
  auto store = [&](int j) {
#pragma unroll
    for (int u = 0; u < CPT; ++u) {
      const int i = tile_of(u, j);
      if (i < 0 || i >= n_coded) continue;   // (uniform in a wave)
      put(i, u, codes8<BF>(raw[u][0], raw[u][1]), codes8<BF>(raw[u][2], raw[u][3]));
    }
    if (t < 4 && j < n_coded) {
      const float v = vs == 0.0f ? kZeroScale : vs < kLeastScale ? kLeastScale : vs;
      s_mul[j & 1][t] = meta_ok ? sc * ks : 0.0f;
      s_base[j & 1][t] = meta_ok ? __builtin_amdgcn_logf(v) : -__builtin_inff();   // hides the group
      s_inv[j & 1][t] = meta_ok ? 1.0f / v : 0.0f;
    }
    // keys coded + 64 j .. of the incomplete page, as they are; past the length zeros
    if (j >= n_coded && j - 1 < n_tiles) {
      const int slot = a.s.slots ? a.s.slots[b] : b;
      const bool ok = slot >= 0 && slot < a.c.n_slots;
      const size_t f = ((size_t)(ok ? slot : 0) * H + h) * page_sz;
#pragma unroll
      for (int u = 0; u < CPT; ++u) {
        const int i = tile_of(u, j), c = t + u * NT;
        if (i < n_coded || i >= n_tiles) continue;
        const int t0 = key0(i), r0 = t0 - coded, n = ok ? min(sq.len - t0, kApTile) : 0;
        v4u x[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {   // two 16-byte pieces
          x[w] = v4u{0, 0, 0, 0};
          if (is_k(u)) {
            const int key = c / (DP / 16), p = c % (DP / 16) * 2 + w;
            if (key < n && p * 8 < D)
              x[w] = *reinterpret_cast<const v4u*>(a.c.kt + f + (size_t)(r0 + key) * D + p * 8);
          } else {
            const int d = (c - CH) >> 2, p = ((c - CH) & 3) * 2 + w, nv = n - p * 8;
            if (nv > 0 && d < D)
              x[w] = *reinterpret_cast<const v4u*>(a.c.vt + f + (size_t)d * P + r0 + p * 8);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              x[w][q] &= (2 * q < nv ? 0xffffu : 0u) | (2 * q + 1 < nv ? 0xffff0000u : 0u);
          }
        }
        put(i, u, x[0], x[1]);
      }
      if (t < 4 && j < n_tiles) {
        s_mul[j & 1][t] = ok ? sc : 0.0f;
        s_base[j & 1][t] = ok ? 0.0f : -__builtin_inff();
        s_inv[j & 1][t] = ok ? 1.0f : 0.0f;
      }
    }
  };

  // ---- a tile ------------------------------------------------------------------
  float m = -__builtin_inff(), l = 0.0f;   // l: this lane's keys
  v16f32 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = v16f32{};
  const int row_k = (l32 & 0x13) | ((l32 & 4) << 1) | ((l32 & 8) >> 1);   // key of score row l32

  v16f32 s[2];
  v4u p[4];
  // S^T of one tile and O^T of the one before it (either may be left out): the
  // fragments come from LDS kAhead products before their use, in program order
  auto multiply = [&](auto with_k, auto with_v, int ik, int iv) {
    constexpr int nk = decltype(with_k)::value ? 2 * NK : 0;
    constexpr int nv = decltype(with_v)::value ? 4 * ND : 0;
    constexpr int kAhead = 6;
    // offsets of the first fragments; the others differ in a constant and in the
    // piece's number, exchanged.  (Opaque: the sums are made here, not kept.)
    uint32_t ak = (uint32_t)(ik & 1) * kBuf + row_k * DP * 2 + ((hf ^ (row_k & KMASK)) << 4);
    uint32_t av = (uint32_t)(iv & 1) * kBuf + kKeys + l32 * kApTile * 2 + ((hf ^ ((l32 >> 1) & 7)) << 4);
    asm volatile("" : "+v"(ak), "+v"(av));
    auto fragment = [&](int n) -> v4u {
      if (n < nk)
        return *reinterpret_cast<const v4u*>(s_kv + (ak ^ ((n >> 1) << 5)) + (n & 1) * 32 * DP * 2);
      const int g = (n - nk) / ND, d = (n - nk) % ND;
      return *reinterpret_cast<const v4u*>(s_kv + (av ^ (g << 5)) + d * 32 * kApTile * 2);
    };
    v4u f[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) f[n] = fragment(n);
    if constexpr (nk > 0) s[0] = s[1] = v16f32{};
#pragma unroll
    for (int n = 0; n < nk + nv; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      if (n < nk) s[n & 1] = mfma32<BF>(f[n % kAhead], qf[n >> 1], s[n & 1]);
      else o[(n - nk) % ND] = mfma32<BF>(f[n % kAhead], p[(n - nk) / ND], o[(n - nk) % ND]);
      if (n + kAhead < nk + nv) f[n % kAhead] = fragment(n + kAhead);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto soften = [&](int i) {   // S^T to weights
    // register 8 w + e of block k: key 32 k + 16 w + 8 hf + e; scores less the maximum
    const int t0 = key0(i);
    const v4f mul = *reinterpret_cast<const v4f*>(s_mul[i & 1]);
    const v4f base0 = *reinterpret_cast<const v4f*>(s_base[i & 1]);
    const v4f inv = *reinterpret_cast<const v4f*>(s_inv[i & 1]);
    const float m0 = m == -__builtin_inff() ? 0.0f : m;
    float top = -__builtin_inff();
    auto scores = [&](auto all) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float base = base0[g] - m0;
        if (ALIBI) base = __builtin_fmaf(slope, (float)(t0 + 16 * g + 8 * hf - pos), base);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x = __builtin_fmaf(s[g >> 1][8 * (g & 1) + e], mul[g], base);
          if (ALIBI) x = __builtin_fmaf(slope, (float)e, x);
          if constexpr (!decltype(all)::value) {
            const int k = t0 + 16 * g + 8 * hf + e;
            x = k >= lo && k < hi ? x : -__builtin_inff();
          }
          s[g >> 1][8 * (g & 1) + e] = x;
          top = __builtin_fmaxf(top, x);
        }
      }
    };
    // every row of the wave sees every key of the tile, or not
    if (t0 >= wv_lo1 && t0 + kApTile <= wv_hi0) scores(std::true_type{});
    else scores(std::false_type{});
    float t_lo, t_hi;
    halves(top, &t_lo, &t_hi);
    top = __builtin_fmaxf(t_lo, t_hi);
    const bool fresh = m == -__builtin_inff();
    if (__any(top > kApSlack || (fresh && top > -__builtin_inff()))) {
      // the maximum moves: by `up` (at first from nothing, to the tile's)
      const float up = fresh ? (top == -__builtin_inff() ? 0.0f : top) : __builtin_fmaxf(top, 0.0f);
      const float f = __builtin_amdgcn_exp2f(-up);
      if (!fresh) {
        l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= f;
        m += up;
      } else if (top > -__builtin_inff()) {
        m = up;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[0][e] -= up;
        s[1][e] -= up;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float add = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w0 = __builtin_amdgcn_exp2f(s[g >> 1][8 * (g & 1) + 2 * u]);
        const float w1 = __builtin_amdgcn_exp2f(s[g >> 1][8 * (g & 1) + 2 * u + 1]);
        p[g][u] = pack2<BF>(w0, w1);
        add += w0 + w1;
      }
      // (a hidden page's scale may be NaN: no 0 * NaN)
      l = __builtin_fmaf(add, add != 0.0f ? inv[g] : 0.0f, l);
    }
  };

  // ---- the loop ----------------------------------------------------------------
  // Step i of a wave: the matrix part, S of tile i and O of tile i - 1, then the
  // vector part, the weights of tile i and its share of the staging.  With eight
  // waves, two on each SIMD, waves 4 .. 7 run half a step behind waves 0 .. 3, so
  // that on every SIMD one wave's matrix part goes with the other's vector part;
  // a barrier ends every half step.  The early waves then stage keys of tile
  // i + 1 and values of tile i, the late ones a tile further: no buffer is
  // written while it is read, and each is whole a half step before its first use.
  if (n_tiles > 0) {
    constexpr bool kPair = NW == 8;
    const bool late = kPair && wave >= 4;
    const int ahead = late ? 2 : 1;
    for (int j = 0; j < ahead; ++j) {
      load_pages(j);
      load_codes(j);
      store(j);
    }
    load_pages(ahead);
    load_codes(ahead);
    load_pages(ahead + 1);
    lds_sync();
    if (late) lds_sync();
    multiply(std::true_type{}, std::false_type{}, 0, 0);
    for (int i = 0; i < n_tiles; ++i) {
      if (kPair) lds_sync();
      store(i + ahead);
      load_codes(i + ahead + 1);
      load_pages(i + ahead + 2);
      soften(i);
      lds_sync();
      // (after the last tile the scores are of whatever the buffer holds, and unused)
      multiply(std::true_type{}, std::true_type{}, i + 1, i);
    }
    if (kPair && !late) lds_sync();
  }

  float l_lo, l_hi;
  halves(l, &l_lo, &l_hi);
  l = l_lo + l_hi;
  if (!live) return;
  const int64_t row_out = (sq.c0 + qi) * H * G + h * G + qg;
  if (a.n_split == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // no key at all: 0
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = 32 * d + 8 * q + 4 * hf;
        if (at < D) {
          uint2 w;
          w.x = pack2<BF>(o[d][4 * q] * inv, o[d][4 * q + 1] * inv);
          w.y = pack2<BF>(o[d][4 * q + 2] * inv, o[d][4 * q + 3] * inv);
          *reinterpret_cast<uint2*>(a.out + row_out * D + at) = w;
        }
      }
    return;
  }
  const size_t at = (((size_t)b * H + h) * ((size_t)G * a.max_q) + rr) * a.n_split + split;
  const size_t n_part = (size_t)a.s.B * H * G * a.max_q * a.n_split;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = 32 * d + 8 * q + 4 * hf;
      if (e < D)
        *reinterpret_cast<v4f*>(a.part + 2 * n_part + at * D + e) =
            v4f{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
    }
  if (hf == 0) {
    a.part[2 * at] = m;
    a.part[2 * at + 1] = l;
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

// Which kernel, how many rows a workgroup takes, and how the keys are split.
struct Plan {
  int rows;      // 16: attn_decode_kernel; 128, 256: attn_run_kernel with 4, 8 waves
  int chunk, n_split;
};
Plan plan(int B, int H, int G, int D, int max_q, int max_len, int window) {
  Plan p;
  int range = max_len;
  if (window > 0) range = (int)std::min((int64_t)max_len, (int64_t)window + max_q + 128);
  const int64_t rows = (int64_t)G * max_q, heads = (int64_t)B * H;
  p.rows = 16;
  if (rows > 16 && D <= 128) p.rows = heads * ((rows + 255) / 256) >= 256 ? 256 : 128;
  const int64_t tiles = heads * ((rows + p.rows - 1) / p.rows);
  // at least 256 keys a workgroup; about four workgroups a compute unit (single
  // rows), or one (runs)
  const int64_t want = std::max<int64_t>((p.rows == 16 ? 1024 : 256) / tiles, 1);
  const int64_t c = std::max<int64_t>(((range + want - 1) / want + 255) / 256 * 256, 256);
  p.chunk = (int)c;
  p.n_split = std::max((int)((range + c - 1) / c), 1);
  return p;
}

template <bool BF, bool ALIBI>
void launch_kernel(const AttnArgs& a, const Plan& p, hipStream_t stream) {
  const int D = a.c.D;
  const dim3 grid(a.c.H * ((a.G * a.max_q + p.rows - 1) / p.rows), a.n_split, a.s.B);
  if (p.rows == 16) {
    const dim3 block(kAdThreads);
    if (D <= 64) hipLaunchKernelGGL((attn_decode_kernel<BF, 64, ALIBI>), grid, block, 0, stream, a);
    else if (D <= 128)
      hipLaunchKernelGGL((attn_decode_kernel<BF, 128, ALIBI>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_kernel<BF, 256, ALIBI>), grid, block, 0, stream, a);
  } else if (p.rows == 128) {
    if (D <= 64)
      hipLaunchKernelGGL((attn_run_kernel<BF, 64, 4, ALIBI>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((attn_run_kernel<BF, 128, 4, ALIBI>), grid, dim3(256), 0, stream, a);
  } else {
    if (D <= 64)
      hipLaunchKernelGGL((attn_run_kernel<BF, 64, 8, ALIBI>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((attn_run_kernel<BF, 128, 8, ALIBI>), grid, dim3(512), 0, stream, a);
  }
}

template <bool BF>
hipError_t launch_typed(const AttnArgs& a, const Plan& p, hipStream_t stream) {
  if (a.alibi) launch_kernel<BF, true>(a, p, stream);
  else launch_kernel<BF, false>(a, p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_split == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<BF>), dim3((a.G * a.max_q + 3) / 4, a.c.H, a.s.B),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t attention_partials(int B, int H, int G, int D, int max_q, int max_len, int window) {
  const Plan p = plan(B, H, G, D, max_q, max_len, window);
  return p.n_split == 1 ? 0 : (size_t)B * H * G * max_q * p.n_split * (size_t)(D + 2);
}

hipError_t launch_attention(AttnArgs a, hipStream_t stream) {
  const Plan p = plan(a.s.B, a.c.H, a.G, a.c.D, a.max_q, a.max_len, a.window);
  a.chunk = p.chunk;
  a.n_split = p.n_split;
  return a.c.bf16 ? launch_typed<true>(a, p, stream) : launch_typed<false>(a, p, stream);
}

}  // namespace i8l
