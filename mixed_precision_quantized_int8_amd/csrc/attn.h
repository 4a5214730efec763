// Attention over the 8-bit key/value cache (internal header; attn.hip and tree.hip have
// the instantiations): attn_decode_kernel for single queries
// and short calls, attn_run_kernel for runs of queries, attn_join_kernel for keys
// that were split over workgroups.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - slope (i - j))
// over the keys j <= i (and i - j < window) of the sequence, k_j = ks c^k_j and
// v_j = vs c^v_j with one ks and vs per page and head.
//
// The value scale of a key's page joins its exponent: with
//   s'_j = s_j + ln vs_j,   m = max_j s'_j,   w_j = exp(s'_j - m) <= 1,
//   o = sum_j w_j c^v_j / sum_j w_j / vs_j,
// so the product on the matrix cores runs on the codes themselves, and the
// rounding of w_j to 16 bits is relative to the largest contribution (it takes the
// error against 64 bits from 2.1e-4 to 2.4e-4 - 2.9e-4 in fp16, from 1.7e-3 to 2.0e-3
// in bf16).  Codes are exact in fp16 and bf16; m and the sums are fp32.  The tokens of the incomplete
// page have 16-bit values and no scale; every kernel takes them last, since weights
// relative to them would lose bits where the codes' scales are small.
//
// TREE: the queries are drafts, a tree of them behind each sequence, whose own keys and
// values are no part of the cache.  Every query sees all of the cache (or a window that
// ends at its position) and the drafts that its mask names.  Drafts are 16-bit values
// too and come last, in the workgroups of the last split.
#pragma once

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
  int n, len;          // queries, tokens held (those that the page table has a place for)
  int first_pos;       // position of its first query; counts the tokens past the table
};
template <bool TREE>
using ArgsOf = std::conditional_t<TREE, TreeArgs, AttnArgs>;
__device__ __forceinline__ Rows rows_of(const AttnArgs& a, int b) {
  Rows r;
  // (lengths end at 2^30, past any page table, so that positions stay in 32 bits)
  const int len = min(max(a.s.lengths[b], 0), 1 << 30);
  int64_t c0 = a.s.cu ? a.s.cu[b] : b, c1 = a.s.cu ? a.s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), a.rows);
  c1 = min(max(c1, c0), a.rows);
  r.c0 = c0;
  r.n = (int)min(c1 - c0, (int64_t)a.max_q);   // (none past max_q is written)
  r.len = min(len, a.s.max_pages << a.c.ps);
  r.first_pos = (int)max(len - (c1 - c0), -((int64_t)1 << 30));
  return r;
}

// Position of query qi of a sequence.  (A tree's matter for a window or a bias only; its
// distances stay in 32 bits.)
template <bool TREE>
__device__ __forceinline__ int position(const ArgsOf<TREE>& a, const Rows& sq, int qi) {
  if constexpr (TREE)
    return a.positions ? min(max(a.positions[sq.c0 + qi], -(1 << 29)), 1 << 30) : sq.len;
  else return sq.first_pos + qi;
}
// Which of the drafts 64 w .. 64 w + 63 query qi's mask names, of the sequence's n.
__device__ __forceinline__ uint64_t draft_mask(const TreeArgs& a, const Rows& sq, int qi, int w) {
  const int left = sq.n - 64 * w;
  return a.masks[(sq.c0 + qi) * a.words + w] & (left >= 64 ? ~0ull : (1ull << left) - 1);
}

__device__ __forceinline__ float xmax16(float v) {   // over the four 16-lane groups
  v = __builtin_fmaxf(v, __shfl_xor(v, 16, 64));
  return __builtin_fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float xsum16(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Partial results of a split launch: (m, l) of every row and split, filled up to 16
// bytes, then its unnormalised output (not written where l is 0 and m -infinity).
__host__ __device__ __forceinline__ size_t part_head(size_t count) { return (2 * count + 3) / 4 * 4; }
__device__ __forceinline__ size_t part_at(const AttnArgs& a, int b, int h, int row, int split) {
  return (((size_t)b * a.c.H + h) * ((size_t)a.G * a.max_q) + row) * a.n_split + split;
}
__device__ __forceinline__ float* part_out(const AttnArgs& a, size_t at) {
  return a.part + part_head((size_t)a.s.B * a.c.H * a.G * a.max_q * a.n_split) + at * a.c.D;
}
__device__ __forceinline__ void say_empty(const AttnArgs& a, int b, int h, int row, int split) {
  const size_t at = part_at(a, b, h, row, split);
  a.part[2 * at] = -__builtin_inff();
  a.part[2 * at + 1] = 0.0f;
}

// How a call with trees is shared out where lengths and drafts are ragged (they are known
// on the device only, and splits that suit the longest sequence leave most compute
// units waiting for it).  Each tile of rows of a sequence counts its blocks of 128 keys, and
// kShareCost more for its start and its drafts; the blocks of all tiles stand in one line,
// and workgroup s of a head takes those from s * each on, a segment of a tile at a time.
// So at most its first segment lacks the tile's start and at most its last the end: two
// places for partial results a workgroup.  Lane b plans sequence b (at most 64).
// 16 sequences of 2 - 8 thousand tokens with 17 to 64 drafts, 32 heads of 128 on 8, bf16:
// 121 us against 148 with splits of equal length; 61 GFLOP, 505 TFLOP/s (the shortest
// drafts leave waves without rows; outputs of split tiles are 13 us of a second launch).
struct SharePlan {
  int first, tiles, blocks;   // where the sequence's blocks begin; of a tile
};
struct Segment {
  int b, tile, begin, end;    // keys
  bool last;                  // the drafts are its too
  int part;                   // place of its partial results, -1: it is the whole tile
  int next;                   // block that the next one begins at
};
constexpr int kShareSeqs = 64, kShareCost = 2;
constexpr int kShareHead = 2 * kShareSeqs + 64;   // words before the partial results, for the join
// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
#define I8L_SCAN(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
  I8L_SCAN(0x111, 0xf);   // by 1, 2, 4, 8 within 16
  I8L_SCAN(0x112, 0xf);
  I8L_SCAN(0x114, 0xf);
  I8L_SCAN(0x118, 0xf);
  I8L_SCAN(0x142, 0xa);   // lane 15 to 16 .. 31, 47 to 48 .. 63
  I8L_SCAN(0x143, 0xc);   // lane 31 to 32 .. 63
#undef I8L_SCAN
  return v;
}
// The first wave's: its lane's plan, and in *each and *total the blocks of a workgroup and
// of all.
__device__ __forceinline__ SharePlan plan_shares(const TreeArgs& a, int rows, int* each, int* total) {
  const int lane = threadIdx.x & 63;
  SharePlan p{0, 0, 0};
  if (lane < a.s.B) {
    const Rows r = rows_of(a, lane);
    p.tiles = (r.n * a.G + rows - 1) / rows;
    p.blocks = (r.len + 127) / 128;
  }
  const int mine = p.tiles * (p.blocks + kShareCost), upto = wave_scan(mine);
  p.first = upto - mine;
  const int all = __builtin_amdgcn_readlane(upto, 63), share = (all + a.shares - 1) / a.shares;
  *each = max(share, 1);
  *total = all;
  if (blockIdx.x == 0) {
    int32_t* table = reinterpret_cast<int32_t*>(a.part);
    table[lane] = p.first;
    table[kShareSeqs + lane] = p.blocks;
    if (lane == 0) table[2 * kShareSeqs] = max(share, 1);
  }
  return p;
}
// The segment that begins at block x of the line (x < total); to: the workgroup's end.
__device__ __forceinline__ Segment segment_at(const SharePlan& p, int x, int to, int s) {
  const int b = __builtin_ctzll(__ballot(p.first + p.tiles * (p.blocks + kShareCost) > x));
  const int blocks = __builtin_amdgcn_readlane(p.blocks, b), c = blocks + kShareCost;
  const int v = x - __builtin_amdgcn_readlane(p.first, b);
  Segment r;
  r.b = b;
  r.tile = v / c;
  const int off = v - r.tile * c, stop = min(c, off + to - x);
  r.begin = 128 * off;
  r.end = 128 * min(stop, blocks);
  r.last = stop == c;
  r.part = off == 0 && r.last ? -1 : 2 * s + (off == 0);
  r.next = x + stop - off;
  return r;
}
// (m, l) and output of row r of the tile of partial results `part`.
__device__ __forceinline__ size_t share_row(const TreeArgs& a, int part, int h, int rows, int r) {
  return ((size_t)part * a.c.H + h) * rows + r;
}
__device__ __forceinline__ float* share_ml(const TreeArgs& a, size_t at) { return a.part + kShareHead + 2 * at; }
__device__ __forceinline__ float* share_out(const TreeArgs& a, int rows, size_t at) {
  return a.part + kShareHead + 4 * (size_t)a.shares * a.c.H * rows + at * a.c.D;
}

// 16 rows (queries of one kv head: token-major, the G heads of a token together)
// against a range of keys.  S^T = K . Q^T and O^T = V^T . P^T on 16x16x32
// matrix instructions; lane l holds query l & 15, and of a tile of 64 keys the
// sixteen 16 g .. 16 g + 15 of group g = l >> 4: row i of score block j is key
// 16 (i / 4) + 4 j + i % 4, so that a lane's sixteen scores are neighbours, lie
// in one page (P >= 16), and are, in order, the lane's operand for the second
// product, whose V^T operand is then 16 contiguous bytes of the [D][P] page.
//
// Bound by the read of the codes: four waves take a tile of 64 keys each, straight
// from memory to registers (no wave shares a key with another, so nothing passes
// through LDS), with the next tile's codes in flight; results of the waves meet in
// LDS at the end.  The matrix cores run 16 columns for however many rows there are;
// converting the codes is the larger part of the vector work, a few times below the
// memory's rate.  One sequence of 131072 tokens, 112 heads of 128: 3.76 GB in
// 617 to 641 us, 5.9 - 6.1 TB/s; 64 sequences of 2 - 8 thousand, 32 heads on 8: 684 MB in
// 153 us, 4.5 TB/s (a large copy reaches 5.15); both in bf16 156 and 645 us; 100 tokens,
// 16 heads of 64: 5.4 us, latency.  (Passes in a captured graph, the join included.)
// A third workgroup a compute unit (168 registers) was slower: 167 and 743 us; two
// blocks of 16 rows a wave too (32 rows, 64 heads, 65536 keys: 321 against 303 us).
//
// DP: head dimension padded to a multiple of 64 (64, 128, 256).
template <bool BF, int DP, bool ALIBI, bool TREE>
__global__ __launch_bounds__(kAdThreads, DP > 128 ? 1 : 2) void attn_decode_kernel(ArgsOf<TREE> a) {
  constexpr int NC = DP / 64, ND = DP / 16;
  __shared__ __attribute__((aligned(16))) float s_o[kAdWaves][16][DP + 4];
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
  const int pos = position<TREE>(a, sq, qi);      // its position; keys <= pos
  const int hi = TREE ? sq.len : min(pos + 1, sq.len);
  const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
  // the tile's range (rows are in the order of their positions, a tree's in any)
  const int q_last = (min(r0 + 16, n_rows) - 1) / G;
  const int all_hi = TREE ? sq.len : min(sq.first_pos + q_last + 1, sq.len);
  int lo_first = a.window > 0 ? max(0, sq.first_pos + r0 / G + 1 - a.window) : 0;
  const int hi_first = TREE ? sq.len : min(sq.first_pos + r0 / G + 1, sq.len);   // seen by every row
  int lo_last = a.window > 0 ? max(0, sq.first_pos + q_last + 1 - a.window) : 0;
  if (TREE && a.window > 0) {
    lo_first = lo_last = lo;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      lo_first = min(lo_first, __shfl_xor(lo_first, off, 64));
      lo_last = max(lo_last, __shfl_xor(lo_last, off, 64));
    }
    lo_first = __builtin_amdgcn_readfirstlane(lo_first);
    lo_last = __builtin_amdgcn_readfirstlane(lo_last);
  }
  // keys of this split: whole pages of any size (128 divides begin and chunk)
  const int first = lo_first & ~127;
  const int begin = first + split * a.chunk;
  const int end = split == a.n_split - 1 ? all_hi : min(begin + a.chunk, all_hi);
  const int coded = sq.len >> ps << ps;            // tokens in complete pages

  // nothing to see here: no more than that is said
  if (begin >= end && a.n_split > 1 && !(TREE && split == a.n_split - 1)) {
    if (t < min(16, n_rows - r0)) say_empty(a, b, h, r0 + t, split);
    return;
  }

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

  // scores of one tile (scaled, in log2 units, base included; top: this lane's highest) to
  // weights, the running maximum and sum; then O
  auto settle = [&](v4f (&s)[4], float top, float inv_vs) {
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
    l = __builtin_fmaf(add, inv_vs, l);
  };
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
    settle(s, top, inv_vs);
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

  // Complete pages: tile i of this wave starts at key c0 + 256 i.  The registers of
  // a tile's keys are free once its scores are formed, those of its values once its
  // outputs are: each then takes the next tile's codes, so that half a tile or more
  // is on its way at any time; the page numbers come a tile before that.
  const int c0 = max(begin, lo_first & ~(kAdTile - 1)) + wave * kAdTile;
  const int c_end = min(end, coded);
  const int sub_k = 16 * (i16 >> 2), sub_v = 16 * grp;   // this lane's keys as K row, as P
  const int8_t* k_at = a.c.kc + h * page_sz + (size_t)(((sub_k & (P - 1)) + (i16 & 3)) * D);
  const int8_t* v_at = a.c.vc + h * page_sz + (size_t)(i16 * P + (sub_v & (P - 1)));
  const uint32_t page_step = (uint32_t)(H * page_sz);   // at most 4096 * 128 * 256
  int pk = 0, pv = 0;          // pages of the tile to load next, as the table has them
  v4u kb[4][NC], vb[ND];       // codes
  float ks = 0.0f, vs0 = 0.0f;
  bool page_ok = false;
  auto load_pages = [&](int t0) {   // (keys past the coded ones: any entry, hidden below)
    pk = table[min((t0 + sub_k) >> ps, a.s.max_pages - 1)];
    pv = table[min((t0 + sub_v) >> ps, a.s.max_pages - 1)];
  };
  auto exists = [&](int page) { return (uint32_t)page < (uint32_t)a.c.n_pages; };
  auto load_k = [&](int t0) {
    const int8_t* at = k_at + (uint64_t)(exists(pk) ? (uint32_t)pk : 0u) * page_step +
                       (t0 & (P - 1) & kAdTile) * D;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (64 * c < D) {   // uniform; a lane past D takes the row's start, which meets zeros of q
          const int d = 64 * c + 16 * grp < D ? 64 * c + 16 * grp : 0;
          kb[j][c] = *reinterpret_cast<const v4u*>(at + 4 * j * D + d);
        }
  };
  auto load_v = [&](int t0) {
    page_ok = exists(pv);
    const uint32_t page = page_ok ? (uint32_t)pv : 0u;
    ks = a.c.ks[(size_t)page * H + h];
    vs0 = a.c.vs[(size_t)page * H + h];
    const int8_t* p = v_at + (uint64_t)page * page_step + (t0 & (P - 1) & kAdTile);
#pragma unroll
    for (int d = 0; d < ND; ++d)
      if (16 * d < D) vb[d] = *reinterpret_cast<const v4u*>(p + (size_t)16 * d * P);   // uniform
  };
  // (no entry of the table depends on the length: the first ones leave with it)
  load_pages(c0);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int c = 0; c < NC; ++c) kb[j][c] = v4u{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < ND; ++d) vb[d] = v4u{0, 0, 0, 0};
  if (c0 < c_end) {
    load_k(c0);
    load_v(c0);
    load_pages(c0 + kAdWaves * kAdTile);
  }
  for (int t0 = c0; t0 < c_end; t0 += kAdWaves * kAdTile) {
    const int next = t0 + kAdWaves * kAdTile;
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
    if (next < c_end) load_k(next);
    const int tv = t0 + sub_v;
    const float vs = vs0 == 0.0f ? kZeroScale : vs0 < kLeastScale ? kLeastScale : vs0;
    const bool all = t0 >= lo_last && t0 + kAdTile <= min(hi_first, coded) && !__any(!page_ok);
    float base = __builtin_amdgcn_logf(vs);
    if (ALIBI) base = __builtin_fmaf(slope, (float)(tv - pos), base);
    // a page of NaNs: its weights are NaN where they are seen, 0 where they are not
    const float inv_vs = vs < __builtin_inff() ? 1.0f / vs : 0.0f;
    soften(s, sc * ks, base, inv_vs, t0, all, lo, min(hi, coded), page_ok);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const v4u p = weights(s, st);
#pragma unroll
      for (int d = 0; d < ND; ++d)
        o[d] = mfma16<BF>(codes8<BF>(vb[d][2 * st], vb[d][2 * st + 1]), p, o[d]);
    }
    if (next < c_end) {
      load_v(next);
      load_pages(next + kAdWaves * kAdTile);
    }
  }

  // keys of the incomplete page, 16 bits each; values past the length are
  // whatever the slot held before and are cleared.  So are infinities and NaNs, which
  // a hidden key's weight of 0 would spread over all rows: where there is one, each lane
  // adds those that its query sees.
  auto tail_tile = [&](int t0) {
    const int slot = a.s.slots ? a.s.slots[b] : b;
    const bool ok = slot >= 0 && slot < a.c.n_slots;
    const size_t f = ((size_t)(ok ? slot : 0) * H + h) * page_sz;
    const int tk = t0 + 16 * (i16 >> 2), tv = t0 + 16 * grp;
    const bool in_k = tk >= coded && tk < coded + P, in_v = ok && tv >= coded && tv < coded + P;
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
    const int from = max(lo, coded);
    soften(s, sc, base, 1.0f, t0, false, from, hi, ok);
    v4u v[2][ND];
    uint32_t odd = 0;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int k0 = tv + 8 * st, nv = in_v ? sq.len - k0 : 0;   // valid keys of these eight
      const uint16_t* vp = a.c.vt + f + (size_t)i16 * P + (in_v ? k0 - coded : 0);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        v[st][d] = v4u{0, 0, 0, 0};
        if (16 * d < D) v[st][d] = *reinterpret_cast<const v4u*>(vp + (size_t)16 * d * P);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[st][d][u] &= (2 * u < nv ? 0xffffu : 0u) | (2 * u + 1 < nv ? 0xffff0000u : 0u);
          odd |= odd_halves<BF>(v[st][d][u]);
        }
    }
    if (__any(odd)) {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t x = v[st][d][u];
            asm volatile("" : "+v"(x));   // (found again here, not kept from above)
            v[st][d][u] = clear_halves(x, odd_halves<BF>(x));
          }
      for (int k = max(t0, from); k < min(t0 + kAdTile, hi); ++k) {
        const uint16_t* vp = a.c.vt + f + (4 * grp << ps) + k - coded;   // of this lane's outputs
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          asm volatile("" : "+v"(vp));   // (an address at a time)
          if (16 * d < D)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] += odd_value<BF>(vp[e << ps]);
          vp += 16 << ps;
        }
      }
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const v4u p = weights(s, st);
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] = mfma16<BF>(v[st][d], p, o[d]);
    }
  };

  if (end > coded && coded >= begin) {
    // The waves whose turn comes after the complete pages' last tile: 100 tokens (one
    // tile of complete pages, one of the tail) 7.4 -> 5.8 us.
    const int n_tiles = max(c_end - (c0 - wave * kAdTile) + kAdTile - 1, 0) / kAdTile;
    const int turn = (wave - n_tiles) & (kAdWaves - 1);
    for (int t0 = (coded & ~(kAdTile - 1)) + turn * kAdTile; t0 < end; t0 += kAdWaves * kAdTile)
      tail_tile(t0);
  }

  // The drafts, a tile of 64 a wave, after the waves' other tiles.  Keys come straight from
  // their rows; values are [draft][D] and the product wants eight drafts of a dimension
  // together: they are transposed 32 drafts at a time through this wave's part of s_o.
  // What is hidden, or no number, is treated as in the incomplete page.
  if constexpr (TREE) {
    auto draft_tile = [&](int t0) {
      const uint64_t word = draft_mask(a, sq, qi, t0 >> 6);
      uint32_t bits = live ? (uint32_t)(word >> (16 * grp)) & 0xffffu : 0u;   // this lane's 16 keys
      // values of step st: drafts 16 g + 8 st + i of the tile are 8 g + i there, two neighbours
      // of 8 dimensions a lane at a time; all on their way before they are needed
      constexpr int NQ = 16 * (DP / 8) / 64;
      v4u v[NQ][2];
      auto load_values = [&](int st) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int q = lane + 64 * n, i = 2 * (q & 15), d = (q >> 4) * 8;
          const int key = t0 + 16 * (i >> 3) + 8 * st + (i & 7);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            v[n][u] = v4u{0, 0, 0, 0};
            if (key + u < sq.n && d < D)
              v[n][u] = *reinterpret_cast<const v4u*>(a.dv + (sq.c0 + key + u) * a.dv_ts + h * a.dv_hs + d);
          }
        }
      };
      load_values(0);
      v4f s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        const int key = min(t0 + 16 * (i16 >> 2) + 4 * j + (i16 & 3), sq.n - 1);
        const uint16_t* kp = a.dk + (sq.c0 + key) * a.dk_ts + h * a.dk_hs;
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
      float top = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[j][e] * sc;
          bool seen = bits >> (4 * j + e) & 1;
          if (ALIBI || a.window > 0) {
            const int back = pos - position<true>(a, sq, min(t0 + 16 * grp + 4 * j + e, sq.n - 1));
            if (ALIBI) x = __builtin_fmaf(-slope, (float)back, x);
            if (a.window > 0 && back >= a.window) {
              seen = false;
              bits &= ~(1u << (4 * j + e));
            }
          }
          s[j][e] = seen ? x : -__builtin_inff();
          top = __builtin_fmaxf(top, s[j][e]);
        }
      settle(s, top, 1.0f);
      uint8_t* turned = reinterpret_cast<uint8_t*>(&s_o[wave][0][0]);   // [d][32 drafts], 64 bytes a row
      uint32_t odd = 0;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int q = lane + 64 * n, i = 2 * (q & 15), d = (q >> 4) * 8;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t bad = odd_halves<BF>(v[n][u][e]);
              odd |= bad;
              v[n][u][e] = clear_halves(v[n][u][e], bad);
            }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint32_t*>(turned + (d + e) * 64 + 2 * i) =
                __builtin_amdgcn_perm(v[n][1][e >> 1], v[n][0][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
        }
        if (st == 0) load_values(1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const v4u p = weights(s, st);
#pragma unroll
        for (int d = 0; d < ND; ++d)
          o[d] = mfma16<BF>(*reinterpret_cast<const v4u*>(turned + (16 * d + i16) * 64 + 16 * grp), p, o[d]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();   // before the next drafts take their place
      }
      if (__any(odd)) {
        // (bits of the four lanes of a query together)
        uint64_t seen = (uint64_t)bits << (16 * grp);
        seen |= __shfl_xor(seen, 16, 64);
        seen |= __shfl_xor(seen, 32, 64);
        for (int key = t0; key < min(t0 + 64, sq.n); ++key) {
          const uint16_t* vp = a.dv + (sq.c0 + key) * a.dv_ts + h * a.dv_hs + 4 * grp;
          if (seen >> (key - t0) & 1)
#pragma unroll
            for (int d = 0; d < ND; ++d)
              if (16 * d < D)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][e] += odd_value<BF>(vp[16 * d + e]);
        }
      }
    };
    if (split == a.n_split - 1) {
      const int n_tiles = max(c_end - (c0 - wave * kAdTile) + kAdTile - 1, 0) / kAdTile + (end > coded ? 1 : 0);
      const int turn = (wave - n_tiles) & (kAdWaves - 1);
      for (int t0 = turn * kAdTile; t0 < sq.n; t0 += kAdWaves * kAdTile) draft_tile(t0);
    }
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
      const size_t at = part_at(a, b, h, R, split);
      *reinterpret_cast<v4f*>(part_out(a, at) + d) = oo;
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
//
// Near what a large fp16 product reaches under the board's power limit (1080 TFLOP/s):
// 4096 queries over 8192 tokens, 32 heads of 128 on 8, in 416 us, 990 TFLOP/s (bf16 405
// us).  No unit is busy throughout: the matrix cores 47 % of the cycles, the vector unit
// 58 %, LDS 38 %, in waves that issue in order, at 1.75 GHz.  Heads of 64 reach 775
// TFLOP/s (the exponentials weigh twice as much), of 80 660 (padded to 128), of 256 855.
// The instantiations for heads of 128 with four waves spill 4 to 7 registers.  What
// carried it there: products and vector work in alternating slots (half_tile) with
// staging that has no branches (638 -> 455 us; two groups of waves half a step
// apart, with barriers, had been slower: 701); eight waves of 32 rows rather than
// four of 64 (which left one wave a SIMD waiting: 752 us; with heads of 256 there is
// no room for more).
constexpr int kApTile = 64;
constexpr float kApSlack = 8.0f;

//
// attn_run: the workgroup's rows r_wg .. of kv head h of sequence b, and its split of the
// keys; SHARE: the segment's keys, without a window.
template <bool BF, int DP, int NW, bool ALIBI, bool TREE, bool SHARE>
__device__ __forceinline__ void attn_run(const ArgsOf<TREE>& a, int b, int h, int r_wg, int split,
                                         const Segment& seg) {
  const int n_split = SHARE ? 1 : a.n_split, chunk = a.chunk;
  constexpr int NT = 64 * NW, kRows = 32 * NW;
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
  __shared__ uint32_t s_odd[2];   // a tile of the incomplete page holds infinities or NaNs
  __shared__ int s_low[TREE ? NW : 1], s_pos[TREE ? kApTile : 1];

  int t = threadIdx.x;
  if (SHARE) asm volatile("" : "+v"(t), "+s"(h));   // (nothing of a segment is formed before it)
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int l32 = lane & 31, hf = lane >> 5;
  const int H = a.c.H, D = a.c.D, ps = a.c.ps, P = 1 << ps, G = a.G;
  const Rows sq = rows_of(a, b);
  const int n_rows = sq.n * G;
  if (r_wg >= n_rows) return;
  const int first_pos = sq.first_pos;

  // this lane's query; rows past the end repeat the last
  const int r_wave = r_wg + 32 * wave;
  const bool live = r_wave + l32 < n_rows;
  const int rr = min(r_wave + l32, n_rows - 1);
  const int qi = rr / G, qg = rr % G;
  const int pos = position<TREE>(a, sq, qi);
  const int hi = TREE ? sq.len : min(pos + 1, sq.len);
  const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
  auto low = [&](int row) -> int {   // first key that a row sees
    const int p = first_pos + row / G;
    return a.window > 0 ? max(0, p + 1 - a.window) : 0;
  };
  auto high = [&](int row) -> int { return TREE ? sq.len : min(first_pos + row / G + 1, sq.len); };
  // what every row of the wave sees, and what some row of the workgroup does
  int wv_lo1 = low(min(r_wave + 32, n_rows) - 1), wg_lo = low(r_wg);
  const int wv_hi0 = high(min(r_wave, n_rows - 1)), wg_hi = high(min(r_wg + kRows, n_rows) - 1);
  if (TREE && !SHARE && a.window > 0) {   // (rows of a tree are in any order)
    wv_lo1 = wg_lo = lo;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      wv_lo1 = max(wv_lo1, __shfl_xor(wv_lo1, off, 64));
      wg_lo = min(wg_lo, __shfl_xor(wg_lo, off, 64));
    }
    wv_lo1 = __builtin_amdgcn_readfirstlane(wv_lo1);
    if (lane == 0) s_low[wave] = wg_lo;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) wg_lo = min(wg_lo, s_low[i]);
    wg_lo = __builtin_amdgcn_readfirstlane(wg_lo);
  }

  const int coded = sq.len >> ps << ps;
  const int first = wg_lo & ~127;
  const int begin = SHARE ? seg.begin : first + split * chunk;
  const int end = SHARE ? min(seg.end, wg_hi) : split == n_split - 1 ? wg_hi : min(begin + chunk, wg_hi);
  const bool drafts = SHARE ? seg.last : TREE && split == n_split - 1;
  // nothing to see here: no more than that is said
  if (begin >= end && (n_split > 1 || SHARE) && !drafts) {
    for (int r = t; r < min(kRows, n_rows - r_wg); r += NT) {
      if constexpr (SHARE) {
        float* ml = share_ml(a, share_row(a, seg.part, h, kRows, r));
        ml[0] = -__builtin_inff();
        ml[1] = 0.0f;
      } else {
        say_empty(a, b, h, r_wg + r, split);
      }
    }
    return;
  }
  // a wave without rows only stages (a tree's rows rarely fill the workgroup)
  const bool idle = TREE && r_wave >= n_rows;
  const int c_begin = max(begin, wg_lo & ~(kApTile - 1));
  const int c_end = min(end, coded);
  const int n_coded = c_end > c_begin ? (c_end - c_begin + kApTile - 1) / kApTile : 0;
  const int n_tail = end > coded && coded >= begin ? (end - coded + kApTile - 1) / kApTile : 0;

  v4u qf[NK];
#pragma unroll
  for (int s = 0; s < NK; ++s) {
    const int d = 16 * s + 8 * hf;
    qf[s] = v4u{0, 0, 0, 0};
    if (live && d < D)
      qf[s] = *reinterpret_cast<const v4u*>(a.q + (sq.c0 + qi) * a.q_ts + (h * G + qg) * a.q_hs + d);
  }
  const float slope = ALIBI ? a.alibi[h * G + qg] * kLog2e : 0.0f;
  const float sc = a.scale * kLog2e;

  // ---- staging -----------------------------------------------------------------
  // No branches: a key past the coded ones repeats the last page, a page that the
  // cache does not have reads page 0, an element past D the page's start; the
  // group's base, the zeros of q and the rows of O that nobody stores hide them.
  const int32_t* table = a.s.table + (size_t)b * a.s.max_pages;
  const size_t page_sz = (size_t)P * D;
  auto exists = [&](int page) { return (uint32_t)page < (uint32_t)a.c.n_pages; };
  // chunk u of this thread: keys (rows of D codes) first, then values (rows of P);
  // its place within a page and its group of 16 keys do not change from tile to
  // tile (tiles start at multiples of 64, and P <= 128: only bit 6 of t0 moves it)
  auto is_k = [&](int u) { return t + u * NT < CH; };
  const int8_t* at0[CPT];   // the chunk in page 0
  int sub[CPT];             // its keys' offset in the tile, a multiple of 16
  uint32_t place[CPT];      // byte offset of its first 16-byte piece in a buffer (the
                            // second: exchanged, ^ 16)
#pragma unroll
  for (int u = 0; u < CPT; ++u) {
    const int c = t + u * NT;
    const int key = is_k(u) ? c / (DP / 16) : ((c - CH) & 3) * 16;
    const int d = is_k(u) ? c % (DP / 16) * 16 : (c - CH) >> 2;
    sub[u] = key & ~15;
    at0[u] = (is_k(u) ? a.c.kc : a.c.vc) + h * page_sz;
    if (d < D) at0[u] += is_k(u) ? (key & (P - 1)) * D + d : d * P + (key & (P - 1));
    place[u] = is_k(u) ? key * DP * 2 + (((d >> 3) ^ (key & KMASK)) << 4)
                       : kKeys + d * kApTile * 2 + (((key >> 3) ^ ((d >> 1) & 7)) << 4);
  }
  const uint32_t page_step = (uint32_t)(H * page_sz);   // at most 4096 * 128 * 256
  // A thread's value chunks run one tile behind its key chunks: step j takes keys of
  // tile j and values of tile j - 1.
  auto tile_of = [&](int u, int j) { return is_k(u) ? j : j - 1; };
  // The last keys come first: with a position bias they have the highest scores, so
  // that the maximum moves at the start and not in every tile.  (The incomplete page
  // comes after them all: its values have no scale, and weights that were relative
  // to them would lose bits where the codes' scales are small.)
  auto tile0 = [&](int i) { return c_begin + (n_coded - 1 - i) * kApTile; };
  int pg[CPT];          // pages of the chunks to load next
  v4u raw[CPT];         // codes in flight
  auto load_page = [&](int u, int j) {
    pg[u] = table[min(max(tile0(tile_of(u, j)) + sub[u], 0), coded - 1) >> ps];
  };
  auto load_chunk = [&](int u, int j) {   // after load_page(u, j)
    const int in_page = tile0(tile_of(u, j)) & (P - 1) & kApTile;
    const uint32_t page = exists(pg[u]) ? (uint32_t)pg[u] : 0u;
    raw[u] = *reinterpret_cast<const v4u*>(at0[u] + (uint64_t)page * page_step +
                                           (is_k(u) ? in_page * D : in_page));
  };
  auto store_piece = [&](int u, int w, int j) {   // piece w of chunk u
    *reinterpret_cast<v4u*>(s_kv + (((uint32_t)(tile_of(u, j) & 1) * kBuf + place[u]) ^ (16 * w))) =
        codes8<BF>(raw[u][2 * w], raw[u][2 * w + 1]);
  };
  // lanes 0 .. 3 of wave 0: page and scales of 16-key group `lane` of a tile
  int pm = -1;
  float ks = 0.0f, vs = 0.0f;
  auto load_meta_page = [&](int i) {
    const int tok = tile0(i) + 16 * lane;
    pm = tok >= 0 && tok < coded ? table[tok >> ps] : -1;
  };
  bool meta_ok = false;
  auto load_scales = [&]() {
    meta_ok = exists(pm);
    const size_t f = (size_t)(meta_ok ? pm : 0) * H + h;
    ks = a.c.ks[f];
    vs = a.c.vs[f];
  };
  auto store_meta = [&](int i, bool ok, float kscale, float vscale) {
    const float v = vscale == 0.0f ? kZeroScale : vscale < kLeastScale ? kLeastScale : vscale;
    s_mul[i & 1][lane] = ok ? sc * kscale : 0.0f;
    s_base[i & 1][lane] = ok ? __builtin_amdgcn_logf(v) : -__builtin_inff();   // hides the group
    // a page of NaNs: its weights are NaN where they are seen, 0 where they are not
    s_inv[i & 1][lane] = ok && v < __builtin_inff() ? 1.0f / v : 0.0f;
  };

  // ---- half a tile, 32 keys -------------------------------------------------------
  // maximum (0 until a key is seen: then limit is -inf) and sum (of this lane's keys)
  float m, limit, l;
  v16f32 s[2], o[ND];
  v4u p[2];
  m = l = 0.0f;
  limit = -__builtin_inff();
  p[0] = p[1] = v4u{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = v16f32{};
  const int row_k = (l32 & 0x13) | ((l32 & 4) << 1) | ((l32 & 8) >> 1);   // key of score row l32
  // LDS offsets of this lane's first fragments: the others differ in a constant and
  // in the piece's number, exchanged
  const uint32_t at_k = (uint32_t)(row_k * DP * 2 + ((hf ^ (row_k & KMASK)) << 4));
  const uint32_t at_v = (uint32_t)(kKeys + l32 * kApTile * 2 + ((hf ^ ((l32 >> 1) & 7)) << 4));
  auto frag_k = [&](uint32_t at, int u, int k) {   // step u of Q . K, half k
    return *reinterpret_cast<const v4u*>(s_kv + (at ^ (u << 5)) + k * 32 * DP * 2);
  };
  auto frag_v = [&](uint32_t at, int n, int k) {   // 16 keys 2 k + n / ND, block n % ND
    return *reinterpret_cast<const v4u*>(s_kv + (at ^ ((2 * k + n / ND) << 5)) +
                                         (n % ND) * 32 * kApTile * 2);
  };
  v4f mul, base0, inv;   // of the tile at hand
  float top;
  // Register 8 g + e of s[k]: key 32 k + 16 g + 8 hf + e.  Pair j (two
  // neighbours): scores less the maximum so far, and the highest of them;
  float bias[2];
  auto bias_of = [&](int t0, int k, int g) {
    const float x = base0[2 * k + g] - m;
    return ALIBI ? __builtin_fmaf(slope, (float)(t0 + 32 * k + 16 * g + 8 * hf - pos), x) : x;
  };
  auto shift = [&](int k, int j) {
#pragma unroll
    for (int e = 2 * j; e < 2 * j + 2; ++e) {
      float x = __builtin_fmaf(s[k][e], mul[2 * k + (e >> 3)], bias[e >> 3]);
      if (ALIBI) x = __builtin_fmaf(slope, (float)(e & 7), x);
      s[k][e] = x;
      top = __builtin_fmaxf(top, x);
    }
  };
  // scores to weights in 16 bits, and their sum.
  float add[2];
  auto weigh = [&](int k, int j) {
    const float w0 = __builtin_amdgcn_exp2f(s[k][2 * j]);
    const float w1 = __builtin_amdgcn_exp2f(s[k][2 * j + 1]);
    uint32_t pair = pack2<BF>(w0, w1);
    asm volatile("" : "+v"(pair));   // formed in its slot, not next to its use
    p[j >> 2][j & 3] = pair;
    add[j >> 2] += w0 + w1;
  };
  auto total = [&](int k) {
#pragma unroll
    for (int g = 0; g < 2; ++g) l = __builtin_fmaf(add[g], inv[2 * k + g], l);
  };
  auto move_top = [&](int k) {   // the maximum, if the scores pass it
    if (__any(top > limit)) {
      float a0, a1;   // both halves of the wave hold the same queries
      halves(top, &a0, &a1);
      const float high = __builtin_fmaxf(a0, a1);
      const bool fresh = limit < 0.0f, some = high > -__builtin_inff();
      // the maximum moves by `up` (at first from nothing, to the tile's)
      const float up = some ? (fresh ? high : __builtin_fmaxf(high, 0.0f)) : 0.0f;
      const float f = fresh ? 1.0f : __builtin_amdgcn_exp2f(-up);
      m += up;
      if (some) limit = kApSlack;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= f;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[k][r] -= up;
    }
  };
  // masks the scores where a row of the wave does not see a key; moves the maximum
  auto settle = [&](int tile0, int k) {
    const int t0 = tile0 + 32 * k;
    if (!(t0 >= wv_lo1 && t0 + 32 <= wv_hi0)) {   // uniform
      top = -__builtin_inff();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int key = t0 + 16 * (r >> 3) + 8 * hf + (r & 7);
        const float x = key >= lo && key < hi ? s[k][r] : -__builtin_inff();
        s[k][r] = x;
        top = __builtin_fmaxf(top, x);
      }
    }
    move_top(k);
  };
  // Half k of tile i.  A wave issues in order, so the matrix cores and the vector
  // unit work at once only where their instructions alternate: the products of the
  // outputs of the half tile before with the shifts of this one's scores, then the
  // products of the next half tile's scores with this one's weights, in slots of
  // one product and its share of the vector work.  Fragments are read kAhead steps
  // before their use; `extra(n)` is more vector work for the first NV slots.
  constexpr int kAhead = 4, NV = 2 * ND;   // (8 pairs over NV, then over NK slots)
  auto half_tile = [&](int i, int k, auto extra) {
    const int t0 = tile0(i);
    uint32_t av = at_v + (uint32_t)((k ? i : i - 1) & 1) * kBuf;
    uint32_t ak = at_k + (uint32_t)((k ? i + 1 : i) & 1) * kBuf;
    asm volatile("" : "+v"(av), "+v"(ak));   // (offsets are formed here, not kept)
    auto fragment = [&](int n) { return n < NV ? frag_v(av, n, k ^ 1) : frag_k(ak, n - NV, k ^ 1); };
    v4u f[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) f[n] = fragment(n);
    top = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < 2; ++g) bias[g] = bias_of(t0, k, g);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      o[n % ND] = mfma32<BF>(f[n % kAhead], p[n / ND], o[n % ND]);
#pragma unroll
      for (int j = n * 8 / NV; j < (n + 1) * 8 / NV; ++j) shift(k, j);
      f[n % kAhead] = fragment(n + kAhead);
      extra(n);
    }
    __builtin_amdgcn_sched_barrier(0);
    settle(t0, k);
    add[0] = add[1] = 0.0f;
    s[k ^ 1] = v16f32{};
#pragma unroll
    for (int n = NV; n < NV + NK; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      s[k ^ 1] = mfma32<BF>(f[n % kAhead], qf[n - NV], s[k ^ 1]);
#pragma unroll
      for (int j = (n - NV) * 8 / NK; j < (n - NV + 1) * 8 / NK; ++j) weigh(k, j);
      if (n + kAhead < NV + NK) f[n % kAhead] = fragment(n + kAhead);
    }
    __builtin_amdgcn_sched_barrier(0);
    total(k);
  };

  auto load_meta = [&](int i) {
    mul = *reinterpret_cast<const v4f*>(s_mul[i & 1]);
    base0 = *reinterpret_cast<const v4f*>(s_base[i & 1]);
    inv = *reinterpret_cast<const v4f*>(s_inv[i & 1]);
  };
  auto first_scores = [&](int i, int k) {
    const uint32_t at = at_k + (uint32_t)(i & 1) * kBuf;
    s[k] = v16f32{};
#pragma unroll
    for (int u = 0; u < NK; ++u) s[k] = mfma32<BF>(frag_k(at, u, k), qf[u], s[k]);
  };
  auto last_outputs = [&](int i, int k) {
    const uint32_t at = at_v + (uint32_t)(i & 1) * kBuf;
#pragma unroll
    for (int n = 0; n < NV; ++n) o[n % ND] = mfma32<BF>(frag_v(at, n, k), p[n / ND], o[n % ND]);
  };

  // ---- the loop over complete pages ----------------------------------------------
  // Step i + 1 (keys of tile i + 1, values of tile i) goes to LDS in the first half
  // of tile i and is read from the second half on; what the first half still reads,
  // keys of tile i and values of tile i - 1, is in the other buffers.
  if (n_coded > 0) {
#pragma unroll
    for (int u = 0; u < CPT; ++u) load_page(u, 0);
#pragma unroll
    for (int u = 0; u < CPT; ++u) load_chunk(u, 0);
#pragma unroll
    for (int u = 0; u < CPT; ++u) load_page(u, 1);
    const bool meta = t < 4;
    if (meta) {
      load_meta_page(0);
      load_scales();
      load_meta_page(1);
    }
#pragma unroll
    for (int u = 0; u < CPT; ++u)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!is_k(u)) raw[u] = v4u{0, 0, 0, 0};   // values of tile -1, multiplied by no weight
        store_piece(u, w, 0);
      }
    if (meta) {
      store_meta(0, meta_ok, ks, vs);
      load_scales();
      load_meta_page(2);
    }
#pragma unroll
    for (int u = 0; u < CPT; ++u) load_chunk(u, 1);
#pragma unroll
    for (int u = 0; u < CPT; ++u) load_page(u, 2);
    lds_sync();
    if (!idle) first_scores(0, 0);
    for (int i = 0; i < n_coded; ++i) {
      load_meta(i);
      if (meta) {
        store_meta(i + 1, meta_ok, ks, vs);
        load_scales();
        load_meta_page(i + 3);
      }
      // the staging in the first slots: convert and store step i + 1, load step i + 2
      auto stage = [&](int n) {
        constexpr int kPer = (4 * CPT + NV - 1) / NV;   // units a slot
#pragma unroll
        for (int x = n * kPer; x < (n + 1) * kPer; ++x) {
          if (x < 2 * CPT) store_piece(x / 2, x % 2, i + 1);
          else if (x < 3 * CPT) load_chunk(x - 2 * CPT, i + 2);
          else if (x < 4 * CPT) load_page(x - 3 * CPT, i + 3);
        }
      };
      if (idle) {
#pragma unroll
        for (int u = 0; u < CPT; ++u) asm volatile("" : "+v"(raw[u]));   // (converted here, not before)
#pragma unroll
        for (int n = 0; n < NV; ++n) stage(n);
      } else {
        half_tile(i, 0, stage);
      }
      lds_sync();
      // (past the last tile the scores are of whatever the buffer holds, and unused)
      if (!idle) half_tile(i, 1, [](int) {});
    }
    if (!idle) last_outputs(n_coded - 1, 1);
  }
  // ---- the keys of the incomplete page, 16 bits each, a tile at a time -------------
  // Infinities and NaNs among the values are cleared, since a hidden key's weight of 0
  // would spread them over all rows; each row then adds those that it sees.
  if (t < 2) s_odd[t] = 0;
  for (int j = 0; j < n_tail; ++j) {
    const int t0 = coded + j * kApTile, r0 = j * kApTile;
    const int slot = a.s.slots ? a.s.slots[b] : b;
    const bool ok = slot >= 0 && slot < a.c.n_slots;
    const size_t f = ((size_t)(ok ? slot : 0) * H + h) * page_sz;
    const int n = ok ? min(sq.len - t0, kApTile) : 0;
    lds_sync();   // buffer 0 has been read
    for (int c = t; c < kApTile * DP / 8; c += NT) {
      const int key = c / (DP / 8), piece = c % (DP / 8);
      v4u x = {0, 0, 0, 0};
      if (key < n && piece * 8 < D)
        x = *reinterpret_cast<const v4u*>(a.c.kt + f + (size_t)(r0 + key) * D + piece * 8);
      *reinterpret_cast<v4u*>(s_kv + key * DP * 2 + ((piece ^ (key & KMASK)) << 4)) = x;
    }
    uint32_t odd = 0;
    for (int c = t; c < DP * kApTile / 8; c += NT) {   // past the length: zeros
      const int d = c >> 3, piece = c & 7, nv = n - piece * 8;
      v4u x = {0, 0, 0, 0};
      if (nv > 0 && d < D)
        x = *reinterpret_cast<const v4u*>(a.c.vt + f + (size_t)d * P + r0 + piece * 8);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] &= (2 * q < nv ? 0xffffu : 0u) | (2 * q + 1 < nv ? 0xffff0000u : 0u);
        const uint32_t bad = odd_halves<BF>(x[q]);
        odd |= bad;
        x[q] = clear_halves(x[q], bad);
      }
      *reinterpret_cast<v4u*>(s_kv + kKeys + d * kApTile * 2 + ((piece ^ ((d >> 1) & 7)) << 4)) = x;
    }
    if (odd) s_odd[j] = 1;   // (at most two tiles)
    if (t < 4) store_meta(0, ok, 1.0f, 1.0f);
    lds_sync();
    load_meta(0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (idle) break;
      first_scores(0, k);
      top = -__builtin_inff();
      add[0] = add[1] = 0.0f;
#pragma unroll
      for (int g = 0; g < 2; ++g) bias[g] = bias_of(t0, k, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) shift(k, e);
      settle(t0, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) weigh(k, e);
      total(k);
      last_outputs(0, k);
    }
    if (s_odd[j] != 0) {   // uniform
      for (int key = max(t0, lo); key < min(t0 + kApTile, hi); ++key) {
        const uint16_t* vp = a.c.vt + f + (4 * hf << ps) + key - coded;   // of this lane's outputs
#pragma unroll
        for (int q = 0; q < 4 * ND; ++q) {
          asm volatile("" : "+v"(vp));   // (an address at a time)
          if (8 * q + 4 * hf < D)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[q >> 2][4 * (q & 3) + e] += odd_value<BF>(vp[e << ps]);
          vp += 8 << ps;
        }
      }
    }
  }

  // ---- the drafts, a tile at a time, in the tail's way: values are transposed on their
  // way into LDS (two drafts' 8 dimensions a thread, as 8 dwords of two drafts)
  if constexpr (TREE) {
    const int n_drafts = drafts ? sq.n : 0;
    for (int t0 = 0; t0 < n_drafts; t0 += kApTile) {
      const int n = min(n_drafts - t0, kApTile);
      lds_sync();   // buffer 0 and s_odd have been read
      if (t == 0) s_odd[0] = 0;
      for (int c = t; c < kApTile * DP / 8; c += NT) {
        const int key = c / (DP / 8), piece = c % (DP / 8);
        v4u x = {0, 0, 0, 0};
        if (key < n && piece * 8 < D)
          x = *reinterpret_cast<const v4u*>(a.dk + (sq.c0 + t0 + key) * a.dk_ts + h * a.dk_hs + piece * 8);
        *reinterpret_cast<v4u*>(s_kv + key * DP * 2 + ((piece ^ (key & KMASK)) << 4)) = x;
      }
      uint32_t odd = 0;
      for (int c = t; c < kApTile / 2 * DP / 8; c += NT) {
        const int key = 2 * (c % (kApTile / 2)), d = c / (kApTile / 2) * 8;
        v4u x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u] = v4u{0, 0, 0, 0};
          if (key + u < n && d < D)
            x[u] = *reinterpret_cast<const v4u*>(a.dv + (sq.c0 + t0 + key + u) * a.dv_ts + h * a.dv_hs + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t bad = odd_halves<BF>(x[u][e]);
            odd |= bad;
            x[u][e] = clear_halves(x[u][e], bad);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint32_t*>(s_kv + kKeys + (d + e) * kApTile * 2 +
                                       (((key >> 3) ^ (((d + e) >> 1) & 7)) << 4) + (key & 7) * 2) =
              __builtin_amdgcn_perm(x[1][e >> 1], x[0][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
      }
      if ((ALIBI || a.window > 0) && t < kApTile)
        s_pos[t] = position<TREE>(a, sq, min(t0 + t, sq.n - 1));
      if (t < 4) store_meta(0, true, 1.0f, 1.0f);
      lds_sync();
      if (odd) s_odd[0] = 1;
      load_meta(0);
      uint64_t word = live ? draft_mask(a, sq, qi, t0 >> 6) : 0;
      if (a.window > 0)
        for (int i = 0; i < n; ++i)
          if (pos - s_pos[i] >= a.window) word &= ~(1ull << i);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (idle) break;
        first_scores(0, k);
        top = -__builtin_inff();
        add[0] = add[1] = 0.0f;
        const uint32_t half = (uint32_t)(word >> (32 * k));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = 16 * (r >> 3) + 8 * hf + (r & 7);
          float x = __builtin_fmaf(s[k][r], sc, -m);
          if (ALIBI) x = __builtin_fmaf(-slope, (float)(pos - s_pos[32 * k + key]), x);
          x = half >> key & 1 ? x : -__builtin_inff();
          s[k][r] = x;
          top = __builtin_fmaxf(top, x);
        }
        move_top(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) weigh(k, e);
        total(k);
        last_outputs(0, k);
      }
      lds_sync();
      if (s_odd[0] != 0) {   // uniform
        for (int key = 0; key < n; ++key) {
          const uint16_t* vp = a.dv + (sq.c0 + t0 + key) * a.dv_ts + h * a.dv_hs + 4 * hf;
          if (word >> key & 1)
#pragma unroll
            for (int q = 0; q < 4 * ND; ++q)
              if (8 * q + 4 * hf < D)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[q >> 2][4 * (q & 3) + e] += odd_value<BF>(vp[8 * q + e]);
        }
      }
    }
  }

  float l_lo, l_hi;
  halves(l, &l_lo, &l_hi);
  const float sum = l_lo + l_hi;
  if (!live) return;
  if (SHARE ? seg.part < 0 : n_split == 1) {
    const int64_t row_out = (sq.c0 + qi) * H * G + h * G + qg;
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;   // no key at all: 0
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = 32 * d + 8 * q + 4 * hf;
        if (at < D) {
          uint2 x;
          x.x = pack2<BF>(o[d][4 * q] * f, o[d][4 * q + 1] * f);
          x.y = pack2<BF>(o[d][4 * q + 2] * f, o[d][4 * q + 3] * f);
          *reinterpret_cast<uint2*>(a.out + row_out * D + at) = x;
        }
      }
    return;
  }
  float *po, *ml;
  if constexpr (SHARE) {
    const size_t at = share_row(a, seg.part, h, kRows, rr - r_wg);
    po = share_out(a, kRows, at);
    ml = share_ml(a, at);
  } else {
    const size_t at = part_at(a, b, h, rr, split);
    po = part_out(a, at);
    ml = a.part + 2 * at;
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = 32 * d + 8 * q + 4 * hf;
      if (e < D)
        *reinterpret_cast<v4f*>(po + e) =
            v4f{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
    }
  if (hf == 0) {
    ml[0] = limit < 0.0f ? -__builtin_inff() : m;
    ml[1] = sum;
  }
}

template <bool BF, int DP, int NW, bool ALIBI, bool TREE>
__global__ __launch_bounds__(64 * NW, DP > 128 ? 1 : 2) void attn_run_kernel(ArgsOf<TREE> a) {
  // the last rows see the most keys: they go first
  const int H = a.c.H, r_wg = ((int)gridDim.x / H - 1 - (int)blockIdx.x / H) * 32 * NW;
  attn_run<BF, DP, NW, ALIBI, TREE, false>(a, blockIdx.z, blockIdx.x % H, r_wg, blockIdx.y, Segment{});
}

template <bool BF, int DP, bool ALIBI>
__global__ __launch_bounds__(512, 2) void attn_share_kernel(TreeArgs a) {
  __shared__ SharePlan s_plan[kShareSeqs];
  __shared__ int s_each, s_total;
  const int H = a.c.H, s = blockIdx.x / H;
  if (threadIdx.x < 64) {
    int each, total;
    s_plan[threadIdx.x] = plan_shares(a, 256, &each, &total);
    if (threadIdx.x == 0) {
      s_each = each;
      s_total = total;
    }
  }
  __syncthreads();
  const int to = __builtin_amdgcn_readfirstlane(min((s + 1) * s_each, s_total));
  for (int x = __builtin_amdgcn_readfirstlane(s * s_each); x < to;) {
    const Segment g = segment_at(s_plan[threadIdx.x & 63], x, to, s);
    attn_run<BF, DP, 8, ALIBI, true, true>(a, g.b, blockIdx.x % H, 256 * g.tile, 0, g);
    x = g.next;
    __syncthreads();   // the segment's tiles have been read
  }
}

// The segments of one row together, where its tile has more than one: `lanes` neighbouring
// lanes a row (a power of two, four elements each), lane s of them weighs segment s; the
// outputs of eight segments are on their way at a time.
template <bool BF>
__global__ __launch_bounds__(256) void share_join_kernel(TreeArgs a, int lanes) {
  constexpr int rows = 256;
  const int D = a.c.D, H = a.c.H, G = a.G, b = blockIdx.z, h = blockIdx.y;
  const int t = threadIdx.x, mine = t & (lanes - 1), d = 4 * mine;
  const int R = (int)blockIdx.x * (256 / lanes) + t / lanes;
  const int32_t* table = reinterpret_cast<const int32_t*>(a.part);
  const Rows sq = rows_of(a, b);
  const int n_rows = sq.n * G;
  if ((int)blockIdx.x * (256 / lanes) >= n_rows) return;   // uniform
  const int r = min(R, n_rows - 1), tile = r / rows;
  const int each = table[2 * kShareSeqs], c = table[kShareSeqs + b] + kShareCost, x0 = table[b] + tile * c;
  const int s_first = x0 / each, n = (x0 + c - 1) / each - s_first + 1;
  if (n < 2) return;   // (a workgroup's rows are of one tile: 256 / lanes divides 256)
  // segment i: of workgroup s_first + i, the first in its place 1, the others in place 0
  auto row_of_part = [&](int i) { return share_row(a, 2 * (s_first + i) + (i == 0), h, rows, r - tile * rows); };
  float m = -__builtin_inff();
  for (int s = mine; s < n; s += lanes) m = __builtin_fmaxf(m, share_ml(a, row_of_part(s))[0]);
  for (int off = 1; off < lanes; off <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, off, 64));
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f;
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < n; s0 += lanes) {
    float f = 0.0f, ls = 0.0f;
    if (s0 + mine < n) {
      const float* ml = share_ml(a, row_of_part(s0 + mine));
      f = __builtin_amdgcn_exp2f(ml[0] - ms);
      ls = ml[1];
      l = __builtin_fmaf(ls, f, l);
    }
    const int left = min(lanes, n - s0);
    for (int j = 0; j < left; j += 8) {
      float fj[8];
      v4f x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int from = (t & 63 & ~(lanes - 1)) + min(j + e, lanes - 1);
        fj[e] = __shfl(f, from, 64);
        // an empty segment has no output; one whose weight underflows counts, by an infinity in it
        const bool some = j + e < left && __shfl(ls, from, 64) != 0.0f;
        x[e] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (some && d < D)
          x[e] = *reinterpret_cast<const v4f*>(share_out(a, rows, row_of_part(s0 + j + e)) + d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[e][i], fj[e], o[i]);
    }
  }
  for (int off = 1; off < lanes; off <<= 1) l += __shfl_xor(l, off, 64);
  if (R >= n_rows || d >= D) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2 w;
  w.x = pack2<BF>(o[0] * inv, o[1] * inv);
  w.y = pack2<BF>(o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2*>(a.out + ((sq.c0 + R / G) * H * G + h * G + R % G) * (int64_t)D + d) = w;
}

// The splits of one row together: one wave per row.  Lane s weighs split s; the
// outputs of eight splits are on their way at a time.
template <bool BF>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63, h = blockIdx.y, b = blockIdx.z;
  const int R = blockIdx.x * 4 + (threadIdx.x >> 6);
  const Rows sq = rows_of(a, b);
  if (R >= sq.n * a.G) return;
  const int H = a.c.H, D = a.c.D;
  const size_t at = part_at(a, b, h, R, 0);
  const float* ml = a.part + 2 * at;
  const float* po = part_out(a, at);
  float m = -__builtin_inff();
  for (int s = lane; s < a.n_split; s += 64) m = __builtin_fmaxf(m, ml[2 * s]);
  m = wave_max(m);
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // elements lane + 64 u
  for (int s0 = 0; s0 < a.n_split; s0 += 64) {
    float f = 0.0f, ls = 0.0f;
    if (s0 + lane < a.n_split) {
      f = __builtin_amdgcn_exp2f(ml[2 * (s0 + lane)] - ms);
      ls = ml[2 * (s0 + lane) + 1];
      l = __builtin_fmaf(ls, f, l);
    }
    // an empty split has no output; one whose weight underflows counts, by an infinity in it
    const uint64_t some = __ballot(ls != 0.0f);
    const int n = min(64, a.n_split - s0);
    for (int j = 0; j < n; j += 8) {
      float fj[8], x[8][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        fj[e] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), j + e));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[e][u] = (some >> (j + e) & 1) && 64 * u < D && lane + 64 * u < D
                        ? po[(size_t)(s0 + j + e) * D + lane + 64 * u]
                        : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = __builtin_fmaf(x[e][u], fj[e], acc[u]);
    }
  }
  for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, 64);
  const int i = R / a.G, g = R % a.G;
  uint16_t* out = a.out + ((sq.c0 + i) * H * a.G + h * a.G + g) * (int64_t)D;
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
  const int64_t rows = (int64_t)G * max_q, heads = (int64_t)B * H;
  // keys that a tile of `n` rows sees (from a multiple of 128 on)
  auto range_of = [&](int n) -> int64_t {
    return window > 0 ? std::min((int64_t)max_len, (int64_t)window + n / G + 129) : max_len;
  };
  // Up to 16 rows are one tile of attn_decode_kernel, which reads the keys once for
  // each 16 rows; more take attn_run_kernel, unless the call is so short that its
  // longer way per tile, or the join of a split, shows (8 kv heads: 256 rows over 1024
  // keys 16.6 against 20.0 us, 2048 rows 32.2 against 39.3; 64 rows over 8192 keys 27.8
  // against 24.2, 256 rows 69 against 37), or it has so few rows more over so many
  // keys that it does not keep memory as busy (64 heads, 32 rows over 65536 keys: 296
  // against 382; 64 rows 487 against 375).
  p.rows = 16;
  const int64_t keys = heads * range_of(16);
  if (rows > 16 &&
      keys * ((rows + 15) / 16) > (range_of(16) <= 1024 ? 1 << 20 : 1 << 18) &&
      !(rows <= 32 && keys >= (1 << 22))) {
    // Wider tiles stage and convert a key for more rows (8 kv heads, 2048 rows over
    // 8192 keys: 128 -> 93 us); narrow ones where the rows, or a short range, would
    // leave compute units idle (64 heads, 512 rows over 1024 keys: 54 -> 37 us).
    const int64_t wide = heads * ((rows + 255) / 256);
    p.rows = rows > 128 && D <= 128 && (wide >= 256 || range_of(256) > 2048) ? 256 : 128;
  }
  // Splits for about 16 (single rows: ragged lengths even out), 2 or 1 workgroups a
  // compute unit; of at least 256 keys, or 1024 where the tiles alone fill the chip
  // (the join is a launch more).
  const int64_t range = range_of(p.rows);
  const int64_t tiles = heads * ((rows + p.rows - 1) / p.rows);
  const int64_t fill = p.rows == 16 ? 4096 : p.rows == 128 ? 512 : 256;
  const int64_t want = std::max<int64_t>(fill / tiles, 1);
  const int64_t c = std::max<int64_t>(((range + want - 1) / want + 255) / 256 * 256,
                                      tiles >= 256 ? 1024 : 256);
  p.chunk = (int)c;
  p.n_split = std::max((int)((range + c - 1) / c), 1);
  return p;
}

template <bool BF, bool ALIBI, bool TREE>
void launch_kernel(const ArgsOf<TREE>& a, const Plan& p, hipStream_t stream) {
  const int D = a.c.D;
  const dim3 grid(a.c.H * ((a.G * a.max_q + p.rows - 1) / p.rows), a.n_split, a.s.B);
  if constexpr (TREE)
    if (a.shares) {
      const dim3 all(a.c.H * a.shares);
      if (D <= 64) hipLaunchKernelGGL((attn_share_kernel<BF, 64, ALIBI>), all, dim3(512), 0, stream, a);
      else hipLaunchKernelGGL((attn_share_kernel<BF, 128, ALIBI>), all, dim3(512), 0, stream, a);
      return;
    }
  if (p.rows == 16) {
    const dim3 block(kAdThreads);
    if (D <= 64) hipLaunchKernelGGL((attn_decode_kernel<BF, 64, ALIBI, TREE>), grid, block, 0, stream, a);
    else if (D <= 128)
      hipLaunchKernelGGL((attn_decode_kernel<BF, 128, ALIBI, TREE>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_decode_kernel<BF, 256, ALIBI, TREE>), grid, block, 0, stream, a);
  } else if (p.rows == 128) {
    if (D <= 64)
      hipLaunchKernelGGL((attn_run_kernel<BF, 64, 4, ALIBI, TREE>), grid, dim3(256), 0, stream, a);
    else if (D <= 128)
      hipLaunchKernelGGL((attn_run_kernel<BF, 128, 4, ALIBI, TREE>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((attn_run_kernel<BF, 256, 4, ALIBI, TREE>), grid, dim3(256), 0, stream, a);
  } else {
    if (D <= 64)
      hipLaunchKernelGGL((attn_run_kernel<BF, 64, 8, ALIBI, TREE>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((attn_run_kernel<BF, 128, 8, ALIBI, TREE>), grid, dim3(512), 0, stream, a);
  }
}

template <bool BF, bool TREE>
hipError_t launch_typed(const ArgsOf<TREE>& a, const Plan& p, hipStream_t stream) {
  if (a.alibi) launch_kernel<BF, true, TREE>(a, p, stream);
  else launch_kernel<BF, false, TREE>(a, p, stream);
  const hipError_t e = hipGetLastError();
  if constexpr (TREE)
    if (e == hipSuccess && a.shares) {
      int lanes = 4;
      while (4 * lanes < a.c.D) lanes *= 2;
      const int per = 256 / lanes;
      hipLaunchKernelGGL((share_join_kernel<BF>), dim3((a.G * a.max_q + per - 1) / per, a.c.H, a.s.B),
                         dim3(256), 0, stream, a, lanes);
      return hipGetLastError();
    }
  if (e != hipSuccess || a.n_split == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<BF>), dim3((a.G * a.max_q + 3) / 4, a.c.H, a.s.B),
                     dim3(256), 0, stream, static_cast<const AttnArgs&>(a));
  return hipGetLastError();
}

// Workgroups a head that a call with trees is shared out to (0: the splits above): one a
// compute unit.  Only where sequences are several and long enough for their lengths to
// matter (64 drafts, 32 heads on 8: 8 sequences of up to 4096 tokens 52 us against 58, 2 of
// them 32 against 36, 48 of them 187 against 210; 16 of up to 1024 tokens 42.5 against 42.1, of
// 2048 78 either way; 32 of up to 1024, 60 drafts of 32 heads on 4, 63 against 49); a window
// bounds the lengths, a plan has room for 64 sequences, and 128 tiles keep the number of
// blocks (of at most 2^30 keys each) in 32 bits.
int tree_shares(const Plan& p, int B, int H, int G, int max_q, int max_len, int window) {
  return p.rows == 256 && B > 1 && B <= kShareSeqs && B * (((int64_t)G * max_q + 255) / 256) <= 128 &&
                 window == 0 && max_len > 2048 && H <= 128
             ? 256 / H
             : 0;
}

// Chooses the kernel and the split, and launches.
template <bool TREE>
hipError_t launch_planned(ArgsOf<TREE> a, hipStream_t stream) {
  const Plan p = plan(a.s.B, a.c.H, a.G, a.c.D, a.max_q, a.max_len, a.window);
  a.chunk = p.chunk;
  a.n_split = p.n_split;
  if constexpr (TREE) a.shares = tree_shares(p, a.s.B, a.c.H, a.G, a.max_q, a.max_len, a.window);
  return a.c.bf16 ? launch_typed<true, TREE>(a, p, stream) : launch_typed<false, TREE>(a, p, stream);
}

}  // namespace

}  // namespace i8l
