// Keys and values into the 8-bit cache with the keys' norm and rotation on the way, and
// the queries' in the same launch: what rotate_heads and cache_write give one after the
// other, bit for bit (the formulas are in rotary.h and kvcache.hip).
//
// A launch has three kinds of workgroups: a page of one head's keys, a page of one head's
// values (kvcache.hip's way), and queries.  Keys are stored as they come, [token][D], so a
// page of them is cut by rotary.h's units: 16 elements of one token a thread, both
// elements of each pair among them, the norm's sum over a few neighbouring lanes.  The
// turned keys are rounded to 16 bits, as the tail keeps them, before they are coded.
//
// Bound by HBM and, for the keys, by the vector unit: every head forms its own angles.
// 24.8 thousand tokens of four sequences, bf16, 32 query heads on 8 of 128, norms on
// both: 560 MB in 132 us, 4.2 TB/s (the queries alone 79 us, 5.1 TB/s; keys and values 62,
// as cache_write without turning 38).  One token each of 16 sequences: 6 us, latency.
#include <algorithm>

#include "pages.h"
#include "rotary.h"

namespace i8l {

// One page of one head of keys; task and tail as for write_page.
template <bool BF, int LAYOUT, int BS, int NU>
__device__ __forceinline__ void append_keys(const Cache& c, const Sequences& s, const CacheRows& x,
                                            const HeadArgs& a, const uint16_t* k_w, int b, int h,
                                            int task, v4u* held, float* row, uint32_t* red) {
  constexpr int NT = 2 * NU;   // tokens a thread
  const int ps = c.ps, P = 1 << ps, D = c.D, t = threadIdx.x, lane = t & 63;
  const int lanes = lanes_of(D), j = t & (lanes - 1);
  const Span sp = seq_span<true>(s, b, ps, x);
  const int p0 = sp.p0;
  if (p0 >= sp.len) return;
  const int g0 = p0 >> ps, gl = (sp.len - 1) >> ps;
  const int g = g0 + task;
  if (g > gl) return;
  const int full = sp.len >> ps;   // complete pages
  const int slot = s.slots ? s.slots[b] : b;
  const bool slot_ok = slot >= 0 && slot < c.n_slots;
  uint16_t* tail = c.kt + ((size_t)(slot_ok ? slot : 0) * c.H + h) * P * D;
  const uint16_t* rows = x.x[0] + h * x.hs[0];
  const Runs at = runs_of<LAYOUT>(a.turn, j);
  const float inv = 1.0f / (float)D;
  // A token's 16 elements, normed and turned (every lane of the wave takes part).  Weights and
  // frequencies come from the cache for each token: kept, their registers would cost waves.
  auto turned = [&](v4u (&p)[2], int pos) {
    int zero = 0;
    asm volatile("" : "+s"(zero));
    float y[16], freq[Angles<LAYOUT>::N];
    v4u w[2];
    if (LAYOUT != kTurnOdd)
#pragma unroll
      for (int e = 0; e < Angles<LAYOUT>::N; ++e)
        freq[e] = a.turn.pairs ? a.turn.freqs[zero + max(Angles<LAYOUT>::pair(a.turn, j, e), 0)] : 0.0f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      w[r] = v4u{0, 0, 0, 0};
      if (k_w && at.at[r] < D) w[r] = *reinterpret_cast<const v4u*>(k_w + zero + at.at[r]);
    }
    unpack<BF>(p, y);
    if (k_w) {
      const Rms m = rms_of<BF>(y, inv, lanes, a.eps);
      float wf[16];
      unpack<BF>(w, wf);
      over_rms(y, m);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] *= wf[e];
    }
    Angles<LAYOUT> angles;
    if constexpr (LAYOUT == kTurnOdd) odd_angles_at(angles, a.turn, lanes, j, pos, row, lane);
    else angles_at(angles, a.turn, j, pos, freq);
    turn<LAYOUT>(y, angles, a.turn, j, row, lane);
    pack<BF>(y, p);
  };
  if (g < full) {
    const int page = s.table[(size_t)b * s.max_pages + g];
    const bool page_ok = page >= 0 && page < c.n_pages;
    // A token at a time, the next two's elements on their way; what is turned waits in LDS
    // for the page's maximum (a thread reads back what it wrote).
    const auto load = [&](int u, v4u (&p)[2]) {
      const int tok = (t + u * BS) / lanes, pos = (g << ps) + tok;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        p[r] = v4u{0, 0, 0, 0};
        if (tok < P && at.at[r] < D) {
          if (pos >= p0)
            p[r] = *reinterpret_cast<const v4u*>(rows + row_of<true>(x, sp.c0 + pos - p0) * x.ts[0] + at.at[r]);
          else if (slot_ok)
            p[r] = *reinterpret_cast<const v4u*>(tail + tok * D + at.at[r]);
        }
      }
    };
    // magnitudes of both types are in the order of their bits, infinities and NaNs last
    u16x2 mag = {0, 0};
    v4u next[2], after[2];
    load(0, next);
    load(1, after);
#pragma unroll 1
    for (int u = 0; u < NT; ++u) {
      v4u p[2] = {next[0], next[1]};
      next[0] = after[0];
      next[1] = after[1];
      if (u + 2 < NT) load(u + 2, after);
      const int pos = (g << ps) + (t + u * BS) / lanes;
      v4u q[2] = {p[0], p[1]};
      turned(q, pos);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (pos >= p0) p[r] = q[r];   // (the tail's tokens are turned already)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mag = __builtin_elementwise_max(mag, __builtin_bit_cast(u16x2, p[r][e] & 0x7fff7fffu));
        held[(u * 2 + r) * BS + t] = p[r];
      }
    }
    uint32_t bits = wave_max_u32(mag[0] > mag[1] ? mag[0] : mag[1]);
    if constexpr (BS > 64) {
      if (lane == 0) red[t >> 6] = bits;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < BS / 64; ++i) bits = max(bits, red[i]);
    }
    const bool finite = bits < (BF ? 0x7f80u : 0x7c00u);
    const float absmax = to_f32<BF>((uint16_t)bits);
    const float top = absmax < kLeastMax ? 0.0f : absmax;
    const float inv65 = (finite ? quant_scale(top) : 0.0f) * 65536.0f;
    int8_t* out = c.kc + ((size_t)(page_ok ? page : 0) * c.H + h) * P * D;
#pragma unroll 1
    for (int u = 0; u < NT; ++u) {
      const int tok = (t + u * BS) / lanes;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const v4u p = held[(u * 2 + r) * BS + t];
        uint32_t z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = to_f32<BF>((uint16_t)(p[e >> 1] >> (16 * (e & 1))));
          z[e] = code_bits(finite ? f : 0.0f, inv65);
        }
        uint2 k;
        k.x = __builtin_amdgcn_perm(z[1], z[0], 0x0c0c0602u) |
              __builtin_amdgcn_perm(z[3], z[2], 0x06020c0cu);
        k.y = __builtin_amdgcn_perm(z[5], z[4], 0x0c0c0602u) |
              __builtin_amdgcn_perm(z[7], z[6], 0x06020c0cu);
        if (page_ok && tok < P && at.at[r] < D)
          *reinterpret_cast<uint2*>(out + tok * D + at.at[r]) = k;
      }
    }
    if (t == 0 && page_ok) c.ks[(size_t)page * c.H + h] = finite ? top / 127.0f : __builtin_nanf("");
  }
  if (task == 0 && gl >= full && slot_ok) {   // the last page stays incomplete
    __syncthreads();   // the old tail has been read
    const int lo = max(p0, full << ps);
    for (int q0 = 0; q0 < (sp.len - lo) * lanes; q0 += BS) {   // uniform
      const int pos = lo + (q0 + t) / lanes;
      const bool live = pos < sp.len;
      v4u p[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        p[r] = v4u{0, 0, 0, 0};
        if (live && at.at[r] < D)
          p[r] = *reinterpret_cast<const v4u*>(
              rows + row_of<true>(x, sp.c0 + pos - p0) * x.ts[0] + at.at[r]);
      }
      turned(p, pos);
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (live && at.at[r] < D)
          *reinterpret_cast<v4u*>(tail + (pos & (P - 1)) * D + at.at[r]) = p[r];
    }
  }
}

// (Pages of up to 8192 elements, NU 1: 80 registers, for six waves a SIMD: 24.8 k tokens, 32
// heads on 8, 132 us, with 93 registers 137; keys kept in registers as values are, 126 of
// them, 148.  Larger pages hold more: NU 2 92 - 101 registers and 32 KB of LDS, four waves,
// NU 4 64 KB, two; queries share the launch and have no more.  8192 tokens, 8 heads: of 128
// on 32 41.6 us with pages of 64 (NU 1), 42.0 of 128 (2); of 256 on 8 51.3 with pages of 32,
// 53.5 of 64 (2), 65.0 of 128 (4).  Halves through LDS do not fit: 132 - 160 registers,
// three waves, one with NU 4.)
template <bool BF, int LAYOUT, int BS, int NU>
__global__ __launch_bounds__(BS) __attribute__((amdgpu_waves_per_eu(LAYOUT == kTurnOdd ? 2 : 6)))
void cache_append_kernel(Cache c, Sequences s, CacheRows x, HeadArgs a, const uint16_t* k_w,
                         uint32_t page_blocks, int n_tok, int groups, int per_wg) {
  // a page of keys in 16 bits, or of values in 8, or the angles of a workgroup's queries
  __shared__ __attribute__((aligned(128))) uint8_t lds[BS * NU * 64];
  static_assert(sizeof(lds) >= 2048, "kTurnTokens * 64 angles; 128 come with twice the threads");
  __shared__ float s_turn[LAYOUT == kTurnOdd ? BS / 64 * kTurnRow : 1];
  __shared__ uint32_t red[BS / 64];
  const int b = blockIdx.z;
  float* row = s_turn + (LAYOUT == kTurnOdd ? (threadIdx.x >> 6) * kTurnRow : 0);
  if (blockIdx.x < page_blocks) {
    // heads first: neighbours in a launch read neighbours in memory
    const uint32_t hk = blockIdx.x % (2 * c.H);
    const int task = blockIdx.x / (2 * c.H), h = hk >> 1;
    if (hk & 1) write_page<BF, true, BS, NU, true>(c, s, x, b, h, task, lds, red);
    else
      append_keys<BF, LAYOUT, BS, NU>(c, s, x, a, k_w, b, h, task, reinterpret_cast<v4u*>(lds), row, red);
    return;
  }
  const uint32_t parts = (groups + per_wg - 1) / per_wg, q = blockIdx.x - page_blocks;
  int64_t c0 = s.cu ? s.cu[b] : b, c1 = s.cu ? s.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), x.rows);
  c1 = min(max(c1, c0), x.rows);
  if (x.counts) c1 = min(c1, c0 + max(x.counts[b], 0));
  const int64_t i0 = (int64_t)(q / parts) * n_tok;
  if (i0 >= c1 - c0) return;
  const int g0 = q % parts * per_wg, pos0 = (int)(max(s.lengths[b], 0) - (c1 - c0) + i0);
  turn_heads<BF, LAYOUT, BS / 64, 1, false>(
      a, c0 + i0, (int)min((int64_t)n_tok, c1 - c0 - i0), [&](int i) { return pos0 + i; }, g0,
      min(per_wg, groups - g0), lanes_of(a.D), reinterpret_cast<float2*>(lds), row);
}

namespace {
template <bool BF, int LAYOUT, int BS, int NU>
void launch_sized(const Cache& c, const Sequences& s, const CacheRows& x, const HeadArgs& a,
                  const uint16_t* k_w, uint32_t page_blocks, int max_q, hipStream_t stream) {
  // The queries' workgroups, as launch_rows has them: a token each, or four where that leaves
  // waves enough and each of them at most eight groups of heads one after the other (40 heads
  // of 128, pages of 64: 16 sequences of 1024 tokens 80 us against 88 with one, 64 of 32 20
  // against 28; pages of 16, where a workgroup is one wave and would have 16 groups, 87
  // against 78 and 22 against 14; of 32, eight groups on two waves, 81 against 81, a quarter
  // of 80 turned 112 against 123, 64 sequences of 64 27 against 24), or where the bound is
  // loose, so that most workgroups have nothing to do (256 sequences of 20 tokens, bounded by
  // their sum: 251 us against 847).
  constexpr int kWaves = BS / 64;
  const int groups = head_groups(a, 0), each = (kTurnTokens * groups + kWaves - 1) / kWaves;
  const int64_t bound = (int64_t)max_q * s.B, rows = std::min(x.rows, bound);
  const int64_t waves = rows / kTurnTokens * kWaves;
  const bool four = max_q >= kTurnTokens &&
                    (bound > 2 * rows ? rows >= 2048
                                      : each <= 8 && waves >= (each <= 4 || kWaves == 4 ? 2048 : 4096));
  const int n_tok = four ? kTurnTokens : 1;
  const int per_wg = n_tok == 1 && groups > BS / 64 && (int64_t)max_q * s.B * groups < 8192 ? BS / 64 : groups;
  const uint32_t q_blocks =
      groups ? (uint32_t)((max_q + n_tok - 1) / n_tok * ((groups + per_wg - 1) / per_wg)) : 0;
  hipLaunchKernelGGL((cache_append_kernel<BF, LAYOUT, BS, NU>), dim3(page_blocks + q_blocks, 1, s.B),
                     dim3(BS), 0, stream, c, s, x, a, k_w, page_blocks, n_tok, groups, per_wg);
}

template <bool BF, int LAYOUT>
void launch_append(const Cache& c, const Sequences& s, const CacheRows& x, const HeadArgs& a,
                   const uint16_t* k_w, int max_new, int max_q, hipStream_t stream) {
  const uint32_t tasks = (max_new + (1 << c.ps) - 2) / (1 << c.ps) + 1;
  const uint32_t page_blocks = tasks * 2 * c.H;
#define I8L_A(BS, NU, _) launch_sized<BF, LAYOUT, BS, NU>(c, s, x, a, k_w, page_blocks, max_q, stream)
  I8L_CACHE_SIZES((lanes_of(c.D) * 16 << c.ps) / 32, I8L_A, 0);
#undef I8L_A
}
}  // namespace

hipError_t launch_cache_append(const Cache& c, const Sequences& s, const AppendRows& r,
                               const HeadArgs& a, int max_new, int max_q, hipStream_t stream) {
  const CacheRows x{{r.k, r.v}, {r.k_ts, r.v_ts}, {r.k_hs, r.v_hs}, r.rows, r.index, r.counts, r.src};
  const TurnLayout layout = turn_layout(a.turn);
#define I8L_L(BF)                                                                            \
  do {                                                                                       \
    if (layout == kTurnHalves) launch_append<BF, kTurnHalves>(c, s, x, a, r.k_w, max_new, max_q, stream); \
    else if (layout == kTurnPairs) launch_append<BF, kTurnPairs>(c, s, x, a, r.k_w, max_new, max_q, stream); \
    else launch_append<BF, kTurnOdd>(c, s, x, a, r.k_w, max_new, max_q, stream);                    \
  } while (0)
  if (c.bf16) I8L_L(true);
  else I8L_L(false);
#undef I8L_L
  return hipGetLastError();
}

}  // namespace i8l
