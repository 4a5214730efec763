// Internal launchers of the serving operators (row norm to codes, product of
// row codes, 8-bit key/value cache, attention over it); the C ABI
// (serve_abi.hip) calls these after validating its arguments on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace i8l {

// Thread-local message buffer behind i8l_last_error (int8lin_abi.hip).
char* error_buffer(size_t* bytes);

// Residual add, root-mean-square norm and row codes (norm.hip).  bf16: the
// element type of X, R, W and H (else fp16).  R, W and H may be NULL.
hipError_t launch_rmsnorm_quant(const uint16_t* X, const uint16_t* R, const uint16_t* W, int M,
                                int K, float eps, bool bf16, int8_t* Xq, float* sx, uint16_t* H,
                                hipStream_t stream);

// The weight-streaming kernel on codes that are already there, M <= kStreamMaxM
// (decode.hip); zeros: at least 16 zero words (no outlier columns).
hipError_t launch_stream_codes(const int8_t* Xq, const float* sx, int M, int K, const int8_t* Wq,
                               const float* sw, int N, const uint16_t* bias, uint16_t* Y,
                               const int32_t* zeros, hipStream_t stream);

// Product of row codes (codes.hip): which kernel, and the partial sums it can use.
struct CodesArgs {
  const int8_t* Xq;
  const float* sx;
  const int8_t* Wq;
  const float* sw;
  const uint16_t* bias;   // fp16 [N] or NULL
  uint16_t* Y;
  int32_t* part;          // p.workspace bytes, or NULL: nothing is split along k
  int M, N, K;
  int n_split;            // set by the launcher
};
struct CodesPlan {
  enum Kind { kStream, kRows, kTiles, kSkinny, kGemm } kind;
  int n_split;
  size_t workspace;       // bytes of partial sums
  int tile_n;             // kTiles: features of a tile, 64 or 128
};
CodesPlan codes_plan(int M, int N, int K);
hipError_t launch_codes(CodesArgs a, const CodesPlan& p, const int32_t* zeros, hipStream_t stream);

// One cache and the sequences of a call.  Pages of P = 1 << ps tokens.
struct Cache {
  int8_t* kc;       // [n_pages][H][P][D]
  int8_t* vc;       // [n_pages][H][D][P]
  float* ks;        // [n_pages][H]
  float* vs;        // [n_pages][H]
  uint16_t* kt;     // [n_slots][H][P][D]
  uint16_t* vt;     // [n_slots][H][D][P]
  int n_pages, n_slots, H, D, ps;
  bool bf16;
};
struct Sequences {
  const int32_t* table;   // [B][max_pages]
  const int32_t* lengths; // [B]
  const int32_t* cu;      // [B + 1] or NULL: one row per sequence
  const int32_t* slots;   // [B] or NULL: slot b
  int B, max_pages;
};

// Rotary positions: pair i of a head turns by position * freqs[i] (rotary.h).
struct Turn {
  const float* freqs;   // [pairs]
  int pairs;
  bool interleaved;
  float factor;         // of cos and sin
};
// Lanes a head: 16 elements each, a power of two (some idle if D is none).
__host__ __device__ inline int lanes_of(int D) {
  int n = 1;
  while (16 * n < D) n *= 2;
  return n;
}
// Heads of two tensors (queries and keys; n 0: none) at the same positions.  x and y:
// element (t, h, d) at t * ts + h * hs + d.
struct HeadArgs {
  struct Side {
    const uint16_t* x;    // input (backward: what went in; NULL without w)
    int64_t x_ts, x_hs;
    const uint16_t* dy;   // backward only
    int64_t dy_ts, dy_hs;
    uint16_t* y;          // output (backward: dx)
    int64_t y_ts, y_hs;
    const uint16_t* w;    // [D] or NULL: no norm
    uint16_t* dw;         // backward: [D], with w
    int n;                // heads
  } side[2];
  Turn turn;
  const int32_t* positions;   // [rows]
  int rows, D;
  float eps;
  bool bf16;
  float* part;          // backward: head_partials floats, where a side has a weight
};
hipError_t launch_rotate_heads(const HeadArgs& a, hipStream_t stream);
// Floats of partial sums that the backward pass needs (0: neither side has a weight).
size_t head_partials(int rows, int D);
hipError_t launch_rotate_heads_backward(const HeadArgs& a, hipStream_t stream);

// kv rows: element (t, h, d) at t * ts + h * hs + d.
hipError_t launch_cache_write(const Cache& c, const Sequences& s, const uint16_t* k,
                              const uint16_t* v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                              int64_t v_hs, int64_t rows, int max_new, hipStream_t stream);
// The same with the keys' norm (k_w, or NULL) and rotation on the way, and the queries'
// in heads.side[0] (n 0: none; heads.positions unused, rows as here); the rows of k and
// v picked by index of their src rows, counts of each sequence's (both may be NULL).
struct AppendRows {
  const uint16_t *k, *v, *k_w;
  int64_t k_ts, k_hs, v_ts, v_hs, src, rows;
  const int32_t *index, *counts;
};
hipError_t launch_cache_append(const Cache& c, const Sequences& s, const AppendRows& x,
                               const HeadArgs& heads, int max_new, int max_q, hipStream_t stream);
// k, v [rows][H][D]; s.cu the first row of each sequence.
hipError_t launch_cache_read(const Cache& c, const Sequences& s, uint16_t* k, uint16_t* v,
                             int64_t rows, int max_len, hipStream_t stream);

struct AttnArgs {
  Cache c;
  Sequences s;
  const uint16_t* q;    // element (t, head, d) at t * q_ts + head * q_hs + d
  int64_t q_ts, q_hs;
  uint16_t* out;        // [rows][H * G][D]
  int64_t rows;
  int G, max_q, max_len, window;
  float scale;          // score factor
  const float* alibi;   // [H * G] or NULL
  // set by the launcher
  float* part;          // partial results, when the keys are split
  int n_split, chunk;
};
// Floats of partial results that launch_attention needs for these sizes (0: none).
size_t attention_partials(int B, int H, int G, int D, int max_q, int max_len, int window);
hipError_t launch_attention(const AttnArgs& a, hipStream_t stream);

// Attention for trees of drafts behind the cached tokens (attn.h): sequence b's drafts
// are its rows; max_q is at least their number.
struct TreeArgs : AttnArgs {
  const uint64_t* masks;      // [rows][words]
  int words;
  const int32_t* positions;   // [rows], or NULL without a window and a bias
  const uint16_t *dk, *dv;    // the drafts' keys and values: element (t, h, d) at
  int64_t dk_ts, dk_hs, dv_ts, dv_hs;   // t * ts + h * hs + d
  // set by the launcher
  int shares;           // workgroups a head that the keys are shared out to, or 0
};
size_t tree_partials(int B, int H, int G, int D, int max_q, int max_len, int window);
hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream);

// A tree of drafts from their parents, and its accepted path (tree.hip).
constexpr int kMaxDrafts = 512;   // of one sequence
struct TreeRows {
  const int32_t *parents, *lengths, *cu;   // cu NULL: one row a sequence
  int64_t rows;
  int n, max_q;
};
hipError_t launch_tree_plan(const TreeRows& r, int32_t* positions, uint64_t* masks, int words,
                            hipStream_t stream);
hipError_t launch_tree_accept(const TreeRows& r, const int64_t* tokens, const int64_t* choices,
                              const int64_t* first, int32_t* path, int32_t* counts,
                              int32_t* new_lengths, int64_t* next, hipStream_t stream);

}  // namespace i8l
