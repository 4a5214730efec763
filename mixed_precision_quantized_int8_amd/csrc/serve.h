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

// kv rows: element (t, h, d) at t * ts + h * hs + d.
hipError_t launch_cache_write(const Cache& c, const Sequences& s, const uint16_t* k,
                              const uint16_t* v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                              int64_t v_hs, int64_t rows, int max_new, hipStream_t stream);
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
hipError_t launch_attention(AttnArgs a, hipStream_t stream);

}  // namespace i8l
