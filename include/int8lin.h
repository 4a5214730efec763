/*
 * int8lin.h -- C ABI of the LLM.int8() quantized linear layer for AMD MI355X
 * (gfx950).  Implemented by libint8lin.so (hand-written HIP kernels).
 *
 * The method is the one described in the blog "A Gentle Introduction to 8-bit
 * Matrix Multiplication for transformers at scale using Hugging Face
 * Transformers, Accelerate and bitsandbytes" (cited as [blog] below):
 *   - vector-wise absmax quantization: one scale per row of the fp16 hidden
 *     states X and one per output column of the weight W
 *     ([blog, "Introduction to model quantization"]);
 *   - mixed-precision decomposition: a column of X holding any value of
 *     magnitude >= threshold (6 in the blog) is an outlier column; outlier
 *     columns are multiplied in fp16 against the matching fp16 rows of W, the
 *     rest in int8 x int8 -> int32; the int8 result is dequantized with the
 *     outer product of the scales over 127^2 and added to the fp16 outlier
 *     product ([blog, "A gentle summary of LLM.int8()"] and
 *     [blog, "A closer look at the MatMul"]).
 *
 * Conventions shared by every entry point
 *   - Tensor pointers are DEVICE pointers (HBM of the current HIP device) and
 *     are row-major.  fp16 tensors are passed as raw IEEE binary16 bits
 *     (uint16_t).  The caller owns and allocates every buffer; the library
 *     allocates no device memory and keeps no state besides a thread-local
 *     error message.
 *   - Every call only enqueues work on `stream` (a hipStream_t; NULL means the
 *     default stream) and returns without synchronizing.  Device-side faults
 *     surface at the caller's next synchronization.
 *   - All argument checks run on the host before any HIP call; on a non-OK
 *     status nothing has been enqueued and i8l_last_error() tells why.
 *   - Shapes: M (rows of X) >= 0, N (output features) >= 0; M == 0 or N == 0
 *     is a valid no-op.  K (input features) must satisfy 16 <= K <= 133136 and
 *     K % 16 == 0 (K * 127^2 must fit in int32).
 *   - Alignment: X, Y, Wq, Xq, acc, X_outliers and workspace pointers must be
 *     16-byte aligned; sw, sx, outlier_idx and n_outliers 4-byte aligned; W and
 *     W_outlier_rows 2-byte aligned.
 *   - Rounding: quantized codes are clamp(round_half_away_from_zero(
 *     fp32(x) * fl32(127 / absmax)), -127, 127), with 127 / absmax an IEEE fp32
 *     division; absmax == 0 gives code 0.
 *   - Functions are reentrant; calls that share a workspace must not overlap.
 */
#ifndef INT8LIN_H
#define INT8LIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  I8L_OK = 0,
  I8L_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad shape, NaN threshold */
  I8L_ERR_K_TOO_LARGE = 2, /* K > 133136: int32 accumulators could overflow */
  I8L_ERR_WORKSPACE = 3,   /* workspace smaller than required */
  I8L_ERR_HIP = 4          /* a HIP launch or runtime call failed */
} i8l_status;

/* Largest supported K (K * 127 * 127 < 2^31, rounded down to a multiple of 16). */
#define I8L_MAX_K 133136

/* Largest K of the zero-point entry points (K * 255 * 127 < 2^31, a multiple
 * of 16): every sum_k (q - zp) * w then fits in int32. */
#define I8L_MAX_K_ZP 66304

/* Byte offsets, inside the int8_linear / int8_quantize_activation workspace, of
 * the intermediates that the call leaves there.  After an int8_linear call
 * (once the stream has reached it) the workspace holds, for that call:
 *   n_outliers   int32 [1]        number of outlier columns n_out
 *   outlier_idx  int32 [K] cap    ascending outlier column indices, first n_out
 *   sx           fp32  [M]        row absmax of X over the regular columns
 *   Xq           int8  [M][K]     row-quantized X, 0 in outlier columns
 *   X_outliers   fp16  [M][K] cap outlier values, element (i, j) at i*K + j,
 *                                 j < n_out, j-th outlier column in ascending order
 *   flags        uint32 [ceil(K/32)] internal: outlier column bitmask
 *   zero_points  int32 [M]        int8_linear_zp only: the row zero points;
 *                                 sx then holds range / 255 and Xq the codes
 *                                 minus 128 (see int8_quantize_activation_zp);
 *                                 internal for absmax codes
 *   act_partials uint32           internal (1 <= M <= 16): per 512-column
 *                                 slice of K, its outlier count and per-row
 *                                 partial maxima / minima of the activation
 *                                 stage (0 bytes for other M)
 *   gemm_counters, gemm_partials   internal (M > 64): a reserved region and
 *                                 int32 partial tiles of the GEMM's split-K
 *                                 tail; gemm_slices partial tiles of 256x256
 * `total` is the size the call requires; it depends on M, K and N. */
typedef struct {
  size_t total;
  size_t n_outliers;
  size_t outlier_idx;
  size_t sx;
  size_t Xq;
  size_t X_outliers;
  size_t flags;
  size_t gemm_counters;
  size_t gemm_partials;
  size_t gemm_slices;
  size_t zero_points;
  size_t act_partials;
} i8l_workspace_layout;

/* Fills *layout for an int8_linear call of this shape.
 * Returns I8L_ERR_INVALID_ARG / I8L_ERR_K_TOO_LARGE on a bad shape. */
i8l_status i8l_linear_workspace(int64_t M, int64_t K, int64_t N, i8l_workspace_layout *layout);

/* Workspace bytes int8_linear needs for this shape (0 on a bad shape). */
size_t i8l_linear_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* Weight quantization ([blog, "A closer look at the MatMul"]: the weight is
 * quantized per column; [blog, "Usage"]: it happens once, when the layer is
 * placed on the GPU, and keeps the int8 weight in nn.Linear's [out][in] layout
 * next to one absmax per output feature).
 *   W   fp16 [K][N]  math layout (Y = X @ W), read only
 *   Wq  int8 [N][K]  out: Wq[n][k] = code(W[k][n], sw[n])
 *   sw  fp32 [N]     out: sw[n] = max_k |W[k][n]| */
i8l_status int8_quantize_weight(const uint16_t *W, int64_t K, int64_t N,
                                int8_t *Wq, float *sw, void *stream);

/* The LLM.int8() linear layer: Y = dequant(int8 part) + fp16 outlier part.
 *   X               fp16 [M][K]  hidden states, read only
 *   Wq, sw          from int8_quantize_weight for the same K, N
 *   W_outlier_rows  fp16 [K][N]  the fp16 weight in math layout; only rows
 *                   that are outlier columns of X are read.  NULL: no fp16
 *                   weight is kept, and each outlier weight value is rebuilt
 *                   from its code as fp16(fl32(Wq[n][k] * sw[n]) / 127)
 *                   ([blog, "Usage"]: the int8 weight times its per-output
 *                   scale over 127 gives the weight back).
 *   threshold       finite > 0: columns of X with any |x| >= threshold are
 *                   outliers; <= 0 or +inf: no decomposition (pure int8);
 *                   NaN: I8L_ERR_INVALID_ARG.
 *   Y               fp16 [M][N]  out: fp16(acc*sx[i]*sw[n]/127^2 + outlier
 *                   product), accumulated in fp32, round-to-nearest-even,
 *                   overflow to +/-inf.
 *   workspace       device scratch of i8l_linear_workspace_bytes(M, K, N)
 *                   bytes; it holds the call's intermediates afterwards (see
 *                   i8l_workspace_layout). */
i8l_status int8_linear(const uint16_t *X, int64_t M, int64_t K,
                       const int8_t *Wq, const float *sw, int64_t N,
                       const uint16_t *W_outlier_rows, float threshold,
                       uint16_t *Y, void *workspace, size_t workspace_bytes,
                       void *stream);

/* int8_linear with a bias, for a linear layer that has one ([blog, "Usage"]:
 * the 8-bit layer takes nn.Linear's bias argument).
 *   bias   fp16 [N], 2-byte aligned, or NULL (then identical to int8_linear);
 *          Y = fp16(acc*sx[i]*sw[n]/127^2 + outlier product + bias[n]), the sum
 *          formed in fp32 and rounded once.
 * Every other argument, and every error, as for int8_linear. */
i8l_status int8_linear_bias(const uint16_t *X, int64_t M, int64_t K,
                            const int8_t *Wq, const float *sw, int64_t N,
                            const uint16_t *W_outlier_rows, const uint16_t *bias,
                            float threshold, uint16_t *Y, void *workspace,
                            size_t workspace_bytes, void *stream);

/* int8_linear_bias without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  The intermediates go to a static scratch
 * array of I8L_STATIC_SCRATCH_BYTES inside the library, one copy per GPU,
 * allocated when the library's code is loaded on that GPU and held until the
 * process ends; the call itself allocates nothing.  Every call on a GPU uses
 * that GPU's one array, so calls that overlap on one GPU (other streams, other
 * host threads) race and must be serialized by the caller; the array keeps the
 * last call's intermediates, and nothing in it needs to start at zero.
 * Arguments, results and errors as for int8_linear_bias, except: a shape
 * whose workspace (i8l_linear_workspace_bytes, less the GEMM's split-K partial
 * tiles if only that makes it fit, in which case every output tile is
 * computed whole) exceeds I8L_STATIC_SCRATCH_BYTES gives I8L_ERR_WORKSPACE
 * with nothing enqueued.  Fits, for example: every M <= 64 with K <= 133136,
 * and M = 2048 with K = 4096. */
#define I8L_STATIC_SCRATCH_BYTES (32u << 20)
i8l_status int8_linear_static(const uint16_t *X, int64_t M, int64_t K,
                              const int8_t *Wq, const float *sw, int64_t N,
                              const uint16_t *W_outlier_rows, const uint16_t *bias,
                              float threshold, uint16_t *Y, void *stream);

/* Activation stage on its own ([blog, "A gentle summary of LLM.int8()"],
 * step 1, and the row-wise quantization of [blog, "A closer look at the
 * MatMul"]); the same kernels int8_linear runs for M > 16.
 *   Xq          int8 [M][K]      out, 0 in outlier columns
 *   sx          fp32 [M]         out
 *   outlier_idx int32 [K] cap    out, ascending, first n_out entries valid
 *   n_outliers  int32 [1]        out
 *   X_outliers  fp16 [M][K] cap  out, element (i, j) at i*K + j for j < n_out
 *   workspace   at least i8l_linear_workspace_bytes(M, K, 0) bytes */
i8l_status int8_quantize_activation(const uint16_t *X, int64_t M, int64_t K, float threshold,
                                    int8_t *Xq, float *sx, int32_t *outlier_idx,
                                    int32_t *n_outliers, uint16_t *X_outliers,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Exact int8 GEMM on its own ([blog, "Introduction to model quantization"]:
 * the normalised int8 matrices are multiplied), the kernel int8_linear uses
 * for M > 64 with its int32 result written out instead of dequantized.
 *   Xq         int8 [M][K]
 *   Wq         int8 [N][K]
 *   acc        int32 [M][N]  out: acc[i][n] = sum_k Xq[i][k] * Wq[n][k]
 *   workspace  NULL: every 256x256 output tile is computed whole.  Otherwise
 *              at least i8l_linear_workspace_bytes(M, K, N) bytes, 16-byte
 *              aligned: the tiles of a partial last round over the compute
 *              units are then split along K, their int32 partials stored in
 *              the workspace and summed by a fix-up launch, exactly as in
 *              int8_linear (too small: I8L_ERR_WORKSPACE).  The result is the
 *              same exact integer either way. */
i8l_status int8_gemm_i32(const int8_t *Xq, const int8_t *Wq, int64_t M, int64_t N, int64_t K,
                         int32_t *acc, void *workspace, size_t workspace_bytes, void *stream);

/* ---- Zero-point variant ----------------------------------------------------
 * [blog, "Introduction to model quantization"] describes, next to absmax, the
 * unsigned int8 scheme: subtract the minimum, scale the range onto [0, 255],
 * and round the image of 0 to an integer, the zero point.  Here X is quantized
 * that way per row (over the regular columns; the outlier decomposition is the
 * same as in int8_linear) and the weight keeps its absmax codes per output
 * feature:
 *   lo = min(0, min_k x), hi = max(0, max_k x) over the row's regular columns,
 *   inv = fl32(255 / fl32(hi - lo))  (0 when hi == lo),
 *   zp = round_half_away(fl32(-lo * inv)),
 *   q = clamp(round_half_away(fl32(x * inv)) + zp, 0, 255),
 *   xscale = fl32(fl32(hi - lo) / 255);
 * outlier columns take q = zp (the code of 0).  Codes are stored as q - 128
 * (int8) so the int8 matrix cores multiply them; the layer uses
 *   sum_k (q - zp) w = sum_k (q - 128) w + (128 - zp) S[n],  S[n] = sum_k Wq[n][k],
 * exact in int32 for K <= I8L_MAX_K_ZP, and
 *   Y = fp16(acc * xscale[i] * sw[n] / 127 + outlier product + bias[n]).
 * X must be finite in its regular columns (a non-finite value there makes the
 * codes of that row unspecified; with the decomposition on, +-inf is always an
 * outlier). */

/* S[n] = sum_k Wq[n][k] (int32), the per-output correction term of the
 * zero-point variant; computed once per layer, like the weight codes.
 *   Wq  int8 [N][K]  16-byte aligned, read only
 *   S   int32 [N]    out, 4-byte aligned
 * Shape rules as for int8_quantize_weight. */
i8l_status int8_weight_code_sums(const int8_t *Wq, int64_t N, int64_t K, int32_t *S,
                                 void *stream);

/* The layer with zero-point activation codes (see above).
 *   wsum   int32 [N] from int8_weight_code_sums for this Wq, 4-byte aligned
 * Every other argument, the workspace size and the errors as for
 * int8_linear_bias; in addition K > I8L_MAX_K_ZP gives I8L_ERR_K_TOO_LARGE.
 * Afterwards the workspace holds Xq (q - 128), sx (xscale), zero_points, the
 * outlier list and X_outliers of this call. */
i8l_status int8_linear_zp(const uint16_t *X, int64_t M, int64_t K,
                          const int8_t *Wq, const float *sw, const int32_t *wsum, int64_t N,
                          const uint16_t *W_outlier_rows, const uint16_t *bias,
                          float threshold, uint16_t *Y, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Activation stage of the zero-point variant on its own.
 *   Xq      int8 [M][K]  out: q - 128, zp - 128 in outlier columns
 *   zp      int32 [M]    out: zero points in [0, 255]
 *   xscale  fp32 [M]     out: fl32(range / 255)
 * Other arguments, alignment, workspace and errors as for
 * int8_quantize_activation; K > I8L_MAX_K_ZP gives I8L_ERR_K_TOO_LARGE. */
i8l_status int8_quantize_activation_zp(const uint16_t *X, int64_t M, int64_t K, float threshold,
                                       int8_t *Xq, int32_t *zp, float *xscale,
                                       int32_t *outlier_idx, int32_t *n_outliers,
                                       uint16_t *X_outliers, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* ---- Mixed int8/fp16 training mode -----------------------------------------
 * [blog, "Usage"]: has_fp16_weights=True (the default) keeps the fp16 weight
 * for training in mixed int8/fp16 precision.  The pages describe no gradient
 * path; the one provided here treats the quantization as the identity: the
 * forward pass is int8_quantize_weight on the current fp16 weight followed by
 * int8_linear_bias with that weight as W_outlier_rows, and the gradients are
 * those of Y = X . W + bias, formed from fp16 operands with fp32 accumulation
 * and rounded once to fp16 (round to nearest even, overflow to +/-inf).
 * Shapes: M >= 0, K as for int8_linear, N >= 0 with N % 8 == 0. */

/* Workspace bytes int8_linear_backward_weight needs (0 on a bad shape):
 * X^T and dY^T with their rows padded to a multiple of 8, and the bias
 * gradient's partial sums. */
size_t i8l_backward_weight_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* dX = dY . W^T.
 *   dY  fp16 [M][N]  gradient of the layer's output, 16-byte aligned
 *   W   fp16 [K][N]  the fp16 weight in math layout, 16-byte aligned
 *   dX  fp16 [M][K]  out, 16-byte aligned
 * M == 0: no-op.  N == 0: dX = 0 (dY and W may then be NULL). */
i8l_status int8_linear_backward_input(const uint16_t *dY, const uint16_t *W, int64_t M,
                                      int64_t K, int64_t N, uint16_t *dX, void *stream);

/* dW = X^T . dY and dbias[n] = sum_i dY[i][n].
 *   X       fp16 [M][K]  the layer's input, 16-byte aligned
 *   dY      fp16 [M][N]  16-byte aligned
 *   dW      fp16 [K][N]  out (the weight's math layout), 16-byte aligned
 *   dbias   fp16 [N]     out, 4-byte aligned, or NULL (not computed)
 *   workspace  at least i8l_backward_weight_workspace_bytes(M, K, N) bytes,
 *              16-byte aligned (may be NULL when M == 0)
 * M == 0: dW = 0 and dbias = 0.  N == 0: no-op. */
i8l_status int8_linear_backward_weight(const uint16_t *X, const uint16_t *dY, int64_t M,
                                       int64_t K, int64_t N, uint16_t *dW, uint16_t *dbias,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* ---- Serving in 8 bits around the layer --------------------------------------
 * What a decoder layer does between its quantized linear layers, with the 8-bit
 * data kept as codes: the norm that feeds a product with row codes, the product
 * of codes that are already there, a key/value cache held in 8 bits, and
 * attention over it.  16-bit tensors are fp16 or bf16 (i8l_dtype), passed as
 * raw bits. */
typedef enum { I8L_FP16 = 0, I8L_BF16 = 1 } i8l_dtype;

/* Residual addition, root-mean-square norm and row codes:
 *   h = round16(X + residual)   (X itself without a residual),
 *   g = h * weight,  a[i] = max_k |g[i][k]|,
 *   Xq = clamp(round_half_away(g * fl32(127 / a)), -127, 127)   (0 where a is 0),
 *   sx = a / sqrt(mean_k h^2 + eps),
 * so that Xq * sx / 127 is the norm's value: the operands of int8_linear_codes.
 * The factor 1 / rms is common to the row and enters the scale alone.  No outlier
 * columns are set apart: a column c times as large as the others leaves those
 * 127 / c steps (int8_linear on 16-bit rows has them).
 *   X         [M][K]  dtype, 16-byte aligned
 *   residual  [M][K]  dtype, or NULL
 *   weight    [K]     dtype, or NULL (ones)
 *   h         [M][K]  out, or NULL (not stored); may be X or residual
 *   Xq        int8 [M][K] out; sx fp32 [M] out
 *   eps       >= 0
 * Statistics in fp32.  A row with a NaN, or an infinity in h, gets the scale NaN
 * (infinity where only g has one); a row whose a is below 2^-93 gets codes and
 * scale 0.  M and K as for int8_linear. */
i8l_status int8_rmsnorm_quant(const uint16_t *X, const uint16_t *residual,
                              const uint16_t *weight, int64_t M, int64_t K, float eps,
                              int dtype, int8_t *Xq, float *sx, uint16_t *h, void *stream);

/* Workspace bytes of int8_linear_codes for this shape (0: none needed). */
size_t i8l_codes_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* Product of row codes with a quantized weight, no outlier columns:
 *   Y = fp16(acc * sx[i] * sw[n] / 127^2 + bias[n]),  acc = sum_k Xq[i][k] Wq[n][k],
 * acc exact in int32, one rounding (to nearest even, overflow to infinity).
 *   Xq  int8 [M][K] and sx fp32 [M], e.g. from int8_rmsnorm_quant
 *   Wq, sw  from int8_quantize_weight;  bias fp16 [N] or NULL
 *   workspace  device scratch of i8l_codes_workspace_bytes, 16-byte aligned
 *              (a smaller one: I8L_ERR_WORKSPACE), or NULL: then nothing is
 *              split along K (same result, more slowly where the output is small)
 * Shapes, alignment and errors as for int8_linear. */
i8l_status int8_linear_codes(const int8_t *Xq, const float *sx, int64_t M, int64_t K,
                             const int8_t *Wq, const float *sw, int64_t N, const uint16_t *bias,
                             uint16_t *Y, void *workspace, size_t workspace_bytes, void *stream);

/* A key/value cache in 8 bits, in pages of page_size tokens; keys and values
 * have one scale for each page and kv head.
 *   scale = fl32(absmax / 127) over the page's page_size * head_dim values,
 *   code = clamp(round_half_away(x * fl32(127 / absmax)), -127, 127),
 *   value = code * scale   (a page with a NaN or an infinity: scale NaN; one
 *   whose absmax is below 2^-93: scale and codes 0).
 * A page's codes are made when its last token arrives; the tokens of a
 * sequence's last, incomplete page are kept in 16 bits in the sequence's slot.
 * So no value is rounded twice, and what the cache holds does not depend on how
 * many calls wrote it.  The caller owns the memory and hands out pages. */
typedef struct {
  int8_t *k_codes;    /* [n_pages][heads][page_size][head_dim], 16-byte aligned */
  int8_t *v_codes;    /* [n_pages][heads][head_dim][page_size], 16-byte aligned */
  float *k_scale;     /* [n_pages][heads] */
  float *v_scale;     /* [n_pages][heads] */
  uint16_t *k_tail;   /* [n_slots][heads][page_size][head_dim] dtype, 16-byte aligned */
  uint16_t *v_tail;   /* [n_slots][heads][head_dim][page_size] dtype, 16-byte aligned */
  int64_t n_pages, n_slots;
  int32_t heads;      /* kv heads, 1 .. 4096 */
  int32_t head_dim;   /* a multiple of 16, 16 .. 256 */
  int32_t page_size;  /* 16, 32, 64 or 128 */
  int32_t dtype;      /* i8l_dtype of the tails and of the 16-bit tensors */
} i8l_kv_cache;

/* The sequences of a call (device arrays).  Entries are clamped to what the
 * tensors hold: a page or slot outside the cache is neither read nor written
 * (its tokens are skipped; attention masks them), tokens past
 * max_pages * page_size are skipped and masked too, but count in the positions. */
typedef struct {
  const int32_t *page_table;  /* [n][max_pages]: page of tokens i * page_size .. */
  const int32_t *lengths;     /* [n]: tokens of each sequence, this call's included */
  const int32_t *cu;          /* [n + 1], ascending: sequence i has rows cu[i] .. cu[i+1] - 1
                                 of the call's packed tensors; NULL: row i alone */
  const int32_t *slots;       /* [n]: its tail slot; NULL: slot i */
  int32_t n;                  /* sequences, 0 .. 65535 */
  int32_t max_pages;          /* max_pages * page_size < 2^30 */
} i8l_sequences;

/* Writes the call's rows as the last tokens of their sequences: row j of a
 * sequence with m rows is its token lengths[i] - m + j.  Tokens before them in
 * the same page must be in the slot (written there by earlier calls).  Sequences
 * may share complete pages, not slots or pages that a call writes.
 *   k, v   [rows][heads][head_dim] dtype; element (t, h, d) at
 *          t * token_stride + h * head_stride + d (strides in elements,
 *          multiples of 8; pointers 16-byte aligned)
 *   max_new  at least the rows of any one sequence */
i8l_status int8_cache_write(const i8l_kv_cache *cache, const i8l_sequences *seqs,
                            const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride,
                            const uint16_t *v, int64_t v_token_stride, int64_t v_head_stride,
                            int64_t rows, int64_t max_new, void *stream);

/* Reads sequences back: rows cu[i] .. cu[i] + lengths[i] - 1 of k and v
 * [rows][heads][head_dim] (dtype, contiguous, 16-byte aligned) receive the
 * tokens of sequence i, complete pages as round16(code * scale), the rest as
 * written.  cu is required.
 *   max_len  at least the longest sequence */
i8l_status int8_cache_read(const i8l_kv_cache *cache, const i8l_sequences *seqs, uint16_t *k,
                           uint16_t *v, int64_t rows, int64_t max_len, void *stream);

/* Workspace bytes of int8_cache_attention for these sizes (0: none needed, or
 * sizes that the call refuses). */
size_t i8l_attention_workspace_bytes(const i8l_kv_cache *cache, int64_t n, int64_t q_heads,
                                     int64_t max_q, int64_t max_len, int64_t window);

/* Causal attention of a call's queries over the cache, which already holds the
 * keys and values of the queries' own tokens (int8_cache_write comes first): row
 * j of a sequence with m rows is the query of token i = lengths - m + j and sees
 * the tokens max(0, i - window + 1) .. i (window 0: all up to i):
 *   out = softmax_t(scale * q . k_t - alibi[head] * (i - t)) . v_t,
 * with the cache's 8-bit values (16-bit in the tail).  Query head h reads kv
 * head h / (q_heads / heads).  A query that sees no token gives 0.  Infinities and
 * NaNs show in the queries that see them (a complete page that holds one reads as NaN
 * as a whole; in the incomplete page they stay in their token and dimension).
 *   q      [rows][q_heads][head_dim] dtype; element (t, h, d) at
 *          t * token_stride + h * head_stride + d (multiples of 8)
 *   alibi  fp32 [q_heads] slopes, or NULL
 *   out    [rows][q_heads][head_dim] dtype, contiguous, 16-byte aligned
 *   max_q  at least the rows of any one sequence (rows past it are not written)
 *   max_len  the longest sequence (sizes the split of the keys; results do
 *          not depend on it beyond the order of sums)
 *   workspace  i8l_attention_workspace_bytes(...) bytes, 16-byte aligned
 * Scores, softmax statistics and sums in fp32; the weights are rounded to
 * dtype, relative to the row's largest contribution, for the matrix cores: value
 * scales that a row sees should be within a factor of 2^90 of each other (a page of
 * zeros counts as 2^-31). */
i8l_status int8_cache_attention(const i8l_kv_cache *cache, const i8l_sequences *seqs,
                                const uint16_t *q, int64_t q_token_stride,
                                int64_t q_head_stride, int64_t q_heads, int64_t rows,
                                int64_t max_q, int64_t max_len, float scale, int64_t window,
                                const float *alibi, uint16_t *out, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Message for the last non-OK status returned on this thread ("" if none). */
const char *i8l_last_error(void);

/* Static build description: target architecture and kernel tile sizes. */
const char *i8l_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* INT8LIN_H */
