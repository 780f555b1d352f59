/*
 * fp8q -- fine-grained E4M3 quantization and the block-scaled FP8 GEMM that
 * consumes it, for AMD Instinct MI355X (gfx950).
 *
 * The method (sources are cited by page title and section):
 *   - "How does the unified E4M3 format contribute to the efficiency of
 *     DeepSeek-V3" (codingmall.com), "Fine-Grained Quantization Strategy":
 *     one E4M3 format for every tensor; activations scaled per 1x128 tile,
 *     weights per 128x128 block.  "Dynamic Scaling and Online Quantization":
 *     each scale is computed from the group's current values.  "Enhanced
 *     Numerical Stability": FP8 partial results are promoted to FP32 at
 *     intervals during accumulation.
 *   - The innerforce.co.kr excerpt of the DeepSeek-V3 report, paragraph on
 *     Figure 7 (a): a group's max-abs is mapped to the largest FP8 value;
 *     1x128 = per token per 128 channels, 128x128 = per 128 input channels
 *     per 128 output channels.  The next paragraph: dequantization is folded
 *     into the FP32 accumulation of the GEMM.
 *   - "DeepSeek FP8 Training" (arcalunar.github.io), the Fprop pipeline, the
 *     weight-gradient list and the input-gradient list: the three products
 *     and their output precisions (BF16 Y and dX, FP32 dW).
 *
 * Numeric conventions (the pages leave these open; the readings taken):
 *   amax' = max(amax, 2^-100); scale s = fl32(amax'/448) is stored; codes are
 *   E4M3FN(fl32(x * fl32(448/amax'))) with round-to-nearest-even, saturation
 *   to +-448 and the sign of zero kept.  Dequantized value = decode(q) * s.
 *   GEMM: for every 128-long chunk kb of the contraction axis an FP8 matrix-
 *   core partial P is formed and added as acc += P * sA(row,kb) * sB(col,kb)
 *   into FP32 registers; the result is stored as BF16 (round-to-nearest-even)
 *   or FP32.  Accuracy of the FP8 variants: within each group of 8 consecutive
 *   K of a chunk the matrix instruction keeps 14 bits below the largest
 *   product's exponent (truncating), so |C - exact| <= 2^-10 * sum|a*b| plus
 *   FP32 rounding; the _exact variants (end of this file) stay within FP32
 *   rounding of the exact contraction.
 *
 * Conventions of every entry point:
 *   - All pointers are DEVICE pointers owned by the caller.  The library
 *     allocates nothing, keeps no pointer after returning and has no global
 *     state beyond the tile setting of fp8q_set_gemm_tile: calls are
 *     re-entrant and thread-safe.  Buffers must stay valid
 *     until the work enqueued on `stream` has completed.
 *   - Work is enqueued asynchronously on `stream` (NULL = the default
 *     stream).  Results are deterministic (no split-K, no atomics but integer
 *     counts, whose sums do not depend on their order).
 *   - The FP8 and MX GEMMs pick a 256x128 or a 256x256 workgroup tile by
 *     problem size (the wide one when its grid has more tiles than half the
 *     device's compute units and the output width is a multiple of 256).
 *     Both run the same arithmetic in the same order, so the choice never
 *     changes a result bit.  fp8q_set_gemm_tile (below) forces either tile
 *     for tests and measurement.
 *   - Arguments are validated on the host before anything is enqueued; a bad
 *     argument returns its status and enqueues nothing.  A zero-size call is
 *     a no-op returning FP8Q_OK.  A launch failure reported by the HIP runtime
 *     returns FP8Q_ERR_LAUNCH.  No exception crosses this interface and the
 *     library never aborts or prints.
 *   - Matrices are row-major; `ld_*` is the distance between rows in
 *     ELEMENTS of that matrix.  Quantizer inputs and code outputs must start on
 *     16-byte boundaries and have row strides that are multiples of 16 bytes
 *     (vector access), else FP8Q_ERR_ALIGN.  Scale arrays need 4-byte alignment.
 *   - Inputs must be finite; NaN or Inf inputs give unspecified codes.
 *   - Device-resident expert offsets (the grouped entry points) are never
 *     read on the host by libfp8q.so.  The same sources compiled with
 *     FP8Q_DEBUG (libfp8q_debug.so) copy them to the host first, wait for
 *     the stream, and return FP8Q_ERR_SHAPE, enqueuing nothing, unless
 *     offsets[0] = 0, they never decrease and offsets[E] = M_total.
 *   - Work is sized for one GPU's share; every size must fit in int64 and the
 *     number of 128-groups of one call must stay below 2^31.  A GEMM's
 *     contraction length is at most 131072 (1024 chunks of 128).
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8Q_OK = 0,
  FP8Q_ERR_NULL = 1,   /* a required pointer is NULL while its size is non-zero */
  FP8Q_ERR_SHAPE = 2,  /* negative size, or a size rule of the entry point broken */
  FP8Q_ERR_STRIDE = 3, /* a leading dimension smaller than the row length */
  FP8Q_ERR_ALIGN = 4,  /* pointer or row stride not aligned as required */
  FP8Q_ERR_DTYPE = 5,  /* unsupported element type */
  FP8Q_ERR_LAUNCH = 6  /* the HIP runtime refused a launch */
} fp8q_status;

typedef enum { FP8Q_BF16 = 0, FP8Q_F32 = 1 } fp8q_dtype;

/* Human-readable name of a status code (static storage, never NULL). */
const char* fp8q_status_string(fp8q_status s);

/* Process-wide choice of the GEMMs' workgroup tile, for tests and
 * measurement: 0 = by problem size (the default), 1 = 256x128, 2 = 256x256
 * where the output width allows it.  The tiles give bit-identical results, so
 * this changes timing only.  It is the library's one piece of state: calls on
 * other threads see the new value from their next launch.  Returns
 * FP8Q_ERR_SHAPE (and changes nothing) for any other value. */
fp8q_status fp8q_set_gemm_tile(int tile);

/*
 * 1x128 activation quantization ("unified E4M3" page, "Fine-Grained
 * Quantization Strategy"; innerforce.co.kr excerpt, Figure 7 (a) item (1)).
 *   x     : [rows, cols] BF16 or FP32 (xt), row stride ld_x >= cols elements
 *   q     : [rows, cols] E4M3 codes (uint8), row stride ld_q >= cols bytes
 *   scale : [rows, ceil(cols/128)] FP32, row stride ld_s >= ceil(cols/128)
 * Group (r, j) = x[r, 128j : min(128j+128, cols)); a trailing partial group
 * uses only the elements present.  Any rows, cols >= 0.
 */
fp8q_status fp8q_quant_act_1x128(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                 uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s, hipStream_t stream);

/*
 * 128x128 weight quantization (same page and section; innerforce.co.kr
 * excerpt, Figure 7 (a) item (2)).
 *   w     : [rows, cols] FP32 (master weights) or BF16 (wt), stride ld_w
 *   q     : [rows, cols] E4M3 codes, stride ld_q
 *   q_t   : optional [cols, rows] E4M3 codes, the exact transpose of q
 *           (stride ld_qt >= rows), or NULL to skip.  A block's scale does not
 *           change under transposition, so q_t with the same scale array is
 *           the weight operand of the input-gradient GEMM.
 *   scale : [ceil(rows/128), ceil(cols/128)] FP32, stride ld_s
 * Block (i, j) = rows [128i, 128i+128) x cols [128j, 128j+128), clipped.
 */
fp8q_status fp8q_quant_weight_128x128(const void* w, fp8q_dtype wt, int64_t rows, int64_t cols, int64_t ld_w,
                                      uint8_t* q, int64_t ld_q, uint8_t* q_t, int64_t ld_qt,
                                      float* scale, int64_t ld_s, hipStream_t stream);

/*
 * Fused quantize + transpose for the weight-gradient operands ("DeepSeek FP8
 * Training", weight-gradient list: both dY and the activation are quantized
 * for the Wgrad GEMM).  The 1x128 rule applied to x^T: a group is 128
 * consecutive rows (tokens) of one column (channel).
 *   x       : [rows, cols] BF16 or FP32, stride ld_x
 *   q_t     : [cols, rows] E4M3 codes, q_t[c, r] = code of x[r, c]; stride ld_qt >= rows
 *   scale_t : [cols, ceil(rows/128)] FP32, stride ld_st
 * The result equals fp8q_quant_act_1x128 applied to the transposed matrix.
 */
fp8q_status fp8q_quant_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                 uint8_t* q_t, int64_t ld_qt, float* scale_t, int64_t ld_st, hipStream_t stream);

/*
 * Dual-output quantizer: fp8q_quant_act_1x128 and fp8q_quant_transpose of the
 * same x in one pass that reads x once (a layer's input X, or its output
 * gradient dY, feeds both a row-quantized GEMM and the weight-gradient GEMM;
 * "DeepSeek FP8 Training", Fprop and weight-gradient lists).  The outputs are
 * byte for byte those of the two separate calls; the arguments and rules are
 * theirs combined (q, scale as fp8q_quant_act_1x128; q_t, scale_t as
 * fp8q_quant_transpose).
 */
fp8q_status fp8q_quant_act_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                     uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s, uint8_t* q_t,
                                     int64_t ld_qt, float* scale_t, int64_t ld_st, hipStream_t stream);

/*
 * Batched quantization: up to FP8Q_MAX_QUANT_JOBS independent quantizations
 * in at most two launches (one for the 1x128 activation jobs, one for the
 * jobs quantizing 128x128 tiles: weight, transpose, act + transpose; the two
 * classes need different register and LDS budgets).  A quantizer of a
 * 25-90 MB tensor spends a few us of its time in the ramp-up and drain of
 * its own HBM stream; in one grid the next job's workgroups start while the
 * previous job's last ones drain.  Online
 * quantization of every tensor right before its use ("How does the unified
 * E4M3 format contribute to the efficiency of DeepSeek-V3", "Dynamic Scaling
 * and Online Quantization") puts several independent quantizations next to
 * each other, e.g. a layer's input X and its weight W before Fprop.
 *   jobs : HOST array of n_jobs descriptions (read during the call only)
 *   kind : FP8Q_QUANT_ACT_1X128       x -> q, scale        (fp8q_quant_act_1x128)
 *          FP8Q_QUANT_WEIGHT_128X128  x -> q, scale, q_t (q_t may be NULL)
 *                                     (fp8q_quant_weight_128x128)
 *          FP8Q_QUANT_TRANSPOSE       x -> q_t, scale_t    (fp8q_quant_transpose)
 *          FP8Q_QUANT_ACT_TRANSPOSE   x -> q, scale, q_t, scale_t
 *                                     (fp8q_quant_act_transpose)
 *   Every field a kind does not use is ignored.  Each job's arguments, rules
 *   and outputs are those of the single entry point named; its outputs are
 *   bit for bit the same.  Jobs must not write memory another job reads or
 *   writes.  All jobs are validated before anything is enqueued: the first
 *   invalid job's status is returned.  n_jobs outside [0, FP8Q_MAX_QUANT_JOBS]
 *   or an unknown kind gives FP8Q_ERR_SHAPE; n_jobs = 0 is a no-op.
 */
#define FP8Q_MAX_QUANT_JOBS 8
typedef enum {
  FP8Q_QUANT_ACT_1X128 = 0,
  FP8Q_QUANT_WEIGHT_128X128 = 1,
  FP8Q_QUANT_TRANSPOSE = 2,
  FP8Q_QUANT_ACT_TRANSPOSE = 3
} fp8q_quant_kind;
typedef struct {
  int32_t kind;            /* fp8q_quant_kind */
  int32_t xt;              /* fp8q_dtype of x */
  const void* x;           /* [rows, cols], row stride ld_x elements */
  int64_t rows, cols, ld_x;
  uint8_t* q;              /* row codes [rows, cols], row stride ld_q bytes */
  int64_t ld_q;
  float* scale;            /* row scales, row stride ld_s */
  int64_t ld_s;
  uint8_t* q_t;            /* transposed codes [cols, rows], row stride ld_qt bytes */
  int64_t ld_qt;
  float* scale_t;          /* transposed scales [cols, ceil(rows/128)], row stride ld_st */
  int64_t ld_st;
} fp8q_quant_job;
fp8q_status fp8q_quant_batch(const fp8q_quant_job* jobs, int n_jobs, hipStream_t stream);

/*
 * Fprop: Y[M,N] = X[M,K] . W[N,K]^T ("DeepSeek FP8 Training", Fprop pipeline:
 * FP8 GEMM with FP32 accumulation, result stored as BF16).
 *   xq : [M, K] codes, contiguous;  xs : [M, K/128] FP32, contiguous
 *   wq : [N, K] codes, contiguous;  ws : [N/128, K/128] FP32, contiguous
 *   y  : [M, N] of type yt (BF16 or FP32), row stride ld_y >= N elements,
 *        ld_y * element size a multiple of 16 bytes, y 16-byte aligned
 * Rules: K % 128 == 0, N % 128 == 0, any M >= 0; xq, wq 16-byte aligned.
 */
fp8q_status fp8q_gemm_fprop(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                            int64_t M, int64_t N, int64_t K, void* y, fp8q_dtype yt, int64_t ld_y,
                            hipStream_t stream);

/*
 * Dgrad: dX[M,K] = dY[M,N] . W[N,K] ("DeepSeek FP8 Training", input-gradient
 * list: FP8 weight and FP8 output gradient, FP32 accumulation, BF16 dX).
 *   dyq  : [M, N] codes (1x128 groups along N), dys : [M, N/128] FP32
 *   wq_t : [K, N] codes = the q_t output of fp8q_quant_weight_128x128
 *   ws   : the SAME [N/128, K/128] block-scale array of that call
 *   dx   : [M, K] of type dxt, row stride ld_dx (rules as y above)
 * Rules: N % 128 == 0 (contraction), K % 128 == 0, any M >= 0.
 */
fp8q_status fp8q_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                            int64_t M, int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                            hipStream_t stream);

/*
 * Wgrad: dW[N,K] (= or +=) dY^T . X over T tokens ("DeepSeek FP8 Training",
 * weight-gradient list: FP32 accumulation, dW stored in FP32).
 *   dyq_t : [N, T] codes, dys_t : [N, T/128]  (fp8q_quant_transpose of dY[T,N])
 *   xq_t  : [K, T] codes, xs_t  : [K, T/128]  (fp8q_quant_transpose of X[T,K])
 *   dw    : [N, K] FP32, row stride ld_dw (multiple of 4 elements)
 *   accumulate : 0 stores the product, 1 adds it to dw
 * Rules: T % 128 == 0, K % 128 == 0, any N >= 0.
 */
fp8q_status fp8q_gemm_wgrad(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t, const float* xs_t,
                            int64_t T, int64_t N, int64_t K, float* dw, int64_t ld_dw, int accumulate,
                            hipStream_t stream);

/*
 * Grouped (MoE) Fprop: for every expert e, rows [o_e, o_{e+1}) of Y are
 * X[o_e:o_{e+1}, :] . W_e^T (the FP8 GEMMs of MoE layers; the expert layout
 * is this library's own, the pages give no grouped algorithm).
 *   xq : [M_total, K] codes, xs : [M_total, K/128]
 *   wq : [E, N, K] codes,    ws : [E, N/128, K/128]
 *   offsets : DEVICE int32 [E+1]; offsets[0] = 0, non-decreasing,
 *             offsets[E] = M_total (it stays on the device and the product
 *             library does not check it: malformed offsets are undefined
 *             behaviour; the FP8Q_DEBUG build rejects them, FP8Q_ERR_SHAPE)
 *   y  : [M_total, N] of type yt, row stride ld_y
 * Rules: K % 128 == 0, N % 128 == 0, 1 <= E <= 65536, any M_total >= 0.
 * Experts with no rows are skipped; no host synchronisation happens.
 */
fp8q_status fp8q_grouped_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                              const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                              void* y, fp8q_dtype yt, int64_t ld_y, hipStream_t stream);

/*
 * MoE backward.  The MoE layers' GEMMs run in FP8 like the dense ones (the
 * innerforce.co.kr excerpt of the DeepSeek-V3 report, the FP8 framework
 * paragraph), with the dense layer's operands per product ("DeepSeek FP8
 * Training", input- and weight-gradient lists).  The expert layouts are this
 * library's own; the pages give no grouped algorithm.  `offsets` is as for
 * fp8q_grouped_gemm (DEVICE int32 [E+1], never read on the host).
 *
 * Token-padded layout of the weight-gradient operands: the tokens of expert
 * e (rows [o_e, o_{e+1}) of the input) occupy token columns [p_e, p_e + m_e)
 * with p_e = 128 * (o_e / 128 + e) (integer division), so that no 128-token
 * group mixes two experts; the columns from p_e + m_e to the end of that
 * 128-token chunk hold code 0.  The padded axis has capacity
 * cap = 128 * (M_total / 128 + E); columns owned by no expert are not written.
 */

/*
 * Grouped quantize + transpose: fp8q_quant_transpose applied to every
 * expert's block of rows on its own (a trailing partial group uses only the
 * expert's tokens), written in the token-padded layout.
 *   x       : [rows = M_total, cols] BF16 or FP32, stride ld_x
 *   q_t     : [cols, ld_qt] E4M3 codes, ld_qt >= cap (multiple of 16)
 *   scale_t : [cols, ld_st] FP32, ld_st >= cap / 128; chunk j = token
 *             columns [128j, 128j + 128)
 * Rules: 1 <= E <= 65536, cap / 128 <= 65535.
 */
fp8q_status fp8q_quant_transpose_grouped(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                         const int32_t* offsets, int64_t E, uint8_t* q_t, int64_t ld_qt,
                                         float* scale_t, int64_t ld_st, hipStream_t stream);

/*
 * Grouped Dgrad: for every expert e, rows [o_e, o_{e+1}) of dX are
 * dY[o_e:o_{e+1}, :] . W_e.
 *   dyq  : [M_total, N] codes (1x128 groups along N), dys : [M_total, N/128]
 *   wq_t : [K, E*N] codes = the q_t output of fp8q_quant_weight_128x128 on the
 *          stacked weights [E*N, K]; W_e^T is columns [eN, (e+1)N)
 *   ws   : the SAME [E*N/128, K/128] scale array of that call
 *   dx   : [M_total, K] of type dxt, row stride ld_dx (rules as fp8q_gemm_dgrad)
 * Rules: N % 128 == 0, K % 128 == 0, 1 <= E <= 65536, E*N <= (2^31-1)/256
 * (the kernels address 256 rows of wq_t with 32-bit offsets), else
 * FP8Q_ERR_SHAPE.
 */
fp8q_status fp8q_grouped_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                    const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                    void* dx, fp8q_dtype dxt, int64_t ld_dx, hipStream_t stream);

/*
 * Grouped Wgrad: dW_e (= or +=) dY[o_e:o_{e+1}]^T . X[o_e:o_{e+1}] for every
 * expert, a contraction over that expert's own tokens.
 *   dyq_t, dys_t : fp8q_quant_transpose_grouped of dY [M_total, N]
 *                  ([N, ld_t] codes, [N, ld_t/128] scales)
 *   xq_t,  xs_t  : fp8q_quant_transpose_grouped of X [M_total, K]
 *                  ([K, ld_t] codes, [K, ld_t/128] scales)
 *   ld_t : the padded token stride of all four, ld_t >= cap, ld_t % 128 == 0
 *   dw   : [E, N, K] FP32, contiguous; an expert with no tokens gets 0
 *          (accumulate = 0) or is left unchanged (accumulate = 1)
 * Rules: K % 128 == 0, any N >= 0, M_total <= 131072, 1 <= E <= 65536,
 * ld_t <= (2^31-1)/256 (the kernels address 256 operand rows with 32-bit
 * offsets), else FP8Q_ERR_SHAPE.
 */
fp8q_status fp8q_grouped_gemm_wgrad(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t,
                                    const float* xs_t, const int32_t* offsets, int64_t E, int64_t M_total,
                                    int64_t N, int64_t K, int64_t ld_t, float* dw, int accumulate,
                                    hipStream_t stream);

/*
 * Fprop and Dgrad with the output's own quantization fused into the epilogue.
 * The BF16 output of each product is the next layer's FP8 input ("DeepSeek
 * FP8 Training", Fprop list: Y leaves the GEMM in BF16 and the following
 * layer's input is quantized 1x128; input-gradient list: dX feeds the layer
 * below), and activations are kept and passed on in FP8 (the innerforce.co.kr
 * excerpt of the DeepSeek-V3 report, paragraph on the FP8 framework).  Each
 * call writes, besides the BF16 output, its 1x128 E4M3 codes and FP32 scales,
 * computed from the BF16-rounded values with the quantizers' arithmetic: the
 * codes and scales are bit for bit those of fp8q_quant_act_1x128 applied to
 * the BF16 output, which this saves reading back.
 *   fprop: arguments as fp8q_gemm_fprop with yt = BF16; yq [M, N] codes (row
 *          stride ld_yq bytes, a multiple of 16, 16-byte aligned), ys
 *          [M, N/128] FP32 (row stride ld_ys >= N/128)
 *   dgrad: arguments as fp8q_gemm_dgrad with dxt = BF16; dxq [M, K], dxs
 *          [M, K/128] likewise
 *   y / dx may be NULL: then only the codes and scales are written.
 *   exact = 0: the FP8 matrix instruction; 1: the exact-accumulation form
 *   (see the _exact variants below); any other value: FP8Q_ERR_SHAPE.
 * Rules and errors otherwise as fp8q_gemm_fprop / fp8q_gemm_dgrad; NULL codes
 * or scales give FP8Q_ERR_NULL.
 */
fp8q_status fp8q_gemm_fprop_quant(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* y, int64_t ld_y, uint8_t* yq,
                                  int64_t ld_yq, float* ys, int64_t ld_ys, int exact, hipStream_t stream);
fp8q_status fp8q_gemm_dgrad_quant(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* dx, int64_t ld_dx, uint8_t* dxq,
                                  int64_t ld_dxq, float* dxs, int64_t ld_dxs, int exact, hipStream_t stream);

/*
 * Promotion-interval study (numerics only; not a step of the method).  The
 * method promotes the FP8 partial of every 128-long K chunk into FP32 ("How
 * does the unified E4M3 format contribute to the efficiency of DeepSeek-V3",
 * "Enhanced Numerical Stability": promotion at fixed intervals; the
 * innerforce.co.kr excerpt of the DeepSeek-V3 report, paragraph after Figure
 * 7 (a), where the interval is lost in the extracted text).  This entry point
 * computes the Fprop product with the partial of each 16x16 output block
 * chained through the matrix instruction's accumulator operand over
 * `interval` elements of K (128, 256, 512 or 1024; 0 = the whole
 * contraction) and promoted only at the end of each interval, with the
 * scales of the interval's last chunk.  The result is the Fprop product only
 * if xs and ws are constant over every interval (for instance all 1, which
 * operands whose groups reach exactly 448 give); the library does not check.
 * interval = 128 is fp8q_gemm_fprop with FP32 output.
 *   Arguments as fp8q_gemm_fprop with yt = FP32 (y, ld_y).
 * Rules: K % 512 == 0 (16-byte scale rows), N % 128 == 0, xs 16-byte
 * aligned, interval as above, else FP8Q_ERR_SHAPE / FP8Q_ERR_ALIGN.
 */
fp8q_status fp8q_gemm_fprop_interval(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                     int64_t M, int64_t N, int64_t K, float* y, int64_t ld_y, int64_t interval,
                                     hipStream_t stream);

/*
 * Exact-accumulation variants.  Same arguments, rules, layouts and results
 * definition as the four GEMMs above; only the in-chunk arithmetic differs.
 * gfx950's FP8 matrix instruction adds the 8 products of each group of 8
 * consecutive K after aligning them to the largest one and truncating the
 * others 13 bits below its exponent (the counterpart of the limited FP8 tensor-
 * core accumulation the innerforce.co.kr excerpt reports for H800, paragraph
 * after Figure 7 (a)).  These variants convert every code exactly to BF16 and
 * use the BF16 matrix instruction, whose products are exact and whose sums are
 * FP32, then promote every 128-K chunk exactly like the FP8 variants.  They
 * run at the BF16 matrix rate (half the FP8 rate) and serve callers who need
 * the result within 1e-5 * sum|a*b| of the exact contraction.
 */
fp8q_status fp8q_gemm_fprop_exact(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* y, fp8q_dtype yt, int64_t ld_y,
                                  hipStream_t stream);
fp8q_status fp8q_gemm_dgrad_exact(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                                  hipStream_t stream);
fp8q_status fp8q_gemm_wgrad_exact(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t,
                                  const float* xs_t, int64_t T, int64_t N, int64_t K, float* dw, int64_t ld_dw,
                                  int accumulate, hipStream_t stream);
fp8q_status fp8q_grouped_gemm_exact(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                    const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                    void* y, fp8q_dtype yt, int64_t ld_y, hipStream_t stream);

/*
 * Microscaling variant (MXFP8 with E4M3 elements, OCP Microscaling v1.0).
 * The pages set the method's FP32 group scales against the small-group
 * power-of-two scaling that newer tensor cores support natively (the
 * innerforce.co.kr excerpt, paragraph on Figure 7 (a)); gfx950's counterpart
 * is the block-scaled matrix instruction.  Numerics differ from the method:
 *   block : 32 consecutive elements along the contraction axis, for BOTH
 *           GEMM operands (so every operand of the three products is
 *           quantized along its own contraction axis, see fp8q_gemm_mx);
 *   scale : one E8M0 byte per block, e = clamp(floor(log2 amax) - 8 + 127,
 *           0, 254), value 2^(e - 127); an all-zero block has e = 0;
 *   codes : E4M3FN(x / 2^(e - 127)), round-to-nearest-even, saturating at
 *           +-448, the sign of zero kept.
 * Scale arrays hold bytes; `ld_s`-type strides are in bytes.
 */

/*
 * 1x32 MX quantization along rows.
 *   x : [rows, cols] BF16 or FP32, stride ld_x (16-byte aligned rows)
 *   q : [rows, cols] codes, stride ld_q (multiple of 16)
 *   s : [rows, ceil(cols/32)] E8M0 bytes, stride ld_s >= ceil(cols/32)
 * A trailing partial block uses the elements present.  Any rows, cols >= 0.
 */
fp8q_status fp8q_quant_mx_1x32(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* q,
                               int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t stream);

/*
 * MX quantization along columns, codes written transposed: the 1x32 rule
 * applied to x^T (a block is 32 consecutive rows of one column).
 *   q_t : [cols, rows] codes, q_t[c, r] = code of x[r, c], stride ld_qt >= rows
 *   s_t : [cols, ceil(rows/32)] E8M0 bytes, stride ld_st
 *   q, s : optional (both NULL, or both set): the fp8q_quant_mx_1x32 outputs
 *          of the same x, produced from the same single read of x.
 * Rules: ceil(rows/128) <= 65535.
 */
fp8q_status fp8q_quant_mx_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                    uint8_t* q_t, int64_t ld_qt, uint8_t* s_t, int64_t ld_st, uint8_t* q,
                                    int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t stream);

/*
 * MX GEMM: C[M,N] (= or +=) A[M,K] . B[N,K]^T with both operands MX-quantized
 * along K.  Fprop: A = X, B = W (fp8q_quant_mx_1x32 of each).  Dgrad: A = dY,
 * B = the q_t / s_t of fp8q_quant_mx_transpose(W).  Wgrad: A = q_t of dY,
 * B = q_t of X (both from fp8q_quant_mx_transpose), K = tokens.
 *   aq : [M, K] codes, stride lda >= K (multiple of 16, aq 16-byte aligned)
 *   as : [M, K/32] E8M0 bytes, stride ld_sa >= K/32, ld_sa % 4 == 0, 4-byte
 *        aligned (16-byte aligned rows load faster)
 *   bq, bs : [N, K], [N, K/32], the same rules with ldb, ld_sb
 *   c  : [M, N] of type ct, stride ld_c (rules as fp8q_gemm_fprop's y)
 *   accumulate : 0 stores, 1 adds to c (FP32 output only)
 * The scales are applied by the matrix instruction to every product, which
 * it accumulates in FP32 (within each group of 8 consecutive K, 14 bits below
 * the largest product are kept, as for the FP8 entry points).
 * Rules: K % 128 == 0, N % 128 == 0, K <= 131072, any M >= 0.
 */
fp8q_status fp8q_gemm_mx(const uint8_t* aq, const uint8_t* as, int64_t lda, int64_t ld_sa, const uint8_t* bq,
                         const uint8_t* bs, int64_t ldb, int64_t ld_sb, int64_t M, int64_t N, int64_t K, void* c,
                         fp8q_dtype ct, int64_t ld_c, int accumulate, hipStream_t stream);

/*
 * Grouped (MoE) MX Fprop: fp8q_gemm_mx per expert over grouped rows, as
 * fp8q_grouped_gemm does for the FP32-scaled codes (the MoE layers' GEMMs
 * run in FP8 like the dense ones, the innerforce.co.kr excerpt of the
 * DeepSeek-V3 report, the FP8 framework paragraph; the expert layout is this
 * library's own).  For every expert e, rows [o_e, o_{e+1}) of Y are
 * X[o_e:o_{e+1}, :] . W_e^T, each product scaled by its two E8M0 scales.
 *   xq : [M_total, K] codes,    xs : [M_total, K/32] E8M0 bytes (contiguous)
 *   wq : [E, N, K] codes,       ws : [E, N, K/32] E8M0 bytes (contiguous)
 *   offsets : DEVICE int32 [E+1], as for fp8q_grouped_gemm (never read on
 *             the host by the product library; malformed offsets are undefined
 *             behaviour, the FP8Q_DEBUG build rejects them)
 *   y  : [M_total, N] of type yt, row stride ld_y
 * Each output element takes the same instructions in the same order as in
 * fp8q_gemm_mx on that expert's rows, so the two agree bit for bit.
 * Rules: K % 128 == 0, N % 128 == 0, K <= 131072, 1 <= E <= 65536, any
 * M_total >= 0; xq, wq 16-byte aligned, xs, ws 4-byte aligned (16-byte
 * aligned scale rows, i.e. K % 512 == 0, load faster).  Experts with no rows
 * are skipped; no host synchronisation happens.
 */
fp8q_status fp8q_grouped_gemm_mx(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                                 const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K, void* y,
                                 fp8q_dtype yt, int64_t ld_y, hipStream_t stream);

/*
 * Grouped (MoE) MX Dgrad: for every expert e, rows [o_e, o_{e+1}) of dX are
 * dY[o_e:o_{e+1}, :] . W_e, as fp8q_grouped_gemm_dgrad with E8M0 block
 * scales (the MoE backward's input gradient, "DeepSeek FP8 Training",
 * input-gradient list; the expert layout is this library's own).
 *   dyq  : [M_total, N] codes, dys : [M_total, N/32] E8M0 bytes
 *          (fp8q_quant_mx_1x32 of dY; contiguous)
 *   wq_t : [K, E*N] codes, ws_t : [K, E*N/32] E8M0 bytes: the q_t / s_t of
 *          fp8q_quant_mx_transpose on the stacked weights [E*N, K]
 *          (contiguous); W_e^T is columns [eN, (e+1)N) of both (N % 32 == 0,
 *          so no scale block mixes two experts)
 *   offsets : DEVICE int32 [E+1], as for fp8q_grouped_gemm
 *   dx   : [M_total, K] of type dxt, row stride ld_dx
 * Each output element takes the same instructions in the same order as
 * fp8q_gemm_mx on that expert's rows with B = the expert's columns of wq_t.
 * Rules: N % 128 == 0, K % 128 == 0, N <= 131072, 1 <= E <= 65536,
 * E*N <= 2^31 / 128, any M_total >= 0; dyq, wq_t 16-byte aligned, dys, ws_t
 * 4-byte aligned.  Experts with no rows are skipped.
 */
fp8q_status fp8q_grouped_gemm_mx_dgrad(const uint8_t* dyq, const uint8_t* dys, const uint8_t* wq_t,
                                       const uint8_t* ws_t, const int32_t* offsets, int64_t E, int64_t M_total,
                                       int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                                       hipStream_t stream);

/*
 * ---- MoE routing: from a router's logits to rows in expert order and back.
 *
 * T tokens choose k of E experts each; pair p = t*k + j is token t's j-th
 * choice and M = T*k the number of rows.  The grouped products above take the
 * rows in expert order; these entry points make that order and undo it, with
 * the gradients of each step.  Limits: 1 <= k <= 32, k <= E <= 1024.
 * Logits, token rows and expert rows may start at any element and have any
 * row stride >= their length (no 16-byte rule here); ids, weights and maps
 * are contiguous [T, k].  Rows have at most 2^30 columns, and T * H / 8 stays
 * below 2^31.  Codes written with a row stride that is a multiple of 16 bytes
 * feed the grouped products and quantizers as they are.
 */
typedef enum { FP8Q_SOFTMAX = 0, FP8Q_SIGMOID = 1 } fp8q_score;

/*
 * Router: the k best experts of every token and their weights.
 *   logits  : [T, E] of type lt, row stride ld; -inf masks an expert for a token
 *   score   : fp8q_score; s = softmax(logits) over the E experts, or sigmoid
 *   bias    : optional [E] finite FP32, added to the score for the CHOICE only
 *             (load balancing), or NULL.  The choice is by logit without it
 *             and by s + bias, both in 64 bits, with it; ties go to the lower
 *             expert.
 *   renormalize : 1 divides the chosen scores by their sum (their ratios hold
 *             where the scores themselves vanish in FP32)
 *   scale   : finite factor of the weights
 *   ids     : [T, k] int32, best first; -1 where a token has fewer than k
 *             experts that are not masked
 *   weights : [T, k] FP32: chosen score (renormalized) * scale, 0 beside id -1
 * Logits are finite or -inf.  A NaN logit is never chosen; it makes the weights
 * of its token's softmax NaN unless they are renormalized.
 */
fp8q_status fp8q_moe_route(const void* logits, fp8q_dtype lt, int64_t T, int64_t E, int64_t ld, int k, int score,
                           const float* bias, int renormalize, float scale, int32_t* ids, float* weights,
                           hipStream_t stream);

/*
 * Gradient of fp8q_moe_route's weights to the logits, for the ids it chose
 * (the choice itself has no gradient).  p = score, g = dweights * scale:
 *   softmax              dl_e = p_e (g_e - sum_j g_j p_j), g_e = 0 if not chosen
 *   softmax, renormalized  dl_j = w_j (g_j - sum g w), w_j = p_j / sum of chosen p
 *   sigmoid              dl_j = g_j p_j (1 - p_j)
 *   sigmoid, renormalized  dl_j = w_j (1 - p_j) (g_j - sum g w)
 * (the last three are 0 for experts not chosen).  Every entry of dlogits
 * [T, E] (type lt, row stride ld_d) is written.  A token's ids differ from
 * each other; entries outside [0, E) are no choice.
 */
fp8q_status fp8q_moe_route_bwd(const float* dweights, const void* logits, fp8q_dtype lt, int64_t T, int64_t E,
                               int64_t ld, const int32_t* ids, int k, int score, int renormalize, float scale,
                               void* dlogits, int64_t ld_d, hipStream_t stream);

/*
 * Stable sort of M pairs by expert.
 *   ids     : [M] int32; a pair whose id is outside [0, E) is dropped
 *   offsets : [E+1]; expert e's rows are [offsets[e], offsets[e+1]).  cover = 0:
 *             offsets[E] is the number of pairs kept.  cover = 1: offsets[E] = M,
 *             the dropped pairs' rows count as the last expert's; they are rows
 *             of zeros (see fp8q_moe_dispatch), so every product over them adds
 *             zeros, and the grouped entry points' rule offsets[E] = M_total
 *             holds without a host read.
 *   dst     : [M]; row of pair p, or -1 - row if it is dropped.  Dropped pairs
 *             take the rows after the kept ones, all in pair order, so the rows
 *             are a permutation of [0, M).
 *   src     : optional [M], the pair of each row (the inverse map), or NULL
 *   workspace : fp8q_moe_sort_workspace(M, E) bytes (NULL if that is 0)
 */
fp8q_status fp8q_moe_sort(const int32_t* ids, int64_t M, int64_t E, int cover, int32_t* offsets, int32_t* dst,
                          int32_t* src, void* workspace, int64_t workspace_bytes, hipStream_t stream);
/* Bytes of workspace that call needs (-1: sizes out of range). */
int64_t fp8q_moe_sort_workspace(int64_t M, int64_t E);

/*
 * Token rows into expert order: row r of pair (t, j) becomes x[t], or zeros if
 * the pair is dropped.
 *   x    : [T, H] of type xt, row stride ld_x
 *   dst  : [T, k] DEVICE map of fp8q_moe_sort (not checked by the product
 *          library: entries that name no row are skipped; the FP8Q_DEBUG build
 *          rejects a map that is no permutation, FP8Q_ERR_SHAPE)
 *   rows : [M, H] of type xt, row stride ld_rows, or NULL
 *   q, scale : [M, H] codes and [M, ceil(H/128)] scales of those rows, bit for
 *          bit what fp8q_quant_act_1x128 makes of them, or NULL
 * At least one of rows and q is wanted.  A token is read and quantized once.
 */
fp8q_status fp8q_moe_dispatch(const void* x, fp8q_dtype xt, int64_t T, int64_t H, int64_t ld_x, const int32_t* dst,
                              int k, void* rows, int64_t ld_rows, uint8_t* q, int64_t ld_q, float* scale,
                              int64_t ld_s, hipStream_t stream);

/* Its gradient: dx[t] = sum over token t's kept pairs, in order and in FP32, of
 * drows[dst[t, j]]; rounded once to dx's type t. */
fp8q_status fp8q_moe_dispatch_bwd(const void* drows, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_rows,
                                  const int32_t* dst, int k, void* dx, int64_t ld_dx, hipStream_t stream);

/* Expert rows back into token order: y[t] = sum over token t's kept pairs, in
 * order and in FP32, of weights[t, j] * yp[dst[t, j]]; rounded once. */
fp8q_status fp8q_moe_combine(const void* yp, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_yp, const int32_t* dst,
                             int k, const float* weights, void* y, int64_t ld_y, hipStream_t stream);

/*
 * Its gradients, from one read of dy and of yp:
 *   rows     : [M, H] of type t, or NULL: weights[t, j] * dy[t] rounded to t at
 *              row dst[t, j], zeros at a dropped pair's row
 *   q, scale : codes and scales of those (rounded) rows, or NULL
 *   dweights : [T, k] FP32, dy[t] . yp[dst[t, j]], 0 for a dropped pair
 */
fp8q_status fp8q_moe_combine_bwd(const void* dy, const void* yp, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_dy,
                                 int64_t ld_yp, const int32_t* dst, int k, const float* weights, void* rows,
                                 int64_t ld_rows, uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s,
                                 float* dweights, hipStream_t stream);

/*
 * Gradient clipping by the global norm: norm = sqrt(sum of g^2 over all
 * tensors), formed in 64 bits, and out = g * c, c = 1 if norm <= max_norm, else
 * max_norm / norm (so a NaN norm gives NaN, an infinite one zeros and NaN); c
 * and the product are in 64 bits too, rounded to FP32 and then to out's type.
 *   grads : HOST array (read during the call only) of n dense FP32 tensors of
 *           any length; out is of type ot, and may be g itself if ot is FP32
 *           (then nothing is written where c = 1)
 *   max_norm : >= 0; +inf only measures and copies
 *   workspace : 8-byte aligned, fp8q_grad_clip_workspace(n) bytes
 *   norm  : one FP32, the norm before clipping (infinite where FP32 cannot hold
 *           it; the outputs are right there too)
 * n = 0 gives norm 0.  Tensors must not overlap each other.
 */
typedef struct {
  const float* g;
  void* out;
  int64_t len;
} fp8q_grad;
fp8q_status fp8q_grad_clip(const fp8q_grad* grads, int64_t n, fp8q_dtype ot, double max_norm, void* workspace,
                           int64_t workspace_bytes, float* norm, hipStream_t stream);
/* Bytes of workspace that call needs (-1: n out of range). */
int64_t fp8q_grad_clip_workspace(int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
