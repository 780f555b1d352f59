// Host-side launchers of the HIP kernels (internal to libfp8q; the C ABI in
// include/fp8q.h validates arguments and calls these).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

hipError_t launch_quant_act(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x,
                            uint8_t* q, int64_t ld_q, float* s, int64_t ld_s, hipStream_t st);

hipError_t launch_quant_weight(const void* w, bool w_bf16, int64_t rows, int64_t cols, int64_t ld_w,
                               uint8_t* q, int64_t ld_q, uint8_t* q_t, int64_t ld_qt,
                               float* s, int64_t ld_s, hipStream_t st);

hipError_t launch_quant_transpose(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x,
                                  uint8_t* q_t, int64_t ld_qt, float* s_t, int64_t ld_st, hipStream_t st);

// quant_act_1x128 and quant_transpose of the same x from one read of it.
hipError_t launch_quant_act_transpose(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x,
                                      uint8_t* q, int64_t ld_q, float* s, int64_t ld_s, uint8_t* q_t,
                                      int64_t ld_qt, float* s_t, int64_t ld_st, hipStream_t st);

// Per expert e (rows [offsets[e], offsets[e+1]) of x), the quantize-transpose
// of that block alone, written at padded token column 128*(offsets[e]/128 + e);
// the tail of an expert's last 128-token chunk is written as code 0.
hipError_t launch_quant_transpose_grouped(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x,
                                          const int32_t* offsets, int64_t E, uint8_t* q_t, int64_t ld_qt,
                                          float* s_t, int64_t ld_st, hipStream_t st);

// One quantization of a batched launch (kinds as fp8q_quant_kind: 0 act 1x128,
// 1 weight 128x128 (q_t optional), 2 transpose, 3 act + transpose); arguments
// as the single entry points, already validated.
struct QuantJob {
  int kind;
  bool x_bf16;
  const void* x;
  int64_t rows, cols, ld_x;
  uint8_t* q;
  int64_t ld_q;
  float* s;
  int64_t ld_s;
  uint8_t* q_t;
  int64_t ld_qt;
  float* s_t;
  int64_t ld_st;
};
constexpr int kMaxQuantJobs = 8;
// All jobs in one grid (each job's blocks form one contiguous range of it).
hipError_t launch_quant_batch(const QuantJob* jobs, int n, hipStream_t st);
// Workgroups that grid has (all must fit one grid dimension).
int64_t quant_batch_blocks(const QuantJob* jobs, int n);

// How the scale of the B operand (rows = output columns) is indexed.
enum SbMode : int {
  kSbBlock = 0,  // one scale per 128 output columns per chunk: sb[(n/128)*sb_rs + kb*sb_cs]
  kSbRow = 1     // one scale per output column per chunk:      sb[n*sb_rs + kb]
};

// What a product's epilogue makes of it for a gated feed-forward block.
enum GatedMode : int { kNotGated = 0, kSwiglu = 1, kDSwiglu = 2 };

// C[m, n] = sum_kb P_kb[m, n] * sa[m*ld_sa + kb] * sB(n, kb), P_kb the FP8
// product of the 128-long chunk kb of A[m, :] and B[n, :] (both row-major
// with the contraction axis contiguous).
struct GemmArgs {
  const uint8_t* A;     // [M, K] codes, row stride lda bytes
  const uint8_t* B;     // [N, K] codes, row stride ldb bytes
  const float* sa;      // [M, K/128]
  const float* sb;      // see SbMode
  void* C;              // [M, N], BF16 or FP32, row stride ldc elements
  int64_t lda, ldb, ld_sa, sb_rs, sb_cs, ldc;
  int64_t M, N, K;
  int sb_mode;          // SbMode
  int out_f32;          // 0 = BF16 output, 1 = FP32 output
  int accumulate;       // FP32 output only: C += result
  int exact;            // 0: FP8 MFMA per chunk; 1: exact BF16 MFMA on the converted codes
  // grouped: rows [offsets[e], offsets[e+1]) use B + e*b_estride, sb + e*sb_estride
  const int32_t* offsets;  // NULL for a plain GEMM
  int64_t E, b_estride, sb_estride;
  // grouped contraction (k_grouped = 1): expert e contracts over the padded
  // chunks [offsets[e]/128 + e, + ceil(m_e/128)) of A and B (token-padded
  // operands), and writes its own output C + e*c_estride; M, N are per expert
  int k_grouped;
  int64_t c_estride;
  // fused output quantization (BF16 output only; qo == NULL: none): the 1x128
  // E4M3 codes qo [M, N] (row stride ld_qo bytes) and scales so [M, N/128]
  // (row stride ld_so) of the BF16-rounded output, as quant_act_1x128 would
  // produce them from C; C may then be NULL (codes only)
  uint8_t* qo;
  float* so;
  int64_t ld_qo, ld_so;
  // gated block: kSwiglu computes h = silu(g) u from gate g and up u, B's
  // rows [0, N) and [N, 2N) (scales likewise), to C (BF16) and / or qo, so;
  // kDSwiglu takes its own product as dh and gu as g and u, and writes
  // their gradients to C [M, 2N] and, if h is given, h again
  int gated;            // GatedMode
  uint16_t* gu;         // [M, 2N] BF16: optional output (SWIGLU), input (DSWIGLU)
  int64_t ld_gu;
  uint16_t* h;          // [M, N] BF16, optional (DSWIGLU)
  int64_t ld_h;
};

hipError_t launch_gemm(const GemmArgs& a, hipStream_t st);

// Workgroup tile of the block-scaled GEMMs: 0 = chosen by problem size,
// 1 = 256 x 128, 2 = 256 x 256 (fp8q_set_gemm_tile; all tiles give the same
// result bits, the gated block's of fewer rows, which only 0 takes, too).
int gemm_tile_setting();
// Compute units of the current device, queried once per device.
int device_cu_count();
// the FP8 matrix-instruction kernel (a.exact == 0)
hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t st);
// the promotion-interval study (block scales, FP32 output): partials chained
// through the matrix instruction over `chunks` chunks (1, 2, 4, 8; 0 = all)
hipError_t launch_gemm_interval(const GemmArgs& a, int chunks, hipStream_t st);

// The gated block of few rows (a.gated == kSwiglu, dense), for sizes of which
// swiglu_few is true on the current device; hf: room for h in FP32 [M, N], needed
// where codes are wanted.
bool swiglu_few(int64_t M, int64_t N, int64_t K);
hipError_t launch_swiglu_few(const GemmArgs& a, float* hf, hipStream_t st);
// The gated block or its gradient (a.gated) in tiles of 32, 64 or 128 rows.
hipError_t launch_gated_small(const GemmArgs& a, int rows, hipStream_t st);
// About what it takes on the current device, and the tiles' rows for that; and what
// the tiles of 256 rows take.
// (experts: 0 of dense rows)
int64_t gated_small_time(int64_t M, int64_t N, int64_t K, int64_t experts, int gated, int* rows);
int64_t gated_large_time(int64_t M, int64_t N, int64_t K, int64_t experts, int gated);

// Microscaling (MXFP8 E4M3) quantizers: one E8M0 scale byte per 32
// consecutive elements, along rows (quant_mx) or along columns with the
// codes transposed (quant_mx_transpose; q, s optional row outputs of the same
// read, NULL to skip).
hipError_t launch_quant_mx(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* q,
                           int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t st);
hipError_t launch_quant_mx_transpose(const void* x, bool x_bf16, int64_t rows, int64_t cols, int64_t ld_x,
                                     uint8_t* q_t, int64_t ld_qt, uint8_t* s_t, int64_t ld_st, uint8_t* q,
                                     int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t st);

// MX GEMM: C = A . B^T, both operands blocked along K with E8M0 bytes
// sa[m*ld_sa + k/32], sb[n*ld_sb + k/32] (strides in bytes).  g carries A, B,
// C, their strides, M, N, K, out_f32 and accumulate; its scale fields are unused.
struct MxArgs {
  GemmArgs g;
  const uint8_t* sa;
  const uint8_t* sb;
  int64_t ld_sa, ld_sb;
  int64_t sb_estride;  // grouped: bytes between experts' B scales (g.b_estride for the codes)
};
hipError_t launch_gemm_mx(const MxArgs& a, hipStream_t st);

// ------------------------------------------------------------ MoE routing
// launch(first, count) for all tokens, a part of them at a time: a grid's threads
// are counted in 32 bits, and 2^26 tokens of 64 threads each are past that.
template <class F>
hipError_t launch_in_parts(int64_t tokens, int64_t threads_per_token, F launch) {
  const int64_t most = ((int64_t)1 << 31) / threads_per_token;
  for (int64_t t = 0; t < tokens; t += most) {
    launch(t, tokens - t < most ? tokens - t : most);
    if (const hipError_t err = hipGetLastError(); err != hipSuccess) return err;
  }
  return hipSuccess;
}

constexpr int kMaxExperts = 1024;  // router and sort (their tables live in LDS)
constexpr int kMaxTopK = 32;       // choices per token

// Router: logits [tokens, experts] (row stride ld elements), k choices.
struct MoeRoute {
  const void* logits;
  bool bf16, sigmoid, renorm;
  int64_t tokens, experts, ld, k;
  float scale;
};
hipError_t launch_moe_route(const MoeRoute& a, const float* bias, int32_t* ids, float* w, hipStream_t st);
hipError_t launch_moe_route_bwd(const MoeRoute& a, const float* dw, const int32_t* ids, void* dl, int64_t ld_dl,
                                hipStream_t st);

// Stable counting sort of n pairs into e bins and one of dropped pairs; ws of
// moe_sort_workspace(n, e) bytes.
int64_t moe_sort_workspace(int64_t n, int64_t e);
hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int64_t e, bool cover, int32_t* offsets, int32_t* dst,
                           int32_t* src, void* ws, hipStream_t st);

// Rows in expert order [tokens * k, cols] and the map to them (moe_rows.hip);
// rows or q may be NULL where an output is not wanted.
struct MoeRows {
  bool bf16;
  int64_t tokens, k, cols;
  const int32_t* dst;  // [tokens, k]
  void* rows;
  int64_t ld_rows;
  uint8_t* q;
  int64_t ld_q;
  float* s;
  int64_t ld_s;
};
hipError_t launch_moe_dispatch(const MoeRows& a, const void* x, int64_t ld_x, hipStream_t st);
// y[t] = sum_j w[t, j] rows[dst[t, j]] (w == NULL: the plain sum)
hipError_t launch_moe_gather(const MoeRows& a, const float* w, void* y, int64_t ld_y, hipStream_t st);
hipError_t launch_moe_combine_bwd(const MoeRows& a, const void* dy, int64_t ld_dy, const void* yp, int64_t ld_yp,
                                  const float* w, float* dw, hipStream_t st);

// ------------------------------------------------------- gradient clipping
constexpr int kMaxClipTensors = 96;  // per launch: the table travels in the kernel's arguments
constexpr int kClipBlocks = 2048;    // most blocks of a launch, and partial sums of all of them
constexpr int kClipChunk = 8192;     // elements of one tensor a block takes at a time
// Up to N tensors, none of them empty.
template <int N>
struct ClipTable {
  const float* g[N];
  void* out[N];
  int cum[N + 1];    // first chunk of each tensor, then their number
  uint16_t last[N];  // elements of a tensor's last chunk
  uint16_t n;
};
typedef ClipTable<kMaxClipTensors> ClipBatch;
// Adds the sums of squares of the batch's chunks to the *held partial sums, of
// which there may then be more; leaves the table in `table` (device memory) for
// the second pass.
hipError_t launch_grad_sumsq(const ClipBatch& b, ClipBatch* table, double* part, int* held, hipStream_t st);
hipError_t launch_grad_scale(const ClipBatch* table, int chunks, bool out_bf16, const double* part, int parts,
                             double max_norm, float* norm, hipStream_t st);

// -------------------------------------------------------------- RMS norm
constexpr int64_t kMaxNormCols = 16384;  // a row stays in a block's registers
// What forward and gradient share: the rows' shape and type, the weights, and
// the outputs (out: y or dx; out or q may be NULL).
struct NormRows {
  bool bf16;
  int64_t rows, cols;
  const float* w;
  void* out;
  int64_t ld_out;
  uint8_t* q;
  int64_t ld_q;
  float* s;
  int64_t ld_s;
};
hipError_t launch_rms_norm(const NormRows& a, const void* x, int64_t ld_x, const void* res, int64_t ld_res, float eps,
                           void* sum, int64_t ld_sum, float* rstd, hipStream_t st);
// Blocks of the gradient's launch, each of which leaves a row of cols partial
// sums of dw.
int64_t rms_norm_parts(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_bwd(const NormRows& a, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                               const float* rstd, const void* dsum, int64_t ld_dsum, float* part, float* dw,
                               hipStream_t st);

// ---------------------------------------------------------------- AdamW
constexpr int kMaxAdamTensors = 60;  // per launch: the table travels in the kernel's arguments, 4 KB at most
constexpr int kAdamChunk = 2048;     // elements of a tensor that a block takes
constexpr int64_t kMaxAdamChunks = ((int64_t(1) << 32) - 1) / 256;  // per launch: its threads are counted in 32 bits
// Consecutive tensors of a call; empty ones among them have no chunk.
template <int N>
struct AdamTable {
  float* p[N];
  const void* g[N];
  void* m[N];
  void* v[N];
  float* m_scale[N];
  float* v_scale[N];
  uint16_t* copy[N];
  int cum[N + 1];    // first chunk of each tensor, then their number
  uint16_t last[N];  // elements of a tensor's last chunk
  uint16_t n;
};
typedef AdamTable<kMaxAdamTensors> AdamBatch;
struct AdamStep {
  float beta1, rest1, beta2, rest2;  // rest = 1 - beta
  float keep;                        // 1 - lr * weight decay
  float step;                        // lr / (1 - beta1^t)
  float root;                        // 1 / sqrt(1 - beta2^t)
  float eps;
  uint32_t seed_lo, seed_hi;         // of the random numbers, with
  uint32_t place;                    // the place of the table's first tensor in the call's list
  const float* norm;                 // of all gradients, or NULL
  double max_norm;
};
hipError_t launch_adamw(const AdamBatch& b, const AdamStep& a, bool g_bf16, bool bits8, hipStream_t st);

}  // namespace fp8q
