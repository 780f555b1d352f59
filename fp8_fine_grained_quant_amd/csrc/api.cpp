// C ABI of libfp8q: host-side argument validation, then the asynchronous
// launch on the caller's stream.  Nothing here allocates, synchronises,
// prints or throws.  The entry points and their rules are documented in
// include/fp8q.h.  (Built with FP8Q_DEBUG, as libfp8q_debug.so, the grouped
// entry points also read the expert offsets back and check them, which
// synchronises the stream.)

#include "../../include/fp8q.h"
#include "launch.h"

#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

namespace fp8q {

namespace {
std::atomic<int> g_gemm_tile{0};  // fp8q_set_gemm_tile
constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];  // compute units per device, 0 = not yet queried
}  // namespace

int gemm_tile_setting() { return g_gemm_tile.load(std::memory_order_relaxed); }

int device_cu_count() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  cus = g_cus[dev].load(std::memory_order_relaxed);
  if (cus > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
  g_cus[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

}  // namespace fp8q

namespace {

using fp8q::GemmArgs;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int esize(fp8q_dtype t) { return t == FP8Q_BF16 ? 2 : 4; }
inline bool valid_dtype(fp8q_dtype t) { return t == FP8Q_BF16 || t == FP8Q_F32; }
inline fp8q_status launched(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_LAUNCH; }

constexpr int64_t kMaxGroups = (int64_t(1) << 31) - 1;

// Expert offsets live on the device and the product library never reads
// them: malformed offsets are undefined behaviour there.  The FP8Q_DEBUG
// build copies them to the host (after the work already on the stream) and
// rejects any that break the rule offsets[0] = 0, non-decreasing,
// offsets[E] = M_total, with FP8Q_ERR_SHAPE and nothing enqueued.
fp8q_status debug_check_offsets(const int32_t* offsets, int64_t E, int64_t M_total, hipStream_t stream) {
#ifdef FP8Q_DEBUG
  std::vector<int32_t> h((size_t)E + 1);
  if (hipMemcpyAsync(h.data(), offsets, h.size() * sizeof(int32_t), hipMemcpyDeviceToHost, stream) != hipSuccess ||
      hipStreamSynchronize(stream) != hipSuccess)
    return FP8Q_ERR_LAUNCH;
  if (h[0] != 0 || h[(size_t)E] != M_total) return FP8Q_ERR_SHAPE;
  for (size_t e = 0; e < (size_t)E; ++e)
    if (h[e + 1] < h[e]) return FP8Q_ERR_SHAPE;
#else
  (void)offsets; (void)E; (void)M_total; (void)stream;
#endif
  return FP8Q_OK;
}
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxContraction = 1024 * 128;  // the GEMM keeps one scale per chunk in LDS

// Checks shared by the three quantizers: input [rows, cols] with stride ld_in
// (elements of size in_es), code output with stride ld_out bytes covering
// out_len bytes per row, scale array of scale_rows x scale_cols with stride
// ld_s.
fp8q_status check_quant(const void* in, int in_es, int64_t rows, int64_t cols, int64_t ld_in,
                        const void* out, int64_t ld_out, int64_t out_len, const void* s, int64_t ld_s,
                        int64_t scale_cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return FP8Q_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP8Q_OK;
  if (!in || !out || !s) return FP8Q_ERR_NULL;
  if (ld_in < cols || ld_out < out_len || ld_s < scale_cols) return FP8Q_ERR_STRIDE;
  if (!aligned16(in) || !aligned16(out) || !aligned4(s)) return FP8Q_ERR_ALIGN;
  if ((ld_in * in_es) % 16 != 0 || ld_out % 16 != 0) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

fp8q_status check_gemm_out(const void* y, fp8q_dtype yt, int64_t ld_y, int64_t ncols) {
  if (!valid_dtype(yt)) return FP8Q_ERR_DTYPE;
  if (!y) return FP8Q_ERR_NULL;
  if (ld_y < ncols) return FP8Q_ERR_STRIDE;
  if (!aligned16(y) || (ld_y * esize(yt)) % 16 != 0) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

}  // namespace

extern "C" {

fp8q_status fp8q_set_gemm_tile(int tile) {
  if (tile < 0 || tile > 2) return FP8Q_ERR_SHAPE;
  fp8q::g_gemm_tile.store(tile, std::memory_order_relaxed);
  return FP8Q_OK;
}

const char* fp8q_status_string(fp8q_status s) {
  switch (s) {
    case FP8Q_OK: return "FP8Q_OK";
    case FP8Q_ERR_NULL: return "FP8Q_ERR_NULL: required pointer is NULL";
    case FP8Q_ERR_SHAPE: return "FP8Q_ERR_SHAPE: negative size or size rule broken";
    case FP8Q_ERR_STRIDE: return "FP8Q_ERR_STRIDE: leading dimension smaller than the row length";
    case FP8Q_ERR_ALIGN: return "FP8Q_ERR_ALIGN: pointer or row stride not aligned as required";
    case FP8Q_ERR_DTYPE: return "FP8Q_ERR_DTYPE: unsupported element type";
    case FP8Q_ERR_LAUNCH: return "FP8Q_ERR_LAUNCH: the HIP runtime refused a launch";
  }
  return "FP8Q: unknown status";
}

fp8q_status fp8q_quant_act_1x128(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                 uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  const fp8q_status c = check_quant(x, esize(xt), rows, cols, ld_x, q, ld_q, cols, scale, ld_s, cdiv(cols, 128));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (rows * cdiv(cols, 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  return launched(fp8q::launch_quant_act(x, xt == FP8Q_BF16, rows, cols, ld_x, q, ld_q, scale, ld_s, stream));
}

fp8q_status fp8q_quant_weight_128x128(const void* w, fp8q_dtype wt, int64_t rows, int64_t cols, int64_t ld_w,
                                      uint8_t* q, int64_t ld_q, uint8_t* q_t, int64_t ld_qt,
                                      float* scale, int64_t ld_s, hipStream_t stream) {
  if (!valid_dtype(wt)) return FP8Q_ERR_DTYPE;
  fp8q_status c = check_quant(w, esize(wt), rows, cols, ld_w, q, ld_q, cols, scale, ld_s, cdiv(cols, 128));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (q_t) {
    if (ld_qt < rows) return FP8Q_ERR_STRIDE;
    if (!aligned16(q_t) || ld_qt % 16 != 0) return FP8Q_ERR_ALIGN;
  }
  if (cdiv(rows, 128) > 65535) return FP8Q_ERR_SHAPE;  // grid y limit
  return launched(fp8q::launch_quant_weight(w, wt == FP8Q_BF16, rows, cols, ld_w, q, ld_q, q_t, ld_qt, scale,
                                            ld_s, stream));
}

fp8q_status fp8q_quant_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                 uint8_t* q_t, int64_t ld_qt, float* scale_t, int64_t ld_st, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  const fp8q_status c =
      check_quant(x, esize(xt), rows, cols, ld_x, q_t, ld_qt, rows, scale_t, ld_st, cdiv(rows, 128));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (cdiv(rows, 128) > 65535) return FP8Q_ERR_SHAPE;
  return launched(
      fp8q::launch_quant_transpose(x, xt == FP8Q_BF16, rows, cols, ld_x, q_t, ld_qt, scale_t, ld_st, stream));
}

fp8q_status fp8q_quant_act_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                     uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s, uint8_t* q_t,
                                     int64_t ld_qt, float* scale_t, int64_t ld_st, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  fp8q_status c = check_quant(x, esize(xt), rows, cols, ld_x, q, ld_q, cols, scale, ld_s, cdiv(cols, 128));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  c = check_quant(x, esize(xt), rows, cols, ld_x, q_t, ld_qt, rows, scale_t, ld_st, cdiv(rows, 128));
  if (c != FP8Q_OK) return c;
  if (cdiv(rows, 128) > 65535) return FP8Q_ERR_SHAPE;
  return launched(fp8q::launch_quant_act_transpose(x, xt == FP8Q_BF16, rows, cols, ld_x, q, ld_q, scale, ld_s,
                                                   q_t, ld_qt, scale_t, ld_st, stream));
}

fp8q_status fp8q_quant_transpose_grouped(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                         const int32_t* offsets, int64_t E, uint8_t* q_t, int64_t ld_qt,
                                         float* scale_t, int64_t ld_st, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (rows < 0 || rows > kMaxDim) return FP8Q_ERR_SHAPE;
  const int64_t cap = 128 * (rows / 128 + E);  // padded token capacity
  const fp8q_status c = check_quant(x, esize(xt), rows, cols, ld_x, q_t, ld_qt, cap, scale_t, ld_st, cap / 128);
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (!offsets) return FP8Q_ERR_NULL;
  if (!aligned4(offsets)) return FP8Q_ERR_ALIGN;
  if (cap / 128 > 65535) return FP8Q_ERR_SHAPE;  // grid y limit
  if (const fp8q_status d = debug_check_offsets(offsets, E, rows, stream); d != FP8Q_OK) return d;
  return launched(fp8q::launch_quant_transpose_grouped(x, xt == FP8Q_BF16, rows, cols, ld_x, offsets, E, q_t, ld_qt,
                                                       scale_t, ld_st, stream));
}

fp8q_status fp8q_quant_batch(const fp8q_quant_job* jobs, int n_jobs, hipStream_t stream) {
  if (n_jobs < 0 || n_jobs > FP8Q_MAX_QUANT_JOBS) return FP8Q_ERR_SHAPE;
  if (n_jobs == 0) return FP8Q_OK;
  if (!jobs) return FP8Q_ERR_NULL;
  fp8q::QuantJob qj[FP8Q_MAX_QUANT_JOBS];
  for (int i = 0; i < n_jobs; ++i) {
    const fp8q_quant_job& J = jobs[i];
    const fp8q_dtype xt = (fp8q_dtype)J.xt;
    if (J.kind < FP8Q_QUANT_ACT_1X128 || J.kind > FP8Q_QUANT_ACT_TRANSPOSE) return FP8Q_ERR_SHAPE;
    if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
    fp8q_status c = FP8Q_OK;
    const int64_t rows = J.rows, cols = J.cols;
    if (J.kind != FP8Q_QUANT_TRANSPOSE)
      c = check_quant(J.x, esize(xt), rows, cols, J.ld_x, J.q, J.ld_q, cols, J.scale, J.ld_s, cdiv(cols, 128));
    if (c == FP8Q_OK && (J.kind == FP8Q_QUANT_TRANSPOSE || J.kind == FP8Q_QUANT_ACT_TRANSPOSE))
      c = check_quant(J.x, esize(xt), rows, cols, J.ld_x, J.q_t, J.ld_qt, rows, J.scale_t, J.ld_st, cdiv(rows, 128));
    if (c == FP8Q_OK && J.kind == FP8Q_QUANT_WEIGHT_128X128 && rows > 0 && cols > 0 && J.q_t) {
      if (J.ld_qt < rows) c = FP8Q_ERR_STRIDE;
      else if (!aligned16(J.q_t) || J.ld_qt % 16 != 0) c = FP8Q_ERR_ALIGN;
    }
    if (c == FP8Q_OK && rows > 0 && cols > 0 && rows * cdiv(cols, 128) > kMaxGroups) c = FP8Q_ERR_SHAPE;
    if (c != FP8Q_OK) return c;
    fp8q::QuantJob& q = qj[i];
    q.kind = J.kind; q.x_bf16 = xt == FP8Q_BF16; q.x = J.x; q.rows = rows; q.cols = cols; q.ld_x = J.ld_x;
    const bool rows_out = J.kind != FP8Q_QUANT_TRANSPOSE, t_out = J.kind != FP8Q_QUANT_ACT_1X128;
    q.q = rows_out ? J.q : nullptr; q.ld_q = J.ld_q; q.s = rows_out ? J.scale : nullptr; q.ld_s = J.ld_s;
    q.q_t = t_out ? J.q_t : nullptr; q.ld_qt = J.ld_qt;
    q.s_t = t_out ? J.scale_t : nullptr; q.ld_st = J.ld_st;
  }
  if (fp8q::quant_batch_blocks(qj, n_jobs) > kMaxGroups) return FP8Q_ERR_SHAPE;  // one grid dimension
  return launched(fp8q::launch_quant_batch(qj, n_jobs, stream));
}

}  // extern "C"

// The fused output quantization's arguments: codes [rows, ncols] (row stride
// ld_q bytes) and scales [rows, ncols/128] (row stride ld_s).
static fp8q_status check_quant_out(const uint8_t* q, int64_t ld_q, const float* s, int64_t ld_s, int64_t ncols) {
  if (!q || !s) return FP8Q_ERR_NULL;
  if (ld_q < ncols || ld_s < ncols / 128) return FP8Q_ERR_STRIDE;
  if (!aligned16(q) || ld_q % 16 != 0 || !aligned4(s)) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

static fp8q_status fp8q_gemm_fprop_impl(int exact, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                            int64_t M, int64_t N, int64_t K, void* y, fp8q_dtype yt, int64_t ld_y,
                            hipStream_t stream, uint8_t* qo = nullptr, int64_t ld_qo = 0, float* so = nullptr,
                            int64_t ld_so = 0, bool quant_out = false) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || K > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(yt)) return FP8Q_ERR_DTYPE;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_SHAPE;  // an empty contraction would leave Y undefined
  if (!xq || !xs || !wq || !ws) return FP8Q_ERR_NULL;
  if (quant_out) {
    const fp8q_status c = check_quant_out(qo, ld_qo, so, ld_so, N);
    if (c != FP8Q_OK) return c;
  }
  if (!quant_out || y != nullptr) {
    const fp8q_status c = check_gemm_out(y, yt, ld_y, N);
    if (c != FP8Q_OK) return c;
  }
  if (!aligned16(xq) || !aligned16(wq) || !aligned4(xs) || !aligned4(ws)) return FP8Q_ERR_ALIGN;
  if (cdiv(M, 256) * (N / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;  // the launch grid
  GemmArgs a{};
  a.A = xq; a.B = wq; a.sa = xs; a.sb = ws; a.C = y;
  a.lda = K; a.ldb = K; a.ld_sa = K / 128; a.sb_rs = K / 128; a.sb_cs = 1; a.ldc = ld_y;
  a.M = M; a.N = N; a.K = K;
  a.sb_mode = fp8q::kSbBlock; a.out_f32 = yt == FP8Q_F32; a.accumulate = 0; a.exact = exact;
  a.qo = qo; a.ld_qo = ld_qo; a.so = so; a.ld_so = ld_so;
  return launched(fp8q::launch_gemm(a, stream));
}

static fp8q_status fp8q_gemm_dgrad_impl(int exact, const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                            int64_t M, int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                            hipStream_t stream, uint8_t* qo = nullptr, int64_t ld_qo = 0, float* so = nullptr,
                            int64_t ld_so = 0, bool quant_out = false) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || N > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(dxt)) return FP8Q_ERR_DTYPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (N == 0) return FP8Q_ERR_SHAPE;
  if (!dyq || !dys || !wq_t || !ws) return FP8Q_ERR_NULL;
  if (quant_out) {
    const fp8q_status c = check_quant_out(qo, ld_qo, so, ld_so, K);
    if (c != FP8Q_OK) return c;
  }
  if (!quant_out || dx != nullptr) {
    const fp8q_status c = check_gemm_out(dx, dxt, ld_dx, K);
    if (c != FP8Q_OK) return c;
  }
  if (!aligned16(dyq) || !aligned16(wq_t) || !aligned4(dys) || !aligned4(ws)) return FP8Q_ERR_ALIGN;
  if (cdiv(M, 256) * (K / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;  // the launch grid
  // NT form over the contraction axis N: A = dY [M, N], B = W^T codes [K, N];
  // the block scale of (output column k, chunk kb over N) is ws[kb, k/128].
  GemmArgs a{};
  a.A = dyq; a.B = wq_t; a.sa = dys; a.sb = ws; a.C = dx;
  a.lda = N; a.ldb = N; a.ld_sa = N / 128; a.sb_rs = 1; a.sb_cs = K / 128; a.ldc = ld_dx;
  a.M = M; a.N = K; a.K = N;
  a.sb_mode = fp8q::kSbBlock; a.out_f32 = dxt == FP8Q_F32; a.accumulate = 0; a.exact = exact;
  a.qo = qo; a.ld_qo = ld_qo; a.so = so; a.ld_so = ld_so;
  return launched(fp8q::launch_gemm(a, stream));
}

static fp8q_status fp8q_gemm_wgrad_impl(int exact, const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t, const float* xs_t,
                            int64_t T, int64_t N, int64_t K, float* dw, int64_t ld_dw, int accumulate,
                            hipStream_t stream) {
  if (T < 0 || N < 0 || K < 0 || T > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (T % 128 != 0 || K % 128 != 0 || T > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return FP8Q_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (T == 0) return FP8Q_ERR_SHAPE;
  if (!dyq_t || !dys_t || !xq_t || !xs_t) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(dw, FP8Q_F32, ld_dw, K);
  if (c != FP8Q_OK) return c;
  if (!aligned16(dyq_t) || !aligned16(xq_t) || !aligned4(dys_t) || !aligned4(xs_t)) return FP8Q_ERR_ALIGN;
  if (cdiv(N, 256) * (K / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;  // the launch grid
  // NT form over the tokens: A = dY^T codes [N, T], B = X^T codes [K, T], one
  // scale per row of each per 128 tokens.
  GemmArgs a{};
  a.A = dyq_t; a.B = xq_t; a.sa = dys_t; a.sb = xs_t; a.C = dw;
  a.lda = T; a.ldb = T; a.ld_sa = T / 128; a.sb_rs = T / 128; a.sb_cs = 1; a.ldc = ld_dw;
  a.M = N; a.N = K; a.K = T;
  a.sb_mode = fp8q::kSbRow; a.out_f32 = 1; a.accumulate = accumulate; a.exact = exact;
  return launched(fp8q::launch_gemm(a, stream));
}

static fp8q_status fp8q_grouped_gemm_impl(int exact, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                              const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                              void* y, fp8q_dtype yt, int64_t ld_y, hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(yt)) return FP8Q_ERR_DTYPE;
  if (M_total == 0 || N == 0) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_SHAPE;
  if (!xq || !xs || !wq || !ws || !offsets) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(y, yt, ld_y, N);
  if (c != FP8Q_OK) return c;
  if (!aligned16(xq) || !aligned16(wq) || !aligned4(xs) || !aligned4(ws) || !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  // the launch grid: a partial m-tile per expert on top of ceil(M_total / 256)
  if (((M_total + 255) / 256 + E) * (N / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  GemmArgs a{};
  a.A = xq; a.B = wq; a.sa = xs; a.sb = ws; a.C = y;
  a.lda = K; a.ldb = K; a.ld_sa = K / 128; a.sb_rs = K / 128; a.sb_cs = 1; a.ldc = ld_y;
  a.M = M_total; a.N = N; a.K = K;
  a.sb_mode = fp8q::kSbBlock; a.out_f32 = yt == FP8Q_F32; a.accumulate = 0; a.exact = exact;
  a.offsets = offsets; a.E = E; a.b_estride = N * K; a.sb_estride = (N / 128) * (K / 128);
  return launched(fp8q::launch_gemm(a, stream));
}


extern "C" {

fp8q_status fp8q_grouped_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                    const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                    void* dx, fp8q_dtype dxt, int64_t ld_dx, hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || N > kMaxContraction) return FP8Q_ERR_SHAPE;
  // the kernels address 256 rows of the stacked transposed codes (E*N bytes
  // each) with 32-bit buffer offsets
  if (E * N > INT32_MAX / 256) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(dxt)) return FP8Q_ERR_DTYPE;
  if (M_total == 0 || K == 0) return FP8Q_OK;
  if (N == 0) return FP8Q_ERR_SHAPE;
  if (!dyq || !dys || !wq_t || !ws || !offsets) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(dx, dxt, ld_dx, K);
  if (c != FP8Q_OK) return c;
  if (!aligned16(dyq) || !aligned16(wq_t) || !aligned4(dys) || !aligned4(ws) || !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  if (((M_total + 255) / 256 + E) * (K / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  // Per expert: the Dgrad NT form (A = dY rows of the expert, contraction N)
  // with B = W_e^T = columns [eN, (e+1)N) of the stacked transposed codes
  // [K, E*N], and the block scale of (output column k, chunk kb) at
  // ws[e*N/128 + kb, k/128].
  GemmArgs a{};
  a.A = dyq; a.B = wq_t; a.sa = dys; a.sb = ws; a.C = dx;
  a.lda = N; a.ldb = E * N; a.ld_sa = N / 128; a.sb_rs = 1; a.sb_cs = K / 128; a.ldc = ld_dx;
  a.M = M_total; a.N = K; a.K = N;
  a.sb_mode = fp8q::kSbBlock; a.out_f32 = dxt == FP8Q_F32; a.accumulate = 0; a.exact = 0;
  a.offsets = offsets; a.E = E; a.b_estride = N; a.sb_estride = (N / 128) * (K / 128);
  return launched(fp8q::launch_gemm(a, stream));
}

fp8q_status fp8q_grouped_gemm_wgrad(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t,
                                    const float* xs_t, const int32_t* offsets, int64_t E, int64_t M_total,
                                    int64_t N, int64_t K, int64_t ld_t, float* dw, int accumulate,
                                    hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (K % 128 != 0 || M_total > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return FP8Q_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (!dyq_t || !dys_t || !xq_t || !xs_t || !offsets || !dw) return FP8Q_ERR_NULL;
  const int64_t cap = 128 * (M_total / 128 + E);
  if (ld_t < cap) return FP8Q_ERR_STRIDE;
  if (ld_t % 128 != 0) return FP8Q_ERR_ALIGN;
  // the kernels address 256 operand rows (ld_t bytes each) with 32-bit buffer offsets
  if (ld_t > INT32_MAX / 256) return FP8Q_ERR_SHAPE;
  if (!aligned16(dyq_t) || !aligned16(xq_t) || !aligned16(dw) || !aligned4(dys_t) || !aligned4(xs_t) ||
      !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  if (E * ((N + 255) / 256) * (K / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  // Per expert: the Wgrad NT form over the expert's padded token chunks
  // (A = dY^T codes [N, ld_t], B = X^T codes [K, ld_t], one scale per row
  // per chunk), written to dw + e*N*K.
  GemmArgs a{};
  a.A = dyq_t; a.B = xq_t; a.sa = dys_t; a.sb = xs_t; a.C = dw;
  a.lda = ld_t; a.ldb = ld_t; a.ld_sa = ld_t / 128; a.sb_rs = ld_t / 128; a.sb_cs = 1; a.ldc = K;
  a.M = N; a.N = K; a.K = ld_t;
  a.sb_mode = fp8q::kSbRow; a.out_f32 = 1; a.accumulate = accumulate; a.exact = 0;
  a.offsets = offsets; a.E = E; a.b_estride = 0; a.sb_estride = 0;
  a.k_grouped = 1; a.c_estride = N * K;
  return launched(fp8q::launch_gemm(a, stream));
}

fp8q_status fp8q_gemm_fprop_quant(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M,
                                  int64_t N, int64_t K, void* y, int64_t ld_y, uint8_t* yq, int64_t ld_yq, float* ys,
                                  int64_t ld_ys, int exact, hipStream_t stream) {
  if (exact != 0 && exact != 1) return FP8Q_ERR_SHAPE;
  return fp8q_gemm_fprop_impl(exact, xq, xs, wq, ws, M, N, K, y, FP8Q_BF16, ld_y, stream, yq, ld_yq, ys, ld_ys, true);
}
fp8q_status fp8q_gemm_dgrad_quant(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* dx, int64_t ld_dx, uint8_t* dxq,
                                  int64_t ld_dxq, float* dxs, int64_t ld_dxs, int exact, hipStream_t stream) {
  if (exact != 0 && exact != 1) return FP8Q_ERR_SHAPE;
  return fp8q_gemm_dgrad_impl(exact, dyq, dys, wq_t, ws, M, N, K, dx, FP8Q_BF16, ld_dx, stream, dxq, ld_dxq, dxs,
                              ld_dxs, true);
}
fp8q_status fp8q_gemm_fprop_interval(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                     int64_t M, int64_t N, int64_t K, float* y, int64_t ld_y, int64_t interval,
                                     hipStream_t stream) {
  int chunks = -1;
  if (interval == 0) chunks = 0;
  else if (interval == 128 || interval == 256 || interval == 512 || interval == 1024) chunks = (int)(interval / 128);
  if (chunks < 0) return FP8Q_ERR_SHAPE;
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 512 != 0 || K > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_SHAPE;
  if (!xq || !xs || !wq || !ws) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(y, FP8Q_F32, ld_y, N);
  if (c != FP8Q_OK) return c;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(xs) || !aligned4(ws)) return FP8Q_ERR_ALIGN;
  if (cdiv(M, 256) * (N / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  GemmArgs a{};
  a.A = xq; a.B = wq; a.sa = xs; a.sb = ws; a.C = y;
  a.lda = K; a.ldb = K; a.ld_sa = K / 128; a.sb_rs = K / 128; a.sb_cs = 1; a.ldc = ld_y;
  a.M = M; a.N = N; a.K = K;
  a.sb_mode = fp8q::kSbBlock; a.out_f32 = 1;
  return launched(fp8q::launch_gemm_interval(a, chunks, stream));
}

fp8q_status fp8q_gemm_fprop(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M,
                            int64_t N, int64_t K, void* y, fp8q_dtype yt, int64_t ld_y, hipStream_t stream) {
  return fp8q_gemm_fprop_impl(0, xq, xs, wq, ws, M, N, K, y, yt, ld_y, stream);
}
fp8q_status fp8q_gemm_fprop_exact(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* y, fp8q_dtype yt, int64_t ld_y,
                                  hipStream_t stream) {
  return fp8q_gemm_fprop_impl(1, xq, xs, wq, ws, M, N, K, y, yt, ld_y, stream);
}
fp8q_status fp8q_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws, int64_t M,
                            int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx, hipStream_t stream) {
  return fp8q_gemm_dgrad_impl(0, dyq, dys, wq_t, ws, M, N, K, dx, dxt, ld_dx, stream);
}
fp8q_status fp8q_gemm_dgrad_exact(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                  int64_t M, int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                                  hipStream_t stream) {
  return fp8q_gemm_dgrad_impl(1, dyq, dys, wq_t, ws, M, N, K, dx, dxt, ld_dx, stream);
}
fp8q_status fp8q_gemm_wgrad(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t, const float* xs_t,
                            int64_t T, int64_t N, int64_t K, float* dw, int64_t ld_dw, int accumulate,
                            hipStream_t stream) {
  return fp8q_gemm_wgrad_impl(0, dyq_t, dys_t, xq_t, xs_t, T, N, K, dw, ld_dw, accumulate, stream);
}
fp8q_status fp8q_gemm_wgrad_exact(const uint8_t* dyq_t, const float* dys_t, const uint8_t* xq_t, const float* xs_t,
                                  int64_t T, int64_t N, int64_t K, float* dw, int64_t ld_dw, int accumulate,
                                  hipStream_t stream) {
  return fp8q_gemm_wgrad_impl(1, dyq_t, dys_t, xq_t, xs_t, T, N, K, dw, ld_dw, accumulate, stream);
}
fp8q_status fp8q_grouped_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                              const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K, void* y,
                              fp8q_dtype yt, int64_t ld_y, hipStream_t stream) {
  return fp8q_grouped_gemm_impl(0, xq, xs, wq, ws, offsets, E, M_total, N, K, y, yt, ld_y, stream);
}
fp8q_status fp8q_grouped_gemm_exact(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                    const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                    void* y, fp8q_dtype yt, int64_t ld_y, hipStream_t stream) {
  return fp8q_grouped_gemm_impl(1, xq, xs, wq, ws, offsets, E, M_total, N, K, y, yt, ld_y, stream);
}

}  // extern "C"

extern "C" {

fp8q_status fp8q_quant_mx_1x32(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* q,
                               int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  const fp8q_status c = check_quant(x, esize(xt), rows, cols, ld_x, q, ld_q, cols, s, ld_s, cdiv(cols, 32));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (rows * cdiv(cols, 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  return launched(fp8q::launch_quant_mx(x, xt == FP8Q_BF16, rows, cols, ld_x, q, ld_q, s, ld_s, stream));
}

fp8q_status fp8q_quant_mx_transpose(const void* x, fp8q_dtype xt, int64_t rows, int64_t cols, int64_t ld_x,
                                    uint8_t* q_t, int64_t ld_qt, uint8_t* s_t, int64_t ld_st, uint8_t* q,
                                    int64_t ld_q, uint8_t* s, int64_t ld_s, hipStream_t stream) {
  if (!valid_dtype(xt)) return FP8Q_ERR_DTYPE;
  if ((q == nullptr) != (s == nullptr)) return FP8Q_ERR_NULL;
  fp8q_status c = check_quant(x, esize(xt), rows, cols, ld_x, q_t, ld_qt, rows, s_t, ld_st, cdiv(rows, 32));
  if (c != FP8Q_OK || rows == 0 || cols == 0) return c;
  if (q) {
    c = check_quant(x, esize(xt), rows, cols, ld_x, q, ld_q, cols, s, ld_s, cdiv(cols, 32));
    if (c != FP8Q_OK) return c;
  }
  if (cdiv(rows, 128) > 65535) return FP8Q_ERR_SHAPE;
  return launched(fp8q::launch_quant_mx_transpose(x, xt == FP8Q_BF16, rows, cols, ld_x, q_t, ld_qt, s_t, ld_st, q,
                                                  ld_q, s, ld_s, stream));
}

fp8q_status fp8q_gemm_mx(const uint8_t* aq, const uint8_t* as, int64_t lda, int64_t ld_sa, const uint8_t* bq,
                         const uint8_t* bs, int64_t ldb, int64_t ld_sb, int64_t M, int64_t N, int64_t K, void* c,
                         fp8q_dtype ct, int64_t ld_c, int accumulate, hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || K > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(ct)) return FP8Q_ERR_DTYPE;
  if (accumulate && ct != FP8Q_F32) return FP8Q_ERR_DTYPE;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_SHAPE;
  if (!aq || !as || !bq || !bs) return FP8Q_ERR_NULL;
  const fp8q_status st = check_gemm_out(c, ct, ld_c, N);
  if (st != FP8Q_OK) return st;
  if (lda < K || ldb < K || ld_sa < K / 32 || ld_sb < K / 32) return FP8Q_ERR_STRIDE;
  if (!aligned16(aq) || !aligned16(bq) || lda % 16 != 0 || ldb % 16 != 0) return FP8Q_ERR_ALIGN;
  if (!aligned4(as) || !aligned4(bs) || ld_sa % 4 != 0 || ld_sb % 4 != 0) return FP8Q_ERR_ALIGN;
  // the kernel's buffer descriptors address one tile's rows with 32-bit offsets
  if (256 * lda > INT32_MAX || 128 * ldb > INT32_MAX) return FP8Q_ERR_SHAPE;
  if (cdiv(M, 256) * (N / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;  // the launch grid
  fp8q::MxArgs a{};
  a.g.A = aq; a.g.B = bq; a.g.C = c;
  a.g.lda = lda; a.g.ldb = ldb; a.g.ldc = ld_c;
  a.g.M = M; a.g.N = N; a.g.K = K;
  a.g.out_f32 = ct == FP8Q_F32; a.g.accumulate = accumulate;
  a.sa = as; a.sb = bs; a.ld_sa = ld_sa; a.ld_sb = ld_sb;
  return launched(fp8q::launch_gemm_mx(a, stream));
}

fp8q_status fp8q_grouped_gemm_mx(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                                 const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K, void* y,
                                 fp8q_dtype yt, int64_t ld_y, hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || K > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(yt)) return FP8Q_ERR_DTYPE;
  if (M_total == 0 || N == 0) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_SHAPE;
  if (!xq || !xs || !wq || !ws || !offsets) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(y, yt, ld_y, N);
  if (c != FP8Q_OK) return c;
  // scale rows are K/32 bytes, a multiple of 4 since K % 128 == 0
  if (!aligned16(xq) || !aligned16(wq) || !aligned4(xs) || !aligned4(ws) || !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  if (((M_total + 255) / 256 + E) * (N / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  fp8q::MxArgs a{};
  a.g.A = xq; a.g.B = wq; a.g.C = y;
  a.g.lda = K; a.g.ldb = K; a.g.ldc = ld_y;
  a.g.M = M_total; a.g.N = N; a.g.K = K;
  a.g.out_f32 = yt == FP8Q_F32; a.g.accumulate = 0;
  a.g.offsets = offsets; a.g.E = E; a.g.b_estride = N * K;
  a.sa = xs; a.sb = ws; a.ld_sa = K / 32; a.ld_sb = K / 32; a.sb_estride = N * (K / 32);
  return launched(fp8q::launch_gemm_mx(a, stream));
}

fp8q_status fp8q_grouped_gemm_mx_dgrad(const uint8_t* dyq, const uint8_t* dys, const uint8_t* wq_t,
                                       const uint8_t* ws_t, const int32_t* offsets, int64_t E, int64_t M_total,
                                       int64_t N, int64_t K, void* dx, fp8q_dtype dxt, int64_t ld_dx,
                                       hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8Q_ERR_SHAPE;
  if (N % 128 != 0 || K % 128 != 0 || N > kMaxContraction) return FP8Q_ERR_SHAPE;
  // the kernel addresses 128 rows of the stacked transposed codes (E*N bytes each) with 32-bit offsets
  if (E * N > INT32_MAX / 128) return FP8Q_ERR_SHAPE;
  if (!valid_dtype(dxt)) return FP8Q_ERR_DTYPE;
  if (M_total == 0 || K == 0) return FP8Q_OK;
  if (N == 0) return FP8Q_ERR_SHAPE;
  if (!dyq || !dys || !wq_t || !ws_t || !offsets) return FP8Q_ERR_NULL;
  const fp8q_status c = check_gemm_out(dx, dxt, ld_dx, K);
  if (c != FP8Q_OK) return c;
  if (!aligned16(dyq) || !aligned16(wq_t) || !aligned4(dys) || !aligned4(ws_t) || !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  if (((M_total + 255) / 256 + E) * (K / 128) > kMaxGroups) return FP8Q_ERR_SHAPE;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  // Per expert: C = dY rows . B^T with B = W_e^T = columns [eN, (e+1)N) of
  // the stacked transposed codes (row stride E*N) and of their scales (E*N/32)
  fp8q::MxArgs a{};
  a.g.A = dyq; a.g.B = wq_t; a.g.C = dx;
  a.g.lda = N; a.g.ldb = E * N; a.g.ldc = ld_dx;
  a.g.M = M_total; a.g.N = K; a.g.K = N;
  a.g.out_f32 = dxt == FP8Q_F32; a.g.accumulate = 0;
  a.g.offsets = offsets; a.g.E = E; a.g.b_estride = N;
  a.sa = dys; a.sb = ws_t; a.ld_sa = N / 32; a.ld_sb = E * N / 32; a.sb_estride = N / 32;
  return launched(fp8q::launch_gemm_mx(a, stream));
}

}  // extern "C"

// ------------------------------------------------------------- MoE routing
namespace {

// Rows accessed at any element alignment (the MoE row kernels).
inline bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }

fp8q_status check_rows(const void* p, fp8q_dtype t, int64_t ld, int64_t cols) {
  if (!p) return FP8Q_ERR_NULL;
  if (ld < cols) return FP8Q_ERR_STRIDE;
  return aligned_to(p, esize(t)) ? FP8Q_OK : FP8Q_ERR_ALIGN;
}

fp8q_status check_route(fp8q_dtype lt, int64_t T, int64_t E, int k, int score, int renormalize, float scale) {
  if (!valid_dtype(lt)) return FP8Q_ERR_DTYPE;
  if (T < 0 || T > kMaxDim || E < 1 || E > fp8q::kMaxExperts || k < 1 || k > fp8q::kMaxTopK || k > E ||
      T * k > kMaxDim)
    return FP8Q_ERR_SHAPE;
  if ((score != FP8Q_SOFTMAX && score != FP8Q_SIGMOID) || (renormalize != 0 && renormalize != 1) ||
      !(scale - scale == 0.f))
    return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

// The sizes of the row entry points: columns, groups and 8-column pieces are
// counted in 32 bits, past a row's end too.  A launch with a thread for each
// piece of a token's columns has at most 1.6 times as many threads, below 2^32;
// those with more go in parts.
fp8q_status check_moe_rows(fp8q_dtype t, int64_t T, int64_t H, int k) {
  if (!valid_dtype(t)) return FP8Q_ERR_DTYPE;
  if (T < 0 || H < 0 || T > kMaxDim || H > kMaxDim || k < 1 || k > fp8q::kMaxTopK || T * k > kMaxDim)
    return FP8Q_ERR_SHAPE;
  if (H > kMaxDim / 2 || T * (cdiv(H, 8) + 15) > kMaxDim) return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

fp8q_status check_codes(const uint8_t* q, int64_t ld_q, const float* s, int64_t ld_s, int64_t H) {
  if (!q || !s) return FP8Q_ERR_NULL;
  if (ld_q < H || ld_s < cdiv(H, 128)) return FP8Q_ERR_STRIDE;
  return aligned4(s) ? FP8Q_OK : FP8Q_ERR_ALIGN;
}

// The map of the row entry points lives on the device, as the expert offsets
// do; the FP8Q_DEBUG build rejects one that is not a permutation of the rows.
fp8q_status debug_check_dst(const int32_t* dst, int64_t m, hipStream_t stream) {
#ifdef FP8Q_DEBUG
  try {
    std::vector<int32_t> h((size_t)m);
    if (hipMemcpyAsync(h.data(), dst, h.size() * sizeof(int32_t), hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
      return FP8Q_ERR_LAUNCH;
    std::vector<bool> seen((size_t)m, false);
    for (const int32_t d : h) {
      const int64_t r = d >= 0 ? (int64_t)d : -1 - (int64_t)d;
      if (r >= m || seen[(size_t)r]) return FP8Q_ERR_SHAPE;
      seen[(size_t)r] = true;
    }
  } catch (const std::bad_alloc&) {  // no memory for the copy: nothing was checked
    return FP8Q_ERR_LAUNCH;
  }
#else
  (void)dst; (void)m; (void)stream;
#endif
  return FP8Q_OK;
}

}  // namespace

extern "C" {

fp8q_status fp8q_moe_route(const void* logits, fp8q_dtype lt, int64_t T, int64_t E, int64_t ld, int k, int score,
                           const float* bias, int renormalize, float scale, int32_t* ids, float* weights,
                           hipStream_t stream) {
  if (const fp8q_status c = check_route(lt, T, E, k, score, renormalize, scale); c != FP8Q_OK || T == 0) return c;
  if (const fp8q_status c = check_rows(logits, lt, ld, E); c != FP8Q_OK) return c;
  if (!ids || !weights) return FP8Q_ERR_NULL;
  if (!aligned4(ids) || !aligned4(weights) || !aligned4(bias)) return FP8Q_ERR_ALIGN;
  const fp8q::MoeRoute a{logits, lt == FP8Q_BF16, score == FP8Q_SIGMOID, renormalize == 1, T, E, ld, k, scale};
  return launched(fp8q::launch_moe_route(a, bias, ids, weights, stream));
}

fp8q_status fp8q_moe_route_bwd(const float* dweights, const void* logits, fp8q_dtype lt, int64_t T, int64_t E,
                               int64_t ld, const int32_t* ids, int k, int score, int renormalize, float scale,
                               void* dlogits, int64_t ld_d, hipStream_t stream) {
  if (const fp8q_status c = check_route(lt, T, E, k, score, renormalize, scale); c != FP8Q_OK || T == 0) return c;
  if (const fp8q_status c = check_rows(logits, lt, ld, E); c != FP8Q_OK) return c;
  if (const fp8q_status c = check_rows(dlogits, lt, ld_d, E); c != FP8Q_OK) return c;
  if (!dweights || !ids) return FP8Q_ERR_NULL;
  if (!aligned4(dweights) || !aligned4(ids)) return FP8Q_ERR_ALIGN;
  const fp8q::MoeRoute a{logits, lt == FP8Q_BF16, score == FP8Q_SIGMOID, renormalize == 1, T, E, ld, k, scale};
  return launched(fp8q::launch_moe_route_bwd(a, dweights, ids, dlogits, ld_d, stream));
}

int64_t fp8q_moe_sort_workspace(int64_t M, int64_t E) {
  if (M < 0 || M > kMaxDim || E < 1 || E > fp8q::kMaxExperts) return -1;
  return fp8q::moe_sort_workspace(M, E);
}

fp8q_status fp8q_moe_sort(const int32_t* ids, int64_t M, int64_t E, int cover, int32_t* offsets, int32_t* dst,
                          int32_t* src, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (M < 0 || M > kMaxDim || E < 1 || E > fp8q::kMaxExperts || (cover != 0 && cover != 1)) return FP8Q_ERR_SHAPE;
  if (!offsets || (M > 0 && (!ids || !dst))) return FP8Q_ERR_NULL;
  if (!aligned4(ids) || !aligned4(offsets) || !aligned4(dst) || !aligned4(src)) return FP8Q_ERR_ALIGN;
  const int64_t need = fp8q::moe_sort_workspace(M, E);
  if (need > 0) {
    if (!workspace) return FP8Q_ERR_NULL;
    if (!aligned4(workspace)) return FP8Q_ERR_ALIGN;
    if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
  }
  return launched(fp8q::launch_moe_sort(ids, M, E, cover == 1, offsets, dst, src, workspace, stream));
}

fp8q_status fp8q_moe_dispatch(const void* x, fp8q_dtype xt, int64_t T, int64_t H, int64_t ld_x, const int32_t* dst,
                              int k, void* rows, int64_t ld_rows, uint8_t* q, int64_t ld_q, float* scale,
                              int64_t ld_s, hipStream_t stream) {
  if (const fp8q_status c = check_moe_rows(xt, T, H, k); c != FP8Q_OK || T == 0 || H == 0) return c;
  if (const fp8q_status c = check_rows(x, xt, ld_x, H); c != FP8Q_OK) return c;
  if (!dst || (!rows && !q)) return FP8Q_ERR_NULL;
  if (!aligned4(dst)) return FP8Q_ERR_ALIGN;
  if (rows)
    if (const fp8q_status c = check_rows(rows, xt, ld_rows, H); c != FP8Q_OK) return c;
  if (q)
    if (const fp8q_status c = check_codes(q, ld_q, scale, ld_s, H); c != FP8Q_OK) return c;
  if (const fp8q_status c = debug_check_dst(dst, T * k, stream); c != FP8Q_OK) return c;
  const fp8q::MoeRows a{xt == FP8Q_BF16, T, k, H, dst, rows, ld_rows, q, ld_q, scale, ld_s};
  return launched(fp8q::launch_moe_dispatch(a, x, ld_x, stream));
}

fp8q_status fp8q_moe_dispatch_bwd(const void* drows, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_rows,
                                  const int32_t* dst, int k, void* dx, int64_t ld_dx, hipStream_t stream) {
  if (const fp8q_status c = check_moe_rows(t, T, H, k); c != FP8Q_OK || T == 0 || H == 0) return c;
  if (const fp8q_status c = check_rows(drows, t, ld_rows, H); c != FP8Q_OK) return c;
  if (const fp8q_status c = check_rows(dx, t, ld_dx, H); c != FP8Q_OK) return c;
  if (!dst) return FP8Q_ERR_NULL;
  if (!aligned4(dst)) return FP8Q_ERR_ALIGN;
  if (const fp8q_status c = debug_check_dst(dst, T * k, stream); c != FP8Q_OK) return c;
  const fp8q::MoeRows a{t == FP8Q_BF16, T, k, H, dst, const_cast<void*>(drows), ld_rows, nullptr, 0, nullptr, 0};
  return launched(fp8q::launch_moe_gather(a, nullptr, dx, ld_dx, stream));
}

fp8q_status fp8q_moe_combine(const void* yp, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_yp, const int32_t* dst,
                             int k, const float* weights, void* y, int64_t ld_y, hipStream_t stream) {
  if (const fp8q_status c = check_moe_rows(t, T, H, k); c != FP8Q_OK || T == 0 || H == 0) return c;
  if (const fp8q_status c = check_rows(yp, t, ld_yp, H); c != FP8Q_OK) return c;
  if (const fp8q_status c = check_rows(y, t, ld_y, H); c != FP8Q_OK) return c;
  if (!dst || !weights) return FP8Q_ERR_NULL;
  if (!aligned4(dst) || !aligned4(weights)) return FP8Q_ERR_ALIGN;
  if (const fp8q_status c = debug_check_dst(dst, T * k, stream); c != FP8Q_OK) return c;
  const fp8q::MoeRows a{t == FP8Q_BF16, T, k, H, dst, const_cast<void*>(yp), ld_yp, nullptr, 0, nullptr, 0};
  return launched(fp8q::launch_moe_gather(a, weights, y, ld_y, stream));
}

fp8q_status fp8q_moe_combine_bwd(const void* dy, const void* yp, fp8q_dtype t, int64_t T, int64_t H, int64_t ld_dy,
                                 int64_t ld_yp, const int32_t* dst, int k, const float* weights, void* rows,
                                 int64_t ld_rows, uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s,
                                 float* dweights, hipStream_t stream) {
  if (const fp8q_status c = check_moe_rows(t, T, H, k); c != FP8Q_OK || T == 0) return c;
  if (!dst || !weights || !dweights) return FP8Q_ERR_NULL;
  if (H > 0) {
    if (!rows && !q) return FP8Q_ERR_NULL;
    if (const fp8q_status c = check_rows(dy, t, ld_dy, H); c != FP8Q_OK) return c;
    if (const fp8q_status c = check_rows(yp, t, ld_yp, H); c != FP8Q_OK) return c;
    if (rows)
      if (const fp8q_status c = check_rows(rows, t, ld_rows, H); c != FP8Q_OK) return c;
    if (q)
      if (const fp8q_status c = check_codes(q, ld_q, scale, ld_s, H); c != FP8Q_OK) return c;
  }
  if (!aligned4(dst) || !aligned4(weights) || !aligned4(dweights)) return FP8Q_ERR_ALIGN;
  if (const fp8q_status c = debug_check_dst(dst, T * k, stream); c != FP8Q_OK) return c;
  const fp8q::MoeRows a{t == FP8Q_BF16, T, k, H, dst, rows, ld_rows, q, ld_q, scale, ld_s};
  return launched(fp8q::launch_moe_combine_bwd(a, dy, ld_dy, yp, ld_yp, weights, dweights, stream));
}

int64_t fp8q_grad_clip_workspace(int64_t n) {
  if (n < 0 || n > kMaxDim) return -1;
  if (n == 0) return 0;
  // partial sums, and for each launch the table the second pass reads
  return fp8q::kClipBlocks * (int64_t)sizeof(double) + cdiv(n, fp8q::kMaxClipTensors) * (int64_t)sizeof(fp8q::ClipBatch);
}

fp8q_status fp8q_grad_clip(const fp8q_grad* grads, int64_t n, fp8q_dtype ot, double max_norm, void* workspace,
                           int64_t workspace_bytes, float* norm, hipStream_t stream) {
  if (!valid_dtype(ot)) return FP8Q_ERR_DTYPE;
  if (n < 0 || n > kMaxDim || !(max_norm >= 0.0)) return FP8Q_ERR_SHAPE;
  if (!norm || (n > 0 && (!grads || !workspace))) return FP8Q_ERR_NULL;
  if (!aligned4(norm) || !aligned_to(workspace, 8)) return FP8Q_ERR_ALIGN;
  if (workspace_bytes < fp8q_grad_clip_workspace(n)) return FP8Q_ERR_SHAPE;
  int64_t chunks = 0;  // of all tensors: counted in 32 bits
  for (int64_t i = 0; i < n; ++i) {
    const fp8q_grad& g = grads[i];
    if (g.len < 0 || (chunks += cdiv(g.len, fp8q::kClipChunk)) > kMaxDim / 2) return FP8Q_ERR_SHAPE;
    if (g.len == 0) continue;
    if (!g.g || !g.out) return FP8Q_ERR_NULL;
    if (!aligned4(g.g) || !aligned_to(g.out, esize(ot))) return FP8Q_ERR_ALIGN;
  }
  // tables of up to kMaxClipTensors non-empty tensors, one launch each and pass
  static_assert(sizeof(fp8q::ClipBatch) % 8 == 0, "tables follow each other");
  double* const part = static_cast<double*>(workspace);
  fp8q::ClipBatch* const tables = reinterpret_cast<fp8q::ClipBatch*>(part + fp8q::kClipBlocks);
  int parts = 0, batches = 0;
  fp8q::ClipBatch b;
  for (int64_t i = 0; i < n;) {
    b.n = 0;
    b.cum[0] = 0;
    for (; i < n && b.n < fp8q::kMaxClipTensors; ++i) {
      const int64_t len = grads[i].len, c = cdiv(len, fp8q::kClipChunk);
      if (c == 0) continue;
      b.g[b.n] = grads[i].g;
      b.out[b.n] = grads[i].out;
      b.last[b.n] = (uint16_t)(len - (c - 1) * fp8q::kClipChunk);
      b.cum[b.n + 1] = b.cum[b.n] + (int)c;
      ++b.n;
    }
    if (b.n == 0) break;
    if (fp8q::launch_grad_sumsq(b, tables + batches, part, &parts, stream) != hipSuccess) return FP8Q_ERR_LAUNCH;
    ++batches;
  }
  // the second pass of the batches before the last: counted again from the sizes
  int64_t i = 0;
  for (int k = 0; k < (batches > 0 ? batches : 1); ++k) {
    int tensors = 0, chunk_count = 0;
    for (; i < n && tensors < fp8q::kMaxClipTensors; ++i) {
      const int c = (int)cdiv(grads[i].len, fp8q::kClipChunk);
      tensors += c > 0;
      chunk_count += c;
    }
    if (fp8q::launch_grad_scale(tables + k, chunk_count, ot == FP8Q_BF16, part, parts, max_norm,
                                k == 0 ? norm : nullptr, stream) != hipSuccess)
      return FP8Q_ERR_LAUNCH;
  }
  return FP8Q_OK;
}

}  // extern "C"

// ---------------------------------------------------- gated feed-forward block
namespace {

// A launch's threads are counted in 32 bits: tiles of 512 threads.
constexpr int64_t kMaxTiles = ((int64_t(1) << 32) - 1) / 512;

// The sizes of the gated block's entry points: outputs of gate and of up each,
// contraction length, 256-row tiles.
fp8q_status check_gated(int64_t M, int64_t width, int64_t inner, int64_t tiles_m) {
  if (M < 0 || width < 0 || inner < 0 || M > kMaxDim || width > kMaxDim / 2 || inner > kMaxDim) return FP8Q_ERR_SHAPE;
  if (width % 128 != 0 || inner % 128 != 0 || inner > kMaxContraction) return FP8Q_ERR_SHAPE;
  if (M == 0 || width == 0) return FP8Q_OK;
  if (inner == 0) return FP8Q_ERR_SHAPE;  // an empty contraction would leave the outputs undefined
  return tiles_m * (width / 128) > kMaxTiles ? FP8Q_ERR_SHAPE : FP8Q_OK;
}

// BF16 matrices of the gated block's entry points, NULL where they are not given.
fp8q_status check_bf16(const void* p, int64_t ld, int64_t cols) {
  return p ? check_gemm_out(p, FP8Q_BF16, ld, cols) : FP8Q_OK;
}

fp8q_status check_swiglu_out(const void* h, int64_t ld_h, const void* gu, int64_t ld_gu, const uint8_t* q, int64_t ld_q,
                             const float* s, int64_t ld_s, int64_t N) {
  if (!h && !gu && !q) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_bf16(h, ld_h, N); c != FP8Q_OK) return c;
  if (const fp8q_status c = check_bf16(gu, ld_gu, 2 * N); c != FP8Q_OK) return c;
  return q || s ? check_quant_out(q, ld_q, s, ld_s, N) : FP8Q_OK;
}

GemmArgs swiglu_args(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M, int64_t N,
                     int64_t K, void* h, int64_t ld_h, void* gu, int64_t ld_gu, uint8_t* q, int64_t ld_q, float* s,
                     int64_t ld_s) {
  GemmArgs a{};
  a.A = xq; a.B = wq; a.sa = xs; a.sb = ws; a.C = h;
  a.lda = K; a.ldb = K; a.ld_sa = K / 128; a.sb_rs = K / 128; a.sb_cs = 1; a.ldc = ld_h;
  a.M = M; a.N = N; a.K = K;
  a.sb_mode = fp8q::kSbBlock; a.gated = fp8q::kSwiglu;
  a.gu = static_cast<uint16_t*>(gu); a.ld_gu = ld_gu;
  a.qo = q; a.ld_qo = ld_q; a.so = s; a.ld_so = ld_s;
  return a;
}

// The gradient's matrices: gu and dgu [rows, 2K], h optional [rows, K].
fp8q_status check_dswiglu(const void* gu, int64_t ld_gu, const void* dgu, int64_t ld_dgu, const void* h, int64_t ld_h,
                          int64_t K) {
  if (!gu || !dgu) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_bf16(gu, ld_gu, 2 * K); c != FP8Q_OK) return c;
  if (const fp8q_status c = check_bf16(dgu, ld_dgu, 2 * K); c != FP8Q_OK) return c;
  return check_bf16(h, ld_h, K);
}

}  // namespace

extern "C" {

int64_t fp8q_gemm_swiglu_workspace(int64_t M, int64_t N, int64_t K, int codes) {
  if (check_gated(M, N, K, cdiv(M, 256)) != FP8Q_OK) return -1;
  return codes && fp8q::swiglu_few(M, N, K) ? M * N * (int64_t)sizeof(float) : 0;
}

fp8q_status fp8q_gemm_swiglu(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M,
                             int64_t N, int64_t K, void* h, int64_t ld_h, void* gu, int64_t ld_gu, uint8_t* q,
                             int64_t ld_q, float* scale, int64_t ld_s, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
  if (const fp8q_status c = check_gated(M, N, K, cdiv(M, 256)); c != FP8Q_OK || M == 0 || N == 0) return c;
  if (!xq || !xs || !wq || !ws) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_swiglu_out(h, ld_h, gu, ld_gu, q, ld_q, scale, ld_s, N); c != FP8Q_OK) return c;
  if (!aligned16(xq) || !aligned16(wq) || !aligned4(xs) || !aligned4(ws)) return FP8Q_ERR_ALIGN;
  const GemmArgs a = swiglu_args(xq, xs, wq, ws, M, N, K, h, ld_h, gu, ld_gu, q, ld_q, scale, ld_s);
  if (fp8q::swiglu_few(M, N, K)) {
    const int64_t need = fp8q_gemm_swiglu_workspace(M, N, K, q != nullptr);
    if (need > 0) {
      if (!workspace) return FP8Q_ERR_NULL;
      if (!aligned16(workspace)) return FP8Q_ERR_ALIGN;
      if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
    }
    return launched(fp8q::launch_swiglu_few(a, q ? static_cast<float*>(workspace) : nullptr, stream));
  }
  return launched(fp8q::launch_gemm(a, stream));
}

fp8q_status fp8q_grouped_gemm_swiglu(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                     const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K, void* h,
                                     int64_t ld_h, void* gu, int64_t ld_gu, uint8_t* q, int64_t ld_q, float* scale,
                                     int64_t ld_s, hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (const fp8q_status c = check_gated(M_total, N, K, cdiv(M_total, 256) + E); c != FP8Q_OK || M_total == 0 || N == 0)
    return c;
  if (!xq || !xs || !wq || !ws || !offsets) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_swiglu_out(h, ld_h, gu, ld_gu, q, ld_q, scale, ld_s, N); c != FP8Q_OK) return c;
  if (!aligned16(xq) || !aligned16(wq) || !aligned4(xs) || !aligned4(ws) || !aligned4(offsets)) return FP8Q_ERR_ALIGN;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  GemmArgs a = swiglu_args(xq, xs, wq, ws, M_total, N, K, h, ld_h, gu, ld_gu, q, ld_q, scale, ld_s);
  a.offsets = offsets; a.E = E; a.b_estride = 2 * N * K; a.sb_estride = (2 * N / 128) * (K / 128);
  return launched(fp8q::launch_gemm(a, stream));
}

fp8q_status fp8q_gemm_dgrad_swiglu(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                   int64_t M, int64_t N, int64_t K, const void* gu, int64_t ld_gu, void* dgu,
                                   int64_t ld_dgu, void* h, int64_t ld_h, hipStream_t stream) {
  if (const fp8q_status c = check_gated(M, K, N, cdiv(M, 256)); c != FP8Q_OK || M == 0 || K == 0) return c;
  if (!dyq || !dys || !wq_t || !ws) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_dswiglu(gu, ld_gu, dgu, ld_dgu, h, ld_h, K); c != FP8Q_OK) return c;
  if (!aligned16(dyq) || !aligned16(wq_t) || !aligned4(dys) || !aligned4(ws)) return FP8Q_ERR_ALIGN;
  GemmArgs a{};  // the product of fp8q_gemm_dgrad
  a.A = dyq; a.B = wq_t; a.sa = dys; a.sb = ws; a.C = dgu;
  a.lda = N; a.ldb = N; a.ld_sa = N / 128; a.sb_rs = 1; a.sb_cs = K / 128; a.ldc = ld_dgu;
  a.M = M; a.N = K; a.K = N;
  a.sb_mode = fp8q::kSbBlock; a.gated = fp8q::kDSwiglu;
  a.gu = static_cast<uint16_t*>(const_cast<void*>(gu)); a.ld_gu = ld_gu;
  a.h = static_cast<uint16_t*>(h); a.ld_h = ld_h;
  return launched(fp8q::launch_gemm(a, stream));
}

fp8q_status fp8q_grouped_gemm_dgrad_swiglu(const uint8_t* dyq, const float* dys, const uint8_t* wq_t, const float* ws,
                                           const int32_t* offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                           const void* gu, int64_t ld_gu, void* dgu, int64_t ld_dgu, void* h,
                                           int64_t ld_h, hipStream_t stream) {
  if (E < 1 || E > 65536) return FP8Q_ERR_SHAPE;
  if (N > 0 && E * N > INT32_MAX / 256) return FP8Q_ERR_SHAPE;  // as fp8q_grouped_gemm_dgrad
  if (const fp8q_status c = check_gated(M_total, K, N, cdiv(M_total, 256) + E); c != FP8Q_OK || M_total == 0 || K == 0)
    return c;
  if (!dyq || !dys || !wq_t || !ws || !offsets) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_dswiglu(gu, ld_gu, dgu, ld_dgu, h, ld_h, K); c != FP8Q_OK) return c;
  if (!aligned16(dyq) || !aligned16(wq_t) || !aligned4(dys) || !aligned4(ws) || !aligned4(offsets))
    return FP8Q_ERR_ALIGN;
  if (const fp8q_status d = debug_check_offsets(offsets, E, M_total, stream); d != FP8Q_OK) return d;
  GemmArgs a{};  // the product of fp8q_grouped_gemm_dgrad
  a.A = dyq; a.B = wq_t; a.sa = dys; a.sb = ws; a.C = dgu;
  a.lda = N; a.ldb = E * N; a.ld_sa = N / 128; a.sb_rs = 1; a.sb_cs = K / 128; a.ldc = ld_dgu;
  a.M = M_total; a.N = K; a.K = N;
  a.sb_mode = fp8q::kSbBlock; a.gated = fp8q::kDSwiglu;
  a.offsets = offsets; a.E = E; a.b_estride = N; a.sb_estride = (N / 128) * (K / 128);
  a.gu = static_cast<uint16_t*>(const_cast<void*>(gu)); a.ld_gu = ld_gu;
  a.h = static_cast<uint16_t*>(h); a.ld_h = ld_h;
  return launched(fp8q::launch_gemm(a, stream));
}

}  // extern "C"

// --------------------------------------------------------------- RMS norm
namespace {

fp8q_status check_norm(fp8q_dtype t, int64_t rows, int64_t cols) {
  if (!valid_dtype(t)) return FP8Q_ERR_DTYPE;
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > fp8q::kMaxNormCols) return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

// The output rows and / or codes of the norm's entry points.
fp8q_status check_norm_out(const void* out, fp8q_dtype t, int64_t ld, const uint8_t* q, int64_t ld_q, const float* s,
                           int64_t ld_s, int64_t cols) {
  if (!out && !q) return FP8Q_ERR_NULL;
  if (out)
    if (const fp8q_status c = check_rows(out, t, ld, cols); c != FP8Q_OK) return c;
  return q || s ? check_codes(q, ld_q, s, ld_s, cols) : FP8Q_OK;
}

}  // namespace

extern "C" {

fp8q_status fp8q_rms_norm(const void* x, fp8q_dtype t, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                          int64_t ld_r, const float* weight, float eps, void* y, int64_t ld_y, uint8_t* q, int64_t ld_q,
                          float* scale, int64_t ld_s, void* sum, int64_t ld_sum, float* rstd, hipStream_t stream) {
  if (const fp8q_status c = check_norm(t, rows, cols); c != FP8Q_OK) return c;
  if (!(eps >= 0.f) || eps - eps != 0.f) return FP8Q_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP8Q_OK;
  if (const fp8q_status c = check_rows(x, t, ld_x, cols); c != FP8Q_OK) return c;
  if (residual) {
    if (const fp8q_status c = check_rows(residual, t, ld_r, cols); c != FP8Q_OK) return c;
    if (const fp8q_status c = check_rows(sum, t, ld_sum, cols); c != FP8Q_OK) return c;
  }
  if (!weight || !rstd) return FP8Q_ERR_NULL;
  if (const fp8q_status c = check_norm_out(y, t, ld_y, q, ld_q, scale, ld_s, cols); c != FP8Q_OK) return c;
  if (!aligned4(weight) || !aligned4(rstd)) return FP8Q_ERR_ALIGN;
  const fp8q::NormRows a{t == FP8Q_BF16, rows, cols, weight, y, ld_y, q, ld_q, scale, ld_s};
  return launched(fp8q::launch_rms_norm(a, x, ld_x, residual, ld_r, eps, sum, ld_sum, rstd, stream));
}

int64_t fp8q_rms_norm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > fp8q::kMaxNormCols) return -1;
  return rows == 0 || cols == 0 ? 0 : fp8q::rms_norm_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

fp8q_status fp8q_rms_norm_bwd(const void* dy, const void* x, fp8q_dtype t, int64_t rows, int64_t cols, int64_t ld_dy,
                              int64_t ld_x, const float* weight, const float* rstd, const void* dsum, int64_t ld_dsum,
                              void* dx, int64_t ld_dx, uint8_t* q, int64_t ld_q, float* scale, int64_t ld_s,
                              float* dweight, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (const fp8q_status c = check_norm(t, rows, cols); c != FP8Q_OK || cols == 0) return c;
  if (!dweight) return FP8Q_ERR_NULL;
  if (!aligned4(dweight)) return FP8Q_ERR_ALIGN;
  if (rows > 0) {
    if (const fp8q_status c = check_rows(dy, t, ld_dy, cols); c != FP8Q_OK) return c;
    if (const fp8q_status c = check_rows(x, t, ld_x, cols); c != FP8Q_OK) return c;
    if (dsum)
      if (const fp8q_status c = check_rows(dsum, t, ld_dsum, cols); c != FP8Q_OK) return c;
    if (!weight || !rstd || !workspace) return FP8Q_ERR_NULL;
    if (const fp8q_status c = check_norm_out(dx, t, ld_dx, q, ld_q, scale, ld_s, cols); c != FP8Q_OK) return c;
    if (!aligned4(weight) || !aligned4(rstd) || !aligned4(workspace)) return FP8Q_ERR_ALIGN;
    if (workspace_bytes < fp8q_rms_norm_bwd_workspace(rows, cols)) return FP8Q_ERR_SHAPE;
  }
  const fp8q::NormRows a{t == FP8Q_BF16, rows, cols, weight, dx, ld_dx, q, ld_q, scale, ld_s};
  return launched(fp8q::launch_rms_norm_bwd(a, dy, ld_dy, x, ld_x, rstd, dsum, ld_dsum, static_cast<float*>(workspace),
                                            dweight, stream));
}

}  // extern "C"

// ------------------------------------------------------------------ AdamW
namespace {

// Whether two tensors of one list share memory (a tensor given twice); list gives
// the first byte of tensor i and its bytes.
template <class F>
bool list_overlaps(int64_t n, F list) {
  // tensors that lie in the order of the list, or in the other one, take one pass
  bool rising = true, falling = true;
  uintptr_t begin = UINTPTR_MAX, end = 0;
  for (int64_t i = 0; i < n; ++i) {
    const auto [at, bytes] = list(i);
    if (at == 0 || bytes == 0) continue;
    rising = rising && at >= end;
    falling = falling && at + bytes <= begin;
    begin = at;
    end = at + bytes;
  }
  if (rising || falling) return false;
  std::vector<std::pair<uintptr_t, uintptr_t>> all;
  all.reserve((size_t)n);
  for (int64_t i = 0; i < n; ++i) {
    const auto [at, bytes] = list(i);
    if (at != 0 && bytes != 0) all.emplace_back(at, bytes);
  }
  std::sort(all.begin(), all.end());
  for (size_t i = 1; i < all.size(); ++i)
    if (all[i].first < all[i - 1].first + all[i - 1].second) return true;
  return false;
}

// Whether a list of what the step writes holds memory twice.
bool adamw_overlaps(const fp8q_adamw_tensor* t, int64_t n, int bits) {
  const int64_t state = bits == 8 ? 1 : 4;
  auto over = [&](auto member, auto bytes) {
    return list_overlaps(n, [&](int64_t i) {
      return std::pair<uintptr_t, uintptr_t>(reinterpret_cast<uintptr_t>(t[i].*member), (uintptr_t)bytes(t[i].len));
    });
  };
  if (over(&fp8q_adamw_tensor::p, [](int64_t len) { return 4 * len; }) ||
      over(&fp8q_adamw_tensor::m, [&](int64_t len) { return state * len; }) ||
      over(&fp8q_adamw_tensor::v, [&](int64_t len) { return state * len; }) ||
      over(&fp8q_adamw_tensor::copy, [](int64_t len) { return 2 * len; }))
    return true;
  auto scales = [](int64_t len) { return 4 * cdiv(len, 128); };
  return bits == 8 && (over(&fp8q_adamw_tensor::m_scale, scales) || over(&fp8q_adamw_tensor::v_scale, scales));
}

}  // namespace

extern "C" {

fp8q_status fp8q_adamw(const fp8q_adamw_tensor* tensors, int64_t n, fp8q_dtype gt, int bits, double lr, double beta1,
                       double beta2, double eps, double weight_decay, int64_t step, uint64_t seed, const float* norm,
                       double max_norm, hipStream_t stream) {
  if (!valid_dtype(gt)) return FP8Q_ERR_DTYPE;
  if (n < 0 || n > kMaxDim || (bits != 8 && bits != 32) || step < 1) return FP8Q_ERR_SHAPE;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !(max_norm >= 0.0) ||
      lr - lr != 0.0 || eps - eps != 0.0 || weight_decay - weight_decay != 0.0)
    return FP8Q_ERR_SHAPE;
  if (n == 0) return FP8Q_OK;
  if (!tensors) return FP8Q_ERR_NULL;
  if (!aligned4(norm)) return FP8Q_ERR_ALIGN;
  for (int64_t i = 0; i < n; ++i) {
    const fp8q_adamw_tensor& t = tensors[i];
    if (t.len < 0 || t.len > fp8q::kMaxAdamChunks * fp8q::kAdamChunk) return FP8Q_ERR_SHAPE;
    if (t.len == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (bits == 8 && (!t.m_scale || !t.v_scale))) return FP8Q_ERR_NULL;
    if (!aligned4(t.p) || !aligned_to(t.g, esize(gt)) || !aligned_to(t.copy, 2)) return FP8Q_ERR_ALIGN;
    if (bits == 32 ? !aligned4(t.m) || !aligned4(t.v) : !aligned4(t.m_scale) || !aligned4(t.v_scale))
      return FP8Q_ERR_ALIGN;
  }
  try {
    if (adamw_overlaps(tensors, n, bits)) return FP8Q_ERR_SHAPE;
  } catch (const std::bad_alloc&) {  // no memory for the check
    return FP8Q_ERR_LAUNCH;
  }
  fp8q::AdamStep a;
  a.beta1 = (float)beta1; a.rest1 = (float)(1.0 - beta1);
  a.beta2 = (float)beta2; a.rest2 = (float)(1.0 - beta2);
  a.keep = (float)(1.0 - lr * weight_decay);
  a.step = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  a.root = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  a.eps = (float)eps;
  if (!std::isfinite(a.keep) || !std::isfinite(a.step) || !std::isfinite(a.root) || !std::isfinite(a.eps))
    return FP8Q_ERR_SHAPE;  // numbers that FP32 does not hold
  a.norm = norm;
  a.max_norm = max_norm;
  a.seed_lo = (uint32_t)seed;
  a.seed_hi = (uint32_t)(seed >> 32);
  fp8q::AdamBatch b;
  for (int64_t i = 0; i < n;) {
    b.n = 0;
    b.cum[0] = 0;
    a.place = (uint32_t)i;
    for (; i < n && b.n < fp8q::kMaxAdamTensors; ++i) {
      const fp8q_adamw_tensor& t = tensors[i];
      const int64_t c = cdiv(t.len, fp8q::kAdamChunk);
      if (b.cum[b.n] + c > fp8q::kMaxAdamChunks) break;
      const int k = b.n++;
      b.p[k] = t.p; b.g[k] = t.g; b.m[k] = t.m; b.v[k] = t.v;
      b.m_scale[k] = t.m_scale; b.v_scale[k] = t.v_scale; b.copy[k] = t.copy;
      b.last[k] = (uint16_t)(t.len - (c - 1) * fp8q::kAdamChunk);
      b.cum[k + 1] = b.cum[k] + (int)c;
    }
    if (b.cum[b.n] > 0 && fp8q::launch_adamw(b, a, gt == FP8Q_BF16, bits == 8, stream) != hipSuccess) return FP8Q_ERR_LAUNCH;
  }
  return FP8Q_OK;
}

}  // extern "C"
