// Rows of an MoE layer between token order and expert order (gfx950).
//
// Pair (t, j) is token t's j-th choice; dst[t*k + j] = r >= 0 says that its
// row in expert order is r, dst = -1 - r that the pair is dropped and row r is
// only padding.
//   dispatch      rows[r] = x[t], zeros for a dropped pair; codes of the same
//   dispatch bwd  dx[t] = sum_j drows[dst[t, j]]
//   combine       y[t] = sum_j w[t, j] yp[dst[t, j]]
//   combine bwd   rows[r] = w[t, j] dy[t], dw[t, j] = dy[t] . yp[dst[t, j]]
// Sums run over j in order in FP32 and are rounded once; a dropped pair's row
// is never used in a sum.  All are HBM-bound.  An entry of dst outside the
// k * T rows is skipped (reads and writes stay in bounds).

#include "launch.h"
#include "row_io.h"

#include <type_traits>

namespace fp8q {

namespace {

constexpr int kJ = 8;  // choices handled together: 8 row loads in flight per lane

__device__ __forceinline__ bool row_ok(int r, int m) { return (uint32_t)r < (uint32_t)m; }

// ---------------------------------------------------------------------------
// Dispatch: 16 lanes own one 128-column group of one token, 8 columns per
// lane, so the group's max-abs is one DPP row reduction (as k_quant_act) and
// a token is read and quantized once however many rows it goes to.
template <class Row, bool ROWS, bool CODES>
__global__ __launch_bounds__(256) void k_dispatch(const typename Row::elem* __restrict__ x, int64_t ld_x,
                                                  const int* __restrict__ dst, int k, int m,
                                                  typename Row::elem* __restrict__ rows, int64_t ld_r,
                                                  uint8_t* __restrict__ q, int64_t ld_q, float* __restrict__ s,
                                                  int64_t ld_s, int cols, int ngr, int total) {
  const int g = (int)((blockIdx.x * 256u + threadIdx.x) >> 4);
  const int lig = threadIdx.x & 15;
  if (g >= total) return;
  const int t = g / ngr, c = g - t * ngr;
  const int c0 = c * 128 + lig * 8;
  float v[8];
  load_cols<Row>(x + (int64_t)t * ld_x, c0, cols, v);
  uint32_t w0 = 0, w1 = 0;
  float sc = 0.f;
  if (CODES) {
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = max(a, abs_bits(v[e]));
    a = row16_max_u32(a);
    float inv;
    group_scale(__uint_as_float(a), sc, inv);
    w0 = pack4_e4m3_grp(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    w1 = pack4_e4m3_grp(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  }
  const int* d = dst + (int64_t)t * k;
  for (int j = 0; j < k; ++j) {
    const int dj = d[j];
    const bool kept = dj >= 0;
    const int r = kept ? dj : -1 - dj;
    if (!row_ok(r, m)) continue;
    if (ROWS) {
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = kept ? v[e] : 0.f;
      store_cols<Row>(rows + (int64_t)r * ld_r, c0, cols, z);
    }
    if (CODES) {
      store_codes(q + (int64_t)r * ld_q, c0, cols, kept ? w0 : 0u, kept ? w1 : 0u);
      if (lig == 0) s[(int64_t)r * ld_s + c] = kept ? sc : kAmaxFloor / kFp8Max;
    }
  }
}

// ---------------------------------------------------------------------------
// Weighted (W) or plain sum of a token's rows: one lane per 8 columns.
template <class Row, bool W>
__global__ __launch_bounds__(256) void k_gather(const typename Row::elem* __restrict__ rows, int64_t ld_r,
                                                const int* __restrict__ dst, const float* __restrict__ w, int k,
                                                int m, typename Row::elem* __restrict__ y, int64_t ld_y, int cols,
                                                int nch, int total) {
  const int i = (int)(blockIdx.x * 256u + threadIdx.x);
  if (i >= total) return;
  const int t = i / nch, c0 = (i - t * nch) * 8;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  const int64_t p0 = (int64_t)t * k;
  for (int j = 0; j < k; ++j) {
    const int r = dst[p0 + j];
    if (!row_ok(r, m)) continue;
    const float wj = W ? w[p0 + j] : 1.f;
    float v[8];
    load_cols<Row>(rows + (int64_t)r * ld_r, c0, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = W ? __builtin_fmaf(wj, v[e], acc[e]) : acc[e] + v[e];
  }
  store_cols<Row>(y + (int64_t)t * ld_y, c0, cols, acc);
}

// ---------------------------------------------------------------------------
// Combine backward: one block per token, so that a token's dw is summed
// inside one block (no atomics; the order is fixed).
template <class Row, bool ROWS, bool CODES>
__global__ __launch_bounds__(256) void k_combine_bwd(const typename Row::elem* __restrict__ dy, int64_t ld_dy,
                                                     const typename Row::elem* __restrict__ yp, int64_t ld_yp,
                                                     const int* __restrict__ dst, const float* __restrict__ w, int k,
                                                     int m, typename Row::elem* __restrict__ rows, int64_t ld_r,
                                                     uint8_t* __restrict__ q, int64_t ld_q, float* __restrict__ s,
                                                     int64_t ld_s, float* __restrict__ dw, int cols, int ngr) {
  __shared__ float red[4][kJ];
  const int t = (int)blockIdx.x, tid = threadIdx.x, lig = tid & 15;
  const int64_t p0 = (int64_t)t * k;
  for (int j0 = 0; j0 < k; j0 += kJ) {
    const int nj = min(kJ, k - j0);
    float acc[kJ];
#pragma unroll
    for (int u = 0; u < kJ; ++u) acc[u] = 0.f;
    for (int c = tid >> 4; c < ngr; c += 16) {
      const int c0 = c * 128 + lig * 8;
      float g[8];
      load_cols<Row>(dy + (int64_t)t * ld_dy, c0, cols, g);
#pragma unroll
      for (int u = 0; u < kJ; ++u) {
        if (u >= nj) break;
        const int d = dst[p0 + j0 + u];
        const bool kept = d >= 0;
        const int r = kept ? d : -1 - d;
        if (!row_ok(r, m)) continue;
        float v[8];
        if (kept) {
          load_cols<Row>(yp + (int64_t)r * ld_yp, c0, cols, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[u] = __builtin_fmaf(g[e], v[e], acc[u]);
        }
        const float wj = w[p0 + j0 + u];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = kept ? g[e] * wj : 0.f;
        const typename Row::Raw raw = Row::pack(v);
        if (ROWS) store_cols<Row>(rows + (int64_t)r * ld_r, c0, cols, v);
        if (CODES) {
          Row::unpack(raw, v);  // the codes are those of the rounded row
          uint32_t a = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) a = max(a, abs_bits(v[e]));
          a = row16_max_u32(a);
          float sc, inv;
          group_scale(__uint_as_float(a), sc, inv);
          store_codes(q + (int64_t)r * ld_q, c0, cols,
                      pack4_e4m3_grp(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      pack4_e4m3_grp(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
          if (lig == 0) s[(int64_t)r * ld_s + c] = sc;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kJ; ++u)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) acc[u] += __shfl_xor(acc[u], o);
    if ((tid & 63) == 0)
#pragma unroll
      for (int u = 0; u < kJ; ++u) red[tid >> 6][u] = acc[u];
    __syncthreads();
    if (tid < nj) dw[p0 + j0 + tid] = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_moe_dispatch(const MoeRows& a, const void* x, int64_t ld_x, hipStream_t st) {
  const int ngr = (int)((a.cols + 127) / 128);
  const int total = (int)(a.tokens * ngr);
  const dim3 grid((uint32_t)(((int64_t)total + 15) / 16));
  auto go = [&](auto row, auto fr, auto fc) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    hipLaunchKernelGGL((k_dispatch<Row, decltype(fr)::value, decltype(fc)::value>), grid, dim3(256), 0, st,
                       (const E*)x, ld_x, a.dst, (int)a.k, (int)(a.tokens * a.k), (E*)a.rows, a.ld_rows, a.q, a.ld_q,
                       a.s, a.ld_s, (int)a.cols, ngr, total);
  };
  using T = std::true_type;
  using F = std::false_type;
  auto pick = [&](auto row) {
    if (a.rows && a.q) go(row, T{}, T{});
    else if (a.q) go(row, F{}, T{});
    else go(row, T{}, F{});
  };
  if (a.bf16) pick(RowBF16{}); else pick(RowF32{});
  return hipGetLastError();
}

hipError_t launch_moe_gather(const MoeRows& a, const float* w, void* y, int64_t ld_y, hipStream_t st) {
  const int nch = (int)((a.cols + 7) / 8);
  const int total = (int)(a.tokens * nch);
  const dim3 grid((uint32_t)(((int64_t)total + 255) / 256));
  auto go = [&](auto row, auto fw) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    hipLaunchKernelGGL((k_gather<Row, decltype(fw)::value>), grid, dim3(256), 0, st, (const E*)a.rows, a.ld_rows,
                       a.dst, w, (int)a.k, (int)(a.tokens * a.k), (E*)y, ld_y, (int)a.cols, nch, total);
  };
  auto pick = [&](auto row) {
    if (w) go(row, std::true_type{}); else go(row, std::false_type{});
  };
  if (a.bf16) pick(RowBF16{}); else pick(RowF32{});
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const MoeRows& a, const void* dy, int64_t ld_dy, const void* yp, int64_t ld_yp,
                                  const float* w, float* dw, hipStream_t st) {
  const int ngr = (int)((a.cols + 127) / 128);
  const dim3 grid((uint32_t)a.tokens);
  auto go = [&](auto row, auto fr, auto fc) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    hipLaunchKernelGGL((k_combine_bwd<Row, decltype(fr)::value, decltype(fc)::value>), grid, dim3(256), 0, st,
                       (const E*)dy, ld_dy, (const E*)yp, ld_yp, a.dst, w, (int)a.k, (int)(a.tokens * a.k),
                       (E*)a.rows, a.ld_rows, a.q, a.ld_q, a.s, a.ld_s, dw, (int)a.cols, ngr);
  };
  using T = std::true_type;
  using F = std::false_type;
  auto pick = [&](auto row) {
    if (a.rows && a.q) go(row, T{}, T{});
    else if (a.q) go(row, F{}, T{});
    else go(row, T{}, F{});
  };
  if (a.bf16) pick(RowBF16{}); else pick(RowF32{});
  return hipGetLastError();
}

}  // namespace fp8q
