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

constexpr int kJ = 8;              // choices handled together: 8 row loads or stores in flight per lane
constexpr int kPair = 2;           // and in the combine gradient
constexpr int kWideThreads = 512;  // most threads of a block that works on one token

__device__ __forceinline__ bool row_ok(int r, int m) { return (uint32_t)r < (uint32_t)m; }
// The row of a map entry, kept or dropped.
__device__ __forceinline__ int row_of(int d) { return d >= 0 ? d : -1 - d; }

template <int J, int I = 0, class F>
__device__ __forceinline__ void each_choice(F f) {
  f(std::integral_constant<int, I>{});
  if constexpr (I + 1 < J) each_choice<J, I + 1>(f);
}

// 16 lanes handle a 128-column group of a row, 8 columns each.  WIDE rows (a
// wave's 512 columns or more) give a block to one token, or to a slice of its
// columns, so the map's entries are uniform: they come by scalar loads and a
// dropped pair is a uniform branch.  Narrow rows put several tokens into a
// wave.  piece counts a token's lanes.
template <bool WIDE>
__device__ __forceinline__ void place(int per_token, int& t, int& piece) {
  if (WIDE) {
    t = (int)(blockIdx.x / (uint32_t)per_token);
    piece = ((int)blockIdx.x - t * per_token) * (int)blockDim.x + (int)threadIdx.x;
  } else {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    t = (int)(i / (uint32_t)per_token);
    piece = (int)(i - (uint32_t)t * (uint32_t)per_token);
  }
}

// The end of the last whole 64-byte segment of a row (of a code row where only
// codes leave).  Kernels that store past the caches leave the waves that hold
// the columns after it to plain stores.
template <class Row, bool ROWS>
__device__ __forceinline__ int whole_end(int cols) {
  return cols & ~(ROWS ? 64 / (int)sizeof(typename Row::elem) - 1 : 63);
}

// First column of a piece.
template <class Row>
__device__ __forceinline__ int piece_col(int piece) { return (piece >> 4) * 128 + (piece & 15) * Row::kLen; }

// ---------------------------------------------------------------------------
// Dispatch: 16 lanes own one 128-column group of one token, so the group's
// max-abs is one DPP row reduction (as k_quant_act) and a token is read and
// quantized once however many rows it goes to.
template <class Row, bool ROWS, bool CODES, bool WIDE, int PAST>
__global__ __launch_bounds__(WIDE ? kWideThreads : 256) void k_dispatch(
    const typename Row::elem* __restrict__ x, int64_t ld_x, const int* __restrict__ dst, int tokens, int k, int m,
    typename Row::elem* __restrict__ rows, int64_t ld_r, uint8_t* __restrict__ q, int64_t ld_q,
    float* __restrict__ s, int64_t ld_s, int cols, int per_token) {
  int t, piece;
  place<WIDE>(per_token, t, piece);
  const int c = piece >> 4, c0 = piece_col<Row>(piece);
  if (t >= tokens || c * 128 >= cols) return;
  const int* d = dst + (int64_t)t * k;
  auto body = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    const typename Row::Raw raw = load_piece<Row, kWhole, !WIDE, 0>(x + (int64_t)t * ld_x, c0, cols);
    uint32_t w0 = 0, w1 = 0;
    float sc = 0.f;
    if (CODES) {
      // a run outside holds values of its own group's last columns: they do not
      // change the group's max-abs
      float v[8], inv;
      Row::unpack(raw, v);
      group_scale(__uint_as_float(row16_max_u32(Row::max_bits(raw))), sc, inv);
      w0 = pack4_e4m3_grp(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      w1 = pack4_e4m3_grp(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    }
    for (int j0 = 0; j0 < k; j0 += kJ) {
      int dj[kJ];
#pragma unroll
      for (int u = 0; u < kJ; ++u) dj[u] = d[min(j0 + u, k - 1)];
#pragma unroll
      for (int u = 0; u < kJ; ++u) {
        if (j0 + u >= k) break;
        const bool kept = dj[u] >= 0;
        const int r = row_of(dj[u]);
        if (!row_ok(r, m)) continue;
        if (ROWS) {
          typename Row::Raw z{};
          if (kept) z = raw;
          store_piece<Row, kWhole, PAST & 1>(rows + (int64_t)r * ld_r, c0, cols, z);
        }
        if (CODES) {
          store_codes<Row, kWhole, PAST / 2>(q + (int64_t)r * ld_q, c0, cols, kept ? w0 : 0u, kept ? w1 : 0u);
          if ((piece & 15) == 0) s[(int64_t)r * ld_s + c] = kept ? sc : kAmaxFloor / kFp8Max;
        }
      }
    }
  };
  if (no_cut<Row>(c0, whole_end<Row, ROWS>(cols), cols)) body(std::true_type{}); else body(std::false_type{});
}

// ---------------------------------------------------------------------------
// Weighted (W) or plain sum of a token's rows; up to kJ rows in flight.
template <class Row, bool W, bool WIDE, int NT>
__global__ __launch_bounds__(WIDE ? kWideThreads : 256) void k_gather(
    const typename Row::elem* __restrict__ rows, int64_t ld_r, const int* __restrict__ dst,
    const float* __restrict__ w, int tokens, int k, int m, typename Row::elem* __restrict__ y, int64_t ld_y, int cols,
    int per_token) {
  int t, piece;
  place<WIDE>(per_token, t, piece);
  const int c0 = piece_col<Row>(piece);
  if (t >= tokens || (piece >> 4) * 128 >= cols) return;
  const int64_t p0 = (int64_t)t * k;
  auto body = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kJ) {
      int r[kJ];
      float wj[kJ];
      typename Row::Raw raw[kJ];
#pragma unroll
      for (int u = 0; u < kJ; ++u) {
        const int64_t at = p0 + min(j0 + u, k - 1);
        r[u] = j0 + u < k ? dst[at] : -1;
        wj[u] = W ? w[at] : 1.f;
      }
#pragma unroll
      for (int u = 0; u < kJ; ++u)
        if (row_ok(r[u], m)) raw[u] = load_piece<Row, kWhole, !WIDE, NT>(rows + (int64_t)r[u] * ld_r, c0, cols);
#pragma unroll
      for (int u = 0; u < kJ; ++u)
        if (row_ok(r[u], m)) {
          float v[8];
          Row::unpack(raw[u], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = W ? __builtin_fmaf(wj[u], v[e], acc[e]) : acc[e] + v[e];
        }
    }
    store_piece<Row, kWhole, 0>(y + (int64_t)t * ld_y, c0, cols, Row::pack(acc));
  };
  if (no_cut<Row>(c0, cols, cols)) body(std::true_type{}); else body(std::false_type{});
}

// ---------------------------------------------------------------------------
// Combine backward: two choices of one token to a block (WIDE) or a 16-lane
// group, whose lanes' products are summed there, without atomics: the order is
// fixed.  dy is read again by the token's other blocks, from the caches; all
// choices in one block need three times the registers and instructions (32768
// rows of 7168 226 us so, 228 with four and 245 with eight; 4905 FP32 rows of
// 2411 with codes 17 us, with eight 29).
template <class Row, bool ROWS, bool CODES, bool WIDE, int PAST, int NTI>
__global__ __launch_bounds__(WIDE ? kWideThreads : 256) void k_combine_bwd(
    const typename Row::elem* __restrict__ dy, int64_t ld_dy, const typename Row::elem* __restrict__ yp,
    int64_t ld_yp, const int* __restrict__ dst, const float* __restrict__ w, int tokens, int k, int m,
    typename Row::elem* __restrict__ rows, int64_t ld_r, uint8_t* __restrict__ q, int64_t ld_q,
    float* __restrict__ s, int64_t ld_s, float* __restrict__ dw, int cols, int parts) {
  constexpr int J = kPair;
  __shared__ float red[kWideThreads / 64][J];
  uint32_t item = WIDE ? blockIdx.x : blockIdx.x * 16 + (threadIdx.x >> 4);
  if (WIDE) {
    // A token's blocks are 8 apart, on one XCD, whose L2 then holds its dy:
    // the last tokens, fewer than 8, keep theirs together.
    const uint32_t eight = 8u * (uint32_t)parts, group = item / eight, at = item - group * eight;
    if ((int)(group * 8) + 8 <= tokens) item = (group * 8 + (at & 7)) * (uint32_t)parts + (at >> 3);
  }
  const int t = (int)(item / (uint32_t)parts), j0 = (int)(item - (uint32_t)t * (uint32_t)parts) * J;
  if (!WIDE && t >= tokens) return;
  const int piece0 = WIDE ? (int)threadIdx.x : (int)threadIdx.x & 15, step = WIDE ? (int)blockDim.x : 16;
  const int64_t p0 = (int64_t)t * k;
  int d[J], r[J];  // a choice's map entry and row; m: no choice
  float wj[J], acc[J];
#pragma unroll
  for (int u = 0; u < J; ++u) {
    const int64_t at = p0 + min(j0 + u, k - 1);
    d[u] = dst[at];
    r[u] = j0 + u < k ? row_of(d[u]) : m;
    wj[u] = w[at];
    acc[u] = 0.f;
  }
  const int mine = j0 + (int)(threadIdx.x & (J - 1));
  const int my_r = CODES && mine < k ? row_of(dst[p0 + mine]) : m;
  auto body = [&](auto whole, int piece) {
    constexpr bool kWhole = decltype(whole)::value;
    const int c = piece >> 4, c0 = piece_col<Row>(piece);
    const typename Row::Raw graw = load_piece<Row, kWhole, !WIDE, 0>(dy + (int64_t)t * ld_dy, c0, cols);
    typename Row::Raw raw[J];
#pragma unroll
    for (int u = 0; u < J; ++u)
      if (d[u] >= 0 && row_ok(r[u], m))
        raw[u] = load_piece<Row, kWhole, !WIDE, NTI>(yp + (int64_t)r[u] * ld_yp, c0, cols);
    bool in[Row::kRuns];
#pragma unroll
    for (int i = 0; i < Row::kRuns; ++i) in[i] = !kWhole || c0 + 64 * i < cols;
    float g[8];
    Row::unpack(graw, g);
    uint32_t am[J];
#pragma unroll
    for (int u = 0; u < J; ++u) {
      am[u] = 0;
      if (!row_ok(r[u], m)) continue;
      float v[8];
      if (d[u] >= 0) {
        Row::unpack(raw[u], v);
#pragma unroll
        for (int i = 0; i < Row::kRuns; ++i) {
          float part = acc[u];
#pragma unroll
          for (int e = i * Row::kLen; e < (i + 1) * Row::kLen; ++e) part = __builtin_fmaf(g[e], v[e], part);
          acc[u] = in[i] ? part : acc[u];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = g[e] * wj[u];
        raw[u] = Row::pack(v);
      } else {
        raw[u] = typename Row::Raw{};
      }
      if (ROWS) store_piece<Row, kWhole, PAST & 1>(rows + (int64_t)r[u] * ld_r, c0, cols, raw[u]);
      if (CODES) am[u] = row16_max_u32(Row::max_bits(raw[u]));  // the codes are those of the rounded row
    }
    if (CODES) {
      // lane u of the group forms the scale of row u
      const int lig = piece & 15;
      uint32_t a = am[0];
#pragma unroll
      for (int u = 1; u < J; ++u) a = (lig & (J - 1)) == u ? +am[u] : a;
      float sc, inv;
      group_scale(__uint_as_float(a), sc, inv);
      if (lig < J && row_ok(my_r, m)) s[(int64_t)my_r * ld_s + c] = sc;
      each_choice<J>([&](auto u) {
        if (!row_ok(r[u.value], m)) return;
        const float iu = row_bcast<u.value>(inv);
        float v[8];
        Row::unpack(raw[u.value], v);
        store_codes<Row, kWhole, PAST / 2>(q + (int64_t)r[u.value] * ld_q, c0, cols,
                                     pack4_e4m3_grp(v[0] * iu, v[1] * iu, v[2] * iu, v[3] * iu),
                                     pack4_e4m3_grp(v[4] * iu, v[5] * iu, v[6] * iu, v[7] * iu));
      });
    }
  };
  for (int piece = piece0; (piece >> 4) * 128 < cols; piece += step) {
    if (no_cut<Row>(piece_col<Row>(piece), whole_end<Row, ROWS>(cols), cols)) body(std::true_type{}, piece);
    else body(std::false_type{}, piece);
  }
  const int nj = min(J, k - j0);
#pragma unroll
  for (int u = 0; u < J; ++u) acc[u] = row16_sum(acc[u]);
  if (WIDE) {
    const int lane = threadIdx.x & 63, waves = (int)blockDim.x >> 6;
#pragma unroll
    for (int u = 0; u < J; ++u) {
      acc[u] += __shfl_xor(acc[u], 16);
      acc[u] += __shfl_xor(acc[u], 32);
    }
    if (lane == 0)
#pragma unroll
      for (int u = 0; u < J; ++u) red[threadIdx.x >> 6][u] = acc[u];
    __syncthreads();
    if ((int)threadIdx.x < nj) {
      float sum = 0.f;
      for (int i = 0; i < waves; ++i) sum += red[i][threadIdx.x];
      dw[p0 + j0 + threadIdx.x] = sum;
    }
  } else {
#pragma unroll
    for (int u = 0; u < J; ++u)
      if ((threadIdx.x & 15) == u && u < nj) dw[p0 + j0 + u] = acc[u];
  }
}

// Blocks of wide rows: the row's pieces in as few slices as blocks of
// kWideThreads allow, of equal length up to a wave (7168 columns: two slices of
// 448 threads, where slices of 512 would leave an eighth of the lanes idle).
// The dispatch to 16384 rows of 7168: 69 us so, 73 with blocks of 256; the
// other kernels differ less.
struct Shape {
  bool wide;
  int slices, threads;
  int64_t pieces;  // of 8 columns, to whole 128-column groups
};
Shape shape_of(int64_t cols) {
  Shape h;
  h.wide = cols >= 512;
  h.pieces = (cols + 127) / 128 * 16;
  h.slices = h.wide ? (int)((h.pieces + kWideThreads - 1) / kWideThreads) : 1;
  h.threads = h.wide ? (int)(((h.pieces + h.slices - 1) / h.slices + 63) / 64 * 64) : 256;
  return h;
}

// Which outputs are stored past the caches (1: rows, 2: codes): those whose
// rows start on 64-byte segments, up to the last whole one; codes beside rows
// only where they fill theirs.  The combine gradient of 32768 rows of 7168
// took 246 us so and 271 us through the caches, the dispatch to 16384 rows 69
// and 81.  Cut segments lose by it: 65000 rows of 864 columns with codes 43 us
// with the codes past the caches, 30 with the rows alone; dense rows of 2047
// BF16 columns 30 us past, 21 through.
int past_caches(const MoeRows& a) {
  auto whole = [](const void* p, int64_t row_bytes) {
    return p && reinterpret_cast<uintptr_t>(p) % 64 == 0 && row_bytes % 64 == 0;
  };
  return (whole(a.rows, a.ld_rows * (a.bf16 ? 2 : 4)) ? 1 : 0) |
         (whole(a.q, a.ld_q) && (!a.rows || a.cols % 64 == 0) ? 2 : 0);
}

template <class F>
void with_flag(bool v, F f) {
  if (v) f(std::true_type{}); else f(std::false_type{});
}
template <class F>
void with_row(bool bf16, F f) {
  if (bf16) f(RowBF16{}); else f(RowF32{});
}
// The outputs asked for (rows, codes or both) and which of them past the
// caches; codes alone of both are stored through them with the rows.
template <class F>
void with_outputs(const MoeRows& a, F f) {
  using T = std::true_type;
  using N = std::false_type;
  const int past = past_caches(a);
  auto go = [&](auto rows, auto codes) {
    constexpr int kBoth = (decltype(rows)::value ? 1 : 0) | (decltype(codes)::value ? 2 : 0);
    if ((past & kBoth) == kBoth) f(rows, codes, std::integral_constant<int, kBoth>{});
    else if (kBoth == 3 && past == 1) f(rows, codes, std::integral_constant<int, kBoth & 1>{});
    else f(rows, codes, std::integral_constant<int, 0>{});
  };
  if (a.rows && a.q) go(T{}, T{});
  else if (a.q) go(N{}, T{});
  else go(T{}, N{});
}

// Rows that cannot all stay in the 256 MiB cache in front of the memory are
// read past the caches: combining 32768 rows of 7168 takes 94 us so and 102 us
// through them.  Rows that may still be there lose by it (34 MB of rows, just
// written: 16 us through the caches, 21 us past them).
bool streamed(const MoeRows& a) { return a.tokens * a.k * a.cols * (a.bf16 ? 2 : 4) > ((int64_t)256 << 20); }

}  // namespace

hipError_t launch_moe_dispatch(const MoeRows& a, const void* x, int64_t ld_x, hipStream_t st) {
  const Shape h = shape_of(a.cols);
  const int per_token = h.wide ? h.slices : (int)h.pieces;
  const uint32_t grid = (uint32_t)(h.wide ? a.tokens * h.slices : (a.tokens * h.pieces + 255) / 256);
  with_row(a.bf16, [&](auto row) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    with_outputs(a, [&](auto fr, auto fc, auto past) {
      with_flag(h.wide, [&](auto wide) {
        hipLaunchKernelGGL((k_dispatch<Row, fr.value, fc.value, wide.value, past.value>), dim3(grid),
                           dim3(h.threads), 0, st, (const E*)x, ld_x, a.dst, (int)a.tokens, (int)a.k,
                           (int)(a.tokens * a.k), (E*)a.rows, a.ld_rows, a.q, a.ld_q, a.s, a.ld_s, (int)a.cols,
                           per_token);
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_moe_gather(const MoeRows& a, const float* w, void* y, int64_t ld_y, hipStream_t st) {
  const Shape h = shape_of(a.cols);
  const int per_token = h.wide ? h.slices : (int)h.pieces;
  const uint32_t grid = (uint32_t)(h.wide ? a.tokens * h.slices : (a.tokens * h.pieces + 255) / 256);
  with_row(a.bf16, [&](auto row) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    with_flag(w != nullptr, [&](auto fw) {
      with_flag(h.wide, [&](auto wide) {
        with_flag(streamed(a), [&](auto nt) {
          hipLaunchKernelGGL((k_gather<Row, fw.value, wide.value, nt.value>), dim3(grid), dim3(h.threads), 0, st,
                             (const E*)a.rows, a.ld_rows, a.dst, w, (int)a.tokens, (int)a.k, (int)(a.tokens * a.k),
                             (E*)y, ld_y, (int)a.cols, per_token);
        });
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const MoeRows& a, const void* dy, int64_t ld_dy, const void* yp, int64_t ld_yp,
                                  const float* w, float* dw, hipStream_t st) {
  const Shape h = shape_of(a.cols);
  const int parts = (int)((a.k + kPair - 1) / kPair);
  hipError_t err = hipSuccess;
  with_row(a.bf16, [&](auto row) {
    typedef decltype(row) Row;
    typedef typename Row::elem E;
    with_outputs(a, [&](auto fr, auto fc, auto past) {
      with_flag(h.wide, [&](auto wide) {
        with_flag(streamed(a), [&](auto nti) {
          err = launch_in_parts(a.tokens, parts * (h.wide ? h.threads : 16), [&](int64_t t, int64_t n) {
            const uint32_t grid = (uint32_t)(h.wide ? n * parts : (n * parts + 15) / 16);
            hipLaunchKernelGGL((k_combine_bwd<Row, fr.value, fc.value, wide.value, past.value, nti.value>),
                               dim3(grid), dim3(h.threads), 0, st, (const E*)dy + t * ld_dy, ld_dy, (const E*)yp,
                               ld_yp, a.dst + t * a.k, w + t * a.k, (int)n, (int)a.k, (int)(a.tokens * a.k),
                               (E*)a.rows, a.ld_rows, a.q, a.ld_q, a.s, a.ld_s, dw + t * a.k, (int)a.cols, parts);
          });
        });
      });
    });
  });
  return err;
}

}  // namespace fp8q
