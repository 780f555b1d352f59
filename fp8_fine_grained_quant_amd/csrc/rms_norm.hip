// Root-mean-square norm of rows, with the residual's addition in front of it
// and 1x128 E4M3 codes behind it, and its gradient (gfx950).
//
//   t = x + residual (rounded to the rows' type: the stream as it is held)
//   r = 1 / sqrt(mean(t^2) + eps),  y = t r w
// and, from dy, t and r,
//   a = dy w,  c = mean(a t r),  dt = r (a - t r c) (+ the stream's own gradient)
//   dw = sum over the rows of dy t r
// All arithmetic is FP32; y and dt are rounded once, to the rows' type or (over
// the unrounded values' scales) to codes.
//
// Both are bound by memory, so a row is read once and stays in registers while
// its sum is formed, and (up to 8192 columns) the weights stay in registers from
// row to row: a block's threads own fixed columns, 8 each, and the block takes
// every gridDim.x-th row.  (Two pieces of 8 columns a thread leave half as many
// waves, and of the gradient only one block a compute unit: 58 us against 54 for
// the norm below, 353 against 208 for its gradient.)
// The gradient's dw needs the same: each block sums its rows' part of it in
// registers and writes it once, and a second launch adds the blocks' parts (in
// a fixed order; no atomics).
//
// 4096 BF16 rows of 7168 with residual, rows and codes: 54 us, 4.9 TB/s, where a
// copy of that many bytes has 5.4; gradient of 16384 rows of 7168 with the
// stream's gradient, rows and codes: 193 to 197 us (the profiler has 206 + 5),
// 5.5 TB/s (a copy: 5.0); of 2999 FP32 rows of 1027: 13.2 us (9.4 and 3.8), bound by
// the latency of three rounds of rows; of 32768 BF16 rows of 128 13.4 us, twice the
// bytes' time: two rounds of rows, the block's 64 rows' sums of dw one after the
// other, and the second launch (3).

#include "launch.h"
#include "row_io.h"

#include <type_traits>

namespace fp8q {

namespace {

// 8-column pieces per thread (V): 1 up to 8192 columns, else 2, with which the
// weights do not fit in the registers and come anew for every row.
constexpr int kNormThreads = 1024;

template <class Row>
__device__ __forceinline__ int norm_col(int piece) { return (piece >> 4) * 128 + (piece & 15) * Row::kLen; }

// The pointer, as one that the compiler has not loaded from before: values that
// are read anew for every row are not to be kept in registers.
__device__ __forceinline__ const float* again(const float* p) {
  asm volatile("" : "+s"(p));
  return p;
}

// The weights of a lane's 8 columns, zeros past the row's end.
template <class Row>
__device__ __forceinline__ void load_weights(const float* w, int c0, int cols, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = Row::kRuns == 1 ? c0 + 4 * h : c0 + 64 * h;
    u32x4 u = {0, 0, 0, 0};
    if (c + 4 <= cols) {
      u = ld16u<0>(w + c);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (c + e < cols) u[e] = __float_as_uint(w[c + e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = __uint_as_float(u[e]);
  }
}

// A lane's 8 columns of a row, zeros in every column past the row's end.
template <class Row, bool TINY, int NT>
__device__ __forceinline__ typename Row::Raw load_row_piece(const typename Row::elem* p, int c0, int cols,
                                                            bool whole) {
  typename Row::Raw raw;
  if (!TINY && whole) {
    raw = load_piece<Row, true, false, NT>(p, c0, cols);
#pragma unroll
    for (int r = 0; r < Row::kRuns; ++r)
      if (c0 + 64 * r >= cols) raw.a[r] = u32x4{0, 0, 0, 0};
  } else {
    raw = load_piece<Row, false, TINY, NT>(p, c0, cols);
  }
  return raw;
}
template <class Row, int NT>
__device__ __forceinline__ void store_row_piece(typename Row::elem* p, int c0, int cols, bool whole,
                                                const typename Row::Raw& raw) {
  if (whole) store_piece<Row, true, NT>(p, c0, cols, raw);
  else store_piece<Row, false, 0>(p, c0, cols, raw);
}

// Codes and scale of a lane's 8 FP32 values; 16 lanes hold a group.
template <class Row>
__device__ __forceinline__ void store_quantized(const float (&y)[8], uint8_t* q, float* s, int piece, int c0, int cols,
                                                bool whole) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, abs_bits(y[e]));
  float sc, inv;
  group_scale(__uint_as_float(row16_max_u32(m)), sc, inv);
  const uint32_t w0 = pack4_e4m3_grp(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
  const uint32_t w1 = pack4_e4m3_grp(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
  if (whole) store_codes<Row, true, 0>(q, c0, cols, w0, w1);
  else store_codes<Row, false, 0>(q, c0, cols, w0, w1);
  if ((piece & 15) == 0 && (piece >> 4) * 128 < cols) s[piece >> 4] = sc;
}

// Which rows a thread works on: a block has as many rows at once as its threads
// hold (row_threads each).  NARROW: rows of 16 or 32 threads, several to a wave;
// otherwise a row's threads are whole waves.
template <bool NARROW>
struct NormPlace {
  int rows_at_once, mine, t;  // the block's rows, this thread's one among them, its place there
  __device__ __forceinline__ explicit NormPlace(int row_threads) {
    rows_at_once = (int)blockDim.x / row_threads;
    mine = (int)threadIdx.x / row_threads;
    if (!NARROW) mine = __builtin_amdgcn_readfirstlane(mine);
    t = (int)threadIdx.x - mine * row_threads;
  }
};

// Sum over a row's threads, the same bits in every thread.  Whole waves: `red`
// holds a value of each wave of the block, and the caller alternates between two
// of them, so that one barrier a call is enough.
template <bool NARROW>
__device__ __forceinline__ float norm_row_sum(float v, float* red, int mine, int row_threads) {
  v = row16_sum(v);
  if (NARROW) return row_threads == 16 ? v : v + __shfl_xor(v, 16);
  const int waves = row_threads >> 6, first = mine * waves;
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  // lane l of every 16 holds the row's wave l's value
  const int l = threadIdx.x & 15;
  return row16_sum(l < waves ? red[first + l] : 0.f);
}

// NT: rows come and go past the caches (see past_caches).
template <class Row, int V, bool TINY, int NT, bool NARROW>
__global__ __launch_bounds__(kNormThreads) void k_rms_norm(const NormRows a, const void* x_, int64_t ld_x,
                                                           const void* res_, int64_t ld_res, float eps, void* sum_,
                                                           int64_t ld_sum, float* rstd_out, int row_threads) {
  typedef typename Row::elem elem;
  __shared__ float red[2][16];
  const elem *x = (const elem*)x_, *res = (const elem*)res_;
  elem *y = (elem*)a.out, *sum = (elem*)sum_;
  const int cols = (int)a.cols;
  const NormPlace<NARROW> at(row_threads);
  int piece[V], c0[V];
  bool whole[V];
  float w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    piece[i] = i * row_threads + at.t;
    c0[i] = norm_col<Row>(piece[i]);
    whole[i] = no_cut<Row>(c0[i], cols, cols);
    if (V == 1) load_weights<Row>(a.w, c0[i], cols, w[i]);
  }
  const float inv_cols = 1.f / (float)cols;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * at.rows_at_once; r0 < a.rows;
       r0 += (int64_t)gridDim.x * at.rows_at_once, turn ^= 1) {
    // rows past the last one repeat it and leave nothing
    const bool on = r0 + at.mine < a.rows;
    const int64_t r = on ? r0 + at.mine : a.rows - 1;
    typename Row::Raw raw[V], other[V];
#pragma unroll
    for (int i = 0; i < V; ++i) raw[i] = load_row_piece<Row, TINY, NT>(x + r * ld_x, c0[i], cols, whole[i]);
    if (res)
#pragma unroll
      for (int i = 0; i < V; ++i) other[i] = load_row_piece<Row, TINY, NT>(res + r * ld_res, c0[i], cols, whole[i]);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v[8];
      Row::unpack(raw[i], v);
      if (res) {
        float o[8];
        Row::unpack(other[i], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += o[e];
        raw[i] = Row::pack(v);
        Row::unpack(raw[i], v);
        if (on) store_row_piece<Row, NT>(sum + r * ld_sum, c0[i], cols, whole[i], raw[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
    }
    ss = norm_row_sum<NARROW>(ss, red[turn], at.mine, row_threads);
    if (!on) continue;
    const float rstd = 1.f / sqrtf(__builtin_fmaf(ss, inv_cols, eps));
    if (at.t == 0) rstd_out[r] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v[8];
      Row::unpack(raw[i], v);
      if (V > 1) load_weights<Row>(again(a.w), c0[i], cols, w[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[i][e];
      if (y) store_row_piece<Row, NT>(y + r * a.ld_out, c0[i], cols, whole[i], Row::pack(v));
      if (a.q) store_quantized<Row>(v, a.q + r * a.ld_q, a.s + r * a.ld_s, piece[i], c0[i], cols, whole[i]);
    }
  }
}

// A block's part of dw is written once however many rows the block has.
template <class Row, int V, bool TINY, int NT, bool NARROW>
__global__ __launch_bounds__(kNormThreads) void k_rms_norm_bwd(const NormRows a, const void* dy_, int64_t ld_dy,
                                                                     const void* x_, int64_t ld_x, const float* rstd_in,
                                                                     const void* dsum_, int64_t ld_dsum,
                                                                     float* __restrict__ part, int row_threads) {
  typedef typename Row::elem elem;
  __shared__ float red[2][16];
  __shared__ float held[V == 1 ? 8 : 1][V == 1 ? kNormThreads : 1];  // dw of the block's rows
  const elem *dy = (const elem*)dy_, *x = (const elem*)x_, *dsum = (const elem*)dsum_;
  elem* dx = (elem*)a.out;
  const int cols = (int)a.cols;
  const NormPlace<NARROW> at(row_threads);
  int piece[V], c0[V];
  bool whole[V];
  float w[V][8], dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    piece[i] = i * row_threads + at.t;
    c0[i] = norm_col<Row>(piece[i]);
    whole[i] = no_cut<Row>(c0[i], cols, cols);
    if (V == 1) load_weights<Row>(a.w, c0[i], cols, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  const float inv_cols = 1.f / (float)cols;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * at.rows_at_once; r0 < a.rows;
       r0 += (int64_t)gridDim.x * at.rows_at_once, turn ^= 1) {
    const bool on = r0 + at.mine < a.rows;
    const int64_t r = on ? r0 + at.mine : a.rows - 1;
    typename Row::Raw rx[V], rd[V], ro[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rx[i] = load_row_piece<Row, TINY, NT>(x + r * ld_x, c0[i], cols, whole[i]);
      rd[i] = load_row_piece<Row, TINY, NT>(dy + r * ld_dy, c0[i], cols, whole[i]);
    }
    // (two pieces of FP32 rows leave no registers for the stream's gradient yet)
    constexpr bool kLate = V > 1 && Row::kRuns == 2;
    if (dsum && !kLate)
#pragma unroll
      for (int i = 0; i < V; ++i) ro[i] = load_row_piece<Row, TINY, NT>(dsum + r * ld_dsum, c0[i], cols, whole[i]);
    const float rstd = rstd_in[r];
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float vx[8], vd[8];
      Row::unpack(rx[i], vx);
      Row::unpack(rd[i], vd);
      if (V > 1) load_weights<Row>(again(a.w), c0[i], cols, w[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = vd[e] * (vx[e] * rstd);
        if (on) dw[i][e] += p;
        c = __builtin_fmaf(p, w[i][e], c);
      }
    }
    c = norm_row_sum<NARROW>(c, red[turn], at.mine, row_threads) * inv_cols;
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float vx[8], vd[8], vo[8];
      Row::unpack(rx[i], vx);
      Row::unpack(rd[i], vd);
      if (dsum && kLate) ro[i] = load_row_piece<Row, TINY, NT>(dsum + r * ld_dsum, c0[i], cols, whole[i]);
      if (dsum) Row::unpack(ro[i], vo);
      if (V > 1) load_weights<Row>(again(a.w), c0[i], cols, w[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = __builtin_fmaf(vx[e] * rstd, -c, vd[e] * w[i][e]) * rstd;
        vd[e] = dsum ? g + vo[e] : g;
      }
      if (dx) store_row_piece<Row, NT>(dx + r * a.ld_out, c0[i], cols, whole[i], Row::pack(vd));
      if (a.q) store_quantized<Row>(vd, a.q + r * a.ld_q, a.s + r * a.ld_s, piece[i], c0[i], cols, whole[i]);
    }
  }
  if (V == 1 && at.rows_at_once > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) held[e][threadIdx.x] = dw[0][e];
    __syncthreads();
    if (at.mine > 0) return;
    for (int k = 1; k < at.rows_at_once; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[0][e] += held[e][k * row_threads + at.t];
  }
  part += (int64_t)blockIdx.x * cols;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = Row::kRuns == 1 ? c0[i] + 4 * h : c0[i] + 64 * h;
      if (c + 4 <= cols) {
        st16u<0>(part + c, u32x4{__float_as_uint(dw[i][4 * h]), __float_as_uint(dw[i][4 * h + 1]),
                                 __float_as_uint(dw[i][4 * h + 2]), __float_as_uint(dw[i][4 * h + 3])});
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (c + e < cols) part[c + e] = dw[i][4 * h + e];
      }
    }
}

// dw[c] = the sum of the blocks' parts: 32 columns and 32 runs of parts a block,
// several of a run's loads in flight.
constexpr int kPartCols = 32, kPartRuns = 32, kPartLoads = 8;
__global__ __launch_bounds__(kPartCols* kPartRuns) void k_norm_parts(const float* __restrict__ part, int parts,
                                                                     int cols, float* __restrict__ dw) {
  __shared__ float red[kPartRuns][kPartCols + 1];
  const int lc = (int)(threadIdx.x & (kPartCols - 1)), run = (int)threadIdx.x / kPartCols;
  const int c = (int)blockIdx.x * kPartCols + lc;
  float s = 0.f;
  if (c < cols) {
    int p = run;
    for (; p + (kPartLoads - 1) * kPartRuns < parts; p += kPartLoads * kPartRuns) {
      float v[kPartLoads];
#pragma unroll
      for (int i = 0; i < kPartLoads; ++i) v[i] = part[(int64_t)(p + i * kPartRuns) * cols + c];
#pragma unroll
      for (int i = 0; i < kPartLoads; ++i) s += v[i];
    }
    for (; p < parts; p += kPartRuns) s += part[(int64_t)p * cols + c];
  }
  red[run][lc] = s;
  __syncthreads();
  // the transposed sums: 32 lanes hold a column's runs
  s = red[lc][run];
  s = row16_sum(s);
  s += __shfl_xor(s, 16);
  const int col = (int)blockIdx.x * kPartCols + run;
  if (lc == 0 && col < cols) dw[col] = s;
}

struct NormShape {
  int v, threads;
};
// A row's pieces of 8 columns, 16 to a group of 128, and as many threads: a quarter
// or half of a wave, or whole waves.
NormShape norm_shape(int64_t cols) {
  const int64_t pieces = (cols + 127) / 128 * 16;
  NormShape n;
  n.v = pieces <= kNormThreads ? 1 : 2;
  n.threads = pieces <= 32 ? (int)pieces : (int)((pieces + 64 * n.v - 1) / (64 * n.v) * 64);
  return n;
}

// Blocks of a launch: as many as the device holds at once, of `waves` waves a
// compute unit.
int64_t norm_blocks(int64_t rows, int threads, int waves) {
  const int per_cu = 64 * waves / threads;
  const int64_t most = (int64_t)device_cu_count() * (per_cu < 1 ? 1 : per_cu);
  return rows < most ? rows : most;
}

// Whether `matrices` matrices of the rows' size are too much for the caches (256
// MB, and what follows finds its rows there if they fit): past them, the norm of
// 16384 rows of 7168 with residual takes 161 us with codes (169 through them), 192
// with rows and codes (209), and its gradient 197 (206); with 4096 rows and codes it
// is 51 (49), with 2048 29 (24).
bool past_caches(const NormRows& a, int matrices) {
  return a.rows * a.cols * (a.bf16 ? 2 : 4) * matrices > ((int64_t)512 << 20);
}

// fn(Row type, pieces per thread, a row may be shorter than a lane's run, past the
// caches, rows narrower than a wave)
template <class F>
hipError_t norm_dispatch(const NormRows& a, const NormShape& n, bool past, F fn) {
  auto with = [&](auto row) {
    typedef decltype(row) Row;
    typedef std::integral_constant<int, 0> Zero;
    typedef std::integral_constant<int, 1> One;
    typedef std::true_type Yes;
    typedef std::false_type No;
    if (a.cols < Row::kLen) return fn(row, One{}, Yes{}, Zero{}, Yes{});
    if (n.threads < 64) return past ? fn(row, One{}, No{}, One{}, Yes{}) : fn(row, One{}, No{}, Zero{}, Yes{});
    if (n.v == 1) return past ? fn(row, One{}, No{}, One{}, No{}) : fn(row, One{}, No{}, Zero{}, No{});
    return fn(row, std::integral_constant<int, 2>{}, No{}, Zero{}, No{});
  };
  return a.bf16 ? with(RowBF16{}) : with(RowF32{});
}

}  // namespace

static_assert(2 * kNormThreads * 8 == kMaxNormCols, "the longest row");

hipError_t launch_rms_norm(const NormRows& a, const void* x, int64_t ld_x, const void* res, int64_t ld_res, float eps,
                           void* sum, int64_t ld_sum, float* rstd, hipStream_t st) {
  const NormShape n = norm_shape(a.cols);
  const int at_once = n.threads < 64 ? 256 / n.threads : 1;
  const int64_t blocks = norm_blocks((a.rows + at_once - 1) / at_once, n.threads * at_once, 32);
  const bool past = past_caches(a, 1 + (res ? 2 : 0) + (a.out ? 1 : 0));
  return norm_dispatch(a, n, past, [&](auto row, auto v, auto tiny, auto nt, auto narrow) {
    hipLaunchKernelGGL((k_rms_norm<decltype(row), decltype(v)::value, decltype(tiny)::value, decltype(nt)::value,
                                   decltype(narrow)::value>),
                       dim3((uint32_t)blocks), dim3(n.threads * at_once), 0, st, a, x, ld_x, res, ld_res, eps, sum,
                       ld_sum, rstd, n.threads);
    return hipGetLastError();
  });
}

// Rows that a block of the gradient works on at once.
static int norm_rows_at_once(const NormShape& n) { return n.v == 1 ? kNormThreads / n.threads : 1; }

// One part for each block that runs at once (the registers leave room for 20 waves
// a compute unit).
int64_t rms_norm_parts(int64_t rows, int64_t cols) {
  const NormShape n = norm_shape(cols);
  const int at_once = norm_rows_at_once(n);
  return norm_blocks((rows + at_once - 1) / at_once, n.threads * at_once, 20);
}

hipError_t launch_rms_norm_bwd(const NormRows& a, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                               const float* rstd, const void* dsum, int64_t ld_dsum, float* part, float* dw,
                               hipStream_t st) {
  const NormShape n = norm_shape(a.cols);
  const int64_t parts = rms_norm_parts(a.rows, a.cols);
  if (parts > 0) {
    const bool past = past_caches(a, 2 + (dsum ? 1 : 0) + (a.out ? 1 : 0));
    const hipError_t err = norm_dispatch(a, n, past, [&](auto row, auto v, auto tiny, auto nt, auto narrow) {
      hipLaunchKernelGGL((k_rms_norm_bwd<decltype(row), decltype(v)::value, decltype(tiny)::value, decltype(nt)::value,
                                         decltype(narrow)::value>),
                         dim3((uint32_t)parts), dim3(n.threads * norm_rows_at_once(n)), 0, st, a, dy, ld_dy, x, ld_x,
                         rstd, dsum, ld_dsum, part, n.threads);
      return hipGetLastError();
    });
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(k_norm_parts, dim3((uint32_t)((a.cols + kPartCols - 1) / kPartCols)), dim3(kPartCols * kPartRuns),
                     0, st, part, (int)parts, (int)a.cols, dw);
  return hipGetLastError();
}

}  // namespace fp8q
