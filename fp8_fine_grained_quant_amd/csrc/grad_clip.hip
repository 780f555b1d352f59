// The global norm of many FP32 gradients and their clipping (gfx950).
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / norm)
//
// Squares are formed and summed in 64 bits, so no finite gradient overflows or
// vanishes in the norm, and it does not depend on how the elements are spread
// over threads beyond the last FP64 bits; the order of every sum is fixed.  The
// factor and its products are in 64 bits as well (the times are the same with
// FP32 products): the only rounding to fewer is the output's.
//
// Two passes over the data, since the factor needs the whole norm first; both
// are bound by memory.  470M gradients (1.88 GB) to BF16: 765 us, 6.1 TB/s over
// the 4.7 GB of both passes (6.2 in the first, which only reads).  The second
// pass reads and writes past the caches (20M gradients 43 us so, 55 us through
// them; the 470M 773 and 851), the first does not, so that the second finds
// there what fits (20M: 49 us where the first passes them too).  Going backwards
// in the second pass, to meet the last gradients read first, measured slower
// (798 us), as did 4 or 16 loads in flight (812, 797).

#include "launch.h"
#include "row_io.h"

#include <math.h>

#include <type_traits>

namespace fp8q {

namespace {

constexpr int kClipThreads = 256, kClipLoads = 8;
constexpr int kClipStep = kClipThreads * 4;  // elements of one load of the whole block
static_assert(kClipStep * kClipLoads == kClipChunk, "a chunk is one round of loads");

// Finds a chunk's tensor: a lane holds two of the tensors' first chunks, so
// that the table is not searched through its memory; the tensor's own entries
// are read from it.
template <int N>
struct ClipFinder {
  const ClipTable<N>& b;
  int first0, first1;
  __device__ __forceinline__ explicit ClipFinder(const ClipTable<N>& t) : b(t) {
    constexpr int kNone = 0x7FFFFFFF;
    const int lane = threadIdx.x & 63, n = t.n;
    first0 = lane < n ? t.cum[lane < N ? lane : 0] : kNone;
    first1 = N > 64 && lane + 64 < n ? t.cum[lane + 64 < N ? lane + 64 : 0] : kNone;
  }
  // The tensor of chunk c, and where in it the chunk starts and how long it is.
  __device__ __forceinline__ int operator()(int c, int64_t& lo, int& len) const {
    const int i = __popcll(__ballot(first0 <= c)) + (N > 64 ? __popcll(__ballot(first1 <= c)) : 0) - 1;
    lo = (int64_t)(c - b.cum[i]) * kClipChunk;
    len = c + 1 < b.cum[i + 1] ? kClipChunk : (int)b.last[i];
    return i;
  }
};

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// A thread's elements of a chunk, all loads in flight together; zeros past the
// tensor's end.
template <int NT>
__device__ __forceinline__ void load_chunk(const float* g, int len, float (&v)[kClipLoads][4]) {
#pragma unroll
  for (int i = 0; i < kClipLoads; ++i) {
    const int e = i * kClipStep + (int)threadIdx.x * 4;
    u32x4 u = {0, 0, 0, 0};
    if (e + 4 <= len) {
      u = ld16u<NT>(g + e);
    } else if (e < len) {
      u[0] = __float_as_uint(g[e]);
      if (e + 1 < len) u[1] = __float_as_uint(g[e + 1]);
      if (e + 2 < len) u[2] = __float_as_uint(g[e + 2]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = __uint_as_float(u[j]);
  }
}

template <int N>
__global__ __launch_bounds__(kClipThreads) void k_grad_sumsq(const ClipTable<N> b, ClipBatch* __restrict__ table,
                                                             double* __restrict__ part, int held) {
  __shared__ double red[4];
  const ClipFinder<N> find(b);
  if (blockIdx.x == gridDim.x - 1) {  // the second pass reads the table from memory
    const int n = b.n;
    for (int i = threadIdx.x; i <= n; i += kClipThreads) {
      table->cum[i] = b.cum[i];
      if (i < n) {
        table->g[i] = b.g[i];
        table->out[i] = b.out[i];
        table->last[i] = b.last[i];
      }
    }
    if (threadIdx.x == 0) table->n = (uint16_t)n;
  }
  double s = 0;
  const int chunks = b.cum[b.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    int64_t lo;
    int len;
    const int i = find(c, lo, len);
    float v[kClipLoads][4];
    load_chunk<0>(b.g[i] + lo, len, v);
#pragma unroll
    for (int l = 0; l < kClipLoads; ++l)
#pragma unroll
      for (int j = 0; j < 4; ++j) s = __builtin_fma((double)v[l][j], (double)v[l][j], s);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = (int)blockIdx.x < held ? part[blockIdx.x] + s : s;
}

template <bool OUT_BF16, int NT>
__device__ __forceinline__ void store_clipped(void* out, int64_t at, const float (&v)[4], int n) {
  if (n >= 4) {
    if (OUT_BF16)
      st8u<NT>((uint16_t*)out + at, u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])});
    else
      st16u<NT>((float*)out + at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                        __float_as_uint(v[3])});
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < n) {
        if (OUT_BF16) ((uint16_t*)out)[at + j] = (uint16_t)pack2_bf16(v[j], 0.f);
        else ((float*)out)[at + j] = v[j];
      }
  }
}

template <bool OUT_BF16>
__global__ __launch_bounds__(kClipThreads) void k_grad_scale(const ClipBatch* __restrict__ table, int chunks,
                                                             const double* __restrict__ part, int parts,
                                                             double max_norm, float* __restrict__ norm_out) {
  __shared__ double red[4];
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += part[i];
  const double norm = sqrt(block_sum(s, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // A NaN norm fails the comparison and gives a NaN factor, an infinite one 0.
  // The factor may be far below FP32's range where its product with a gradient
  // is not, so it and the product are in 64 bits.
  const double f = norm <= max_norm ? 1.0 : max_norm / norm;
  if (chunks == 0) return;  // no table, and a null pointer to it: no reference before this
  const ClipBatch& b = *table;
  const ClipFinder<kMaxClipTensors> find(b);
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    int64_t lo;
    int len;
    const int i = find(c, lo, len);
    if (!OUT_BF16 && f == 1.0 && b.out[i] == b.g[i]) continue;  // in place, and nothing to clip
    float v[kClipLoads][4];
    load_chunk<1>(b.g[i] + lo, len, v);
#pragma unroll
    for (int l = 0; l < kClipLoads; ++l) {
      const int e = l * kClipStep + (int)threadIdx.x * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[l][j] = (float)((double)v[l][j] * f);
      store_clipped<OUT_BF16, 1>(b.out[i], lo + e, v[l], len - e);
    }
  }
}

// Blocks of one launch: at most kClipBlocks.  A batch's blocks add to the
// partial sums of the batches before it (launches of one stream follow each
// other), so that all of them, which every scaling block adds up, stay that few
// whatever the number of tensors (4000 of 100000 elements to BF16: 1077 us; 2230
// with a batch's sums beside the others').
int clip_blocks(int chunks) { return chunks < 1 ? 1 : chunks < kClipBlocks ? chunks : kClipBlocks; }

template <int N>
hipError_t sumsq(const ClipBatch& b, ClipBatch* table, double* part, int held, int blocks, hipStream_t st) {
  ClipTable<N> t;
  t.n = b.n;
  for (int i = 0; i < b.n; ++i) {
    t.g[i] = b.g[i];
    t.out[i] = b.out[i];
    t.cum[i] = b.cum[i];
    t.last[i] = b.last[i];
  }
  t.cum[b.n] = b.cum[b.n];
  hipLaunchKernelGGL(k_grad_sumsq<N>, dim3(blocks), dim3(kClipThreads), 0, st, t, table, part, held);
  return hipGetLastError();
}

}  // namespace

// The table's size is that of a few classes: a launch takes 2.9 us on the host
// with 16 bytes of arguments, 3.4 with the table of 32 tensors (712 bytes), 3.7
// with that of 64 (1416) and 3.9 with that of 96 (2120).
hipError_t launch_grad_sumsq(const ClipBatch& b, ClipBatch* table, double* part, int* held, hipStream_t st) {
  const int blocks = clip_blocks(b.cum[b.n]), before = *held;
  if (blocks > before) *held = blocks;
  if (b.n <= 8) return sumsq<8>(b, table, part, before, blocks, st);
  if (b.n <= 32) return sumsq<32>(b, table, part, before, blocks, st);
  if (b.n <= 64) return sumsq<64>(b, table, part, before, blocks, st);
  return sumsq<kMaxClipTensors>(b, table, part, before, blocks, st);
}

hipError_t launch_grad_scale(const ClipBatch* table, int chunks, bool out_bf16, const double* part, int parts,
                             double max_norm, float* norm, hipStream_t st) {
  const dim3 grid(clip_blocks(chunks));
  if (out_bf16)
    hipLaunchKernelGGL(k_grad_scale<true>, grid, dim3(kClipThreads), 0, st, table, chunks, part, parts, max_norm, norm);
  else
    hipLaunchKernelGGL(k_grad_scale<false>, grid, dim3(kClipThreads), 0, st, table, chunks, part, parts, max_norm,
                       norm);
  return hipGetLastError();
}

}  // namespace fp8q
