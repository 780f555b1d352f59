// The global norm of many FP32 gradients and their clipping (gfx950).
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / norm)
//
// Squares are formed and summed in 64 bits, so no finite gradient overflows or
// vanishes and the norm does not depend on how the elements are spread over
// threads beyond the last FP64 bits; the order of every sum is fixed.  Two
// passes over the data, since the factor needs the whole norm first; both are
// bound by memory.  470M gradients (1.88 GB) to BF16: 773 us, 6.1 TB/s over the
// 4.7 GB of both passes.  The second pass reads and writes past the caches
// (20M gradients 43 us so, 55 us through them; the 470M 773 and 851), the first
// does not, so that the second finds there what fits (20M: 49 us if it does).
// Going backwards in the second pass, to meet the last gradients read first,
// measured slower (798 us), as did 4 or 16 loads in flight (812, 797).

#include "launch.h"
#include "row_io.h"

#include <math.h>

#include <type_traits>

namespace fp8q {

namespace {

constexpr int kClipThreads = 256, kClipLoads = 8;
constexpr int kClipStep = kClipThreads * 4;            // elements of one load of the whole block
constexpr int kClipChunk = kClipStep * kClipLoads;     // elements of one tensor a block takes at a time

// The tensor that chunk c belongs to: cum[i] is the first chunk of tensor i.
__device__ __forceinline__ int clip_find(const ClipBatch& b, int c) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c >= b.cum[mid]) lo = mid; else hi = mid;
  }
  return lo;
}

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

__global__ __launch_bounds__(kClipThreads) void k_grad_sumsq(const ClipBatch b, double* __restrict__ part) {
  __shared__ double red[4];
  double s = 0;
  for (int c = blockIdx.x; c < b.cum[b.n]; c += gridDim.x) {
    const int i = clip_find(b, c);
    const int64_t lo = (int64_t)(c - b.cum[i]) * kClipChunk;
    float v[kClipLoads][4];
    load_chunk<0>(b.g[i] + lo, (int)min((int64_t)kClipChunk, b.len[i] - lo), v);
#pragma unroll
    for (int l = 0; l < kClipLoads; ++l)
#pragma unroll
      for (int j = 0; j < 4; ++j) s = __builtin_fma((double)v[l][j], (double)v[l][j], s);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
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
__global__ __launch_bounds__(kClipThreads) void k_grad_scale(const ClipBatch b, const double* __restrict__ part,
                                                             int parts, double max_norm,
                                                             float* __restrict__ norm_out) {
  __shared__ double red[4];
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += part[i];
  const double norm = sqrt(block_sum(s, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // a NaN norm fails the comparison and gives a NaN factor, an infinite one 0
  const float f = norm <= max_norm ? 1.f : (float)(max_norm / norm);
  const int chunks = b.cum[b.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = clip_find(b, c);
    if (!OUT_BF16 && f == 1.f && b.out[i] == b.g[i]) continue;  // in place, and nothing to clip
    const int64_t lo = (int64_t)(c - b.cum[i]) * kClipChunk;
    const int len = (int)min((int64_t)kClipChunk, b.len[i] - lo);
    float v[kClipLoads][4];
    load_chunk<1>(b.g[i] + lo, len, v);
#pragma unroll
    for (int l = 0; l < kClipLoads; ++l) {
      const int e = l * kClipStep + (int)threadIdx.x * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[l][j] *= f;
      store_clipped<OUT_BF16, 1>(b.out[i], lo + e, v[l], len - e);
    }
  }
}

// Blocks of one launch: at most kClipBlocks, so that the partial sums every
// scaling block adds up stay few.
int clip_blocks(const ClipBatch& b) {
  const int c = b.cum[b.n];
  return c < 1 ? 1 : c < kClipBlocks ? c : kClipBlocks;
}

}  // namespace

int64_t clip_chunks(int64_t len) { return (len + kClipChunk - 1) / kClipChunk; }

hipError_t launch_grad_sumsq(const ClipBatch& b, double* part, int* blocks, hipStream_t st) {
  *blocks = clip_blocks(b);
  hipLaunchKernelGGL(k_grad_sumsq, dim3(*blocks), dim3(kClipThreads), 0, st, b, part);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const ClipBatch& b, bool out_bf16, const double* part, int parts, double max_norm,
                             float* norm, hipStream_t st) {
  if (out_bf16)
    hipLaunchKernelGGL(k_grad_scale<true>, dim3(clip_blocks(b)), dim3(kClipThreads), 0, st, b, part, parts, max_norm, norm);
  else
    hipLaunchKernelGGL(k_grad_scale<false>, dim3(clip_blocks(b)), dim3(kClipThreads), 0, st, b, part, parts, max_norm, norm);
  return hipGetLastError();
}

}  // namespace fp8q
