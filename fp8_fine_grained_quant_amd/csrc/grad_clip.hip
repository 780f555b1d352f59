// The global norm of many FP32 gradients and their clipping (gfx950).
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / norm)
//
// Squares are formed and summed in 64 bits, so no finite gradient overflows or
// vanishes and the norm does not depend on how the elements are spread over
// threads beyond the last FP64 bits; the order of every sum is fixed.  Two
// passes over the data: the factor needs the whole norm first.

#include "launch.h"
#include "row_io.h"

#include <math.h>

#include <type_traits>

namespace fp8q {

namespace {

constexpr int kClipChunk = 8192;  // elements of one tensor a block takes at a time

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

__global__ __launch_bounds__(256) void k_grad_sumsq(const ClipBatch b, double* __restrict__ part) {
  __shared__ double red[4];
  double s = 0;
  for (int c = blockIdx.x; c < b.cum[b.n]; c += gridDim.x) {
    const int i = clip_find(b, c);
    const int64_t lo = (int64_t)(c - b.cum[i]) * kClipChunk;
    const int len = (int)min((int64_t)kClipChunk, b.len[i] - lo);
    const float* g = b.g[i] + lo;
    for (int e = threadIdx.x * 4; e < len; e += 1024) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (e + 4 <= len) {
        const u32x4 u = ld16u<0>(g + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(u[j]);
      } else {
        for (int j = 0; j < len - e; ++j) v[j] = g[e + j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s = __builtin_fma((double)v[j], (double)v[j], s);
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <bool OUT_BF16>
__global__ __launch_bounds__(256) void k_grad_scale(const ClipBatch b, const double* __restrict__ part, int parts,
                                                    double max_norm, float* __restrict__ norm_out) {
  __shared__ double red[4];
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
  const double norm = sqrt(block_sum(s, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // a NaN norm fails the comparison and gives a NaN factor, an infinite one 0
  const float f = norm <= max_norm ? 1.f : (float)(max_norm / norm);
  for (int c = blockIdx.x; c < b.cum[b.n]; c += gridDim.x) {
    const int i = clip_find(b, c);
    const int64_t lo = (int64_t)(c - b.cum[i]) * kClipChunk;
    const int len = (int)min((int64_t)kClipChunk, b.len[i] - lo);
    const float* g = b.g[i] + lo;
    for (int e = threadIdx.x * 4; e < len; e += 1024) {
      float v[4];
      if (e + 4 <= len) {
        const u32x4 u = ld16u<0>(g + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(u[j]) * f;
        if (OUT_BF16)
          st8u<0>((uint16_t*)b.out[i] + lo + e, u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])});
        else
          st16u<0>((float*)b.out[i] + lo + e, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                   __float_as_uint(v[2]), __float_as_uint(v[3])});
      } else {
        for (int j = 0; j < len - e; ++j) {
          const float o = g[e + j] * f;
          if (OUT_BF16) ((uint16_t*)b.out[i])[lo + e + j] = (uint16_t)pack2_bf16(o, 0.f);
          else ((float*)b.out[i])[lo + e + j] = o;
        }
      }
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
  hipLaunchKernelGGL(k_grad_sumsq, dim3(*blocks), dim3(256), 0, st, b, part);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const ClipBatch& b, bool out_bf16, const double* part, int parts, double max_norm,
                             float* norm, hipStream_t st) {
  if (out_bf16)
    hipLaunchKernelGGL(k_grad_scale<true>, dim3(clip_blocks(b)), dim3(256), 0, st, b, part, parts, max_norm, norm);
  else
    hipLaunchKernelGGL(k_grad_scale<false>, dim3(clip_blocks(b)), dim3(256), 0, st, b, part, parts, max_norm, norm);
  return hipGetLastError();
}

}  // namespace fp8q
