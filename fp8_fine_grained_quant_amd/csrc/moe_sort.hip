// Stable counting sort of (token, choice) pairs by expert (gfx950).
//
// Bins 0 .. E-1 are the experts, bin E collects the dropped pairs (ids outside
// [0, E)), which therefore come last.  Pair i of bin b goes to row
//   base[b] + (pairs of bin b before i),
// base the exclusive sum of the bin counts.  The pairs are cut into chunks of
// consecutive ones, a block each, and every chunk into tiles that the block's
// waves share, kSteps * 64 pairs each; the pairs before i are those of the
// chunks before (chunk counts from a first launch), of the tiles and waves
// before (LDS), of the wave's earlier steps, and of the lower lanes holding the
// same bin.  Integer counts only: the result does not depend on the order in
// which anything runs.

#include "device_common.h"
#include "launch.h"

namespace fp8q {

namespace {

constexpr int kSortWaves = 8, kSteps = 4;
constexpr int kSortThreads = kSortWaves * 64;
constexpr int kTile = kSortThreads * kSteps;  // pairs a block ranks together
constexpr int kOneBlock = 4096;   // most pairs that one block sorts by itself
constexpr int kMostBlocks = 256;  // most chunks: every block reads all their counts

// Ints between the blocks' counts: whole 16-byte pieces.
__host__ __device__ constexpr int sort_stride(int e) { return (e + 4) / 4 * 4; }

__device__ __forceinline__ int sort_bin(const int* ids, int i, int e) {
  const int b = ids[i];
  return (uint32_t)b < (uint32_t)e ? b : e;
}

// Chunk counts: cnt[block][bin].
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const int* __restrict__ ids, int n, int e, int chunk,
                                                             int* __restrict__ cnt) {
  __shared__ int h[kMaxExperts + 1];
  for (int b = threadIdx.x; b <= e; b += kSortThreads) h[b] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int hi = (int)min((int64_t)n, lo + chunk);
  for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += kTile) {
    int b[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) b[u] = sort_bin(ids, (int)min(i0 + u * kSortThreads, (int64_t)hi - 1), e);
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (i0 + u * kSortThreads < hi) atomicAdd(&h[b[u]], 1);
  }
  __syncthreads();
  int* const c = cnt + (int64_t)blockIdx.x * sort_stride(e);
  for (int b = threadIdx.x; b < sort_stride(e); b += kSortThreads) c[b] = b <= e ? h[b] : 0;
}

// Rows of one chunk's pairs.  cnt == NULL: the only chunk.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const int* __restrict__ ids, int n, int e, int bits,
                                                             int chunk, const int* __restrict__ cnt, int cover,
                                                             int* __restrict__ offsets, int* __restrict__ dst,
                                                             int* __restrict__ src) {
  __shared__ int wh[kSortWaves][kMaxExperts + 1];  // pairs of the tile per wave and bin, then the wave's next row
  __shared__ int base[kMaxExperts + 4];            // pairs in the chunks before, then the bin's next row
  __shared__ int tot[kMaxExperts + 4];             // bin counts of all pairs
  __shared__ int part[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, e1 = e + 1;
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int hi = (int)min((int64_t)n, lo + chunk);
  for (int b = tid; b < sort_stride(e); b += kSortThreads) base[b] = tot[b] = 0;
  for (int b = tid; b < kSortWaves * e1; b += kSortThreads) wh[b / e1][b % e1] = 0;
  __syncthreads();
  if (cnt) {
    // a thread adds up 4 bins of every rows-th block
    const int quads = sort_stride(e) / 4, rows = kSortThreads / quads;
    const int row = tid / quads, q = tid - row * quads;
    if (row < rows) {
      typedef int i32x4 __attribute__((ext_vector_type(4)));
      typedef i32x4 i32x4_u __attribute__((aligned(4)));
      i32x4 before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
      const int blocks = (int)gridDim.x;
#pragma unroll 8
      for (int c = row; c < blocks; c += rows) {
        const i32x4 v = *reinterpret_cast<const i32x4_u*>(cnt + (int64_t)c * quads * 4 + q * 4);
        all += v;
        before += c < (int)blockIdx.x ? v : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        atomicAdd(&base[q * 4 + i], before[i]);
        atomicAdd(&tot[q * 4 + i], all[i]);
      }
    }
  } else {
    for (int i = tid; i < hi; i += kSortThreads) atomicAdd(&tot[sort_bin(ids, i, e)], 1);
  }
  __syncthreads();
  // base += the exclusive sum of tot over the bins
  int carry = 0;
  for (int b0 = 0; b0 < e1; b0 += kSortThreads) {
    const int b = b0 + tid;
    const int v = b < e1 ? tot[b] : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 63) part[wave] = inc;
    __syncthreads();
    int first = carry;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) first += part[w];
      carry += part[w];
    }
    if (b < e1) {
      base[b] += first + inc - v;
      if (blockIdx.x == 0) offsets[b] = cover && b == e ? n : first + inc - v;
    }
    __syncthreads();
  }
  for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
    // each pair's rank among its wave's pairs of the same bin
    const int64_t i0 = t0 + wave * (kSteps * 64) + lane;
    int bin[kSteps], rank[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) bin[u] = i0 + u * 64 < hi ? sort_bin(ids, (int)(i0 + u * 64), e) : -1;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const bool on = bin[u] >= 0;
      uint64_t same = __ballot(on);  // lanes with this lane's bin
      if (same == 0) break;
      for (int bit = 0; bit < bits; ++bit) {
        const uint64_t set = __ballot((bin[u] >> bit) & 1);
        same &= ((bin[u] >> bit) & 1) ? set : ~set;
      }
      const int lead = on ? __ffsll((unsigned long long)same) - 1 : lane;
      int first = 0;
      if (on && lane == lead) first = atomicAdd(&wh[wave][bin[u]], __popcll(same));
      first = __shfl(first, lead);
      rank[u] = first + __popcll(same & ((1ull << lane) - 1));
    }
    __syncthreads();
    for (int b = tid; b < e1; b += kSortThreads) {
      int run = base[b];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = wh[w][b];
        wh[w][b] = run;
        run += v;
      }
      base[b] = run;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      if (bin[u] < 0) continue;
      const int i = (int)(i0 + u * 64), row = wh[wave][bin[u]] + rank[u];
      dst[i] = bin[u] == e ? -1 - row : row;
      if (src) src[row] = i;
    }
    if (t0 + kTile < hi) {  // another tile
      __syncthreads();
      for (int b = tid; b < kSortWaves * e1; b += kSortThreads) wh[b / e1][b % e1] = 0;
      __syncthreads();
    }
  }
}

// Pairs per block: one block up to kOneBlock pairs, which saves a launch (4096
// pairs: 10.3 us by one block, 10.2 us by two launches and 5 us more on the
// host; 8192 pairs: 20.2 us and 11.3 us); above, a tile each (262144 pairs of
// 256 experts: 14.1 us, with half a tile 15.9, with two 16.8), and more per
// block once that would make over kMostBlocks of them.  What is left is the
// two launches and one block's chain of steps; the pairs' bytes alone would
// take 1 us.
int sort_chunk(int64_t n) {
  if (n <= kOneBlock) return kOneBlock;
  const int64_t c = (n + kMostBlocks - 1) / kMostBlocks;
  return (int)((c + kTile - 1) / kTile * kTile);
}

}  // namespace

int64_t moe_sort_workspace(int64_t n, int64_t e) {
  const int64_t chunk = sort_chunk(n), blocks = (n + chunk - 1) / chunk;
  return blocks <= 1 ? 0 : blocks * sort_stride((int)e) * (int64_t)sizeof(int);
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int64_t e, bool cover, int32_t* offsets, int32_t* dst,
                           int32_t* src, void* ws, hipStream_t st) {
  const int chunk = sort_chunk(n);
  const int blocks = n == 0 ? 1 : (int)((n + chunk - 1) / chunk);
  int bits = 1;
  while ((e >> bits) != 0) ++bits;
  int* cnt = nullptr;
  if (blocks > 1) {
    cnt = (int*)ws;
    hipLaunchKernelGGL(k_sort_count, dim3(blocks), dim3(kSortThreads), 0, st, ids, (int)n, (int)e, chunk, cnt);
    if (const hipError_t err = hipGetLastError(); err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(k_sort_place, dim3(blocks), dim3(kSortThreads), 0, st, ids, (int)n, (int)e, bits, chunk,
                     (const int*)cnt, (int)cover, offsets, dst, src);
  return hipGetLastError();
}

}  // namespace fp8q
