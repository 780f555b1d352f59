// Stable counting sort of (token, choice) pairs by expert (gfx950).
//
// Bins 0 .. E-1 are the experts, bin E collects the dropped pairs (ids outside
// [0, E)), which therefore come last.  Pair i of bin b goes to row
//   base[b] + (pairs of bin b before i),
// base the exclusive sum of the bin counts.  The pairs are cut into chunks of
// consecutive ones, a block each, and every block's into spans, a wave each;
// the pairs before i are those of the chunks before (chunk counts from a first
// launch), of the block's waves before (LDS), of the wave's earlier steps, and
// of the lower lanes holding the same bin.  Integer counts only: the result
// does not depend on the order in which anything runs.

#include "device_common.h"
#include "launch.h"

namespace fp8q {

namespace {

constexpr int kSortWaves = 8;
constexpr int kSortThreads = kSortWaves * 64;

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
  for (int i = (int)lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&h[sort_bin(ids, i, e)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b <= e; b += kSortThreads) cnt[(int64_t)blockIdx.x * (e + 1) + b] = h[b];
}

// Rows of one chunk's pairs.  cnt == NULL: the only chunk.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const int* __restrict__ ids, int n, int e, int bits,
                                                             int chunk, const int* __restrict__ cnt, int cover,
                                                             int* __restrict__ offsets, int* __restrict__ dst,
                                                             int* __restrict__ src) {
  __shared__ int wh[kSortWaves][kMaxExperts + 1];  // counts, then next row, per wave and bin
  __shared__ int tot[kMaxExperts + 1];             // bin counts of all pairs, then their exclusive sum
  __shared__ int part[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, e1 = e + 1;
  for (int b = tid; b < kSortWaves * e1; b += kSortThreads) wh[b / e1][b % e1] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int hi = (int)min((int64_t)n, lo + chunk);
  const int span = ((chunk + kSortWaves * 64 - 1) / (kSortWaves * 64)) * 64;
  const int wlo = (int)min((int64_t)hi, lo + (int64_t)wave * span), whi = (int)min((int64_t)hi, (int64_t)wlo + span);
  for (int i = wlo + lane; i < whi; i += 64) atomicAdd(&wh[wave][sort_bin(ids, i, e)], 1);
  __syncthreads();
  for (int b = tid; b < e1; b += kSortThreads) {
    int before = 0, all = 0;
    if (cnt) {
      for (int c = 0; c < (int)gridDim.x; ++c) {
        const int v = cnt[(int64_t)c * e1 + b];
        if (c < (int)blockIdx.x) before += v;
        all += v;
      }
    }
    int run = before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = wh[w][b];
      wh[w][b] = run;
      run += v;
    }
    tot[b] = cnt ? all : run;
  }
  __syncthreads();
  // exclusive sum of tot over the bins
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
    int base = carry;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) base += part[w];
      carry += part[w];
    }
    if (b < e1) {
      tot[b] = base + inc - v;
      if (blockIdx.x == 0) offsets[b] = cover && b == e ? n : base + inc - v;
    }
    __syncthreads();
  }
  for (int b = tid; b < kSortWaves * e1; b += kSortThreads) wh[b / e1][b % e1] += tot[b % e1];
  __syncthreads();
  for (int i0 = wlo; i0 < whi; i0 += 64) {
    const int i = i0 + lane;
    const bool on = i < whi;
    const int b = on ? sort_bin(ids, i, e) : 0;
    uint64_t same = __ballot(on);  // lanes with this lane's bin
    for (int bit = 0; bit < bits; ++bit) {
      const uint64_t set = __ballot((b >> bit) & 1);
      same &= ((b >> bit) & 1) ? set : ~set;
    }
    const int lead = on ? __ffsll((unsigned long long)same) - 1 : lane;
    int first = 0;
    if (on && lane == lead) first = atomicAdd(&wh[wave][b], __popcll(same));
    first = __shfl(first, lead);
    if (on) {
      const int row = first + __popcll(same & ((1ull << lane) - 1));
      dst[i] = b == e ? -1 - row : row;
      if (src) src[row] = i;
    }
  }
}

// Pairs per block: one block up to 4096 pairs; above, 4096 each, and more per
// block once that would make over 256 of them (every block reads all counts).
int sort_chunk(int64_t n) {
  constexpr int64_t kLeast = 4096, kMostBlocks = 256;
  const int64_t c = (n + kMostBlocks - 1) / kMostBlocks;
  return (int)(c < kLeast ? kLeast : c);
}

}  // namespace

int64_t moe_sort_workspace(int64_t n, int64_t e) {
  const int64_t chunk = sort_chunk(n), blocks = (n + chunk - 1) / chunk;
  return blocks <= 1 ? 0 : blocks * (e + 1) * (int64_t)sizeof(int);
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
