// The gated feed-forward block h = silu(x Wg^T) (x Wu^T) for few rows (gfx950):
// tokens being generated.
//
// With few rows the block's time is that of reading its 2 N K weight codes, and
// the 256-row tiles of the large products would do it with N / 128 workgroups, an
// eighth or less of the chip.  Here a workgroup owns 8 gate
// columns and the 8 up columns of the same outputs, which together are the 16
// rows of one matrix instruction's operand, and its waves share the chunks of
// 128 K.  Each wave brings its chunks of the weights and of x to its own part of
// LDS by direct loads, several of them in flight, and waits for nobody; the
// waves' sums meet at the end, in the order of the waves.  (Loads straight to the
// registers, in the matrix instruction's layout, have neighbouring lanes in
// different rows, and the cache takes each lane's 16 bytes on its own: 13
// accesses' time for one.  64 rows of 2048 x 7168 took 25 us that way.)
//
// Every chunk's partial is formed with BF16 matrix instructions on the exactly
// converted codes (exact products, FP32 sums), as the _exact products do.

#include "device_common.h"
#include "gemm_tile.h"
#include "launch.h"

#include <type_traits>

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kFewCols = 8;  // output columns of a workgroup

// 32 codes (the lane's K positions of a chunk) as four groups of 8 BF16 values.
__device__ __forceinline__ void widen(const u32x4 (&f)[2], v8bf (&out)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int a = (int)f[q >> 1][2 * (q & 1)], b = (int)f[q >> 1][2 * (q & 1) + 1];
    const v2bf c0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const v2bf c1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const v2bf c2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const v2bf c3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    out[q] = v8bf{c0[0], c0[1], c1[0], c1[1], c2[0], c2[1], c3[0], c3[1]};
  }
}

// MT: 16-row tiles of x that a workgroup works on; W: waves; BATCH: chunks whose
// scales a wave fetches together (8 or 4).  A wave has two chunks in flight, which
// leaves room for a second workgroup where MT is 1 (four, with one workgroup a
// compute unit: 8.0 us against 7.3 for 8 rows of 2048 x 7168, 19 against 13 for 16
// of 8192 x 4096).
template <int MT, int W, int BATCH>
__global__ __launch_bounds__(64 * W) void k_swiglu_few(const GemmArgs p, float* __restrict__ hf) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kChunk = 2048 * (MT + 1);        // a chunk's 16 weight rows, then its x rows
  constexpr int kScRows = 16 * MT + 2, kScPitch = BATCH + 1;
  // one LDS object a stage, so that no wait for one covers another
  __shared__ __attribute__((aligned(16))) uint8_t st0[W * kChunk];
  __shared__ __attribute__((aligned(16))) uint8_t st1[W * kChunk];
  __shared__ float scales[W][kScRows * kScPitch];
  static_assert(W * 1024 * MT <= W * kChunk, "the waves' sums fit in a stage");
  static_assert(BATCH % 2 == 0, "a batch ends with the second stage");
  static_assert(32 * MT <= 64 * W, "a thread for every 4 outputs");

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);  // first row of this workgroup
  const int rows = (int)min(p.M - row0, (int64_t)(16 * MT));
  const int n0 = (int)blockIdx.x * kFewCols, nk = (int)(p.K / 128);
  const int first = w * nk / W, last = (w + 1) * nk / W;  // this wave's chunks
  const int64_t u0 = p.N + n0;                            // first up row

  auto rsrc = [](const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t rG = rsrc(p.B + n0 * p.ldb, (uint32_t)(kFewCols * p.ldb));
  const __amdgpu_buffer_rsrc_t rU = rsrc(p.B + u0 * p.ldb, (uint32_t)(kFewCols * p.ldb));
  const __amdgpu_buffer_rsrc_t rA = rsrc(p.A + row0 * p.lda, (uint32_t)(rows * p.lda));  // rows past the last one: no access
  // a load brings 8 rows of 128 bytes: lane 8 r + c the 16 bytes c ^ r of row r
  const int r8 = lane >> 3, c16 = 16 * ((lane & 7) ^ r8);
  const uint32_t vB = (uint32_t)(r8 * p.ldb + c16), vA = (uint32_t)(r8 * p.lda + c16);
  constexpr int kLoads = 2 * (MT + 1);  // of a chunk
  // Whole pairs of chunks are worked on, so that every wait has the same loads
  // behind it: a chunk past the wave's last one repeats that, with a scale of zero,
  // and past the last pair as many loads are issued without access.
  const int pairs_end = first + (last - first + 1) / 2 * 2;
  auto issue = [&](int kb, uint8_t* stage) {
    uint8_t* const to = stage + w * kChunk;
    const bool on = kb < pairs_end;
    const uint32_t k = on ? (uint32_t)min(kb, last - 1) * 128 : 0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rG, (lds_ptr)to, 16, on ? vB : kNoAccess, k, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rU, (lds_ptr)(to + 1024), 16, on ? vB : kNoAccess, k, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr)(to + 2048 + 1024 * i), 16,
                                               on ? vA + (uint32_t)(8 * i * p.lda) : kNoAccess, k, 0, 0);
  };

  // The scales of a batch of chunks: row i < 16 MT of x, then gate's and up's
  // block; lane BATCH r + c holds chunk c of rows r, r + 64 / BATCH, ...
  constexpr int kScAtOnce = 64 / BATCH, kScLoads = 16 * MT / kScAtOnce;
  const int sr = lane / BATCH, sk = lane % BATCH;
  float sx[kScLoads], sb = 0.f;
  auto load_scales = [&](int kb) {
    const int k = min(kb + sk, nk - 1);
#pragma unroll
    for (int i = 0; i < kScLoads; ++i)
      sx[i] = p.sa[(row0 + min(kScAtOnce * i + sr, rows - 1)) * p.ld_sa + k];
    sb = p.sb[((sr & 1 ? u0 : (int64_t)n0) / 128) * p.sb_rs + k * p.sb_cs];
  };
  float* const sc = scales[w];
  auto keep_scales = [&] {
#pragma unroll
    for (int i = 0; i < kScLoads; ++i) sc[(kScAtOnce * i + sr) * kScPitch + sk] = sx[i];
    if (sr < 2) sc[(16 * MT + sr) * kScPitch + sk] = sb;
  };

  v4f acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = v4f{0.f, 0.f, 0.f, 0.f};

  auto fence = [] { asm volatile("" ::: "memory"); };
  load_scales(first);
  fence();
  issue(first, st0);
  issue(first + 1, st1);
  keep_scales();

  const int sw = l16 & 7;
  const int lo = l16 * 128 + 16 * (g ^ sw), hi = l16 * 128 + 16 * ((4 + g) ^ sw);
  auto step = [&](int kb, int j, uint8_t* stage) {
    __builtin_amdgcn_s_waitcnt(0x0F70 | (kLoads & 15) | ((kLoads >> 4) << 14));  // the stage's loads have landed
    fence();
    const uint8_t* const at = stage + w * kChunk;
    u32x4 b[2], a[MT][2];
    b[0] = *reinterpret_cast<const u32x4*>(at + lo);
    b[1] = *reinterpret_cast<const u32x4*>(at + hi);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      a[m][0] = *reinterpret_cast<const u32x4*>(at + 2048 * (m + 1) + lo);
      a[m][1] = *reinterpret_cast<const u32x4*>(at + 2048 * (m + 1) + hi);
    }
    // lane 16 g + l16 will hold the sums of x's row l16 and weight rows 4 g + r:
    // gate for g < 2, up behind
    const float sw_ = kb < last ? sc[(16 * MT + (g >> 1)) * kScPitch + j] : 0.f;
    float s[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) s[m] = sc[(16 * m + l16) * kScPitch + j] * sw_;
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the stage is read
    fence();
    issue(kb + 2, stage);
    v8bf wb[4], xb[4];
    widen(b, wb);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      widen(a[m], xb);
      v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], xb[q], c, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(c[r], s[m], acc[m][r]);
    }
  };
  for (int k0 = first; k0 < last; k0 += BATCH) {
    const bool more = k0 + BATCH < last;
    if (more) load_scales(k0 + BATCH);
    for (int j = 0; j < BATCH && k0 + j < last; j += 2) {
      step(k0 + j, j, st0);
      step(k0 + j + 1, j + 1, st1);
    }
    if (more) keep_scales();
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();  // no load is to come into what the sums take
  float4* const red = reinterpret_cast<float4*>(st0);
#pragma unroll
  for (int m = 0; m < MT; ++m) red[(w * MT + m) * 64 + lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  // a thread makes 4 outputs: rows l16, gate columns 4 g (g < 2) of lane 16 g +
  // l16 and the up columns of lane 16 (g + 2) + l16
  const int m = (int)threadIdx.x >> 5, at = threadIdx.x & 31;
  if (m >= MT) return;
  float4 vg = red[m * 64 + at], vu = red[m * 64 + at + 32];
#pragma unroll
  for (int i = 1; i < W; ++i) {
    const float4 x = red[(i * MT + m) * 64 + at], y = red[(i * MT + m) * 64 + at + 32];
    vg.x += x.x; vg.y += x.y; vg.z += x.z; vg.w += x.w;
    vu.x += y.x; vu.y += y.y; vu.z += y.z; vu.w += y.w;
  }
  if (16 * m + (at & 15) >= rows) return;
  const int64_t row = row0 + 16 * m + (at & 15);
  const int col = n0 + 4 * (at >> 4);
  auto pack = [](const float4& v) { return make_uint2(pack2_bf16(v.x, v.y), pack2_bf16(v.z, v.w)); };
  if (p.gu != nullptr) {
    *reinterpret_cast<uint2*>(p.gu + row * p.ld_gu + col) = pack(vg);
    *reinterpret_cast<uint2*>(p.gu + row * p.ld_gu + p.N + col) = pack(vu);
  }
  vg.x *= sigmoid_f32(vg.x) * vu.x;
  vg.y *= sigmoid_f32(vg.y) * vu.y;
  vg.z *= sigmoid_f32(vg.z) * vu.z;
  vg.w *= sigmoid_f32(vg.w) * vu.w;
  if (p.C != nullptr) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.C) + row * p.ldc + col) = pack(vg);
  if (hf != nullptr) *reinterpret_cast<float4*>(hf + row * p.N + col) = vg;
#endif  // __HIP_DEVICE_COMPILE__
}

template <int MT, int W, int BATCH>
hipError_t few(const GemmArgs& a, float* hf, hipStream_t st) {
  const dim3 grid((uint32_t)(a.N / kFewCols), (uint32_t)((a.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((k_swiglu_few<MT, W, BATCH>), grid, dim3(64 * W), 0, st, a, hf);
  return hipGetLastError();
}

// 16-row tiles of a workgroup.
int few_tiles(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : M <= 64 ? 4 : 8; }

}  // namespace

// By the times of the kernels in ns, of rounds of workgroups: here 4 us and 40 + 31
// mt ns a chunk (8, 32, 64 and 128 rows of 2048 x 7168: 7.3, 8.7, 12.1 and 19.4 us;
// tiles of 32 rows take 28 there up to 256 rows, the large ones 50 to 70).  Up to 16
// rows only the large tiles' time is asked, not the small ones', so that what is
// generated for a few sequences mostly has the exact products' accuracy: with K = 128
// up to a width of 4096, with K = 1024 of 8192 (but for 6272), with K = 7168 of 22528
// (and at some widths above), from K = 16384 on of any.  Wider blocks fill the device
// with FP8 tiles (the small ones, once they are not taken here), which are faster
// with a short K: 8 rows of 8192, 16384 and 32768 x 128 take 5.4 us (here 7.2, 12 and
// 23), of 24576 x 1024 12 (24), of 32768 x 7168 80 (88), but of 24576 x 4096 45 (40)
// and of 28672 x 8192 82 (79).
bool swiglu_few(int64_t M, int64_t N, int64_t K) {
  const int64_t mt = few_tiles(M), nk = K / 128, cus = device_cu_count();
  const int64_t rounds = ((M + 16 * mt - 1) / (16 * mt) * (N / kFewCols) + cus - 1) / cus;
  const int64_t here = rounds * (4000 + nk * (40 + 31 * mt));
  int rows;
  return here <= gated_large_time(M, N, K, 0, kSwiglu) &&
         (M <= 16 || here <= gated_small_time(M, N, K, 0, kSwiglu, &rows));
}

// The codes of a 128-column group need 16 workgroups' outputs: they are made by
// a second launch from h in FP32 (hf).
hipError_t launch_swiglu_few(const GemmArgs& a, float* hf, hipStream_t st) {
  const int mt = few_tiles(a.M);
  const hipError_t err = mt == 1   ? few<1, 8, 8>(a, hf, st)
                         : mt == 2 ? few<2, 8, 8>(a, hf, st)
                         : mt == 4 ? few<4, 7, 8>(a, hf, st)
                                   : few<8, 4, 4>(a, hf, st);
  if (err != hipSuccess || a.qo == nullptr) return err;
  return launch_quant_act(hf, false, a.M, a.N, a.N, a.qo, a.ld_qo, a.so, a.ld_so, st);
}

}  // namespace fp8q
