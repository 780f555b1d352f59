// The gated feed-forward block h = silu(x Wg^T) (x Wu^T) for few rows (gfx950):
// tokens being generated.
//
// With up to 64 rows the block's time is that of reading its 2 N K weight
// codes, and the 256-row tiles of the large products would do it with N / 128
// workgroups, an eighth or less of the chip.  Here a workgroup owns 8 gate
// columns and the 8 up columns of the same outputs, which together are the 16
// rows of one matrix instruction's operand, and its 8 waves take the chunks of
// 128 K in turn, several of them in flight, straight from memory to registers:
// no weight is used twice, so none goes through LDS.  The waves' sums meet in
// LDS, in the order of the waves.  x is read by every workgroup, from the
// caches.
//
// Every chunk's partial is formed with BF16 matrix instructions on the exactly
// converted codes (exact products, FP32 sums), as the _exact products do: twice
// the matrix time, which the weights' reading hides.

#include "device_common.h"
#include "gemm_tile.h"
#include "launch.h"

#include <type_traits>

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kFewWaves = 8, kFewCols = 8;

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

// MT: 16-row tiles of x; U: chunks of a wave in flight.
template <int MT, int U>
__global__ __launch_bounds__(64 * kFewWaves) void k_swiglu_few(const GemmArgs p, float* __restrict__ hf) {
  __shared__ float4 red[kFewWaves][MT][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * kFewCols, nk = (int)(p.K / 128);
  // weight row of this lane: gate n0 + l16, or up n0 + l16 - 8
  const int64_t brow = l16 < kFewCols ? n0 + l16 : p.N + n0 + (l16 - kFewCols);
  const uint8_t* const B = p.B + brow * p.ldb + 16 * g;
  // lane 16 g + l16 holds the sums of x's row l16 and weight rows 4 g + r: gate
  // for g < 2, up behind
  const float* const sb = p.sb + (g < 2 ? n0 / 128 : (p.N + n0) / 128) * p.sb_rs;
  const uint8_t* A[MT];
  const float* sa[MT];
  v4f acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = min((int64_t)(16 * m + l16), p.M - 1);  // rows past the last repeat it and are not stored
    A[m] = p.A + row * p.lda + 16 * g;
    sa[m] = p.sa + row * p.ld_sa;
    acc[m] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  for (int k0 = w; k0 < nk; k0 += kFewWaves * U) {
    u32x4 b[U][2], a[U][MT][2];
    float s[U][MT], sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + kFewWaves * u, nk - 1);
      b[u][0] = ld_stream16<0>(B + (int64_t)kb * 128);
      b[u][1] = ld_stream16<0>(B + (int64_t)kb * 128 + 64);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        a[u][m][0] = ld_stream16<0>(A[m] + (int64_t)kb * 128);
        a[u][m][1] = ld_stream16<0>(A[m] + (int64_t)kb * 128 + 64);
        s[u][m] = sa[m][kb];
      }
      sw[u] = sb[kb * p.sb_cs];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + kFewWaves * u >= nk) break;
      v8bf wb[4], xb[4];
      widen(b[u], wb);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        widen(a[u][m], xb);
        v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], xb[q], c, 0, 0, 0);
        const float sc = s[u][m] * sw[u];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(c[r], sc, acc[m][r]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) red[w][m][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  // a thread makes 4 outputs: rows l16, gate columns 4 g (g < 2) of lane 16 g +
  // l16 and the up columns of lane 16 (g + 2) + l16
  const int m = (int)threadIdx.x >> 5, at = threadIdx.x & 31;
  if (m >= MT) return;
  float4 vg = red[0][m][at], vu = red[0][m][at + 32];
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) {
    const float4 x = red[i][m][at], y = red[i][m][at + 32];
    vg.x += x.x; vg.y += x.y; vg.z += x.z; vg.w += x.w;
    vu.x += y.x; vu.y += y.y; vu.z += y.z; vu.w += y.w;
  }
  const int64_t row = 16 * m + (at & 15);
  const int col = n0 + 4 * (at >> 4);
  if (row >= p.M) return;
  auto pack = [](const float4& v) {
    return make_uint2(pack2_bf16(v.x, v.y), pack2_bf16(v.z, v.w));
  };
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
}

}  // namespace

// The codes of a 128-column group need 16 workgroups' outputs: they are made by
// a second launch from h in FP32 (hf).
hipError_t launch_swiglu_few(const GemmArgs& a, float* hf, hipStream_t st) {
  const dim3 grid((uint32_t)(a.N / kFewCols)), block(64 * kFewWaves);
  if (a.M <= 16) hipLaunchKernelGGL((k_swiglu_few<1, 8>), grid, block, 0, st, a, hf);
  else if (a.M <= 32) hipLaunchKernelGGL((k_swiglu_few<2, 4>), grid, block, 0, st, a, hf);
  else hipLaunchKernelGGL((k_swiglu_few<4, 2>), grid, block, 0, st, a, hf);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.qo == nullptr) return err;
  return launch_quant_act(hf, false, a.M, a.N, a.N, a.qo, a.ld_qo, a.so, a.ld_so, st);
}

}  // namespace fp8q
