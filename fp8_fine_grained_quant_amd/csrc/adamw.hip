// An AdamW step over many tensors (gfx950).
//
//   g' = g * min(1, max_norm / norm)          (where a norm is given)
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in FP32 (the clipped gradient in 64 bits, as grad_clip forms it).  The states
// are m and v in FP32, or the E4M3 codes of m and of sqrt(v) with an FP32 scale
// per 128 elements each.  sqrt(v) has half of v's binades, so that a block's
// 2^17.8 of E4M3 hold 2^35.6 of v; what is above zero never becomes zero, since
// m / sqrt(v) would then grow without bound.  Codes are rounded at random, with
// probabilities that make the rounding's mean the value itself: to the nearest
// code, a change of v by 1 - b2 of itself would be less than half a step and v
// would never move.  It is the root's mean that is kept; the mean of its square, v
// of the next step, is above it by the rounding's variance, which adds up over the
// 1 / (1 - b2) steps that v remembers: 1.026 of the 32-bit state in the mean with
// b2 = 0.95, 1.047 with 0.99, 1.052 with 0.999 (a million elements, normal gradients
// of one size; 1.023, 1.047 and 1.055 with sizes that spread by a factor of e either
// way), and the steps' mean size, in which m's rounding counts as well, 1.007, 1.013
// and 1.016 of that with 32-bit states.  The random
// bits are a hash of the element's place and a key of the tensor, so a step is
// repeatable and no state is kept for them.
//
// Bound by memory: every value is read and written once, 28 bytes an element
// with FP32 gradients and states, 16.1 with 8-bit states and two more for a BF16
// copy.  Parameters, gradients, copies and FP32 states pass the caches: 235M
// parameters with 8-bit states and copies 735 us a pass (724 to 766 by card and
// timer), 5.8 TB/s; 200M with FP32 states 972, 5.8 TB/s.  In turn with the other
// ways: 724 and 977 us, all through the caches 794 and 1052 (only the stores past
// them 770 where that was 728).  A block has one piece of a tensor, 8 elements a
// thread, and ends: what the device holds is then made up by the pieces that begin
// as others end (in turn, 2048 blocks that took 8192 elements at a time 816 and 1045
// us against 728 and 972; 200 tensors of 100 to 2000000 elements, whose last blocks
// ran alone, 160 against 139).

#include "launch.h"
#include "row_io.h"

namespace fp8q {

namespace {

constexpr int kAdamThreads = 256;
static_assert(kAdamChunk == kAdamThreads * 8 && kAdamChunk % 128 == 0, "8 elements of every thread, whole groups");

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6C8E9CF5u;
  x = (x ^ (x >> 15)) * 0xB2D05E13u;
  return x ^ (x >> 16);
}

// y (at most 448 and a rounding in magnitude) to one of the two E4M3 values
// around it, away from zero where the fraction of their distance and u in [0, 1)
// reach 1.  POSITIVE: what is above zero stays so.
template <bool POSITIVE>
__device__ __forceinline__ float round_e4m3(float y, float u) {
  const uint32_t a = __float_as_uint(y) & 0x7FFFFFFFu;
  const uint32_t e = max(a & 0x7F800000u, 121u << 23);          // exponent, at least -6
  const float up = __uint_as_float((257u << 23) - e);            // 2^(3 - exponent)
  const float down = __uint_as_float(e - (3u << 23));            // 2^(exponent - 3)
  float n = floorf(__builtin_fmaf(__uint_as_float(a), up, u));
  if (POSITIVE) n = a != 0 ? __builtin_fmaxf(n, 1.f) : n;
  return __builtin_copysignf(__builtin_fminf(n * down, kFp8Max), y);
}

// A lane's 8 elements: two runs of 4, 64 apart, as RowF32 has them.  n counts
// the elements from the run's first on that exist (any number).
__device__ __forceinline__ void load_f32(const float* p, int n, float* v) {
  u32x4 u = {0, 0, 0, 0};
  if (n >= 4) {
    u = ld16u<1>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) u[e] = __float_as_uint(p[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(u[e]);
}
__device__ __forceinline__ void store_f32(float* p, int n, const float* v) {
  if (n >= 4) {
    st16u<1>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void load_bf16(const uint16_t* p, int n, float* v) {
  u32x2 u = {0, 0};
  if (n >= 4) {
    u = *reinterpret_cast<const u32x2_u*>(p);
  } else {
    if (n > 0) u[0] = p[0];
    if (n > 1) u[0] |= (uint32_t)p[1] << 16;
    if (n > 2) u[1] = p[2];
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_bf16(uint16_t* p, int n, const float* v) {
  const u32x2 u = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
  if (n >= 4) {
    st8u<1>(p, u);
  } else {
    if (n > 0) p[0] = (uint16_t)u[0];
    if (n > 1) p[1] = (uint16_t)(u[0] >> 16);
    if (n > 2) p[2] = (uint16_t)u[1];
  }
}
__device__ __forceinline__ uint32_t load_code4(const uint8_t* p, int n) {
  if (n >= 4) return *reinterpret_cast<const u32_u*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) w |= (uint32_t)p[e] << (8 * e);
  return w;
}
__device__ __forceinline__ void store_code4(uint8_t* p, int n, uint32_t w) {
  if (n >= 4) {
    st4u<0>(p, w);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) p[e] = (uint8_t)(w >> (8 * e));
  }
}
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0] * s;
  v[1] = lo[1] * s;
  v[2] = hi[0] * s;
  v[3] = hi[1] * s;
}

// The group's scale; a value that is not finite makes it NaN, and with it the
// group's values.
__device__ __forceinline__ float state_scale(const float (&x)[8], float& inv) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[e]));
  m = max(row16_max_u32(m), __float_as_uint(kAmaxFloor));
  if (m >= 0x7F800000u) m = 0x7FC00000u;
  inv = 1.f / __uint_as_float(m) * kFp8Max;
  return __uint_as_float(m) / kFp8Max;
}

template <int N, bool G_BF16, bool BITS8>
__global__ __launch_bounds__(kAdamThreads) void k_adamw(const AdamTable<N> t, const AdamStep a) {
  // finds a chunk's tensor: lane i holds the first chunk of tensor i (an empty
  // tensor has that of the one behind it, which is found)
  const int lane = threadIdx.x & 63;
  const int first = lane < t.n ? t.cum[lane < N ? lane : 0] : 0x7FFFFFFF;
  const double norm = a.norm ? (double)*a.norm : 0.0;
  const double factor = norm <= a.max_norm ? 1.0 : a.max_norm / norm;  // a NaN norm gives a NaN factor
  const int at = ((int)threadIdx.x >> 4) * 128 + ((int)threadIdx.x & 15) * 4;
  const int c = blockIdx.x, i = __popcll(__ballot(first <= c)) - 1;
  const int64_t lo = (int64_t)(c - t.cum[i]) * kAdamChunk;
  const int len = c + 1 < t.cum[i + 1] ? kAdamChunk : (int)t.last[i];
  const uint32_t key = mix(mix(a.seed_lo + 0x9E3779B1u * (a.place + (uint32_t)i)) + a.seed_hi) +
                       (uint32_t)((uint64_t)lo >> 32) * 0x27D4EB2Fu;
  if (((int)threadIdx.x >> 4) * 128 >= len) return;  // a group's 16 lanes stay together
  float p[8], g[8], m[8], v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t o = lo + at + 64 * h;
    const int n = len - at - 64 * h;
    load_f32(t.p[i] + o, n, p + 4 * h);
    if (G_BF16) load_bf16((const uint16_t*)t.g[i] + o, n, g + 4 * h);
    else load_f32((const float*)t.g[i] + o, n, g + 4 * h);
    if (!BITS8) {
      load_f32((const float*)t.m[i] + o, n, m + 4 * h);
      load_f32((const float*)t.v[i] + o, n, v + 4 * h);
    }
  }
  const int64_t group = (lo + at) >> 7;
  if (BITS8) {
    const float sm = t.m_scale[i][group], sv = t.v_scale[i][group];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t o = lo + at + 64 * h;
      const int n = len - at - 64 * h;
      decode4(load_code4((const uint8_t*)t.m[i] + o, n), sm, m + 4 * h);
      decode4(load_code4((const uint8_t*)t.v[i] + o, n), sv, v + 4 * h);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (BITS8) v[e] *= v[e];
    if (a.norm) g[e] = (float)((double)g[e] * factor);
    // every product and sum rounded on its own: a state in 8 bits goes by the
    // last bits of its value where that is near a border of the rounding, and
    // these are the bits that the formula gives, term by term
    m[e] = a.beta1 * m[e] + a.rest1 * g[e];
    v[e] = a.beta2 * v[e] + a.rest2 * (g[e] * g[e]);
    const float root = sqrtf(v[e]);
    p[e] = __builtin_fmaf(p[e], a.keep, -(a.step * m[e] / __builtin_fmaf(root, a.root, a.eps)));
    if (BITS8) v[e] = root;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t o = lo + at + 64 * h;
    const int n = len - at - 64 * h;
    store_f32(t.p[i] + o, n, p + 4 * h);
    if (t.copy[i]) store_bf16(t.copy[i] + o, n, p + 4 * h);
    if (!BITS8) {
      store_f32((float*)t.m[i] + o, n, m + 4 * h);
      store_f32((float*)t.v[i] + o, n, v + 4 * h);
    }
  }
  if (BITS8) {
    float inv_m, inv_v;
    const float sm = state_scale(m, inv_m), sv = state_scale(v, inv_v);
    if ((threadIdx.x & 15) == 0) {
      t.m_scale[i][group] = sm;
      t.v_scale[i][group] = sv;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t o = lo + at + 64 * h;
      const int n = len - at - 64 * h;
      float ym[4], yv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = mix((uint32_t)(o + e) * 0x85297A4Du + key);
        ym[e] = round_e4m3<false>(m[4 * h + e] * inv_m, (float)(r & 0xFFFFu) * 0x1p-16f);
        yv[e] = round_e4m3<true>(v[4 * h + e] * inv_v, (float)(r >> 16) * 0x1p-16f);
      }
      store_code4((uint8_t*)t.m[i] + o, n, pack4_e4m3_grp(ym[0], ym[1], ym[2], ym[3]));
      store_code4((uint8_t*)t.v[i] + o, n, pack4_e4m3_grp(yv[0], yv[1], yv[2], yv[3]));
    }
  }
}

template <int N>
hipError_t adamw(const AdamBatch& b, const AdamStep& a, bool g_bf16, bool bits8, hipStream_t st) {
  AdamTable<N> t;
  t.n = b.n;
  for (int i = 0; i < b.n; ++i) {
    t.p[i] = b.p[i];
    t.g[i] = b.g[i];
    t.m[i] = b.m[i];
    t.v[i] = b.v[i];
    t.m_scale[i] = b.m_scale[i];
    t.v_scale[i] = b.v_scale[i];
    t.copy[i] = b.copy[i];
    t.cum[i] = b.cum[i];
    t.last[i] = b.last[i];
  }
  t.cum[b.n] = b.cum[b.n];
  const dim3 grid(b.cum[b.n]), block(kAdamThreads);
  if (bits8) {
    if (g_bf16) hipLaunchKernelGGL((k_adamw<N, true, true>), grid, block, 0, st, t, a);
    else hipLaunchKernelGGL((k_adamw<N, false, true>), grid, block, 0, st, t, a);
  } else {
    if (g_bf16) hipLaunchKernelGGL((k_adamw<N, true, false>), grid, block, 0, st, t, a);
    else hipLaunchKernelGGL((k_adamw<N, false, false>), grid, block, 0, st, t, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamBatch& b, const AdamStep& a, bool g_bf16, bool bits8, hipStream_t st) {
  return b.n <= 8 ? adamw<8>(b, a, g_bf16, bits8, st) : adamw<kMaxAdamTensors>(b, a, g_bf16, bits8, st);
}

}  // namespace fp8q
