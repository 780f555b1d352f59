// Row access shared by the MoE row kernels and gradient clipping: elements of a
// row as 16-byte accesses at ANY element alignment.  gfx950 global
// memory instructions take multi-dword accesses at any byte address, so rows
// whose length is odd use the same instructions as aligned ones; only the
// alignment the compiler may assume differs.
#pragma once

#include "device_common.h"

namespace fp8q {

typedef u32x4 u32x4_u __attribute__((aligned(1)));
typedef u32x2 u32x2_u __attribute__((aligned(1)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef uint16_t u16_u __attribute__((aligned(1)));

template <int NT>
__device__ __forceinline__ u32x4 ld16u(const void* p) {
  if (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_u*>(p));
  return *reinterpret_cast<const u32x4_u*>(p);
}
template <int NT>
__device__ __forceinline__ void st16u(void* p, u32x4 v) {
  if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_u*>(p));
  else *reinterpret_cast<u32x4_u*>(p) = v;
}
template <int NT>
__device__ __forceinline__ void st8u(void* p, u32x2 v) {
  if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_u*>(p));
  else *reinterpret_cast<u32x2_u*>(p) = v;
}

template <int NT>
__device__ __forceinline__ void st4u(void* p, uint32_t v) {
  if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32_u*>(p));
  else *reinterpret_cast<u32_u*>(p) = v;
}

// Two FP32 values -> two BF16 values in one dword, round to nearest even (the
// conversion instruction; a NaN stays a NaN).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Row element types.  A lane holds 8 columns of a 128-column group as runs of
// 16 bytes: one of 8 BF16 columns, or two of 4 FP32 columns 64 apart, so that
// 16 lanes always access a contiguous 256 bytes (FP32 pieces of 8 neighbouring
// columns made every store instruction write half of each 32 bytes, which
// halved the rate of stores past the caches).  Raw is the runs as loaded;
// unpack widens them to FP32, pack rounds them to the type.
struct RowBF16 {
  typedef uint16_t elem;
  static constexpr int kRuns = 1, kLen = 8;
  struct Raw { u32x4 a[kRuns]; };
  __device__ __forceinline__ static void unpack(const Raw& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.a[0][i] << 16);
      v[2 * i + 1] = __uint_as_float(r.a[0][i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static Raw pack(const float v[8]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[0][i] = pack2_bf16(v[2 * i], v[2 * i + 1]);
    return r;
  }
  // The largest magnitude as FP32 bits (a NaN is larger than all).
  __device__ __forceinline__ static uint32_t max_bits(const Raw& r) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = __builtin_bit_cast(u16x2, r.a[0][0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.a[0][i] & 0x7FFF7FFFu));
    return (uint32_t)max(m[0], m[1]) << 16;
  }
  __device__ __forceinline__ static float load1(const elem* p) { return bf16_to_f32(*p); }
};

struct RowF32 {
  typedef float elem;
  static constexpr int kRuns = 2, kLen = 4;
  struct Raw { u32x4 a[kRuns]; };
  __device__ __forceinline__ static void unpack(const Raw& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.a[i >> 2][i & 3]);
  }
  __device__ __forceinline__ static Raw pack(const float v[8]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.a[i >> 2][i & 3] = __float_as_uint(v[i]);
    return r;
  }
  __device__ __forceinline__ static uint32_t max_bits(const Raw& r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, r.a[i >> 2][i & 3] & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ static float load1(const elem* p) { return *p; }
};

// True if no lane of the wave has a run that column `end` cuts or that lies
// between it and the row's end; end is the row's end, or that of its last whole
// 64 columns.  Then the wave's runs are inside or outside as a whole.  The
// branch on it is uniform, so loads and stores inside carry no masks of single
// columns.
template <class Row>
__device__ __forceinline__ bool no_cut(int c0, int end, int cols) {
  bool ok = true;
#pragma unroll
  for (int r = 0; r < Row::kRuns; ++r) {
    const int cr = c0 + 64 * r;
    ok = ok && (cr + Row::kLen <= end || cr >= cols);
  }
  return __all(ok);
}

// v >> bits of a 128-bit number; bits a multiple of 16, 128 and more give 0.
__device__ __forceinline__ u32x4 shift_right(u32x4 v, int bits) {
  const int w = bits >> 5;
  v = (w & 1) ? u32x4{v[1], v[2], v[3], 0u} : v;
  v = (w & 2) ? u32x4{v[2], v[3], 0u, 0u} : v;
  v = w >= 4 ? u32x4{0u, 0u, 0u, 0u} : v;
  return u32x4{__builtin_amdgcn_alignbit(v[1], v[0], bits & 16), __builtin_amdgcn_alignbit(v[2], v[1], bits & 16),
               __builtin_amdgcn_alignbit(v[3], v[2], bits & 16), v[3] >> (bits & 16)};
}

// A lane's runs from column c0, zeros past the row's end.  WHOLE: no_cut
// holds; a run outside reads the row's last columns (of the same group), and
// its lane drops it.  Otherwise a run that the end cuts or that lies past it
// reads the row's last columns and shifts them into place, so that no lane
// loads single columns (800 columns of 65645 BF16 rows combined in 24 us: 799
// took 60 us that way).  TINY: the row may be shorter than a run.
template <class Row, bool WHOLE, bool TINY, int NT>
__device__ __forceinline__ typename Row::Raw load_piece(const typename Row::elem* p, int c0, int cols) {
  typename Row::Raw raw;
#pragma unroll
  for (int r = 0; r < Row::kRuns; ++r) {
    const int cr = c0 + 64 * r;
    if (!WHOLE && TINY && cols < Row::kLen) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < Row::kLen && cr + e < cols ? Row::load1(p + cr + e) : 0.f;
      raw.a[r] = Row::pack(v).a[0];
    } else {
      const int at = min(cr, cols - Row::kLen);
      raw.a[r] = ld16u<NT>(p + at);
      if (!WHOLE) raw.a[r] = shift_right(raw.a[r], (cr - at) * (8 * (int)sizeof(typename Row::elem)));
    }
  }
  return raw;
}

// The first n bytes of v, n below 16 (a multiple of 2).
__device__ __forceinline__ void store_bytes(void* to, u32x4 v, int n) {
  uint8_t* p = reinterpret_cast<uint8_t*>(to);
  if (n & 8) {
    st8u<0>(p, u32x2{v[0], v[1]});
    p += 8;
    v[0] = v[2];
    v[1] = v[3];
  }
  if (n & 4) {
    st4u<0>(p, v[0]);
    p += 4;
    v[0] = v[1];
  }
  if (n & 2) *reinterpret_cast<u16_u*>(p) = (uint16_t)v[0];
}

// NT: past the caches, for whole pieces only.
template <class Row, bool WHOLE, int NT>
__device__ __forceinline__ void store_piece(typename Row::elem* p, int c0, int cols, const typename Row::Raw& raw) {
#pragma unroll
  for (int r = 0; r < Row::kRuns; ++r) {
    const int cr = c0 + 64 * r;
    if (WHOLE ? cr < cols : cr + Row::kLen <= cols)
      st16u<WHOLE && NT>(p + cr, raw.a[r]);
    else if (!WHOLE && cr < cols)
      store_bytes(p + cr, raw.a[r], (cols - cr) * (int)sizeof(typename Row::elem));
  }
}

// The codes of a lane's 8 columns (two dwords) to a code row.
template <class Row, bool WHOLE, int NT>
__device__ __forceinline__ void store_codes(uint8_t* p, int c0, int cols, uint32_t w0, uint32_t w1) {
#pragma unroll
  for (int r = 0; r < Row::kRuns; ++r) {
    const int cr = c0 + 64 * r;
    uint32_t w = r == 0 ? w0 : w1;
    if (WHOLE ? cr < cols : cr + Row::kLen <= cols) {
      if (Row::kRuns == 1) st8u<WHOLE && NT>(p + cr, u32x2{w0, w1});
      else st4u<WHOLE && NT>(p + cr, w);
    } else if (!WHOLE && cr < cols) {
      const int n = cols - cr;
      uint8_t* q = p + cr;
      if (Row::kRuns == 1 && (n & 4)) {
        st4u<0>(q, w);
        q += 4;
        w = w1;
      }
      if (n & 2) {
        *reinterpret_cast<u16_u*>(q) = (uint16_t)w;
        q += 2;
        w >>= 16;
      }
      if (n & 1) *q = (uint8_t)w;
    }
  }
}

}  // namespace fp8q
