// Row access shared by the MoE row kernels and gradient clipping: 8 elements
// of a row as 16-byte accesses at ANY element alignment.  gfx950 global
// memory instructions take multi-dword accesses at any byte address, so rows
// whose length is odd use the same instructions as aligned ones; only the
// alignment the compiler may assume differs.
#pragma once

#include "device_common.h"

namespace fp8q {

typedef u32x4 u32x4_u __attribute__((aligned(1)));
typedef u32x2 u32x2_u __attribute__((aligned(1)));

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

// Two FP32 values -> two BF16 values in one dword, round to nearest even (the
// conversion instruction; a NaN stays a NaN).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Row element types.  Raw is 8 elements as loaded; unpack widens them to
// FP32, pack rounds them to the type.
struct RowBF16 {
  typedef uint16_t elem;
  struct Raw { u32x4 a; };
  template <int NT = 0>
  __device__ __forceinline__ static Raw load8(const elem* p) { return Raw{ld16u<NT>(p)}; }
  __device__ __forceinline__ static void unpack(const Raw& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.a[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static Raw pack(const float v[8]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = pack2_bf16(v[2 * i], v[2 * i + 1]);
    return r;
  }
  template <int NT = 0>
  __device__ __forceinline__ static void store8(elem* p, const Raw& r) { st16u<NT>(p, r.a); }
  __device__ __forceinline__ static float load1(const elem* p) { return bf16_to_f32(*p); }
  __device__ __forceinline__ static void store1(elem* p, float v) { *p = (elem)pack2_bf16(v, 0.f); }
};

struct RowF32 {
  typedef float elem;
  struct Raw { u32x4 a, b; };
  template <int NT = 0>
  __device__ __forceinline__ static Raw load8(const elem* p) { return Raw{ld16u<NT>(p), ld16u<NT>(p + 4)}; }
  __device__ __forceinline__ static void unpack(const Raw& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(r.a[i]);
      v[4 + i] = __uint_as_float(r.b[i]);
    }
  }
  __device__ __forceinline__ static Raw pack(const float v[8]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = __float_as_uint(v[i]);
      r.b[i] = __float_as_uint(v[4 + i]);
    }
    return r;
  }
  template <int NT = 0>
  __device__ __forceinline__ static void store8(elem* p, const Raw& r) {
    st16u<NT>(p, r.a);
    st16u<NT>(p + 4, r.b);
  }
  __device__ __forceinline__ static float load1(const elem* p) { return *p; }
  __device__ __forceinline__ static void store1(elem* p, float v) { *p = v; }
};

// 8 elements from column c0 of a row of `cols`, zeros past its end.
template <class Row, int NT = 0>
__device__ __forceinline__ void load_cols(const typename Row::elem* p, int c0, int cols, float v[8]) {
  if (c0 + 8 <= cols) {
    Row::unpack(Row::template load8<NT>(p + c0), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < cols ? Row::load1(p + c0 + e) : 0.f;
  }
}

template <class Row, int NT = 0>
__device__ __forceinline__ void store_cols(typename Row::elem* p, int c0, int cols, const float v[8]) {
  if (c0 + 8 <= cols) {
    Row::template store8<NT>(p + c0, Row::pack(v));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < cols) Row::store1(p + c0 + e, v[e]);
  }
}

// 8 codes (two dwords) to column c0 of a code row of `cols`.
template <int NT = 0>
__device__ __forceinline__ void store_codes(uint8_t* p, int c0, int cols, uint32_t w0, uint32_t w1) {
  if (c0 + 8 <= cols) {
    st8u<NT>(p + c0, u32x2{w0, w1});
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < cols) p[c0 + e] = (uint8_t)(((e < 4 ? w0 : w1) >> (8 * (e & 3))) & 0xFF);
  }
}

}  // namespace fp8q
