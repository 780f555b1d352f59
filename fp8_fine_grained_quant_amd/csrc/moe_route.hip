// The router of an MoE layer: the k best experts of every token, their
// weights, and the gradient to the logits (gfx950).
//
// Scores are softmax(logits) or sigmoid(logits); an expert whose logit is -inf
// is masked for that token.  Without a bias the logits decide (both scores
// grow with them), with one the score plus the bias does, in 64 bits: two
// experts' sums may differ by less than FP32 resolves, and the choice must not
// depend on how a score was rounded.  Equal keys go to the lower expert.
//
// Up to kShort choices: 16 lanes (8 for up to 64 experts) work on a token, 8
// experts at a time each.  A key and its expert make one unique number, held
// as a double, since an FP64 maximum and minimum are one instruction each: a
// lane sorts its 8 by a network, merges them into its 8 largest so far, and
// the lanes' lists merge over DPP steps.  More choices: a wave per token; each
// lane sorts its own keys once, and each choice is the largest of the lanes'
// first keys, which its lane drops (16384 tokens, 256 experts, no bias: 7.4 us
// the first way, 11.3 the second).  Both are bound by these instructions, not
// by the logits' bytes.
//
// With a bias the keys are formed in FP32, and only a token where two of its
// first k + 1 are too close to be told apart takes them to 64 bits (16384
// tokens of 256 FP32 logits, 8 choices, biases of normal distribution: 12.8 us;
// 41.8 with every key in 64 bits).  Equal keys are too close by definition, so
// the time depends on how many there are: of BF16 logits with such a bias 0.1 %
// of the tokens have some and take 11 us, with a bias of zeros 34 % and 17 us,
// with all logits equal every token and 47 us.

#include "device_common.h"
#include "launch.h"
#include "row_io.h"

#include <math.h>

#include <type_traits>

namespace fp8q {

namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr int kRouteThreads = 256;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u));
}

// Step i of a token's lanes meeting each other: after the steps every lane has
// met all G, each once.  16 lanes: rotations by 8, 4, 2, 1; 8 lanes: mirrored,
// then by exchanges of neighbours and of pairs.
template <int G, int I, class T>
__device__ __forceinline__ T meet(T v) {
  constexpr int kCtrl16[4] = {0x128, 0x124, 0x122, 0x121}, kCtrl8[3] = {0x141, 0xB1, 0x4E};
  return dpp<G == 8 ? kCtrl8[I % 3] : kCtrl16[I]>(v);
}

// Sum and maximum over a token's G lanes; the same bits in every lane.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += meet<G, 0>(v);
  v += meet<G, 1>(v);
  v += meet<G, 2>(v);
  if (G >= 16) v += meet<G, 3>(v);
  if (G == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// G == 64: the rows' maxima travel up by row broadcasts to the last lane.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, meet<G, 0>(v));
  v = max(v, meet<G, 1>(v));
  v = max(v, meet<G, 2>(v));
  if (G >= 16) v = max(v, meet<G, 3>(v));
  if (G == 64) {
    v = max(v, dpp<0x142>(v));
    v = max(v, dpp<0x143>(v));
    v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
  return v;
}

// Keys as unsigned integers in the same order (both zeros the same); 0 for what
// is never chosen: a masked expert, a NaN.  Integers, since their maximum is
// one DPP instruction, where FP32's carries a NaN rule.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const int u = __float_as_int(v + 0.f);
  return v > -kInf ? (uint32_t)(u ^ ((u >> 31) | (int)0x80000000)) : 0u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return u == 0 ? -kInf : __int_as_float((int)u < 0 ? (int)u ^ (int)0x80000000 : ~(int)u);
}

// The largest of a token's values, -inf if there is none (a NaN is none).
template <int G>
__device__ __forceinline__ float group_max(float v) { return order_value(group_max<G>(order_bits(v))); }

// What the wave's lanes wrote to LDS is seen by all of them, in this order.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// True for the lanes whose token has a lane where `p` holds.
template <int G>
__device__ __forceinline__ bool group_any(bool p) {
  const uint64_t all = __ballot(p);
  return G == 64 ? all != 0 : ((all >> (threadIdx.x & (64 - G))) & ((1 << (G & 31)) - 1)) != 0;
}

// exp of a value that is not positive: 1 + exp(-x) would overflow, and the
// score with it vanish, long before the score leaves FP32.
__device__ __forceinline__ float sigmoid(float x) {
  const float z = expf(-__builtin_fabsf(x));
  return (x < 0.f ? z : 1.f) / (1.f + z);
}

// The same within 4 units of 2^-24, with hardware exp2 and reciprocal (1 ulp
// each): the exponent's rounding and exp2 bring at most 0.7, the sum and the
// reciprocal 1 each, the product 0.5.
__device__ __forceinline__ float sigmoid_near(float x) {
  const float z = __builtin_amdgcn_exp2f(-__builtin_fabsf(x) * 1.44269504f);
  const float r = __builtin_amdgcn_rcpf(1.f + z);
  return x < 0.f ? z * r : r;
}

// A chosen score up to a factor common to the token's choices, for weights
// that are divided by their sum: score / e^c with c the largest chosen logit
// (for sigmoids at most 0), so that scores which vanish in FP32 keep their
// ratio.  `top` is the largest chosen logit.
template <bool SIG>
__device__ __forceinline__ float scaled_score(float x, float top) {
  if (!SIG) return expf(x - top);
  return x < 0.f ? expf(x - __builtin_fminf(top, 0.f)) / (1.f + expf(x)) : sigmoid(x);
}

struct LogitBF16 {
  typedef uint16_t elem;
  __device__ __forceinline__ static float load(const elem* p) { return bf16_to_f32(*p); }
  __device__ __forceinline__ static void store(elem* p, float v) { *p = (elem)pack2_bf16(v, 0.f); }
  __device__ __forceinline__ static void load4(const elem* p, float* v) {
    const u32x2 u = *reinterpret_cast<const u32x2_u*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static void store4(elem* p, const float* v) {
    st8u<0>(p, u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])});
  }
};
struct LogitF32 {
  typedef float elem;
  __device__ __forceinline__ static float load(const elem* p) { return *p; }
  __device__ __forceinline__ static void store(elem* p, float v) { *p = v; }
  __device__ __forceinline__ static void load4(const elem* p, float* v) {
    const u32x4 u = ld16u<0>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  }
  __device__ __forceinline__ static void store4(elem* p, const float* v) {
    st16u<0>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
  }
};

// The V entries from `first` of a row of e, `none` past its end.
template <class L, int V>
__device__ __forceinline__ void load_experts(const typename L::elem* p, int first, int e, float none, float x[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (first + i + 4 <= e) {
      L::load4(p + first + i, x + i);
    } else {
#pragma unroll
      for (int u = i; u < i + 4; ++u) x[u] = first + u < e ? L::load(p + first + u) : none;
    }
  }
}

// Score + bias in FP32, -inf for a masked expert or a NaN.  top, inv: the
// largest logit and 1 / sum of a softmax.
template <bool SIG>
__device__ __forceinline__ float near_key(float x, float b, float top, float inv) {
  const float s = SIG ? sigmoid_near(x) : expf(x - top) * inv;
  const float key = s + b;
  return x > -kInf ? key : -kInf;
}
// How far apart two such keys have to be for their order to be the true one,
// where the one is `key`.  A sigmoid is off by at most 4 units of 2^-24, a
// softmax by 2^-17 of itself (the sum of up to 1024 terms; no score is above
// inv), a key by 2^-24 of itself besides.
template <bool SIG>
__device__ __forceinline__ float key_tol(float key, float inv) {
  return (SIG ? 0x1p-20f : 0x1p-16f * inv) + 0x1p-22f * __builtin_fabsf(key);
}

constexpr int kNear = 64;  // experts that FP32 may leave undecided: a lane each

// The choice by score + bias in 64 bits, for a token where FP32 cannot tell the
// order; the whole wave works on it, and its lane j returns choice j, or -1.
// kth is the k-th largest FP32 key: only experts within the tolerance of it or
// above it can be chosen.  Up to kNear of them get a lane each, which counts
// the larger ones; more (many equal keys) are chosen one after the other.
// list: kNear ints of LDS of the wave's own.
template <class L, int V, bool SIG>
__device__ __forceinline__ int choose64(const typename L::elem* p, const float* bias, int e, int k, float top,
                                        float inv, float kth, int* list) {
  const int lane = threadIdx.x & 63, first = lane * V;
  float x[V], b[V];
  load_experts<L, V>(p, first, e, -kInf, x);
  load_experts<LogitF32, V>(bias, first, e, 0.f, b);
  const float least = kth - key_tol<SIG>(kth, inv);
  double total = 1.0;
  if (!SIG) {
    total = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) total += x[i] > -kInf ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  }
  auto key64 = [&](float xi, float bi) {
    const double s = SIG ? 1.0 / (1.0 + exp(-(double)xi)) : exp((double)xi - (double)top) / total;
    return xi > -kInf ? s + (double)bi : -(double)kInf;
  };
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool on = near_key<SIG>(x[i], b[i], top, inv) >= least && x[i] > -kInf;
    const uint64_t all = __ballot(on);
    const int at = n + __popcll(all & ((1ull << lane) - 1));
    if (on && at < kNear) list[at] = first + i;
    n += __popcll(all);
  }
  wave_fence();
  if (n <= kNear) {
    const int id = lane < n ? list[lane] : -1;
    const double key = id < 0 ? -(double)kInf : key64(L::load(p + id), bias[id]);
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, j);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), j);
      const double other = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
      rank += other > key || (other == key && __builtin_amdgcn_readlane(id, j) < id);
    }
    wave_fence();
    list[lane] = -1;
    wave_fence();
    if (id >= 0 && rank < kNear) list[rank] = id;
    wave_fence();
    const int got = list[lane];
    wave_fence();
    return got;
  }
  double key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = key64(x[i], b[i]);
  int id = -1;
  for (int j = 0; j < k; ++j) {
    double best = -(double)kInf;
    int at = -1;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = first + i;
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double ob = __shfl_xor(best, o);
      const int oa = __shfl_xor(at, o);
      if (ob > best || (ob == best && oa >= 0 && (at < 0 || oa < at))) {
        best = ob;
        at = oa;
      }
    }
    if (lane == j) id = at;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (first + i == at) key[i] = -(double)kInf;
  }
  return id;
}

// A lane's keys in descending order, equal ones in theirs: pass A carries the
// largest of the entries from A on up to A.
template <int V, int A = 0>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[V], int (&loc)[V]) {
  if constexpr (A + 1 < V) {
#pragma unroll
    for (int i = V - 1; i > A; --i) {
      const uint32_t k0 = key[i - 1], k1 = key[i];
      const int l0 = loc[i - 1], l1 = loc[i];
      const bool up = k1 > k0;
      key[i - 1] = max(k0, k1);
      key[i] = min(k0, k1);
      loc[i - 1] = up ? l1 : l0;
      loc[i] = up ? l0 : l1;
    }
    sort_lane<V, A + 1>(key, loc);
  }
}

// The weight of this lane's choice from the largest logit `top` and the sum
// `total` of a token's softmax, and the store of both.
template <class L, int G, bool SIG>
__device__ __forceinline__ void finish(const typename L::elem* p, int id, float top, float total, int renorm,
                                       float scale, bool store, int64_t at, int* __restrict__ ids,
                                       float* __restrict__ w) {
  const float x = id < 0 ? -kInf : L::load(p + id);
  float s = 0.f;
  if (renorm) {
    top = group_max<G>(x);
    s = id < 0 ? 0.f : scaled_score<SIG>(x, top);
    total = group_sum<G>(s);
  } else if (id >= 0) {
    s = SIG ? sigmoid(x) : expf(x - top);
  }
  const float out = id < 0 ? 0.f : SIG && !renorm ? s : s / total;
  if (store) {
    ids[at] = id;
    w[at] = out * scale;
  }
}

// Eight descending keys.
constexpr int kShort = 8;
struct Short {
  double v[kShort];

  template <int A, int B>
  __device__ __forceinline__ void order() {
    const double a = v[A], b = v[B];
    v[A] = __builtin_fmax(a, b);
    v[B] = __builtin_fmin(a, b);
  }
  __device__ __forceinline__ void sort() {
    order<0, 2>(); order<1, 3>(); order<4, 6>(); order<5, 7>();
    order<0, 4>(); order<1, 5>(); order<2, 6>(); order<3, 7>();
    order<0, 1>(); order<2, 3>(); order<4, 5>(); order<6, 7>();
    order<2, 4>(); order<3, 5>();
    order<1, 4>(); order<3, 6>();
    order<1, 2>(); order<3, 4>(); order<5, 6>();
  }
  // The largest 8 of both lists; `left` (REST) becomes the high half of the
  // largest key that any merge left out.
  template <bool REST>
  __device__ __forceinline__ void merge(const Short& o, uint32_t& left) {
#pragma unroll
    for (int i = 0; i < kShort; ++i) {
      const double a = v[i], b = o.v[kShort - 1 - i];
      if (REST) left = max(left, min(high(a), high(b)));
      v[i] = __builtin_fmax(a, b);
    }
    order<0, 4>(); order<1, 5>(); order<2, 6>(); order<3, 7>();
    order<0, 2>(); order<1, 3>(); order<4, 6>(); order<5, 7>();
    order<0, 1>(); order<2, 3>(); order<4, 5>(); order<6, 7>();
  }
  template <int G, int I, bool REST>
  __device__ __forceinline__ void meet_merge(uint32_t& left) {
    Short o;
#pragma unroll
    for (int i = 0; i < kShort; ++i) o.v[i] = meet<G, I>(v[i]);
    if (REST) left = max(left, meet<G, I>(left));
    merge<REST>(o, left);
  }

  __device__ __forceinline__ static uint32_t high(double d) {
    return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 32);
  }
  __device__ __forceinline__ static uint32_t key(double d) {
    return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 30);
  }
  // Key bits, then the expert's complement (the lower expert is the larger
  // number): finite, not negative and different from each other.
  __device__ __forceinline__ static double make(uint32_t key, int expert) {
    return __builtin_bit_cast(double, (uint64_t)(key >> 2) << 32 | (uint32_t)(key << 30 | (0x3FFFFFFF - expert)));
  }
};

// CHUNKS: how often a lane takes 8 experts, its logits then in registers; 0: any
// number of times, its logits read again for each use.  V64: experts per lane
// where the whole wave takes one token.
template <class L, int G, int CHUNKS, int V64, bool SIG, bool BIAS>
__global__ __launch_bounds__(kRouteThreads) void k_route_short(const typename L::elem* __restrict__ logits,
                                                               int64_t ld, const float* __restrict__ bias,
                                                               int tokens, int e, int k, int renorm, float scale,
                                                               int* __restrict__ ids, float* __restrict__ w) {
  const int gl = threadIdx.x & (G - 1);
  const int mine = (int)(blockIdx.x * (kRouteThreads / G) + threadIdx.x / G);
  // a wave's lanes stay together: tokens past the end repeat the last one
  const int t = min(mine, tokens - 1);
  const typename L::elem* p = logits + (int64_t)t * ld;
  float held[CHUNKS > 0 ? CHUNKS : 1][8], held_bias[CHUNKS > 0 ? CHUNKS : 1][8];
  if (CHUNKS > 0) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      load_experts<L, 8>(p, (c * G + gl) * 8, e, -kInf, held[c]);
      if (BIAS) load_experts<LogitF32, 8>(bias, (c * G + gl) * 8, e, 0.f, held_bias[c]);
    }
  }
  // f(first expert, its 8 logits, a chunk's number) for every chunk
  auto each_chunk = [&](auto f) {
    if (CHUNKS > 0) {
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) f((c * G + gl) * 8, held[c], held_bias[c], c);
    } else {
      for (int c = 0; c * G * 8 < e; ++c) {
        float x[8], b[8];
        load_experts<L, 8>(p, (c * G + gl) * 8, e, -kInf, x);
        if (BIAS) load_experts<LogitF32, 8>(bias, (c * G + gl) * 8, e, 0.f, b);
        f((c * G + gl) * 8, x, b, c);
      }
    }
  };
  float top = -kInf, total = 1.f, inv = 1.f;
  if (!SIG && (BIAS || !renorm)) {
    bool nan = false;
    each_chunk([&](int, const float (&x)[8], const float (&)[8], int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top = __builtin_fmaxf(top, x[i]);
        nan |= x[i] != x[i];
      }
    });
    top = group_max<G>(top);
    total = 0.f;
    each_chunk([&](int, const float (&x)[8], const float (&)[8], int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) total += x[i] > -kInf ? expf(x[i] - top) : 0.f;
    });
    total = group_sum<G>(total);
    inv = __builtin_amdgcn_rcpf(total);
    if (group_any<G>(nan)) total = __builtin_nanf("");
  }
  Short best;
  uint32_t left = 0;
  each_chunk([&](int first, const float (&x)[8], const float (&b)[8], int c) {
    Short some;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float key = BIAS ? near_key<SIG>(x[i], b[i], top, inv) : x[i];
      some.v[i] = Short::make(order_bits(key), first + i);
    }
    some.sort();
    if (c == 0) best = some;
    else best.merge<BIAS>(some, left);
  });
  best.meet_merge<G, 0, BIAS>(left);
  best.meet_merge<G, 1, BIAS>(left);
  best.meet_merge<G, 2, BIAS>(left);
  if (G == 16) best.meet_merge<G, 3, BIAS>(left);
  double pick = best.v[0];
#pragma unroll
  for (int i = 1; i < kShort; ++i) {
    const double v = best.v[i];
    pick = gl == i ? v : pick;
  }
  const uint32_t hi = Short::high(pick);
  int id = hi == 0 || gl >= k ? -1 : 0x3FFFFFFF - (int)((uint32_t)__builtin_bit_cast(uint64_t, pick) & 0x3FFFFFFF);
  if (BIAS) {
    __shared__ int lists[kRouteThreads];
    const float key = order_value(Short::key(pick));
    const float next = gl == kShort - 1 ? order_value(left << 2 | 3) : dpp<0x101>(key);
    uint64_t near = __ballot(gl < k && key - next <= key_tol<SIG>(key, inv));
    while (near != 0) {  // one token after the other
      const int lane0 = __builtin_ctzll(near) & ~(G - 1);
      near &= ~(((1ull << G) - 1) << lane0);
      auto of = [&](float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
      const int at = choose64<L, V64, SIG>(logits + (int64_t)__builtin_amdgcn_readlane(t, lane0) * ld, bias, e, k,
                                           of(top, lane0), of(inv, lane0), of(key, lane0 + k - 1),
                                           lists + (threadIdx.x & ~63));
      const int mine64 = __shfl(at, gl);
      if ((int)(threadIdx.x & (64 - G)) == lane0) id = gl < k ? mine64 : -1;
    }
  }
  finish<L, G, SIG>(p, id, top, total, renorm, scale, gl < k && mine < tokens, (int64_t)t * k + gl, ids, w);
}

// More than kShort choices: a wave per token, lane j keeps choice j.
template <class L, int V, bool SIG, bool BIAS>
__global__ __launch_bounds__(kRouteThreads) void k_route(const typename L::elem* __restrict__ logits, int64_t ld,
                                                         const float* __restrict__ bias, int tokens, int e, int k,
                                                         int renorm, float scale, int* __restrict__ ids,
                                                         float* __restrict__ w) {
  constexpr int G = 64;
  const int gl = threadIdx.x & 63;
  const int t = (int)(blockIdx.x * (kRouteThreads / G) + threadIdx.x / G);
  if (t >= tokens) return;
  const typename L::elem* p = logits + (int64_t)t * ld;
  float x[V], b[V];
  load_experts<L, V>(p, gl * V, e, -kInf, x);
  if (BIAS) load_experts<LogitF32, V>(bias, gl * V, e, 0.f, b);
  float top = -kInf, total = 1.f, inv = 1.f;
  if (!SIG && (BIAS || !renorm)) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      top = __builtin_fmaxf(top, x[i]);
      nan |= x[i] != x[i];
    }
    top = group_max<G>(top);
    total = 0.f;
    float ex[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = x[i] > -kInf ? expf(x[i] - top) : 0.f;
      total += ex[i];
    }
    total = group_sum<G>(total);
    if (BIAS) {
      inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = near_key<SIG>(x[i], b[i], top, inv);
    }
    if (group_any<G>(nan)) total = __builtin_nanf("");
  }
  if (SIG && BIAS) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = near_key<SIG>(x[i], b[i], top, inv);
  }
  uint32_t key[V];
  int loc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = order_bits(x[i]);
    loc[i] = gl * V + i;
  }
  sort_lane<V>(key, loc);
  int my_id = -1;
  uint32_t my_key = 0;
  // with a bias one choice more, to see how close it came
  for (int j = 0; j < k + (BIAS ? 1 : 0); ++j) {
    const uint32_t best = group_max<G>(key[0]);
    if (best == 0) break;
    const int at = __builtin_amdgcn_readlane(loc[0], __builtin_ctzll(__ballot(key[0] == best)));
    if (gl == j) {
      my_id = at;
      my_key = best;
    }
    const bool drop = at == loc[0];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t k0 = key[i], k1 = i + 1 < V ? +key[i + 1] : 0u;
      const int l0 = loc[i], l1 = i + 1 < V ? +loc[i + 1] : l0;
      key[i] = drop ? k1 : k0;
      loc[i] = drop ? l1 : l0;
    }
  }
  if (BIAS) {
    __shared__ int lists[kRouteThreads];
    const float key0 = order_value(my_key), key1 = __shfl_down(key0, 1);
    if (__any(gl < k && key0 - key1 <= key_tol<SIG>(key0, inv)))
      my_id = choose64<L, V, SIG>(p, bias, e, k, top, inv,
                                  __int_as_float(__builtin_amdgcn_readlane(__float_as_int(key0), k - 1)),
                                  lists + (threadIdx.x & ~63));
  }
  finish<L, G, SIG>(p, gl < k ? my_id : -1, top, total, renorm, scale, gl < k, (int64_t)t * k + gl, ids, w);
}

// Lane j of a token computes what choice j needs; the few chosen entries find
// their experts' lanes through the wave's own part of LDS.  Only softmax
// without renormalization has a gradient to every expert.
template <class L, int G, int V, bool SIG>
__global__ __launch_bounds__(kRouteThreads) void k_route_bwd(const float* __restrict__ dw,
                                                             const typename L::elem* __restrict__ logits, int64_t ld,
                                                             const int* __restrict__ ids, int tokens, int e, int k,
                                                             int renorm, float scale,
                                                             typename L::elem* __restrict__ dl, int64_t ld_dl) {
  __shared__ float rows[kRouteThreads * V];
  const int gl = threadIdx.x & (G - 1);
  const int mine = (int)(blockIdx.x * (kRouteThreads / G) + threadIdx.x / G), t = min(mine, tokens - 1);
  float* const r = rows + (threadIdx.x / G) * (G * V);
  const typename L::elem* p = logits + (int64_t)t * ld;
  const bool dense = !SIG && !renorm;
  int id = -1;
  float x = -kInf, g = 0.f;
  if (gl < k) {
    id = ids[(int64_t)t * k + gl];
    g = dw[(int64_t)t * k + gl] * scale;
  }
  float xs[V];
  if (dense) load_experts<L, V>(p, gl * V, e, -kInf, xs);
  if ((uint32_t)id < (uint32_t)e) x = L::load(p + id);
  if (x == -kInf) {  // no choice, or a masked expert: no gradient
    id = -1;
    g = 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) r[gl * V + i] = 0.f;
  wave_fence();
  float top = x, total = 0.f, ex[V];
  if (dense) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, xs[i]);
  }
  top = group_max<G>(top);
  if (dense) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = xs[i] == -kInf ? 0.f : expf(xs[i] - top);
      total += ex[i];
    }
  }
  float s = 0.f;
  if (id >= 0) s = SIG && !renorm ? sigmoid(x) : scaled_score<SIG>(x, top);
  total = dense ? group_sum<G>(total) : renorm ? group_sum<G>(s) : 1.f;
  const float wj = id < 0 ? 0.f : s / total;  // the weight before `scale`
  const float mean = group_sum<G>(g * wj);
  float d;
  if (SIG) {
    const float rest = sigmoid(-x);  // 1 - s without cancellation
    d = renorm ? (g - mean) * wj * rest : g * s * rest;
  } else {
    d = dense ? g : (g - mean) * wj;
  }
  if (id >= 0) r[id] = d;
  wave_fence();
  if (mine >= tokens) return;
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    out[i] = r[gl * V + i];
    if (dense) out[i] = xs[i] == -kInf ? 0.f : ex[i] / total * (out[i] - mean);
  }
  typename L::elem* o = dl + (int64_t)t * ld_dl;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const int at = gl * V + i;
    if (at + 4 <= e) {
      L::store4(o + at, out + i);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at + u < e) L::store(o + at + u, out[i + u]);
    }
  }
}

using I4 = std::integral_constant<int, 4>;
using I8 = std::integral_constant<int, 8>;
using I16 = std::integral_constant<int, 16>;
using I64 = std::integral_constant<int, 64>;

// f(lanes per token, experts per lane) of the gradient.  Up to 128 experts a
// row of 16 lanes holds a token (it needs a lane for each choice).
template <class F>
void with_layout(const MoeRoute& a, F f) {
  if (a.k <= 16 && a.experts <= 64) f(I16{}, I4{});
  else if (a.k <= 16 && a.experts <= 128) f(I16{}, I8{});
  else if (a.experts <= 256) f(I64{}, I4{});
  else if (a.experts <= 512) f(I64{}, I8{});
  else f(I64{}, I16{});
}
template <class F>
void with_flag(bool v, F f) {
  if (v) f(std::true_type{}); else f(std::false_type{});
}
template <class F>
void with_logits(bool bf16, F f) {
  if (bf16) f(LogitBF16{}); else f(LogitF32{});
}
dim3 route_grid(int64_t tokens, int lanes) {
  const int per_block = kRouteThreads / lanes;
  return dim3((uint32_t)((tokens + per_block - 1) / per_block));
}

}  // namespace

hipError_t launch_moe_route(const MoeRoute& a, const float* bias, int32_t* ids, float* w, hipStream_t st) {
  hipError_t err = hipSuccess;
  with_logits(a.bf16, [&](auto l) {
    typedef decltype(l) L;
    with_flag(a.sigmoid, [&](auto sig) {
      with_flag(bias != nullptr, [&](auto bi) {
        auto go = [&](auto kernel, int lanes) {
          err = launch_in_parts(a.tokens, lanes, [&](int64_t t, int64_t n) {
            hipLaunchKernelGGL(kernel, route_grid(n, lanes), dim3(kRouteThreads), 0, st,
                               (const typename L::elem*)a.logits + t * a.ld, a.ld, bias, (int)n, (int)a.experts,
                               (int)a.k, (int)a.renorm, a.scale, ids + t * a.k, w + t * a.k);
          });
        };
        if (a.k <= kShort) {
          // A softmax uses its logits three times: held in registers, 177 tokens of
          // 161 experts take 6.8 us, read again 8.9.  A sigmoid uses them once.
          constexpr int kTwo = decltype(sig)::value ? 0 : 2;
          if (a.experts <= 64) go(k_route_short<L, 8, 1, 4, sig.value, bi.value>, 8);
          else if (a.experts <= 128) go(k_route_short<L, 16, 1, 4, sig.value, bi.value>, 16);
          else if (a.experts <= 256) go(k_route_short<L, 16, kTwo, 4, sig.value, bi.value>, 16);
          else go(k_route_short<L, 16, 0, kMaxExperts / 64, sig.value, bi.value>, 16);
        } else {
          if (a.experts <= 256) go(k_route<L, 4, sig.value, bi.value>, 64);
          else go(k_route<L, 16, sig.value, bi.value>, 64);
        }
      });
    });
  });
  return err;
}

hipError_t launch_moe_route_bwd(const MoeRoute& a, const float* dw, const int32_t* ids, void* dl, int64_t ld_dl,
                                hipStream_t st) {
  hipError_t err = hipSuccess;
  with_logits(a.bf16, [&](auto l) {
    typedef decltype(l) L;
    typedef typename L::elem E;
    with_layout(a, [&](auto lanes, auto v) {
      with_flag(a.sigmoid, [&](auto sig) {
        err = launch_in_parts(a.tokens, lanes.value, [&](int64_t t, int64_t n) {
          hipLaunchKernelGGL((k_route_bwd<L, lanes.value, v.value, sig.value>), route_grid(n, lanes.value),
                             dim3(kRouteThreads), 0, st, dw + t * a.k, (const E*)a.logits + t * a.ld, a.ld,
                             ids + t * a.k, (int)n, (int)a.experts, (int)a.k, (int)a.renorm, a.scale,
                             (E*)dl + t * ld_dl, ld_dl);
        });
      });
    });
  });
  return err;
}

}  // namespace fp8q
