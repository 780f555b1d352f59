// The router of an MoE layer: the k best experts of every token, their
// weights, and the gradient to the logits (gfx950).
//
// Scores are softmax(logits) or sigmoid(logits); an expert whose logit is -inf
// is masked for that token.  Without a bias the logits decide (both scores
// grow with them), with one the score plus the bias does, in 64 bits: two
// experts' sums may differ by less than FP32 resolves, and the choice must not
// depend on how a score was rounded.  Equal keys go to the lower expert.

#include "device_common.h"
#include "launch.h"

#include <math.h>

#include <type_traits>

namespace fp8q {

namespace {

constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o));
  return v;
}

// exp of a value that is not positive: 1 + exp(-x) would overflow, and the
// score with it vanish, long before the score leaves FP32.
__device__ __forceinline__ float sigmoid(float x) {
  const float z = expf(-__builtin_fabsf(x));
  return (x < 0.f ? z : 1.f) / (1.f + z);
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
  __device__ __forceinline__ static void store(elem* p, float v) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
};
struct LogitF32 {
  typedef float elem;
  __device__ __forceinline__ static float load(const elem* p) { return *p; }
  __device__ __forceinline__ static void store(elem* p, float v) { *p = v; }
};

// One wave per token; lane l holds experts l, l + 64, ...
template <class L, int V, bool SIG, bool BIAS>
__global__ __launch_bounds__(256) void k_route(const typename L::elem* __restrict__ logits, int64_t ld,
                                               const float* __restrict__ bias, int tokens, int e, int k, int renorm,
                                               float scale, int* __restrict__ ids, float* __restrict__ w) {
  const int t = (int)(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63;
  if (t >= tokens) return;
  const typename L::elem* p = logits + (int64_t)t * ld;
  float x[V];
  double key[V];
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ex = i * 64 + lane;
    x[i] = ex < e ? L::load(p + ex) : -kInf;
    top = __builtin_fmaxf(top, x[i]);
  }
  top = wave_max(top);
  float total = 1.f;
  if (!SIG && !renorm) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) total += x[i] == -kInf ? 0.f : expf(x[i] - top);
    total = wave_sum(total);
  }
  if (BIAS) {
    double dt = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (SIG) key[i] = 1.0 / (1.0 + exp(-(double)x[i]));
      else key[i] = x[i] == -kInf ? 0.0 : exp((double)x[i] - (double)top);
      dt += key[i];
    }
    if (!SIG) dt = wave_sum(dt);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ex = i * 64 + lane;
      const double sc = SIG ? key[i] : key[i] / dt;
      key[i] = x[i] == -kInf ? -(double)kInf : sc + (ex < e ? (double)bias[ex] : 0.0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = (double)x[i];
  }
  int my_id = -1;
  float my_x = -kInf;  // lane j keeps choice j
  for (int j = 0; j < k; ++j) {
    double best = -(double)kInf;
    int at = -1;
    float bx = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 64 + lane;
        bx = x[i];
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double ob = __shfl_xor(best, o);
      const int oa = __shfl_xor(at, o);
      const float ox = __shfl_xor(bx, o);
      if (ob > best || (ob == best && oa >= 0 && (at < 0 || oa < at))) {
        best = ob;
        at = oa;
        bx = ox;
      }
    }
    if (at < 0) break;
    if (lane == j) {
      my_id = at;
      my_x = bx;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 64 + lane == at) key[i] = -(double)kInf;
  }
  float s = 0.f;
  if (renorm) {
    top = wave_max(my_x);
    s = my_id < 0 ? 0.f : scaled_score<SIG>(my_x, top);
    total = wave_sum(s);
  } else if (my_id >= 0) {
    s = SIG ? sigmoid(my_x) : expf(my_x - top);
  }
  const float out = my_id < 0 ? 0.f : SIG && !renorm ? s : s / total;
  if (lane < k) {
    ids[(int64_t)t * k + lane] = my_id;
    w[(int64_t)t * k + lane] = out * scale;
  }
}

// One wave per token: lane j computes what choice j needs, the row of
// gradients is put together in LDS (its chosen entries are few) and leaves
// once.  Only softmax without renormalization has a gradient to every expert.
template <class L, bool SIG>
__global__ __launch_bounds__(256) void k_route_bwd(const float* __restrict__ dw,
                                                   const typename L::elem* __restrict__ logits, int64_t ld,
                                                   const int* __restrict__ ids, int tokens, int e, int k, int renorm,
                                                   float scale, typename L::elem* __restrict__ dl, int64_t ld_dl) {
  __shared__ float row[4][kMaxExperts];
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = (int)(blockIdx.x * 4 + wv);
  float* r = row[wv];
  for (int i = lane; i < e; i += 64) r[i] = 0.f;
  __syncthreads();
  const bool live = t < tokens;
  const typename L::elem* p = logits + (int64_t)(live ? t : 0) * ld;
  int id = -1;
  float x = -kInf, g = 0.f;
  if (live && lane < k) {
    id = ids[(int64_t)t * k + lane];
    if ((uint32_t)id < (uint32_t)e) x = L::load(p + id);
    if (x == -kInf) id = -1;  // no choice, or a masked expert: no gradient
    else g = dw[(int64_t)t * k + lane] * scale;
  }
  const bool dense = !SIG && !renorm;
  float top = x, total = 0.f;
  if (dense && live)
    for (int i = lane; i < e; i += 64) top = __builtin_fmaxf(top, L::load(p + i));
  top = wave_max(top);
  if (dense && live)
    for (int i = lane; i < e; i += 64) {
      const float v = L::load(p + i);
      total += v == -kInf ? 0.f : expf(v - top);
    }
  float s = 0.f;
  if (id >= 0) s = SIG && !renorm ? sigmoid(x) : scaled_score<SIG>(x, top);
  total = dense ? wave_sum(total) : renorm ? wave_sum(s) : 1.f;
  const float wj = id < 0 ? 0.f : s / total;  // the weight before `scale`
  const float mean = wave_sum(g * wj);
  float d;
  if (SIG) {
    const float rest = sigmoid(-x);  // 1 - s without cancellation
    d = renorm ? (g - mean) * wj * rest : g * s * rest;
  } else {
    d = dense ? g : (g - mean) * wj;
  }
  if (id >= 0) r[id] = d;
  __syncthreads();
  if (!live) return;
  typename L::elem* o = dl + (int64_t)t * ld_dl;
  for (int i = lane; i < e; i += 64) {
    float v = r[i];
    if (dense) {
      const float xi = L::load(p + i);
      v = xi == -kInf ? 0.f : expf(xi - top) / total * (v - mean);
    }
    L::store(o + i, v);
  }
}

}  // namespace

hipError_t launch_moe_route(const MoeRoute& a, const float* bias, int32_t* ids, float* w, hipStream_t st) {
  const dim3 grid((uint32_t)((a.tokens + 3) / 4));
  auto go = [&](auto l, auto v, auto sig, auto bi) {
    typedef decltype(l) L;
    hipLaunchKernelGGL((k_route<L, decltype(v)::value, decltype(sig)::value, decltype(bi)::value>), grid, dim3(256),
                       0, st, (const typename L::elem*)a.logits, a.ld, bias, (int)a.tokens, (int)a.experts, (int)a.k,
                       (int)a.renorm, a.scale, ids, w);
  };
  auto pick_score = [&](auto l, auto v) {
    if (a.sigmoid) bias ? go(l, v, std::true_type{}, std::true_type{}) : go(l, v, std::true_type{}, std::false_type{});
    else bias ? go(l, v, std::false_type{}, std::true_type{}) : go(l, v, std::false_type{}, std::false_type{});
  };
  auto pick_v = [&](auto l) {
    if (a.experts <= 256) pick_score(l, std::integral_constant<int, 4>{});
    else pick_score(l, std::integral_constant<int, kMaxExperts / 64>{});
  };
  if (a.bf16) pick_v(LogitBF16{}); else pick_v(LogitF32{});
  return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const MoeRoute& a, const float* dw, const int32_t* ids, void* dl, int64_t ld_dl,
                                hipStream_t st) {
  const dim3 grid((uint32_t)((a.tokens + 3) / 4));
  auto go = [&](auto l, auto sig) {
    typedef decltype(l) L;
    typedef typename L::elem E;
    hipLaunchKernelGGL((k_route_bwd<L, decltype(sig)::value>), grid, dim3(256), 0, st, dw, (const E*)a.logits, a.ld,
                       ids, (int)a.tokens, (int)a.experts, (int)a.k, (int)a.renorm, a.scale, (E*)dl, ld_dl);
  };
  auto pick = [&](auto l) {
    if (a.sigmoid) go(l, std::true_type{}); else go(l, std::false_type{});
  };
  if (a.bf16) pick(LogitBF16{}); else pick(LogitF32{});
  return hipGetLastError();
}

}  // namespace fp8q
