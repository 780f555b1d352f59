// Output-tile assignment and LDS-staged epilogue shared by the GEMM kernels.
#pragma once

#include "device_common.h"
#include "launch.h"
#include "row_io.h"

namespace fp8q {

constexpr int kGroupM = 4;  // m-tiles per band of the tile order

struct TileCoord {
  int64_t m0;    // first output row of the tile
  int64_t mend;  // end of the rows this tile may write (M, or the expert's end)
  int n0;        // first output column
  int e;         // expert (grouped launches), else 0
};

// Maps this workgroup to an output tile; false when it has none (grouped
// launches size the grid for the worst case).
//
// Dispatch hands consecutive workgroup ids to the 8 XCDs in turn, so the ids
// are first renumbered to give each XCD one contiguous run of tile numbers;
// tile numbers then walk bands of kGroupM m-tiles column by column.  The
// workgroups of one XCD thus cover a compact block of the output and share
// their A rows and B columns in that XCD's L2.
// The coordinates depend only on the workgroup id, the launch arguments and
// the expert offsets, so they are the same in every lane; the compiler cannot
// always prove that through the expert walks below, and then keeps them in
// vector registers and wraps every buffer load that uses them in a loop over
// lanes (measured: 52 such loops in the grouped weight-gradient kernel).
// Reading them back from lane 0 makes them scalar again.
__device__ __forceinline__ int64_t uniform_i64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ void make_uniform(TileCoord& tc) {
  tc.m0 = uniform_i64(tc.m0);
  tc.mend = uniform_i64(tc.mend);
  tc.n0 = __builtin_amdgcn_readfirstlane(tc.n0);
  tc.e = __builtin_amdgcn_readfirstlane(tc.e);
}

template <int BM, int BN, bool GROUPED>
__device__ __forceinline__ bool tile_coord(const GemmArgs& p, TileCoord& tc) {
  const int G = gridDim.x, bid = blockIdx.x;
  const int xcd = bid & 7, q8 = G >> 3, r8 = G & 7;
  const int t = xcd * q8 + min(xcd, r8) + (bid >> 3);
  const int tiles_n = (int)(p.N / BN);
  if (!GROUPED) {
    const int tiles_m = (int)((p.M + BM - 1) / BM);
    const int band = kGroupM * tiles_n;
    const int b = t / band, first_m = b * kGroupM;
    const int gm = min(tiles_m - first_m, kGroupM);
    const int in_band = t - b * band;
    tc.m0 = (int64_t)(first_m + in_band % gm) * BM;
    tc.n0 = (in_band / gm) * BN;
    tc.mend = p.M;
    tc.e = 0;
    return true;
  }
  if (p.k_grouped) {
    // grouped contraction: every expert owns a full M x N grid of tiles, and
    // tiles of different experts differ in work (the expert's token count).
    // Each XCD takes an equal share of every expert: the expert's tiles in
    // n-major order (m-tiles innermost) are cut into 8 contiguous runs whose
    // lengths differ by at most one, run x on XCD x, walked expert by expert,
    // so an XCD reads about 1/8 of each expert's X^T column blocks once and
    // shares the expert's dY^T rows among its workgroups.  (Taking the
    // experts in turns tile by tile instead measured 1.6x slower: the XCD's
    // L2 then holds no expert's operands long enough.  Whole n-slices per
    // XCD leave an XCD idle when the n-tile count is not a multiple of 8, as
    // with 28 tiles of 256 columns.)
    const int tiles_m = (int)((p.M + BM - 1) / BM);
    const int per_ex = tiles_m * tiles_n;
    const int slots = (per_ex + 7) / 8;  // workgroups per expert per XCD
    const int ew = (bid >> 3) / slots;   // position in this XCD's walk over the experts
    if (ew >= (int)p.E) return false;
    const int tl = (bid >> 3) - ew * slots;
    // each XCD starts its walk E/8 experts after the previous one, so that
    // at any moment the XCDs work on different experts (some storing a small
    // expert's gradient while others compute a large one's; measured 626 ->
    // 618 us for the 32-expert weight gradient)
    const int e = (int)((ew + (int64_t)xcd * ((p.E + 7) / 8)) % p.E);
    const int q = per_ex >> 3, r = per_ex & 7;
    if (tl >= q + (xcd < r ? 1 : 0)) return false;
    const int t = xcd * q + min(xcd, r) + tl;
    tc.m0 = (int64_t)(t % tiles_m) * BM;
    tc.n0 = (t / tiles_m) * BN;
    tc.mend = p.M;
    tc.e = e;
    make_uniform(tc);
    return true;
  }
  // grouped rows: tiles never straddle experts.  The grid is sized for the
  // worst case (a partial m-tile per expert), so the real tiles are counted
  // first and cut into 8 contiguous runs of near-equal length, run x on XCD x
  // (cutting the whole grid instead left the last XCDs without work: 616 real
  // tiles of 768 slots filled XCDs 0-5 and part of 6).
  int64_t total = 0;
  for (int e = 0; e < (int)p.E; ++e) total += (p.offsets[e + 1] - p.offsets[e] + BM - 1) / BM;
  total *= tiles_n;
  const int64_t q = total >> 3, rem = total & 7, slot = bid >> 3;
  if (slot >= q + (xcd < rem ? 1 : 0)) return false;
  const int64_t tg = xcd * q + min((int64_t)xcd, rem) + slot;
  int64_t base = 0, lo = 0, hi = 0, mt = 0;
  int e = 0;
  for (; e < (int)p.E; ++e) {
    lo = p.offsets[e];
    hi = p.offsets[e + 1];
    mt = (hi - lo + BM - 1) / BM;
    const int64_t cnt = mt * tiles_n;
    if (tg < base + cnt) break;
    base += cnt;
  }
  if (e >= (int)p.E) return false;
  const int64_t local = tg - base;
  tc.m0 = lo + (local % mt) * BM;
  tc.n0 = (int)(local / mt) * BN;
  tc.mend = hi;
  tc.e = e;
  make_uniform(tc);
  return true;
}

// NTS = 1 writes non-temporally: for outputs that are written once and read
// much later (the weight gradients), so they do not fill the caches with
// dirty lines that the kernels after them must write back (measured:
// grouped Wgrad 796 -> 618 us, and the kernel after it 521 -> 465 us).
//
// Writes one wave's WM x WN accumulator block to C, staged through the
// wave's private LDS region `ep` in passes of ER rows so that every global
// access is a full 16-byte row segment.  Rows at or beyond `mend` are not
// written.  Accumulator layout of sub-tile (i, j), lane l = 16 g + l16:
// TRL = 0 (A the matrix instruction's first operand): rows 16 i + 4 g + r,
// column 16 j + l16; TRL = 1 (B first): row 16 i + l16, columns
// 16 j + 4 g + r.
template <int TM, int TN, int OUT_F32, int ER, int NTS = 0, bool TRL = false>
__device__ __forceinline__ void store_tile(const float (&acc)[TM][TN][4], uint8_t* ep, const GemmArgs& p,
                                           int64_t row0, int64_t mend, int col0, int lane) {
  constexpr int WM = 16 * TM, WN = 16 * TN;
  constexpr int ES = OUT_F32 ? 4 : 2;
  constexpr int P = WN * ES + 16;       // padded LDS row pitch
  constexpr int CPR = WN * ES / 16;     // 16-byte chunks per row
  constexpr int RPI = 64 / CPR;         // rows per store instruction
  constexpr int PASSES = WM / ER;
  static_assert(64 % CPR == 0 && ER % RPI == 0 && ER % 16 == 0 && WM % ER == 0, "epilogue store shape");
  const int g = lane >> 4, l16 = lane & 15;
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    if (pass) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the previous pass's LDS reads are done
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int i = pass * (ER / 16); i < (pass + 1) * (ER / 16); ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if constexpr (TRL) {
          const int rl = 16 * i + l16 - pass * ER, cl = 16 * j + 4 * g;
          if (OUT_F32) {
            *reinterpret_cast<float4*>(ep + rl * P + 4 * cl) =
                make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
          } else {
            const uint32_t lo = f32_to_bf16_rne(acc[i][j][0]) | (f32_to_bf16_rne(acc[i][j][1]) << 16);
            const uint32_t hi = f32_to_bf16_rne(acc[i][j][2]) | (f32_to_bf16_rne(acc[i][j][3]) << 16);
            *reinterpret_cast<uint2*>(ep + rl * P + 2 * cl) = make_uint2(lo, hi);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int rl = 16 * i + 4 * g + r - pass * ER, cl = 16 * j + l16;
            if (OUT_F32)
              *reinterpret_cast<float*>(ep + rl * P + 4 * cl) = acc[i][j][r];
            else
              *reinterpret_cast<uint16_t*>(ep + rl * P + 2 * cl) = (uint16_t)f32_to_bf16_rne(acc[i][j][r]);
          }
        }
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes are done
    __builtin_amdgcn_wave_barrier();
    // (row addresses by pointer increments: a 64-bit multiply per store was
    // most of the epilogue's address arithmetic)
    uint8_t* dst = reinterpret_cast<uint8_t*>(p.C) +
                   ((row0 + pass * ER + lane / CPR) * p.ldc + col0) * ES + 16 * (lane % CPR);
    const int64_t it_step = (int64_t)RPI * p.ldc * ES;
#pragma unroll
    for (int it = 0; it < ER / RPI; ++it, dst += it_step) {
      const int rl = it * RPI + lane / CPR, ch = lane % CPR;
      const int64_t row = row0 + pass * ER + rl;
      if (row >= mend) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(ep + rl * P + 16 * ch);
      if (OUT_F32 && p.accumulate) {
        const float4 o = *reinterpret_cast<const float4*>(dst);
        float4 f = *reinterpret_cast<const float4*>(&v);
        f.x += o.x; f.y += o.y; f.z += o.z; f.w += o.w;
        *reinterpret_cast<float4*>(dst) = f;
      } else {
        st_stream16<NTS>(dst, v.x, v.y, v.z, v.w);
      }
    }
  }
}

// The epilogue with the output's own quantization fused in (BF16 output,
// accumulators in the TRL = 1 layout of store_tile: lane 16 g + l16 holds row
// 16 i + l16, columns 16 j + 4 g + r): every wave's strip is 128 columns wide
// and starts on a multiple of 128, so each of its rows holds exactly one 1x128
// group of the output, spread over the four lanes l16, l16 + 16, l16 + 32,
// l16 + 48.  Each value is first rounded to BF16 (RNE); the group's max-abs,
// scale and codes are then taken from those BF16 values with the quantizers'
// own arithmetic (group_scale, pack4_e4m3_grp), so the codes and scales equal
// what quant_act_1x128 computes from the stored BF16 output.  The BF16 values
// leave through store_tile (skipped when p.C is NULL); the scaled values are
// staged through the wave's LDS region in passes of 16 rows so that every
// code store is a full 16-byte row segment.  The accumulators are only read.
template <int TM, int TN, int ER>
__device__ __forceinline__ void store_tile_q(const float (&acc)[TM][TN][4], uint8_t* ep, const GemmArgs& p,
                                             int64_t row0, int64_t mend, int col0, int lane) {
  static_assert(TN == 8, "a wave's strip is one 128-column group wide");
  constexpr int P = 128 * 4 + 16;  // padded LDS row pitch of the scaled values
  const int g = lane >> 4, l16 = lane & 15;
  auto rounded = [](float v) { return bf16_to_f32(f32_to_bf16_rne(v)); };
  if (p.C != nullptr) {
    store_tile<TM, TN, 0, ER, 0, true>(acc, ep, p, row0, mend, col0, lane);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the staging area is read out
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {  // one 16-row sub-tile per pass
    if (i) {
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_wave_barrier();
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) m = max(m, abs_bits(rounded(acc[i][j][r])));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));  // the row's other three lanes
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    float sc, inv;
    group_scale(__uint_as_float(m), sc, inv);
    const int64_t row = row0 + 16 * i + l16;
    if (g == 0 && row < mend) p.so[row * p.ld_so + (col0 >> 7)] = sc;
#pragma unroll
    for (int j = 0; j < TN; ++j)
      *reinterpret_cast<float4*>(ep + l16 * P + 4 * (16 * j + 4 * g)) =
          make_float4(rounded(acc[i][j][0]) * inv, rounded(acc[i][j][1]) * inv, rounded(acc[i][j][2]) * inv,
                      rounded(acc[i][j][3]) * inv);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
    // lane (rl = lane / 8, ch = lane % 8): 16 consecutive values of row rl
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int rl = it * 8 + (lane >> 3), ch = lane & 7;
      const int64_t orow = row0 + 16 * i + rl;
      const float4* src = reinterpret_cast<const float4*>(ep + rl * P + 64 * ch);
      const float4 v0 = src[0], v1 = src[1], v2 = src[2], v3 = src[3];
      if (orow >= mend) continue;
      const uint32_t w0 = pack4_e4m3_grp(v0.x, v0.y, v0.z, v0.w), w1 = pack4_e4m3_grp(v1.x, v1.y, v1.z, v1.w);
      const uint32_t w2 = pack4_e4m3_grp(v2.x, v2.y, v2.z, v2.w), w3 = pack4_e4m3_grp(v3.x, v3.y, v3.z, v3.w);
      st_stream16<0>(p.qo + orow * p.ld_qo + col0 + 16 * ch, w0, w1, w2, w3);
    }
  }
}

// ---------------------------------------------------------------------------
// Epilogues of the gated feed-forward block h = silu(g) u, silu(g) = g s with
// s = 1 / (1 + exp(-g)).

// By the exponential that cannot overflow, so that s keeps its relative accuracy
// down to the least numbers (1 / (1 + exp(-g)) is 0 from g = -89 on):
// e = exp(-|g|) = (2^-t)^2 with t = |g| log2(e) / 2, whose rounding is made good
// to first order (the exponential instruction gives no numbers below 2^-126; its
// square does), and 1 / (1 + e) by the reciprocal instruction.  Each of the two
// is off by one unit: s by 11 half units in all.  (With the library's expf and
// an IEEE division the epilogues' arithmetic took twice as long, 81 us against
// 76 for the gradient of 4096 x 2048 x 7168.)
__device__ __forceinline__ float sigmoid_f32(float g) {
  constexpr float kHalfLog2e = 0.72134752044448170f, kRest = (float)(0.72134752044448170 - (double)kHalfLog2e);
  constexpr float kLn2 = 0.69314718055994531f;
  const float a = fmaxf(-fabsf(g), -512.f), t = a * kHalfLog2e;  // e is 0 long before; finite for an infinite g
  const float lost = __builtin_fmaf(a, kRest, __builtin_fmaf(a, kHalfLog2e, -t));
  const float h = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(h, lost * kLn2, h), e = r * r;
  return (g < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e);
}

// One wave's 16 TM x 16 TN values (layout of store_tile with TRL = 1) as BF16 to
// a matrix of row stride ld, a full 16-byte row segment at a time.
template <int TM, int TN>
__device__ __forceinline__ void store_bf16(const float (&v)[TM][TN][4], uint8_t* ep, uint16_t* out, int64_t ld,
                                           int64_t row0, int64_t mend, int lane) {
  constexpr int P = 16 * TN * 2 + 16;            // padded LDS row pitch
  constexpr int CPR = 2 * TN, RPI = 64 / CPR;    // segments per row, rows per store instruction
  constexpr int SUB = 12288 / (16 * P) < TM ? 12288 / (16 * P) : TM;  // sub-tiles staged at once
  static_assert(TM % SUB == 0, "whole passes");
  const int lg = lane >> 4, l16 = lane & 15;
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += SUB) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the staging area is read out
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = i0; i < i0 + SUB; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<uint2*>(ep + (16 * (i - i0) + l16) * P + 2 * (16 * j + 4 * lg)) =
            make_uint2(pack2_bf16(v[i][j][0], v[i][j][1]), pack2_bf16(v[i][j][2], v[i][j][3]));
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int it = 0; it < 16 * SUB / RPI; ++it) {
      const int rl = it * RPI + lane / CPR, ch = lane % CPR;
      const int64_t row = row0 + 16 * i0 + rl;
      const uint4 x = *reinterpret_cast<const uint4*>(ep + rl * P + 16 * ch);
      if (row < mend) st_stream16<0>(out + row * ld + 8 * ch, x.x, x.y, x.z, x.w);
    }
  }
}

// One wave's gate and up accumulators of the same 16 TM x 16 TN outputs (layout of
// store_tile with TRL = 1): gate and up as they are to p.gu (BF16, up N columns
// after gate) if given, h to p.C (BF16) if given, and h's codes and scales,
// over the unrounded values, to p.qo and p.so if given.  A 128-column group is
// held by 8 / TN waves, which exchange their rows' max-abs through
// `maxima` [8 / TN][256]: with p.qo every wave of the workgroup makes this call.
// row_in_tile is the strip's first row in the tile, part the wave's part of the group.
template <int TM, int TN>
__device__ __forceinline__ void store_tile_swiglu(float (&g)[TM][TN][4], const float (&u)[TM][TN][4], uint8_t* ep,
                                                  const GemmArgs& p, int64_t row0, int64_t mend, int col0, int lane,
                                                  float* maxima, int row_in_tile, int part) {
  const int lg = lane >> 4, l16 = lane & 15;
  if (p.gu != nullptr) {
    store_bf16<TM, TN>(g, ep, p.gu + col0, p.ld_gu, row0, mend, lane);
    store_bf16<TM, TN>(u, ep, p.gu + col0 + p.N, p.ld_gu, row0, mend, lane);
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) g[i][j][r] = g[i][j][r] * sigmoid_f32(g[i][j][r]) * u[i][j][r];
  if (p.C != nullptr) store_bf16<TM, TN>(g, ep, reinterpret_cast<uint16_t*>(p.C) + col0, p.ldc, row0, mend, lane);
  if (p.qo == nullptr) return;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) m = max(m, abs_bits(g[i][j][r]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));  // the row's other three lanes
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (lg == 0) maxima[part * 256 + row_in_tile + 16 * i + l16] = __uint_as_float(m);
  }
  __syncthreads();  // (the staging area is read out as well)
  constexpr int P = 16 * TN + 16;     // padded LDS row pitch of the codes
  constexpr int RPI = 64 / TN;        // rows per store instruction, of TN 16-byte segments
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int rt = row_in_tile + 16 * i + l16;
    float sc, inv;
    float most = maxima[rt];
#pragma unroll
    for (int k = 1; k < 8 / TN; ++k) most = __builtin_fmaxf(most, maxima[256 * k + rt]);
    group_scale(most, sc, inv);
    const int64_t row = row0 + 16 * i + l16;
    if (part == 0 && lg == 0 && row < mend) p.so[row * p.ld_so + (col0 >> 7)] = sc;
#pragma unroll
    for (int j = 0; j < TN; ++j)
      *reinterpret_cast<uint32_t*>(ep + (16 * i + l16) * P + 16 * j + 4 * lg) =
          pack4_e4m3_grp(g[i][j][0] * inv, g[i][j][1] * inv, g[i][j][2] * inv, g[i][j][3] * inv);
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int it = 0; it < 16 * TM / RPI; ++it) {
    const int rl = it * RPI + lane / TN, ch = lane % TN;
    const int64_t row = row0 + rl;
    if (row >= mend) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(ep + rl * P + 16 * ch);
    st_stream16<0>(p.qo + row * p.ld_qo + col0 + 16 * ch, v.x, v.y, v.z, v.w);
  }
}

// The gradient's: the accumulators are dh (the output projection's Dgrad), g and
// u come from p.gu, and
//   dg = dh u (s + g s (1 - s)),   du = dh g s
// go to p.C [M, 2N] (BF16, du N columns after dg) and h = g s u to p.h if given.
// g and u are read as full 16-byte row segments, a 16-row sub-tile of them a
// GateUp, AHEAD of them before their use (the narrow tile's kernel loads all
// before its last chunks, when the memory has little to do).  dh goes through
// the wave's staging area into the segments' layout, in which the outputs leave
// from the registers.
template <int TN>
struct GateUp {
  static constexpr int kSegs = 16 * TN * 2 / 16;  // 16-byte segments per row
  static constexpr int kRows = 64 / kSegs;        // rows per load instruction
  u32x4 g[16 / kRows], u[16 / kRows];

  __device__ __forceinline__ void load(const GemmArgs& p, int64_t first, int64_t mend, int col0, int lane) {
#pragma unroll
    for (int it = 0; it < 16 / kRows; ++it) {
      // rows past the last one repeat it and are not stored
      const int64_t row = min(first + it * kRows + lane / kSegs, mend - 1);
      const uint16_t* src = p.gu + row * p.ld_gu + col0 + 8 * (lane % kSegs);
      g[it] = ld_stream16<0>(src);
      u[it] = ld_stream16<0>(src + p.N);
    }
  }
};

template <int TM, int TN, int AHEAD>
__device__ __forceinline__ void store_tile_dswiglu(const float (&dh)[TM][TN][4], uint8_t* ep, const GemmArgs& p,
                                                   int64_t row0, int64_t mend, int col0, int lane,
                                                   GateUp<TN> (&held)[AHEAD]) {
  typedef GateUp<TN> Held;
  constexpr int P = 16 * TN * 4 + 16;  // padded LDS row pitch of 16 rows of FP32
  static_assert(16 * P <= 12288, "a sub-tile fits a wave's staging area");
  const int lg = lane >> 4, l16 = lane & 15;
  auto lds_done = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_wave_barrier();
  };
  uint16_t* const C = reinterpret_cast<uint16_t*>(p.C);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t first = row0 + 16 * i;
    if (i) lds_done();
#pragma unroll
    for (int j = 0; j < TN; ++j)
      *reinterpret_cast<float4*>(ep + l16 * P + 4 * (16 * j + 4 * lg)) =
          make_float4(dh[i][j][0], dh[i][j][1], dh[i][j][2], dh[i][j][3]);
    lds_done();
    Held& gu = held[i % AHEAD];
#pragma unroll
    for (int it = 0; it < 16 / Held::kRows; ++it) {
      const int rl = it * Held::kRows + lane / Held::kSegs, ch = lane % Held::kSegs;
      const float4 lo = *reinterpret_cast<const float4*>(ep + rl * P + 32 * ch);
      const float4 hi = *reinterpret_cast<const float4*>(ep + rl * P + 32 * ch + 16);
      const float d[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      u32x4 wg, wu, wh;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float dg[2], du[2], h[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float g = __uint_as_float(r ? gu.g[it][k] & 0xFFFF0000u : gu.g[it][k] << 16);
          const float u = __uint_as_float(r ? gu.u[it][k] & 0xFFFF0000u : gu.u[it][k] << 16);
          const float s = sigmoid_f32(g), gs = g * s;
          dg[r] = d[2 * k + r] * u * __builtin_fmaf(gs, 1.f - s, s);
          du[r] = d[2 * k + r] * gs;
          h[r] = gs * u;
        }
        wg[k] = pack2_bf16(dg[0], dg[1]);
        wu[k] = pack2_bf16(du[0], du[1]);
        wh[k] = pack2_bf16(h[0], h[1]);
      }
      const int64_t row = first + rl;
      if (row >= mend) continue;
      uint16_t* dst = C + row * p.ldc + col0 + 8 * ch;
      st_stream16<0>(dst, wg[0], wg[1], wg[2], wg[3]);
      st_stream16<0>(dst + p.N, wu[0], wu[1], wu[2], wu[3]);
      if (p.h != nullptr) st_stream16<0>(p.h + row * p.ld_h + col0 + 8 * ch, wh[0], wh[1], wh[2], wh[3]);
    }
    if (i + AHEAD < TM) gu.load(p, first + 16 * AHEAD, mend, col0, lane);
  }
}

}  // namespace fp8q
