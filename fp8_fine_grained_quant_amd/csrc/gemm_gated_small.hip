// The gated feed-forward block and its gradient of a few hundred rows (gfx950),
// in all or an expert: too many for the kernel of few rows, and too few for the
// 256-row tiles to give every compute unit one.
//
// Tiles of 16 TM rows (32, 64 or 128) by 64 TN rows of B: of the block TN is 4, 128
// gate and the 128 up rows of the same outputs (a whole group of h's codes); of the
// gradient 2, 128 columns of dh.  Four waves share a tile's columns, every wave
// reading all of its rows: wave w has gate and up of outputs 32 w to 32 w + 31 of
// the tile, or columns 32 w to 32 w + 31 of dh.  A chunk's operands and scales come
// to LDS by direct loads, three stages of them; while a chunk is multiplied, the
// next one's fragments replace its own in the registers.  One barrier a chunk:
// behind it the next chunk is there for all waves, and the stage of this one, whose
// fragments are read, takes the loads of the third one after it.
//
// Products, scales and their sums are those of the large tiles, chunk by chunk,
// with the same bits.
//
// 512 rows of 2048 x 7168 with gate and up kept: 31 us (the large tiles 72), 1024
// rows 38 (75), 2048 rows 62 (76); their gradients 20 (55), 26 (57), 41 (59).  The
// time of a chunk is that of the loads to LDS that a compute unit's waves put out
// for it, about 27 cycles each (24 to 52 loads; with 128 rows the block's matrix
// instructions take longer).  More stages change nothing, nor does reading all
// fragments first; a chunk's loads one by one behind its matrix instructions instead
// of together before them take 33 us instead of 37 with 64 rows, 53 instead of 65
// with 128 (a chunk's fragments read at its own begin: 54 and 91).

#include "device_common.h"
#include "gemm_tile.h"
#include "launch.h"

#include <algorithm>

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kSmallNT = 256;

template <bool GRADIENT, int TM, bool GROUPED>
__global__ __launch_bounds__(kSmallNT) void k_gated_small(const GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int TN = GRADIENT ? 2 : 4, BM = 16 * TM;
  constexpr int kA = BM * 128, kB = 64 * TN * 128, kStage = kA + kB + 1024;
  constexpr int kIA = BM / 32, kIB = 2 * TN, kLoads = kIA + kIB + 1;  // a wave's loads of a chunk
  // one LDS object a stage, so that no wait for one covers another
  __shared__ __attribute__((aligned(16))) uint8_t st0[kStage], st1[kStage], st2[kStage];
  TileCoord tc;
  if (!tile_coord<BM, 128, GROUPED>(p, tc)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int nk = (int)(p.K / 128), rows = (int)min(tc.mend - tc.m0, (int64_t)BM);
  const uint8_t* const B = p.B + (GROUPED ? tc.e * p.b_estride : 0);
  const float* const sb = p.sb + (GROUPED ? tc.e * p.sb_estride : 0);

  auto rsrc = [](const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  // the wave's 16 TN rows of B, and its scales: waves 0 and 1 the rows', 2 and 3
  // gate's and up's block (the gradient's one, twice)
  const int64_t b0 = GRADIENT ? tc.n0 + 32 * w : tc.n0 + 64 * (w & 1) + (w >> 1) * p.N;
  const int64_t s0 = GRADIENT || w == 2 ? tc.n0 : tc.n0 + p.N;
  const __amdgpu_buffer_rsrc_t rA = rsrc(p.A + tc.m0 * p.lda, (uint32_t)(rows * p.lda));  // rows past the last one: no access
  const __amdgpu_buffer_rsrc_t rB = rsrc(B + b0 * p.ldb, (uint32_t)(16 * TN * p.ldb));
  const __amdgpu_buffer_rsrc_t rS =
      w < 2 ? rsrc(p.sa + tc.m0 * p.ld_sa, (uint32_t)(rows * p.ld_sa * 4))
            : rsrc(sb + s0 / 128 * p.sb_rs, (uint32_t)(((int64_t)(nk - 1) * p.sb_cs + 1) * 4));
  const int r8 = lane >> 3, c16 = 16 * ((lane & 7) ^ r8);
  const uint32_t vA = (uint32_t)((w * kIA * 8 + r8) * p.lda + c16), vB = (uint32_t)(r8 * p.ldb + c16);
  const uint32_t stepA = (uint32_t)(8 * p.lda), stepB = (uint32_t)(8 * p.ldb);
  const uint32_t vS = w < 2 ? (uint32_t)(min(64 * w + lane, rows - 1) * p.ld_sa * 4) : 0u;
  const uint32_t stepS = w < 2 ? 4u : (uint32_t)(4 * p.sb_cs);
  // load d of a wave's kLoads of chunk kb; past the last chunk one without access
  auto issue_one = [&](int kb, uint8_t* st, int d) __attribute__((always_inline)) {
    const bool on = kb < nk;
    const uint32_t k = on ? (uint32_t)kb : 0u;
    if (d < kIA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr)(st + (w * kIA + d) * 1024), 16,
                                               on ? vA + d * stepA : kNoAccess, k * 128, 0, 0);
    else if (d < kIA + kIB)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr)(st + kA + (w * kIB + d - kIA) * 1024), 16,
                                               on ? vB + (d - kIA) * stepB : kNoAccess, k * 128, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_ptr)(st + kA + kB + w * 256), 4, on ? vS : kNoAccess, k * stepS,
                                               0, 0);
  };
  auto issue = [&](int kb, uint8_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < kLoads; ++d) issue_one(kb, st, d);
  };

  const int sw = l16 & 7;
  const int lo = l16 * 128 + 16 * (g ^ sw), hi = l16 * 128 + 16 * ((4 + g) ^ sw);
  auto frag = [&](const uint8_t* at) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(at + lo), b = *reinterpret_cast<const u32x4*>(at + hi);
    return v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  };
  float acc[TM][TN][4];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.f;

  auto fence = [] { asm volatile("" ::: "memory"); };
  v8i a[TM], b0s[TN], b1s[TN];     // fragments of A, of B of this chunk and the next one (by turns)
  float sg[TM], su[TM];            // a chunk's row scales times gate's (the gradient's) and up's block
  v4f pp[2][TN];                   // partials of a row sub-tile and of the one before
  float lg = 0.f, lu = 0.f;        // scales of the chunk before's last sub-tile
  auto rd_b = [&](const uint8_t* st, int j) {
    return frag(st + kA + 128 * (GRADIENT ? 32 * w + 16 * j : (j >> 1) * 128 + 32 * w + 16 * (j & 1)));
  };
  auto rd_a = [&](const uint8_t* st, int i) { return frag(st + 128 * 16 * i); };
  auto promote = [&](int i, float g_, float u_) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = __builtin_fmaf(pp[i & 1][j][r], !GRADIENT && j >= 2 ? u_ : g_, acc[i][j][r]);
  };
  // Chunk kb, whose fragments and scales are in registers: those of the next one
  // come from `next` meanwhile, each after its predecessor's use, and a sub-tile is
  // added to the sums behind the matrix instructions of the one after it.
  auto step = [&](int kb, const uint8_t* next, uint8_t* free, v8i (&b)[TN], v8i (&bn)[TN]) __attribute__((always_inline)) {
    // the next chunk's loads have landed (the one after it may be under way), and
    // this one's fragments are read
    __builtin_amdgcn_s_waitcnt(0x0070 | (kLoads & 15) | ((kLoads >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    fence();
    const float* const sc = reinterpret_cast<const float*>(next + kA + kB);
    const float sb0 = sc[128], sb1 = sc[192];
    float sn[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      constexpr int kSlots = TM * TN;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int slot = i * TN + j;
        pp[i & 1][j] =
            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[i], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int d = slot * kLoads / kSlots; d < (slot + 1) * kLoads / kSlots; ++d) issue_one(kb + 3, free, d);
        if (j < TN - 1) __builtin_amdgcn_sched_barrier(0);
      }
      a[i] = rd_a(next, i);
      sn[i] = sc[16 * i + l16];
#pragma unroll
      for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) bn[j] = rd_b(next, j);
      if (i == 0) promote(TM - 1, lg, lu);
      else promote(i - 1, sg[i - 1], su[i - 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    lg = sg[TM - 1];
    lu = su[TM - 1];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      sg[i] = sn[i] * sb0;
      su[i] = sn[i] * sb1;
    }
    fence();
  };

  issue(0, st0);
  issue(1, st1);
  issue(2, st2);
  static_assert(2 * kLoads < 64, "loads that a wait can count");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * kLoads & 15) | ((2 * kLoads >> 4) << 14));  // the first chunk's loads
  __builtin_amdgcn_s_barrier();
  fence();
  {
    const float* const sc = reinterpret_cast<const float*>(st0 + kA + kB);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      a[i] = rd_a(st0, i);
      sg[i] = sc[16 * i + l16] * sc[128];
      su[i] = sc[16 * i + l16] * sc[192];
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      b0s[j] = rd_b(st0, j);
      pp[0][j] = pp[1][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
  }
  int c = 0;
  constexpr int kAhead = GRADIENT ? TM : 1;
  GateUp<2> gate_up[kAhead];
  // six chunks: three stages, two sets of B's fragments
  auto turns = [&](int end) __attribute__((always_inline)) {
    for (; c + 6 <= end; c += 6) {
      step(c, st1, st0, b0s, b1s);
      step(c + 1, st2, st1, b1s, b0s);
      step(c + 2, st0, st2, b0s, b1s);
      step(c + 3, st1, st0, b1s, b0s);
      step(c + 4, st2, st1, b0s, b1s);
      step(c + 5, st0, st2, b1s, b0s);
    }
  };
  if constexpr (GRADIENT) {
    // gate and up, which only the epilogue needs, before the last chunks (the waits
    // in front of these only get stricter)
    turns(nk - 6);
#pragma unroll
    for (int i = 0; i < TM; ++i) gate_up[i].load(p, tc.m0 + 16 * i, tc.mend, tc.n0 + 32 * w, lane);
  }
  turns(nk);
  if (c < nk) step(c, st1, st0, b0s, b1s);
  if (c + 1 < nk) step(c + 1, st2, st1, b1s, b0s);
  if (c + 2 < nk) step(c + 2, st0, st2, b0s, b1s);
  if (c + 3 < nk) step(c + 3, st1, st0, b1s, b0s);
  if (c + 4 < nk) step(c + 4, st2, st1, b0s, b1s);
  promote(TM - 1, lg, lu);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  fence();

  // a wave's staging area is its quarter of a stage
  static_assert((GRADIENT ? 16 * (16 * 2 * 4 + 16) : 16 * TM * (16 * 2 * 2 + 16)) <= kStage / 4, "the epilogue's staging area");
  uint8_t* const ep = st0 + w * (kStage / 4 / 16 * 16);
  if constexpr (GRADIENT) {
    store_tile_dswiglu<TM, TN, TM>(acc, ep, p, tc.m0, tc.mend, tc.n0 + 32 * w, lane, gate_up);
  } else {
    float gate[TM][2][4], up[TM][2][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          gate[i][j][r] = acc[i][j][r];
          up[i][j][r] = acc[i][j + 2][r];
        }
    store_tile_swiglu<TM, 2>(gate, up, ep, p, tc.m0, tc.mend, tc.n0 + 32 * w, lane, reinterpret_cast<float*>(st1), 0, w);
  }
#endif  // __HIP_DEVICE_COMPILE__
}

template <bool GRADIENT, int TM, bool GROUPED>
hipError_t small(const GemmArgs& a, hipStream_t st) {
  const int64_t tiles_m = (a.M + 16 * TM - 1) / (16 * TM) + (GROUPED ? a.E : 0);  // grouped: upper bound
  hipLaunchKernelGGL((k_gated_small<GRADIENT, TM, GROUPED>), dim3((uint32_t)(tiles_m * (a.N / 128))), dim3(kSmallNT), 0,
                     st, a);
  return hipGetLastError();
}
template <bool GRADIENT, bool GROUPED>
hipError_t small(const GemmArgs& a, int rows, hipStream_t st) {
  return rows == 32   ? small<GRADIENT, 2, GROUPED>(a, st)
         : rows == 64 ? small<GRADIENT, 4, GROUPED>(a, st)
                      : small<GRADIENT, 8, GROUPED>(a, st);
}

// What a kernel's workgroups take, in ns: a start, and a chunk's time, which grows by
// `full` where every compute unit has one.
struct TileTime {
  int rows, cols, start, chunk, full;
};
// About how many there are: an expert's last tile of rows is half full on average,
// and no expert has none.
int64_t tile_count(const TileTime& t, int64_t M, int64_t N, int64_t experts) {
  int64_t tiles_m = (M + t.rows - 1) / t.rows;
  if (experts > 0) tiles_m = std::min(M, std::max(experts, tiles_m + experts / 2));
  return tiles_m * (N / t.cols);
}
int64_t tile_time(const TileTime& t, int64_t tiles, int64_t nk) {
  const int64_t cus = device_cu_count(), rounds = tiles / cus, rest = tiles % cus;
  return rounds * (t.start + nk * (t.chunk + t.full)) + (rest ? t.start + nk * (t.chunk + t.full * rest / cus) : 0);
}

}  // namespace

// Measured, of 2048 x 7168 with gate and up kept: tiles of 32 rows (512 rows) 31 us,
// of 64 (1024) 38, of 128 (2048) 62, the large tiles 72, 75 and 76; the gradient's
// 20, 26 and 41, the large ones 55, 57 and 59.  4096 rows: 128 and 97, 85 and 69.
int64_t gated_small_time(int64_t M, int64_t N, int64_t K, int64_t experts, int gated, int* rows) {
  static constexpr TileTime kBlock[3] = {
      {32, 128, 5100, 420, 40}, {64, 128, 6200, 490, 70}, {128, 128, 8200, 800, 150}};
  static constexpr TileTime kGradient[3] = {
      {32, 128, 4900, 235, 40}, {64, 128, 5700, 320, 50}, {128, 128, 8500, 500, 80}};
  int64_t best = INT64_MAX;
  *rows = 0;
  // Many experts' weights are a matter of the memory, which more tiles of rows ask for
  // them more often: here up to two rounds of the lowest tiles (32 experts of 2048 x
  // 7168: 256 rows in all 158 us, 184 with the large tiles; 1024 rows, in 3 rounds, 205
  // and 196; 2048 rows 231 and 205.  8 experts of 1024 x 2048, 1000 rows: 15 and 30).
  if (experts > 0 && tile_count(kBlock[0], M, N, experts) > 2 * device_cu_count()) return best;
  for (const TileTime& t : gated == kSwiglu ? kBlock : kGradient) {
    // a launch's threads are counted in 32 bits
    if (((M + t.rows - 1) / t.rows + experts) * (N / t.cols) > ((int64_t(1) << 32) - 1) / kSmallNT) continue;
    const int64_t time = tile_time(t, tile_count(t, M, N, experts), K / 128);
    if (time < best) {
      best = time;
      *rows = t.rows;
    }
  }
  return best;
}

int64_t gated_large_time(int64_t M, int64_t N, int64_t K, int64_t experts, int gated) {
  // (the gradient's 256 x 256 tiles where they are taken)
  const bool wide = N % 256 == 0 && 2 * ((M + 255) / 256) * (N / 256) > device_cu_count();
  const TileTime t = gated == kSwiglu ? TileTime{256, 128, 8700, 1100, 500}
                     : wide           ? TileTime{256, 256, 15000, 1300, 700}
                                      : TileTime{256, 128, 13000, 730, 280};
  return tile_time(t, tile_count(t, M, N, experts), K / 128);
}

hipError_t launch_gated_small(const GemmArgs& a, int rows, hipStream_t st) {
  const bool grouped = a.offsets != nullptr;
  if (a.gated == kSwiglu) return grouped ? small<false, true>(a, rows, st) : small<false, false>(a, rows, st);
  return grouped ? small<true, true>(a, rows, st) : small<true, false>(a, rows, st);
}

}  // namespace fp8q
