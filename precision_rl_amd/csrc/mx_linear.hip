// Dense product of MX operands on gfx950: y[t, n] = bf16(sum_k (c 2^X)_x (c 2^X)_w)
// with x MXFP8 (E4M3) or MXFP4 (E2M1) and w MXFP4, one E8M0 scale per 32 of K,
// on v_mfma_scale_f32_16x16x128_f8f6f4 with FP32 accumulation.
//
// The weights are the matrix instruction's A operand and the activations its B
// operand, so that a lane's four accumulators are consecutive columns of one
// row of y.  Every output element is one chain of these instructions over K in
// ascending steps of 128, whatever the tile: the bits of a token's result
// depend neither on the batch size nor on the other tokens, and no variant
// splits K.
//
// Operand lanes (checked on the device with one-hot inputs): lane l holds row
// l % 16.  FP4: elements 32 (l / 16) .. +31 of the 128; FP8: elements 16 (l /
// 16) .. +15 and 64 + 16 (l / 16) .. +15.  In both the lane supplies the scale
// of its row's 32-block l / 16.

#include <algorithm>

#include "gemm_common.h"
#include "internal.h"

namespace w4a4 {
namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));

constexpr int kLinBK = 128;   // K per stage: one matrix instruction

// A tile of BM tokens x BN columns by WM x WN waves, a ring of S stages.
template <bool X8_, int BM_, int BN_, int WM_, int WN_, int S_, int OCC_>
struct LinCfg {
  static constexpr bool X8 = X8_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, OCC = OCC_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int TM = BM / WM, TN = BN / WN;   // a wave's tokens and columns
  static constexpr int FT = TM / 16, FN = TN / 16;   // its 16-wide operand blocks
  static constexpr int kXRow = X8 ? 128 : 64, kWRow = 64;   // bytes per staged row
  // 1 KB pieces (one copy of a wave) per stage and per wave; where there are
  // fewer pieces than waves, some waves copy the same piece (the same bytes
  // to the same place), so that every wave has the same count outstanding
  static constexpr int NX = BM * kXRow / 1024, NW = BN * kWRow / 1024, NS = (BM + BN + 63) / 64;
  static constexpr int PX = (NX + kWaves - 1) / kWaves, PW = (NW + kWaves - 1) / kWaves,
                       PS = (NS + kWaves - 1) / kWaves;
  static constexpr int kCopies = PX + PW + PS;
  static constexpr int kW = BM * kXRow, kScales = kW + BN * kWRow, kStage = kScales + NS * 256;
  static constexpr int kLds = S * kStage;
  static_assert(NX * 1024 == BM * kXRow && NW * 1024 == BN * kWRow, "whole pieces");
  static_assert((S - 1) * kCopies <= 63, "the vector-memory counter has six bits");
  static_assert(FN == 1 || FN % 2 == 0, "columns are paired");
};

// 16-byte chunk slot of chunk c of staged row r: the 16 rows that one phase of
// a 16-byte read touches lie in distinct banks.
template <class C>
__device__ __forceinline__ int x_slot(int r, int c) {
  return C::X8 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
}
template <class C>
__device__ __forceinline__ int w_slot(int r, int c) {
  return C::FN == 1 ? c ^ ((r >> 2) & 3) : c ^ ((r >> 3) & 3);
}
// Column (within the wave's TN) of row i of column block f.  Blocks come in
// pairs: a lane's accumulators of the two are 8 consecutive columns, a 16-byte
// store, and the four lane groups of a row together store 64 bytes.
template <class C>
__device__ __forceinline__ int col_of(int f, int i) {
  return C::FN == 1 ? i : 32 * (f / 2) + 8 * (i / 4) + 4 * (f % 2) + i % 4;
}

template <int P, int MAX>
__device__ __forceinline__ void wait_stages(int later) {   // at most `later` later stages outstanding
  if (later >= MAX) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(P * MAX) : "memory");
  } else if constexpr (MAX > 0) {
    wait_stages<P, MAX - 1>(later);
  }
}

struct LinArgs {
  int64_t T;
  int K, N;
  const uint8_t *x, *xs, *w, *ws;
  uint16_t* y;
  int64_t y_stride;
  int m_tiles, n_tiles;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::OCC)
mx_linear_kernel(LinArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int r16 = lane & 15, g = lane >> 4;

  // Tiles are dealt to the XCDs in contiguous runs; within a run, groups of
  // up to 8 token tiles with the column tiles running over them, so that the
  // tiles that run together share both operands in the XCD's L2.
  int64_t tile;
  {
    const int64_t total = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    const int64_t per_xcd = (total + kXcds - 1) / kXcds;
    const int64_t b = blockIdx.x;
    tile = (b % kXcds) * per_xcd + b / kXcds;
    if (b / kXcds >= per_xcd || tile >= total) return;
  }
  constexpr int kGroup = 8;
  const int64_t group = tile / (static_cast<int64_t>(kGroup) * a.n_tiles);
  const int in_group = static_cast<int>(tile - group * kGroup * a.n_tiles);
  const int gm = static_cast<int>(min<int64_t>(kGroup, a.m_tiles - group * kGroup));
  const int64_t m0 = (group * kGroup + in_group % gm) * C::BM;
  const int64_t n0 = static_cast<int64_t>(in_group / gm) * C::BN;
  const int rows = static_cast<int>(min<int64_t>(C::BM, a.T - m0));   // >= 1
  const int cols = static_cast<int>(min<int64_t>(C::BN, a.N - n0));

  const int x_pitch = C::X8 ? a.K : a.K / 2, w_pitch = a.K / 2, s_pitch = a.K / 32;
  const uint8_t* x_base = a.x + m0 * x_pitch;
  const uint8_t* w_base = a.w + n0 * w_pitch;
  // Copy sources; rows past the operand are clamped to its last (they feed
  // only outputs that are not stored).
  uint32_t x_off[C::PX], w_off[C::PW];
  const uint8_t* s_src[C::PS];
#pragma unroll
  for (int j = 0; j < C::PX; ++j) {
    const int piece = (wave + j * C::kWaves) % C::NX;
    const int row = C::X8 ? 8 * piece + (lane >> 3) : 16 * piece + (lane >> 2);
    const int chunk = x_slot<C>(row, C::X8 ? lane & 7 : lane & 3);
    x_off[j] = static_cast<uint32_t>(min(row, rows - 1)) * static_cast<uint32_t>(x_pitch) + chunk * 16;
  }
#pragma unroll
  for (int j = 0; j < C::PW; ++j) {
    const int row = 16 * ((wave + j * C::kWaves) % C::NW) + (lane >> 2);
    w_off[j] = static_cast<uint32_t>(min(row, cols - 1)) * static_cast<uint32_t>(w_pitch) +
               w_slot<C>(row, lane & 3) * 16;
  }
#pragma unroll
  for (int j = 0; j < C::PS; ++j) {
    const int q = 64 * ((wave + j * C::kWaves) % C::NS) + lane;
    s_src[j] = q < C::BM ? a.xs + (m0 + min(q, rows - 1)) * s_pitch
                         : a.ws + (n0 + min(q - C::BM, cols - 1)) * s_pitch;
  }
  const uint32_t lds0 = lds_addr(lds);
  auto issue = [&](int kt) {
    const uint32_t st = lds0 + (kt % C::S) * C::kStage;
#pragma unroll
    for (int j = 0; j < C::PX; ++j)
      dma16_off(x_base + static_cast<int64_t>(kt) * C::kXRow, x_off[j], st + ((wave + j * C::kWaves) % C::NX) * 1024);
#pragma unroll
    for (int j = 0; j < C::PW; ++j)
      dma16_off(w_base + static_cast<int64_t>(kt) * C::kWRow, w_off[j],
                st + C::kW + ((wave + j * C::kWaves) % C::NW) * 1024);
#pragma unroll
    for (int j = 0; j < C::PS; ++j)
      dma4(s_src[j] + kt * 4, st + C::kScales + ((wave + j * C::kWaves) % C::NS) * 256);
  };

  floatx4_t acc[C::FN][C::FT];
#pragma unroll
  for (int f = 0; f < C::FN; ++f)
#pragma unroll
    for (int t = 0; t < C::FT; ++t) acc[f][t] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // The lane's LDS offsets within a stage.  Blocks lie 16 rows (a pair of
  // column blocks: 32) apart, where the slots repeat.
  const int xr = wm * C::TM + r16;
  const int x_lane = xr * C::kXRow + x_slot<C>(xr, g) * 16;
  const int x_lane_hi = xr * C::kXRow + x_slot<C>(xr, 4 + g) * 16;   // FP8: the upper 64 of K
  const int wr0 = wn * C::TN + col_of<C>(0, r16), wr1 = wn * C::TN + (C::FN == 1 ? 0 : col_of<C>(1, r16));
  const int w_lane[2] = {C::kW + wr0 * C::kWRow + w_slot<C>(wr0, g) * 16,
                         C::kW + wr1 * C::kWRow + w_slot<C>(wr1, g) * 16};
  const int xs_lane = C::kScales + xr * 4 + g;
  const int ws_lane[2] = {C::kScales + (C::BM + wr0) * 4 + g, C::kScales + (C::BM + wr1) * 4 + g};

  struct Frags {
    u32x4_t x[C::FT][C::X8 ? 2 : 1];
    u32x4_t w[C::FN];
    int xs[C::FT], ws[C::FN];
  };
  auto read = [&](int kt, Frags& f) {
    const uint32_t st = opaque_sgpr(lds0 + (kt % C::S) * C::kStage);
#pragma unroll
    for (int t = 0; t < C::FT; ++t) {
      f.x[t][0] = *lds_ptr<u32x4_t>(st + x_lane + t * 16 * C::kXRow);
      if constexpr (C::X8) f.x[t][1] = *lds_ptr<u32x4_t>(st + x_lane_hi + t * 16 * C::kXRow);
      f.xs[t] = *lds_ptr<uint8_t>(st + xs_lane + t * 16 * 4);
    }
#pragma unroll
    for (int n = 0; n < C::FN; ++n) {
      f.w[n] = *lds_ptr<u32x4_t>(st + w_lane[n % 2] + (n / 2) * 32 * C::kWRow);
      f.ws[n] = *lds_ptr<uint8_t>(st + ws_lane[n % 2] + (n / 2) * 32 * 4);
    }
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int t = 0; t < C::FT; ++t) {
      i32x8_t xv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xv[i] = static_cast<int>(f.x[t][0][i]);
        xv[4 + i] = C::X8 ? static_cast<int>(f.x[t][C::X8 ? 1 : 0][i]) : 0;
      }
#pragma unroll
      for (int n = 0; n < C::FN; ++n) {
        const i32x8_t wv = {static_cast<int>(f.w[n][0]), static_cast<int>(f.w[n][1]), static_cast<int>(f.w[n][2]),
                            static_cast<int>(f.w[n][3]), 0, 0, 0, 0};
        // formats: 4 = FP4 E2M1, 0 = FP8 E4M3; scale bytes in bits 7:0
        acc[n][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, acc[n][t], 4, C::X8 ? 0 : 4, 0,
                                                                     f.ws[n], 0, f.xs[t]);
      }
    }
  };

  // Stage kt + 1 is read into registers while the matrix instructions of
  // stage kt run; a stage's slot is free once every wave holds it in
  // registers, at the barrier of the step that multiplies it.
  const int nk = a.K / kLinBK;
  for (int s = 0; s < C::S && s < nk; ++s) issue(s);
  Frags even, odd;
  wait_stages<C::kCopies, C::S - 1>(min(C::S, nk) - 1);
  read(0, even);
  auto step = [&](int kt, const Frags& cur, Frags& next) {
    if (kt + 1 < nk) {
      wait_stages<C::kCopies, C::S - 2>(min(C::S - 2, nk - 2 - kt));
      if (kt + C::S < nk) issue(kt + C::S);
      read(kt + 1, next);
    }
    multiply(cur);
  };
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, even, odd);
    if (kt + 1 < nk) step(kt + 1, odd, even);
  }

#pragma unroll
  for (int t = 0; t < C::FT; ++t) {
    const int tr = wm * C::TM + 16 * t + r16;
    if (tr >= rows) continue;
    uint16_t* yr = a.y + (m0 + tr) * a.y_stride + n0;
    if constexpr (C::FN == 1) {
      const int n = wn * C::TN + 4 * g;
      if (n < cols)
        *reinterpret_cast<u32x2_t*>(yr + n) =
            u32x2_t{pack_bf16x2(acc[0][t][0], acc[0][t][1]), pack_bf16x2(acc[0][t][2], acc[0][t][3])};
    } else {
#pragma unroll
      for (int f = 0; f < C::FN; f += 2) {
        const int n = wn * C::TN + 16 * f + 8 * g;
        if (n < cols)
          *reinterpret_cast<u32x4_t*>(yr + n) =
              u32x4_t{pack_bf16x2(acc[f][t][0], acc[f][t][1]), pack_bf16x2(acc[f][t][2], acc[f][t][3]),
                      pack_bf16x2(acc[f + 1][t][0], acc[f + 1][t][1]), pack_bf16x2(acc[f + 1][t][2], acc[f + 1][t][3])};
      }
    }
  }
}

template <class C>
bool launch_cfg(LinArgs a, hipStream_t s) {
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_linear_kernel<C>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
  if (attr != hipSuccess) return launch_ok("mx_linear") && false;
  a.m_tiles = static_cast<int>((a.T + C::BM - 1) / C::BM);
  a.n_tiles = (a.N + C::BN - 1) / C::BN;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
  launch_kernel("mx_linear", mx_linear_kernel<C>, dim3(xcd_grid(tiles)), dim3(C::kThreads), C::kLds, s, a);
  return launch_ok("mx_linear");
}

template <bool X8>
bool launch_format(const LinArgs& a, hipStream_t s) {
  if (a.T <= 16) return launch_cfg<LinCfg<X8, 16, 16, 1, 1, 8, 1>>(a, s);
  if (a.T <= 64) return launch_cfg<LinCfg<X8, 64, 64, 1, 4, 4, 1>>(a, s);
  return launch_cfg<LinCfg<X8, 128, 128, 2, 2, 4, 1>>(a, s);
}

}  // namespace

bool launch_mx_linear(int64_t T, int K, int N, bool x_fp8, const uint8_t* x, const uint8_t* xs, const uint8_t* w,
                      const uint8_t* ws, uint16_t* y, int64_t y_stride, hipStream_t s) {
  if (T == 0) return true;
  const LinArgs a{T, K, N, x, xs, w, ws, y, y_stride, 0, 0};
  return x_fp8 ? launch_format<true>(a, s) : launch_format<false>(a, s);
}

}  // namespace w4a4
