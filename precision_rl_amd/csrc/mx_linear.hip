// Dense product of MX operands on gfx950: y[t, n] = bf16(sum_k (c 2^X)_x (c 2^X)_w)
// with x MXFP8 (E4M3) or MXFP4 (E2M1) and w MXFP4, one E8M0 scale per 32 of K,
// on v_mfma_scale_f32_32x32x64_f8f6f4 with FP32 accumulation.
//
// The weights are the matrix instruction's A operand and the activations its B
// operand, so that a lane's accumulators are consecutive columns of one row of
// y.  Every output element is one chain of these instructions over K in
// ascending steps of 64, whatever the tile: the bits of a token's result
// depend neither on the batch size nor on the other tokens, and no variant
// splits K.  With FP8 the instruction itself adds 8 adjacent products at a time
// and cuts each below 2^-13 of the largest before they reach the FP32
// accumulator, which costs about 5e-5 of the output's root mean square, a
// twentieth of the bf16 rounding; taken because the exact way, elements as
// bf16 with the scales applied, runs at about a third of the rate (a large bf16
// product 1.60 PFLOP/s, the FP8 x FP4 instruction 4.6 with operands in registers).
//
// Operand lanes (checked on the device with one-hot inputs): lane l holds row
// l % 32, half h = l / 32.  FP4: elements 32 h .. +31 of the 64; FP8: elements
// 16 h .. +15 and 32 + 16 h .. +15.  In both the lane supplies the scale of its
// row's 32-block h.
//
// A stage of both operands and of their scales is copied to LDS while the one
// before is multiplied.  At T = 16384, K = 2048, N = 4096 FP4 takes 88 us
// (3.1 PFLOP/s) and FP8 112 (2.5).  Of the former's 64 us a doubling of K adds
// (4.3 PFLOP/s), the matrix instructions alone take 43, the copies alone 41
// (one stage of 64 KB in flight a CU) and the operand reads alone 37; the
// stores, which a round's tiles make together at the memory's rate, take 20 us
// of the 88.  At T = 1 (N = 4096) a call takes 4.8 us (5.3 with FP8): 8 stages in a
// row of one wave, each a chain of four instructions on one accumulator, the
// operands' LDS latency and the next copies' issue.

#include <algorithm>

#include "gemm_common.h"
#include "internal.h"
#include "launch_parts.h"

namespace w4a4 {
namespace {

constexpr int kStep = 128;        // K per step: two matrix instructions, four scale bytes a row
constexpr int kScaleSteps = 4;    // scales are copied for four steps at a time

// A tile of BM tokens x BN columns by WM x WN waves, a ring of S stages of SK
// steps each.  AHEAD: a part of a stage is read into registers while the matrix
// instructions of the part before it run (a second set of operand registers).
template <bool X8_, int BM_, int BN_, int WM_, int WN_, int S_, int OCC_, int SK_ = 2, bool AHEAD_ = true>
struct LinCfg {
  static constexpr bool X8 = X8_, AHEAD = AHEAD_;
  static constexpr int SK = SK_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, OCC = OCC_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int TM = BM / WM, TN = BN / WN;   // a wave's tokens and columns
  static constexpr int FT = TM / 32, FN = TN / 32;   // its 32-wide operand blocks
  static constexpr int kXRow = (X8 ? 128 : 64) * SK, kWRow = 64 * SK;   // bytes per staged row
  static constexpr int kXLanes = kXRow / 16, kWLanes = kWRow / 16;   // lanes that copy one row
  // 1 KB pieces (one copy of a wave) per stage and per wave; where there are
  // fewer pieces than waves, some waves copy the same piece (the same bytes
  // to the same place), so that every wave has the same count outstanding.
  // Scales: 16 rows x four steps x 4 bytes per copy (four lanes a row), read
  // one word per row and step; against one copy per step and a byte read per
  // matrix instruction 2 to 15% of the time (T = 1024, N = 4096: 12.8 -> 11.1
  // us as 64 x 64 with FP4; T = 16384: 130 -> 126 as 256 x 256 with FP8).
  static constexpr int NX = BM * kXRow / 1024, NW = BN * kWRow / 1024, NS = (BM + BN) / 16;
  static constexpr int PX = (NX + kWaves - 1) / kWaves, PW = (NW + kWaves - 1) / kWaves,
                       PS = (NS + kWaves - 1) / kWaves;
  static constexpr int kCopies = PX + PW;
  static constexpr int kW = BM * kXRow, kStage = kW + BN * kWRow;
  // Scales: a ring of groups of kScaleSteps steps, GS stages.  Those of a
  // group are copied when the stage S before its first has been read, by
  // when the last stage of the group kScaleGroups before it has been, too.
  static constexpr int GS = kScaleSteps / SK, kScaleGroups = (S + 2 * GS - 2) / GS;
  static constexpr int kScales = S * kStage, kScaleRow = kScaleSteps * 4, kScaleGroup = (BM + BN) * kScaleRow;
  static constexpr int kLds = kScales + kScaleGroups * kScaleGroup;
  static_assert(NX % PX == 0 && NW % PW == 0, "a wave's pieces follow each other");
  static_assert(FT >= 1 && FN >= 1 && FT * 32 * WM == BM && FN * 32 * WN == BN, "whole blocks");
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
  static_assert((S - 2) * kCopies + ((S - 2) / GS + 1) * PS + (AHEAD ? kCopies + PS : 0) <= 63, "the vector-memory counter has six bits");
};

// 16-byte chunk slot of chunk c of staged row r: the 16 rows that one phase of
// a 16-byte read touches lie in distinct banks.
template <int ROW>
__device__ __forceinline__ int slot_of(int r, int c) {
  return c ^ (ROW == 256 ? r & 15 : ROW == 128 ? (r >> 1) & 7 : (r >> 2) & 3);
}

// Column (within a block of 32) of the matrix instruction's row i = 8 a + 4 h + b:
// a lane of half h holds the columns 8 h .. +7 (a = 0, 1) and 16 + 8 h .. +7 (a =
// 2, 3), two 16-byte stores.
__device__ __forceinline__ int col_of(int i) { return 16 * (i / 16) + 8 * (i / 4 % 2) + 4 * (i / 8 % 2) + i % 4; }

// A per-lane LDS address as one register, so that the reads from it differ in
// their constant offsets alone.
__device__ __forceinline__ uint32_t opaque_vgpr(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ __attribute__((address_space(3))) u32x4_t* lds_out(uint32_t a) {
  return reinterpret_cast<__attribute__((address_space(3))) u32x4_t*>(static_cast<uintptr_t>(a));
}

// Every LDS operation of this wave is done.  The builtin, not assembly: the
// compiler has to know it, or it would wait for the following stage's reads
// before the matrix instructions.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0) alone
  asm volatile("" ::: "memory");
}
// Behind a barrier the next copies, or the results, overwrite what was read
// last: this wave's reads are done at it, wherever the compiler puts the matrix
// instructions that wait for them.  No cost where they are done already (the
// counter is at zero).
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Waits until everything up to a stage has landed, `later` stages (at most
// MAX) having been issued after it: COPIES copies each, and SCALES more for
// every GS-th, one more of those if `extra`.
template <int MAX, int COPIES, int SCALES, int GS>
__device__ __forceinline__ void wait_stages(int later, bool extra) {
  if (later >= MAX) {
    if (extra) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MAX * COPIES + (MAX / GS + 1) * SCALES) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MAX * COPIES + MAX / GS * SCALES) : "memory");
  } else if constexpr (MAX > 0) {
    wait_stages<MAX - 1, COPIES, SCALES, GS>(later, extra);
  }
}

// N copies of 1 KB to consecutive places in LDS, lane offsets off[0 .. N).  The
// instruction's offset moves both of its addresses, so four copies share one
// LDS base; off[j] leaves out what the instruction adds: the caller puts `base`
// 3 KB before the tile and 3 KB less j % 4 KB into off[j]; the s_nop as in
// dma16.  Against an address per copy a stage of one wave takes 16 instructions
// fewer (T = 1, N = 4096, K = 2048: 5.7 -> 5.3 us with FP8), 128 x 128 with FP4
// at T = 16384 98 -> 92.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // M0 is reserved; nothing else here uses it
template <int N>
__device__ __forceinline__ void copy_pieces(const uint8_t* base, const uint32_t* off, uint32_t to) {
  const void* b = uniform_ptr(base);
  const uint32_t m = __builtin_amdgcn_readfirstlane(to);
  if constexpr (N == 1) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off[0]), "s"(b), "s"(m) : "memory", "m0");
  } else if constexpr (N == 2) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024"
                 ::"v"(off[0]), "v"(off[1]), "s"(b), "s"(m) : "memory", "m0");
  } else if constexpr (N == 4) {
    asm volatile("s_mov_b32 m0, %5\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %4\n\tglobal_load_lds_dwordx4 %1, %4 offset:1024\n\t"
                 "global_load_lds_dwordx4 %2, %4 offset:2048\n\tglobal_load_lds_dwordx4 %3, %4 offset:%6"
                 ::"v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(b), "s"(m), "n"(3 * 1024) : "memory", "m0");
  } else {
    static_assert(N % 4 == 0, "1, 2 or a multiple of 4");
#pragma unroll
    for (int j = 0; j < N; j += 4) copy_pieces<4>(base, off + j, to + j * 1024);
  }
}
#pragma clang diagnostic pop

struct LinArgs {
  int64_t T;
  int K, N;
  const uint8_t *x, *xs, *w, *ws;
  uint16_t* y;
  int64_t y_stride;
  int m_tiles, n_tiles;
  int64_t first, count;   // the launch's tiles
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::OCC)
mx_linear_kernel(LinArgs a) {
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];   // rows of at most 256 bytes
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int r32 = lane & 31, h = lane >> 5;

  // Tiles are dealt to the XCDs in contiguous runs; within a run, groups of
  // up to 8 token tiles with the column tiles running over them, so that the
  // tiles that run together share both operands in the XCD's L2.
  int64_t tile;
  {
    const int64_t per_xcd = (a.count + kXcds - 1) / kXcds;
    const int64_t b = blockIdx.x;
    tile = (b % kXcds) * per_xcd + b / kXcds;
    if (b / kXcds >= per_xcd || tile >= a.count) return;
    tile += a.first;
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
  const int steps = a.K / kStep, stages = (steps + C::SK - 1) / C::SK;
  const uint8_t* x_base = a.x + m0 * x_pitch - 3 * 1024;
  const uint8_t* w_base = a.w + n0 * w_pitch - 3 * 1024;
  // Copy sources and destinations; rows past the operand are clamped to its
  // last (they feed only outputs that are not stored).
  const uint32_t lds0 = lds_addr(lds);
  uint32_t x_off[C::PX], w_off[C::PW], s_off[C::PS], s_dst[C::PS];
  const int x_piece = wave * C::PX % C::NX, w_piece = wave * C::PW % C::NW;   // the wave's first
  const uint32_t x_dst = lds0 + x_piece * 1024, w_dst = lds0 + C::kW + w_piece * 1024;
  const uint8_t* s_base[C::PS];
  int s_flip[C::PS];
  uint32_t x_upper = 0, w_upper = 0;   // bit j: the lane's chunk of copy j lies in the stage's second step
#pragma unroll
  for (int j = 0; j < C::PX; ++j) {
    const int row = (x_piece + j) * (kWave / C::kXLanes) + lane / C::kXLanes;
    const int chunk = slot_of<C::kXRow>(row, lane % C::kXLanes);
    x_off[j] = static_cast<uint32_t>(min(row, rows - 1)) * static_cast<uint32_t>(x_pitch) + chunk * 16 + (3 - j % 4) * 1024;
    x_upper |= (chunk >= C::kXLanes / 2 ? 1u : 0u) << j;
  }
#pragma unroll
  for (int j = 0; j < C::PW; ++j) {
    const int row = (w_piece + j) * (kWave / C::kWLanes) + lane / C::kWLanes;
    const int chunk = slot_of<C::kWRow>(row, lane % C::kWLanes);
    w_off[j] = static_cast<uint32_t>(min(row, cols - 1)) * static_cast<uint32_t>(w_pitch) + chunk * 16 + (3 - j % 4) * 1024;
    w_upper |= (chunk >= C::kWLanes / 2 ? 1u : 0u) << j;
  }
#pragma unroll
  for (int j = 0; j < C::PS; ++j) {
    const int piece = (wave + j * C::kWaves) % C::NS;
    const bool of_x = piece < C::BM / 16;
    s_base[j] = of_x ? a.xs + m0 * s_pitch : a.ws + n0 * s_pitch;
    s_off[j] = min((of_x ? piece : piece - C::BM / 16) * 16 + lane / 4, (of_x ? rows : cols) - 1) * s_pitch;
    s_dst[j] = lds0 + C::kScales + piece * 256;
    s_flip[j] = 2 * (piece & 1);   // the upper 16 of 32 rows: steps 2 3 0 1, so that 32 rows' reads miss each other's banks
  }
  // Issues the copies of the next stage (stages are issued in order).
  int next = 0;
  uint32_t next_slot = 0, next_group = 0;
  auto issue = [&]() {
    if (next % C::GS == 0) {
#pragma unroll
      for (int j = 0; j < C::PS; ++j)
        dma4_off(s_base[j], s_off[j] + min(next * C::SK + ((lane & 3) ^ s_flip[j]), steps - 1) * 4,
                 s_dst[j] + next_group);
      next_group += C::kScaleGroup;
      if (next_group == C::kScaleGroups * C::kScaleGroup) next_group = 0;
    }
    const uint8_t* xb = x_base + static_cast<int64_t>(next) * C::kXRow;
    const uint8_t* wb = w_base + static_cast<int64_t>(next) * C::kWRow;
    if (C::SK == 2 && next * 2 + 1 == steps) {
      // an odd number of steps: the last stage's second half lies behind the
      // row and is filled from the first (never multiplied)
      uint32_t x_last[C::PX], w_last[C::PW];
#pragma unroll
      for (int j = 0; j < C::PX; ++j) x_last[j] = (x_upper >> j) & 1u ? x_off[j] - C::kXRow / 2 : x_off[j];
#pragma unroll
      for (int j = 0; j < C::PW; ++j) w_last[j] = (w_upper >> j) & 1u ? w_off[j] - C::kWRow / 2 : w_off[j];
      copy_pieces<C::PX>(xb, x_last, x_dst + next_slot);
      copy_pieces<C::PW>(wb, w_last, w_dst + next_slot);
    } else {
      copy_pieces<C::PX>(xb, x_off, x_dst + next_slot);
      copy_pieces<C::PW>(wb, w_off, w_dst + next_slot);
    }
    ++next;
    next_slot += C::kStage;
    if (next_slot == C::S * C::kStage) next_slot = 0;
  };
  // Stage st has landed in this wave: at most the stages issued after it, up
  // to `next`, are outstanding.
  auto wait_stage = [&](int st, auto most) {
    constexpr int kMost = decltype(most)::value;
    if constexpr (kMost == 0) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
      const int later = min(kMost, stages - 1 - st);
      wait_stages<kMost, C::kCopies, C::PS, C::GS>(later, (st + later) / C::GS - st / C::GS > later / C::GS);
    }
  };

  floatx16_t acc[C::FN][C::FT];
#pragma unroll
  for (int f = 0; f < C::FN; ++f)
#pragma unroll
    for (int t = 0; t < C::FT; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[f][t][v] = 0.0f;

  // The lane's rows, and its LDS offsets within a stage per step and matrix
  // instruction (and for FP8 per half of its 32 bytes).  Blocks lie 32 rows
  // apart, where the slots repeat.
  const int xr = wm * C::TM + r32, wr = wn * C::TN + col_of(r32);
  const uint32_t x_lane = lds0 + xr * C::kXRow + slot_of<C::kXRow>(xr, h) * 16;
  const uint32_t w_lane = lds0 + C::kW + wr * C::kWRow + slot_of<C::kWRow>(wr, h) * 16;
  const uint32_t xs_lane = lds0 + C::kScales + xr * C::kScaleRow + (xr & 16) / 2;
  const uint32_t ws_lane = lds0 + C::kScales + (C::BM + wr) * C::kScaleRow + (wr & 16) / 2;
  using u32_steps = uint32_t __attribute__((ext_vector_type(C::SK)));
  struct Frags {   // one matrix instruction's worth of K
    u32x4_t x[C::FT][C::X8 ? 2 : 1], w[C::FN];
  };
  struct Scales {   // a stage's: per step the 4 bytes of the rows' 128 elements
    u32_steps x[C::FT], w[C::FN];
  };
  uint32_t slot = 0, sc = 0;   // LDS offsets of the stage being read and of its first step's scales
  auto advance = [&]() {
    slot += C::kStage;
    if (slot == C::S * C::kStage) slot = 0;
    sc += C::SK * 4;
    if (sc % C::kScaleRow == 0) sc += C::kScaleGroup - C::kScaleRow;   // the next group's first step
    if (sc == C::kScaleGroups * C::kScaleGroup) sc = 0;
  };
  auto read = [&](auto part, Frags& f) {   // part of the stage: step part / 2, instruction part % 2
    constexpr int kSub = decltype(part)::value / 2, kHalf = decltype(part)::value % 2;
    // chunk c ^ (h ^ row) of the row's slots: h is bit 0 of the chunk, the part its upper bits
    const uint32_t wa = opaque_vgpr((w_lane + slot) ^ (4 * kSub + 2 * kHalf) * 16);
    const uint32_t xa = opaque_vgpr((x_lane + slot) ^ (C::X8 ? 8 * kSub + 4 * kHalf : 4 * kSub + 2 * kHalf) * 16);
    const uint32_t xb = C::X8 ? opaque_vgpr((x_lane + slot) ^ (8 * kSub + 4 * kHalf + 2) * 16) : 0u;
#pragma unroll
    for (int n = 0; n < C::FN; ++n) f.w[n] = *lds_ptr<u32x4_t>(wa + n * 32 * C::kWRow);
#pragma unroll
    for (int t = 0; t < C::FT; ++t) {
      f.x[t][0] = *lds_ptr<u32x4_t>(xa + t * 32 * C::kXRow);
      if constexpr (C::X8) f.x[t][1] = *lds_ptr<u32x4_t>(xb + t * 32 * C::kXRow);
    }
  };
  auto read_scales = [&](Scales& g) {
    const uint32_t at = sc % C::kScaleRow, group = sc - at;   // exchanged halves: see the copies
    const uint32_t xs = opaque_vgpr((xs_lane ^ at) + group), ws = opaque_vgpr((ws_lane ^ at) + group);
#pragma unroll
    for (int n = 0; n < C::FN; ++n) g.w[n] = *lds_ptr<u32_steps>(ws + n * 32 * C::kScaleRow);
#pragma unroll
    for (int t = 0; t < C::FT; ++t) g.x[t] = *lds_ptr<u32_steps>(xs + t * 32 * C::kScaleRow);
  };
  // The lane's byte of a matrix instruction becomes byte 0 or 2, which the
  // instruction selects.
  auto shift_scales = [&](const Scales& g, Scales& o) {
#pragma unroll
    for (int n = 0; n < C::FN; ++n) o.w[n] = g.w[n] >> (8u * h);
#pragma unroll
    for (int t = 0; t < C::FT; ++t) o.x[t] = g.x[t] >> (8u * h);
  };
  auto multiply = [&](auto part, const Frags& f, const Scales& g) {
    constexpr int kSub = decltype(part)::value / 2, kHalf = decltype(part)::value % 2;
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
        // formats: 4 = FP4 E2M1, 0 = FP8 E4M3; scale byte 0 or 2 of the register
        acc[n][t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wv, xv, acc[n][t], 4, C::X8 ? 0 : 4, 2 * kHalf, static_cast<int>(g.w[n][kSub]), 2 * kHalf,
            static_cast<int>(g.x[t][kSub]));
      }
    }
  };
  constexpr std::integral_constant<int, 0> p0{};
  constexpr std::integral_constant<int, 1> p1{};
  constexpr std::integral_constant<int, 2> p2{};
  constexpr std::integral_constant<int, 3> p3{};
  const bool odd_steps = C::SK == 2 && steps % 2 != 0;

  if constexpr (C::AHEAD) {
    // A stage's slot is free once every wave has its last part in registers:
    // at the barrier in front of that part's matrix instructions.
    Frags even, odd;
    Scales scales, loaded;
    constexpr std::integral_constant<int, 2 * C::SK - 1> last{};
    for (int s = 0; s < C::S && s < stages; ++s) issue();
    wait_stage(0, std::integral_constant<int, C::S - 1>{});
    barrier();
    read_scales(loaded);
    read(p0, even);
    for (int st = 0; st < stages; ++st) {
      read(p1, odd);
      shift_scales(loaded, scales);
      multiply(p0, even, scales);
      if constexpr (C::SK == 2) {
        if (!odd_steps || st + 1 < stages) {
          read(p2, even);
          multiply(p1, odd, scales);
          read(p3, odd);
          multiply(p2, even, scales);
        } else {   // the last part's scales are those of the only step
#pragma unroll
          for (int n = 0; n < C::FN; ++n) scales.w[n][1] = scales.w[n][0];
#pragma unroll
          for (int t = 0; t < C::FT; ++t) scales.x[t][1] = scales.x[t][0];
        }
      }
      wait_lds();
      if (st + 1 < stages) {
        wait_stage(st + 1, std::integral_constant<int, C::S - 2>{});
        barrier();
        if (next < stages) issue();
        advance();
        read_scales(loaded);
        read(p0, even);
      }
      multiply(last, odd, scales);
    }
  } else {
    for (int s = 0; s < C::S - 1 && s < stages; ++s) issue();
    for (int st = 0; st < stages; ++st) {
      // stage st has landed in every wave, and every wave has stage st - 1 in registers
      wait_stage(st, std::integral_constant<int, C::S - 2>{});
      barrier();
      if (next < stages) issue();
      Frags f;
      Scales scales;
      read_scales(scales);
      read(p0, f);
      shift_scales(scales, scales);
      multiply(p0, f, scales);
      read(p1, f);
      multiply(p1, f, scales);
      if constexpr (C::SK == 2) {
        if (!odd_steps || st + 1 < stages) {
          read(p2, f);
          multiply(p2, f, scales);
          read(p3, f);
          multiply(p3, f, scales);
        }
      }
      advance();
    }
  }

  // The wave's results, rounded, go through its own part of the ring 32 rows
  // at a time and leave as whole rows of its columns (16-byte chunks, slots as
  // the operands'): against 16-byte stores from the accumulators, of which two
  // make 32 bytes of a row, 4 to 10% of the time of 8192 x 2048 columns.
  // Non-temporal: y is not read again here, and the operands stay in the L2.
  constexpr int kOutRow = C::TN * 2, kOutChunks = kOutRow / 16, kOutRows = kWave / kOutChunks;
  static_assert(C::kWaves * 32 * kOutRow <= C::kScales, "the staged rows fit in the ring");
  barrier();   // every wave is past its last read of the ring, and every copy has landed
  const uint32_t out = lds0 + wave * (32 * kOutRow);
  const int out_row = lane / kOutChunks, out_chunk = lane % kOutChunks;
  const int n = wn * C::TN + out_chunk * 8;
#pragma unroll
  for (int t = 0; t < C::FT; ++t) {
#pragma unroll
    for (int f = 0; f < C::FN; ++f)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const floatx16_t& v = acc[f][t];
        *lds_out(out + r32 * kOutRow + slot_of<kOutRow>(r32, 4 * f + 2 * q + h) * 16) =
            u32x4_t{pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                    pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7])};
      }
    wait_lds();
#pragma unroll
    for (int p = 0; p < 32 / kOutRows; ++p) {
      const int row = p * kOutRows + out_row, tr = wm * C::TM + 32 * t + row;
      const u32x4_t o = *lds_ptr<u32x4_t>(out + row * kOutRow + slot_of<kOutRow>(row, out_chunk) * 16);
      if (tr < rows && n < cols)
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(a.y + (m0 + tr) * a.y_stride + n0 + n));
    }
  }
}

template <class C>
bool launch_cfg(LinArgs a, hipStream_t s) {
  static OncePerDevice lds;
  if (!set_lds(lds, &mx_linear_kernel<C>, C::kLds)) return launch_ok("mx_linear") && false;
  a.m_tiles = static_cast<int>((a.T + C::BM - 1) / C::BM);
  a.n_tiles = (a.N + C::BN - 1) / C::BN;
  launch_parts(static_cast<int64_t>(a.m_tiles) * a.n_tiles, C::kThreads, [&](int64_t first, int64_t count) {
    a.first = first;
    a.count = count;
    launch_kernel("mx_linear", mx_linear_kernel<C>, dim3(xcd_grid(count)), dim3(C::kThreads), C::kLds, s, a);
  });
  return launch_ok("mx_linear");
}

// Tiles of BM x BN in a product.
int64_t tiles_of(const LinArgs& a, int bm, int bn) {
  return (a.T + bm - 1) / bm * static_cast<int64_t>((a.N + bn - 1) / bn);
}

// The tile: the larger, the fewer bytes a product copies, but every CU wants
// one.
//   32 x 32 up to 512 tiles (two a CU; up to 1024 for at most 32 tokens, half of
//     whose rows a tile of 64 would leave empty: T = 1, N = 32768, K = 4096 12.2
//     us against 13.7 with FP8, 12.0 against 12.4), then 64 x 64 up to 640: N = 4096, K =
//     2048, T = 1: 5.3 us against 6.0 with 64 x 64 (FP8; 4.8 against 5.1 with
//     FP4); T = 128: 5.8 against 6.2; T = 200: 6.6 against 6.4; T = 500: 8.8 (64 x
//     64) against 10.9 (128 x 128); T = 1024: 16.1 against 13.2.
//   64 x 128 for at most 64 tokens beyond that, half of whose rows a tile of
//     128 would leave empty: T = 48, N = 65536: 13.3 us, as 64 x 64, with FP4,
//     14.0 against 16.4 with FP8.
//   FP4: 128 x 128 or 256 x 256 by rounds over the chip: two of the former run
//     on a CU at once, and a round of 512 takes 1 / 1.6 of a round of 256 of the
//     latter, its last one 0.65 of that where it has at most one tile a CU.  T
//     = 5001, K = 4096, N = 2048 (1.25 against 0.6 rounds): 35 against 32 us;
//     T = 10000, K = 2048 (2.5 against 1.25): 29 against 35; T = 1500, N =
//     4096: 13 against 17; T = 16384: 92 against 88.
//   FP8, whose instructions take twice as long per byte of w: 128 x 128 with
//     stages of two steps for at most one tile a CU (256 tiles 12.8 us against
//     16.9 with 128 x 256), beyond that the smallest of 128 x 256, 192 x 256 and
//     256 x 256 of which one round over the chip does: N = 4096, K = 2048, T =
//     2048 18.6, 22.2, 24.0 us, T = 2560 24.5, 22.4, 25.2; N = 2048, K = 4096, T
//     = 5001 46.1, 39.4, 42.5, T = 8192 55.9, 77.4, 53.6.  Beyond one round 128 x
//     256, two of which run on a CU at once: T = 10000, N = 4096, K = 2048 69,
//     87, 81; T = 16384 113, 133, 121.
template <bool X8>
bool launch_format(const LinArgs& a, hipStream_t s) {
  if (tiles_of(a, 32, 32) <= (a.T <= 32 ? 1024 : 512)) return launch_cfg<LinCfg<X8, 32, 32, 1, 1, 2, 2>>(a, s);
  if (tiles_of(a, 64, 64) <= 640) return launch_cfg<LinCfg<X8, 64, 64, 2, 2, 2, 2>>(a, s);
  if (a.T <= 64) return launch_cfg<LinCfg<X8, 64, 128, 2, 2, 2, 2>>(a, s);
  const int64_t n128 = tiles_of(a, 128, 128), n256 = tiles_of(a, 256, 256);
  if constexpr (X8) {
    if (n128 <= 256) return launch_cfg<LinCfg<true, 128, 128, 4, 2, 2, 2>>(a, s);
    if (tiles_of(a, 128, 256) > 256 && n256 <= 256) {
      if (tiles_of(a, 192, 256) <= 256) return launch_cfg<LinCfg<true, 192, 256, 3, 4, 2, 1, 1, false>>(a, s);
    } else {
      return launch_cfg<LinCfg<true, 128, 256, 2, 4, 2, 2, 1, false>>(a, s);
    }
  } else {
    const double rounds128 = static_cast<double>(n128 / 512) + (n128 % 512 > 256 ? 1.0 : n128 % 512 > 0 ? 0.65 : 0.0);
    if (rounds128 <= 1.6 * static_cast<double>((n256 + 255) / 256))
      return launch_cfg<LinCfg<false, 128, 128, 2, 2, 2, 2>>(a, s);
  }
  // 16 waves of 64 x 64, whose registers a second set of operands would not
  // fit in; with FP8 stages of one step, for the ring to fit in LDS
  return launch_cfg<LinCfg<X8, 256, 256, 4, 4, 2, 1, X8 ? 1 : 2, false>>(a, s);
}

}  // namespace

bool launch_mx_linear(int64_t T, int K, int N, bool x_fp8, const uint8_t* x, const uint8_t* xs, const uint8_t* w,
                      const uint8_t* ws, uint16_t* y, int64_t y_stride, hipStream_t s) {
  if (T == 0) return true;
  const LinArgs a{T, K, N, x, xs, w, ws, y, y_stride, 0, 0, 0, 0};
  return x_fp8 ? launch_format<true>(a, s) : launch_format<false>(a, s);
}

}  // namespace w4a4
