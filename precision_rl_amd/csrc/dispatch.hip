// Token dispatch around separate expert calls on gfx950: tokens sorted by
// expert and back with the router's weights applied, and both gradients.
//
//   permute         xp[row_map[t,j]] = x[t];  pad rows zero
//   its gradient    dx[t] = rnd(sum_j dxp[row_map[t,j]])
//   unpermute       y[t] = rnd(sum_j p[t,j] o[row_map[t,j]])
//   its gradient    do[row_map[t,j]] = rnd(p[t,j] dy[t]);  pad rows zero
//                   dp[t,j] = sum_h dy[t,h] o[row_map[t,j],h]
//
// Sums run in FP32, those over j in ascending j, and are rounded once.  A slot
// whose expert id lies outside [0, E) is not dispatched: its row_map entry is
// -1 and it adds nothing.  Every row index is checked against the buffer's rows
// before it is used.
//
// All four move rows and compute next to nothing: HBM binds them, every row is
// read or written once, and a token's row is read once for its k destinations.
// Linear copies of 1 GiB reach 6.5 TB/s on this card, rows of 4 KB in the order
// of the tokens 5.5 to 5.9: 16384 tokens of 2048 in bf16 with 8 of 128 experts
// each take 110 us sorted (101 the copy, 9 the maps), 102 combined, 202 for the
// combination's gradients (100 dp, 101 do).  Two kernels that went by expert rows
// instead, so that those are streamed and the tokens' come from the memory-side
// cache, took 140 for 101 (the copy) and 220 for 207 (both gradients in one).
// One token takes 3.4 us sorted, 48 3.3 combined, 61 4.2 for the gradients.
//
// The quantising permute's routing (quantize.hip) and the expert path's own
// gather, scatter and pad rows (elementwise.hip) are not built on these: they take
// bf16 rows of calls whose every slot is dispatched, quantise in the same pass,
// and their layout, which is the same, is pinned by their own tests.

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"
#include "launch_parts.h"
#include "row_walk.h"

namespace w4a4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxK = 8;
constexpr int kMaxE = 1024;
// Entries (token, slot) that one workgroup of the counting kernel ranks.
constexpr int kRankChunk = 1024;

int64_t rank_chunks(int64_t T, int k) { return (T * k + kRankChunk - 1) / kRankChunk; }

// Whether every workgroup counts all entries itself, in one launch: T / 8
// workgroups of T k entries each.  Against count, scan and copy in three launches
// (rows of 512 bytes, on the device): 2048 tokens with 8 experts each 8.7 us
// against 10.5, 4096 with one 7.6 against 10.1; 8192 with two 24.5 against 11.3.
bool one_launch(int64_t T, int k) { return T <= 5792 && T * T * k <= int64_t{1} << 25; }
// Up to how many tokens a workgroup takes one of them instead of eight: 256
// tokens 4.9 us against 5.3, 512 6.2 against 5.8.
constexpr int kOneTokenAWorkgroup = 256;

// A 16-byte chunk of a row.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {   // bf16
  static constexpr int N = 8;
  u32x4_t w;
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = pack_bf16x2(v[2 * d], v[2 * d + 1]);
  }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  u32x4_t w;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ void put(const float (&v)[4]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = __float_as_uint(v[d]);
  }
};

// --------------------------------------------------------------- the maps
// Lanes of the wave with the same e (below 1024) as this one, among `live` ones:
// one vote per bit of e.
__device__ __forceinline__ uint64_t same_lanes(int e, bool live) {
  uint64_t m = __ballot(live);
#pragma unroll
  for (int bit = 0; bit < 10; ++bit) {
    const uint64_t v = __ballot((e >> bit) & 1);
    m &= (e >> bit) & 1 ? v : ~v;
  }
  return m;
}
__device__ __forceinline__ uint64_t lanes_below() {
  return (uint64_t{1} << (threadIdx.x % kWave)) - 1;
}
__device__ __forceinline__ bool in_range(int e, int E) { return static_cast<uint32_t>(e) < static_cast<uint32_t>(E); }

// Per chunk of 1024 entries, one thread each: an entry's rank within the chunk
// among those of its expert (ascending t * k + j, also where a token names an
// expert twice), parked in row_map, and the chunk's counts.  The waves' counts
// per expert meet in LDS.  Count and scan take 3.4 to 4.9 us each for 131072
// entries of 128 experts; adding the chunks' counts up in every workgroup of the
// copy instead of a scan saves nothing there and costs 14 us with rows of 256
// bytes.
__global__ void __launch_bounds__(kRankChunk)
permute_count_kernel(int64_t n, int E, const int32_t* __restrict__ idx, int32_t* __restrict__ row_map,
                     int32_t* __restrict__ counts) {
  constexpr int W = kRankChunk / kWave;
  extern __shared__ __attribute__((aligned(16))) uint16_t s_count[];   // [W][E]
  const int tid = threadIdx.x;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRankChunk + tid;
  const int e = i < n ? idx[i] : -1;
  const bool live = in_range(e, E);
  for (int c = tid; c < W * E / 2; c += kRankChunk) reinterpret_cast<uint32_t*>(s_count)[c] = 0u;
  __syncthreads();
  const uint64_t same = same_lanes(e, live);
  uint16_t* const mine = s_count + tid / kWave * E + e;
  if (live && (same & lanes_below()) == 0) *mine = static_cast<uint16_t>(__popcll(same));
  __syncthreads();
  if (tid < E) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = s_count[w * E + tid];
      s_count[w * E + tid] = static_cast<uint16_t>(run);
      run += v;
    }
    counts[static_cast<int64_t>(blockIdx.x) * E + tid] = run;
  }
  __syncthreads();
  if (live) row_map[i] = *mine + __popcll(same & lanes_below());
}
inline uint32_t count_lds_bytes(int E) { return static_cast<uint32_t>(kRankChunk / kWave * E) * 2u; }

// One workgroup of 1024 threads: thread (s, e) sums a segment of the chunks'
// counts of expert e (the first kKeep stay in registers), the segments of an
// expert are scanned in LDS, the chunks' running sums written over the counts,
// and the experts' padded totals scanned by a thread each.  cols: E rounded up
// to a power of two.  131072 entries take 4.3 us with 32 experts, 4.6 with 128, and
// with more, whose segments are longer than kKeep, 10.5 with 256, 22 with 512 and
// 47 with 1024.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads)
permute_scan_kernel(int32_t* __restrict__ counts, int n_chunks, int E, int cols, int align,
                    int32_t* __restrict__ offsets, int32_t* __restrict__ expert_count) {
  constexpr int kKeep = 16;
  __shared__ int32_t s_sum[kScanThreads], s_wave[kScanThreads / kWave];
  const int tid = threadIdx.x, e = tid & (cols - 1), seg = tid / cols, segs = kScanThreads / cols;
  const int per = (n_chunks + segs - 1) / segs;
  const int c0 = min(n_chunks, seg * per), c1 = e < E ? min(n_chunks, c0 + per) : c0;
  int keep[kKeep];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    keep[i] = c0 + i < c1 ? counts[static_cast<int64_t>(c0 + i) * E + e] : 0;
    sum += keep[i];
  }
  for (int c = c0 + kKeep; c < c1; ++c) sum += counts[static_cast<int64_t>(c) * E + e];
  int run = sum;
  for (int d = cols; d < kScanThreads; d <<= 1) {
    s_sum[tid] = run;
    __syncthreads();
    const int u = tid >= d ? s_sum[tid - d] : 0;
    __syncthreads();
    run += u;
  }
  s_sum[tid] = run;
  run -= sum;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    if (c0 + i < c1) counts[static_cast<int64_t>(c0 + i) * E + e] = run;
    run += keep[i];
  }
  for (int c = c0 + kKeep; c < c1; ++c) {
    const int64_t i = static_cast<int64_t>(c) * E + e;
    const int v = counts[i];
    counts[i] = run;
    run += v;
  }
  __syncthreads();
  const int total = tid < E ? s_sum[kScanThreads - cols + tid] : 0;
  const int padded = (total + align - 1) / align * align;
  int incl = padded;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int u = __shfl_up(incl, d, kWave);
    if (tid % kWave >= d) incl += u;
  }
  if (tid % kWave == kWave - 1) s_wave[tid / kWave] = incl;
  __syncthreads();
  for (int w = 0; w < tid / kWave; ++w) incl += s_wave[w];
  if (tid < E) {
    expert_count[tid] = total;
    offsets[tid + 1] = incl;
    if (tid == 0) offsets[0] = 0;
  }
}

struct PermuteArgs {
  int64_t T;
  int chunks, k, E, align;             // chunks: 16-byte chunks of a row
  const uint8_t* x;
  int64_t x_pitch;                     // bytes
  const int32_t* idx;
  uint8_t* xp;                         // null: the maps alone
  int32_t *offsets, *row_map, *src_row;
  const int32_t *counts, *expert_count;
  int64_t token_blocks, first;         // workgroups of tokens (those of pad rows follow); this launch's first
  int pad_parts;                       // workgroups of pad rows per expert
  bool pads_past;                      // pad rows are stored past the caches
};

// Workgroups that clear the pad rows of an expert, of which there may be `rows`:
// 64 KiB to each, `most` for all experts (two of 256 threads a compute unit; fewer
// of those that count all entries first: 512 tokens of 4 KB in groups of 128 for
// 128 experts 14.3 us with 128, 15.4 with 512).  A workgroup an expert took 14.4
// us against 5.7 for the combination's gradients of 52 tokens of 7 KB in groups of
// 128 for 16 experts, 19.0 against 14.4 for 512 of 4 KB and 128 experts.
int pad_parts(int64_t rows, int chunks, int E, int most = 512) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((rows * chunks + 4095) / 4096, most / E)));
}

// A wave's zeros in row r, past the caches where the rows that the call may write,
// pads among them, are more than they hold: 1478 tokens of 14 KB sorted in groups
// of 64 for 171 experts 42 us against 53, 16384 of 4 KB in groups of 128 for 128
// 117 against 128; 64 of 8 KB 18.4 against 16.6.
__device__ __forceinline__ void clear_row(void* rows, int64_t r, int chunks, bool past) {
  u32x4_t* row = static_cast<u32x4_t*>(rows) + r * chunks;
  const u32x4_t zero{0u, 0u, 0u, 0u};
  if (past) {
    for (int c = threadIdx.x % kWave; c < chunks; c += kWave) __builtin_nontemporal_store(zero, row + c);
  } else {
    for (int c = threadIdx.x % kWave; c < chunks; c += kWave) row[c] = zero;
  }
}

// A part's share of the zeros in the pad rows [r0, r1) of an expert.
template <int THREADS>
__device__ __forceinline__ void clear_pad_rows(const PermuteArgs& a, int r0, int r1, int part) {
  const int tid = static_cast<int>(threadIdx.x);
  if (part == 0) walk_rows(r0, r1, tid, THREADS, [&](int64_t r) { a.src_row[r] = -1; });
  if (a.xp == nullptr) return;
  constexpr int W = THREADS / kWave;
  walk_rows(r0, r1, part * W + tid / kWave, a.pad_parts * W,
            [&](int64_t r) { clear_row(a.xp, r, a.chunks, a.pads_past); });
}

// Rows of a length that 64 bytes do not divide start anywhere in a line, and a
// wave's 64 chunks would write parts of the lines at both of its ends.  Where many
// are written, every destination gets its chunks in lanes counted from a line's
// start, so that only a row's own ends are written in parts.  A lane's chunk then
// differs from destination to destination: each loads its own, all before the
// first is stored (from the caches after the first).  16384 tokens of 2056 with 5
// experts each 88 us against 103 (of 2048: 71), 6760 of 6008 94 against 121; writes
// of less than 64 bytes are 2.2% of all against 5.0 (of 2048: 0.7).  With half of the
// slots dispatched 50 us against 58, with a quarter 38 against 35; not worth it
// with one destination (16384 of 2056 34 against 31), short rows (16384
// of 264 with 5 23.6 against 22.8), what the caches hold (2000 of 2056 with 5 17.0
// against 16.2) and in the one launch for few tokens (2500 of 4104 40 against 36).
bool by_lines(int64_t T, int k, int chunks) {
  return chunks % 4 != 0 && chunks >= 64 && k > 1 && T * k * chunks >= int64_t{1} << 22;
}
__device__ __forceinline__ int line_offset(const u32x4_t* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 4) & 7;
}

// For each destination row_of(j), j < k, that is one: store(j, p, chunk c of src)
// for all c, TEAM lanes.
template <int TEAM, class Row, class Store>
__device__ __forceinline__ void to_lines(const u32x4_t* src, u32x4_t* dst, int chunks, int k, int lane, Row row_of,
                                         Store store) {
  u32x4_t* to[kMaxK];
  int at[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    const int64_t r = j < k ? row_of(j) : -1;
    to[j] = dst + (r < 0 ? 0 : r) * chunks;
    at[j] = r < 0 ? 1 << 30 : lane - line_offset(to[j]);
  }
  for (int c0 = 0; c0 < chunks + 7; c0 += TEAM) {
    u32x4_t v[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (static_cast<uint32_t>(at[j] + c0) < static_cast<uint32_t>(chunks)) v[j] = src[at[j] + c0];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (static_cast<uint32_t>(at[j] + c0) < static_cast<uint32_t>(chunks)) store(j, to[j] + at[j] + c0, v[j]);
  }
}

// x[t]'s chunk `lane` where there is one, loaded ahead of the row indices.
__device__ __forceinline__ u32x4_t first_chunk(const PermuteArgs& a, int64_t t, int lane) {
  u32x4_t v{0u, 0u, 0u, 0u};
  if (a.xp != nullptr && t < a.T && lane < a.chunks)
    v = reinterpret_cast<const u32x4_t*>(a.x + t * a.x_pitch)[lane];
  return v;
}
template <int TEAM, bool LINES>
__device__ __forceinline__ void copy_token(const PermuteArgs& a, int64_t t, int lane, u32x4_t v, const int32_t* rows) {
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.x + t * a.x_pitch);
  u32x4_t* dst = reinterpret_cast<u32x4_t*>(a.xp);
  if constexpr (LINES) {
    to_lines<TEAM>(src, dst, a.chunks, a.k, lane, [&](int j) { return rows[j]; },
                   [](int, u32x4_t* p, const u32x4_t& w) { __builtin_nontemporal_store(w, p); });
    return;
  }
  for (int c = lane; c < a.chunks; c += TEAM) {
    if (c != lane) v = src[c];
    for (int j = 0; j < a.k; ++j) {
      const int r = rows[j];
      if (r >= 0) __builtin_nontemporal_store(v, dst + static_cast<int64_t>(r) * a.chunks + c);
    }
  }
}

// Few entries in one launch: each workgroup counts all of them by expert in LDS,
// those before its own G tokens apart, scans the padded group sizes, and copies
// its tokens, 256 threads each.
template <int THREADS, int G>
__global__ void __launch_bounds__(THREADS)
permute_few_kernel(PermuteArgs a) {
  constexpr int W = THREADS / kWave, kTeams = THREADS / kThreads;
  static_assert(G * kMaxK <= kWave && G % kTeams == 0, "one wave ranks the workgroup's entries");
  __shared__ int32_t s_before[kMaxE], s_after[kMaxE], s_off[kMaxE + 1], s_wave[W], s_row[G * kMaxK];
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, team = tid / kThreads, tl = tid % kThreads;
  const bool pads = blockIdx.x >= a.token_blocks;
  const int64_t t0 = pads ? a.T : static_cast<int64_t>(blockIdx.x) * G;
  const u32x4_t v = first_chunk(a, t0 + team, tl);
  for (int e = tid; e < a.E; e += THREADS) s_before[e] = s_after[e] = 0;
  const int n = static_cast<int>(a.T) * a.k, own0 = static_cast<int>(t0) * a.k;
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const int e = a.idx[i];
    if (in_range(e, a.E)) atomicAdd(i < own0 ? &s_before[e] : &s_after[e], 1);
  }
  __syncthreads();
  // exclusive scan of the padded group sizes: a thread's consecutive experts,
  // the wave's lanes, the waves
  const int per = (a.E + THREADS - 1) / THREADS, e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
  auto padded = [&](int e) { return (s_before[e] + s_after[e] + a.align - 1) / a.align * a.align; };
  int mine = 0;
  for (int e = e0; e < e1; ++e) mine += padded(e);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int u = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += u;
  }
  if (lane == kWave - 1) s_wave[wave] = incl;
  __syncthreads();
  int run = incl - mine;
  for (int w = 0; w < wave; ++w) run += s_wave[w];
  for (int e = e0; e < e1; ++e) {
    s_off[e] = run;
    run += padded(e);
  }
  if (tid == THREADS - 1) s_off[a.E] = run;   // the last thread's sum is the total
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = tid; e <= a.E; e += THREADS) a.offsets[e] = s_off[e];
  if (pads) {
    const int b = static_cast<int>(blockIdx.x - a.token_blocks), e = b / a.pad_parts;
    clear_pad_rows<THREADS>(a, s_off[e] + s_before[e] + s_after[e], s_off[e + 1], b % a.pad_parts);
    return;
  }
  if (wave == 0) {
    const int i = own0 + lane;
    const bool own = lane < G * a.k && i < n;
    const int e = own ? a.idx[i] : -1;
    const bool live = in_range(e, a.E);
    const uint64_t same = same_lanes(e, live);
    int row = -1;
    if (live) {
      row = s_off[e] + s_before[e] + __popcll(same & lanes_below());
      a.src_row[row] = static_cast<int32_t>(t0) + lane / a.k;
    }
    if (own) {
      a.row_map[i] = row;
      s_row[lane] = row;
    }
  }
  __syncthreads();
  if (a.xp == nullptr) return;
#pragma unroll
  for (int g = 0; g < G / kTeams; ++g) {
    const int own = g * kTeams + team;
    const int64_t t = t0 + own;
    if (t < a.T) copy_token<kThreads, false>(a, t, tl, g == 0 ? v : first_chunk(a, t, tl), s_row + own * a.k);
  }
}

// After the counts and their scan: TEAM lanes per token.
template <int TEAM, bool LINES>
__global__ void __launch_bounds__(kThreads)
permute_rows_kernel(PermuteArgs a) {
  constexpr int kTeams = kThreads / TEAM;
  __shared__ int32_t s_row[kTeams * kMaxK];
  const int tid = threadIdx.x, lane = tid % TEAM;
  const int64_t block = a.first + blockIdx.x;
  if (block >= a.token_blocks) {
    const int b = static_cast<int>(block - a.token_blocks), e = b / a.pad_parts;
    clear_pad_rows<kThreads>(a, a.offsets[e] + a.expert_count[e], a.offsets[e + 1], b % a.pad_parts);
    return;
  }
  const int64_t t0 = block * kTeams, t = t0 + tid / TEAM;
  const u32x4_t v = first_chunk(a, t, lane);
  const int64_t i = t0 * a.k + tid;
  if (tid < kTeams * a.k && i < a.T * a.k) {
    const int e = a.idx[i];
    int row = -1;
    if (in_range(e, a.E)) {
      row = a.offsets[e] + a.counts[i / kRankChunk * a.E + e] + a.row_map[i];
      a.src_row[row] = static_cast<int32_t>(t0 + tid / a.k);
    }
    a.row_map[i] = row;
    s_row[tid] = row;
  }
  __syncthreads();
  if (t < a.T && a.xp != nullptr) copy_token<TEAM, LINES>(a, t, lane, v, s_row + tid / TEAM * a.k);
}

__global__ void __launch_bounds__(kThreads)
clear_offsets_kernel(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) offsets[i] = 0;
}

// ------------------------------------------------------------ back to tokens
// NT: expert rows loaded past the caches, where streams() says so of the bytes of
// all slots: 16384 tokens of 2048 with 8 experts each combined in 102 us against
// 111, 2048 of them in 14.4 against 13.1; dp of 16384 in 100 against 109; both
// gradients in one pass of 8000 in 99 against 104, of 2048 in 28 against 24.  How
// many slots are dispatched is not known on the host: with a quarter of them the
// rule takes the slower side in between (8192 combined 18.4 us against 16.1, the
// gradients of 6144 25.4 against 22.9), and the faster one from there on (16384
// combined 33.8 against 37.5).  A choice at run time around each load keeps a lane's
// loads from being in flight together (110 us for 102), so both kernels are built
// both ways.  Tokens' rows are loaded through the caches: past them the sort takes
// as long (110 us).
template <bool NT>
__device__ __forceinline__ u32x4_t load16(const u32x4_t* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}

struct GatherArgs {
  int64_t T;
  int chunks, k;
  uint32_t magic, rows;       // magic: 2^32 / chunks, rounded up
  const void* src;            // [rows, H]
  const int32_t* row_map;
  const float* w;             // null: 1
  void* out;
  int64_t out_pitch;          // bytes
  int64_t first;
};

// A lane per output chunk, in flat order over the tokens' rows: its k loads (at
// most K) are all in flight, no lane is idle whatever the row length, and a wide
// row is work for several workgroups.
template <typename T, int K, bool NT>
__global__ void __launch_bounds__(kThreads)
gather_rows_kernel(GatherArgs a) {
  constexpr int N = Chunk<T>::N;
  const int64_t base = (a.first + blockIdx.x) * kThreads, t0 = base / a.chunks;
  // below chunks + 256, where magic divides exactly
  const uint32_t i = static_cast<uint32_t>(base - t0 * a.chunks) + threadIdx.x;
  const uint32_t q = a.chunks > 1 ? __umulhi(i, a.magic) : i;
  const int64_t t = t0 + q;
  const int c = static_cast<int>(i - q * a.chunks);
  if (t >= a.T) return;
  const u32x4_t* src = static_cast<const u32x4_t*>(a.src) + c;
  int32_t row[K];
  float w[K];
  Chunk<T> v[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    row[j] = j < a.k ? a.row_map[t * a.k + j] : -1;
    w[j] = a.w != nullptr && j < a.k ? a.w[t * a.k + j] : 1.0f;
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (static_cast<uint32_t>(row[j]) < a.rows) v[j].w = load16<NT>(src + static_cast<int64_t>(row[j]) * a.chunks);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (static_cast<uint32_t>(row[j]) < a.rows) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(w[j], v[j].get(i), acc[i]);
    }
  }
  Chunk<T> o;
  o.put(acc);
  __builtin_nontemporal_store(o.w, reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) + t * a.out_pitch) + c);
}

// ------------------------------------------------- gradient of the unpermute
struct UnpermuteBwdArgs {
  int64_t T;
  int chunks, k, E;
  uint32_t rows;
  const void* dy;
  int64_t dy_pitch;           // bytes
  const void* o;
  const int32_t* row_map;
  const float* w;
  const int32_t *offsets, *src_row;   // either may be null where no group is padded
  void* d_o;                  // null: dp alone
  float* dw;                  // null: do alone
  uint32_t apart;             // rows in use from which do is made by tokens and not beside dp
  int64_t main_blocks, first; // workgroups of entries or tokens (those of pad rows follow); this launch's first
  int pad_parts;              // workgroups of pad rows per expert
  bool pads_past;             // pad rows are stored past the caches
};

// Rows in use: entries of row_map at or past this are not dispatched.
__device__ __forceinline__ uint32_t used_rows(const UnpermuteBwdArgs& a) {
  return a.offsets != nullptr ? min(a.rows, static_cast<uint32_t>(max(a.offsets[a.E], 0))) : a.rows;
}

template <typename T>
__device__ __forceinline__ void store_scaled(const Chunk<T>& g, float w, u32x4_t* to) {
  constexpr int N = Chunk<T>::N;
  float p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = w * g.get(i);
  Chunk<T> q;
  q.put(p);
  __builtin_nontemporal_store(q.w, to);
}

// A part's share of the pad rows of an expert: up to 127 rows before its group's
// end (or the buffer's) with src_row -1, none where the last row is a slot's.
__device__ __forceinline__ void clear_pad_rows(const UnpermuteBwdArgs& a, int b) {
  const int e = b / a.pad_parts, part = b % a.pad_parts;
  const int64_t lo = max(a.offsets[e], 0);
  const int64_t hi = min(static_cast<int64_t>(a.offsets[e + 1]), static_cast<int64_t>(a.rows));
  if (lo >= hi || a.src_row[hi - 1] >= 0) return;
  walk_rows(max(lo, hi - 127), hi, part * kWaves + static_cast<int>(threadIdx.x) / kWave, a.pad_parts * kWaves,
            [&](int64_t r) {
              if (a.src_row[r] < 0) clear_row(a.d_o, r, a.chunks, a.pads_past);
            });
}

// LANES lanes: do[r] = w[i] dy[t] and dp[i] = <dy[t], o[r]> of entry i = t k + j.
// Lane l takes the chunks l, l + LANES, ... in order (four in flight), each summed
// by itself, the lanes join by halves: dp's bits depend on the row's length and
// type alone.
template <typename T, int LANES, bool NT>
__device__ __forceinline__ void entry_grad(const UnpermuteBwdArgs& a, int64_t t, int64_t i, uint32_t r, bool store) {
  constexpr int N = Chunk<T>::N, kAhead = 4;
  const int lane = threadIdx.x % LANES;
  const u32x4_t* dy = reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(a.dy) + t * a.dy_pitch);
  const u32x4_t* o = static_cast<const u32x4_t*>(a.o) + static_cast<int64_t>(r) * a.chunks;
  u32x4_t* d_o = static_cast<u32x4_t*>(a.d_o) + static_cast<int64_t>(r) * a.chunks;
  const float w = a.w[i];
  float sum = 0.0f;
  for (int c0 = lane; c0 < a.chunks; c0 += kAhead * LANES) {
    Chunk<T> g[kAhead], v[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int c = c0 + n * LANES;
      if (c >= a.chunks) continue;
      v[n].w = load16<NT>(o + c);
      g[n].w = dy[c];
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int c = c0 + n * LANES;
      if (c >= a.chunks) continue;
      if (store) store_scaled<T>(g[n], w, d_o + c);
      float part = g[n].get(0) * v[n].get(0);
#pragma unroll
      for (int q = 1; q < N; ++q) part = fmaf(g[n].get(q), v[n].get(q), part);
      sum += part;
    }
  }
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) a.dw[i] = sum;
}

// LANES lanes per entry; pad rows by workgroups of their own.
template <typename T, int LANES, bool NT>
__global__ void __launch_bounds__(kThreads)
unpermute_bwd_entries_kernel(UnpermuteBwdArgs a) {
  const int64_t block = a.first + blockIdx.x;
  if (block >= a.main_blocks) {
    clear_pad_rows(a, static_cast<int>(block - a.main_blocks));
    return;
  }
  int slot = threadIdx.x / LANES;
  if constexpr (LANES == kWave) slot = __builtin_amdgcn_readfirstlane(slot);
  const int64_t i = block * (kThreads / LANES) + slot;
  if (i >= a.T * a.k) return;
  const uint32_t r = static_cast<uint32_t>(a.row_map[i]), used = used_rows(a);
  if (r < used) entry_grad<T, LANES, NT>(a, i / a.k, i, r, a.d_o != nullptr && used < a.apart);
  else if (threadIdx.x % LANES == 0) a.dw[i] = 0.0f;
}

// do by itself: a workgroup per token, dy read once from memory (16384 tokens
// with 8 experts each 17 us with rows of up to 128, 26 with 512, 101 with 2048).
template <typename T, bool LINES>
__global__ void __launch_bounds__(kThreads)
unpermute_bwd_scatter_kernel(UnpermuteBwdArgs a) {
  const int64_t t = a.first + blockIdx.x;
  if (t >= a.main_blocks) {
    clear_pad_rows(a, static_cast<int>(t - a.main_blocks));
    return;
  }
  const uint32_t used = used_rows(a);
  if (used < a.apart) return;
  const u32x4_t* dy = reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(a.dy) + t * a.dy_pitch);
  if constexpr (LINES) {
    to_lines<kThreads>(
        dy, static_cast<u32x4_t*>(a.d_o), a.chunks, a.k, threadIdx.x,
        [&](int j) {
          const uint32_t r = static_cast<uint32_t>(a.row_map[t * a.k + j]);
          return r < used ? static_cast<int64_t>(r) : -1;
        },
        [&](int j, u32x4_t* p, const u32x4_t& w) { store_scaled<T>(Chunk<T>{w}, a.w[t * a.k + j], p); });
    return;
  }
  for (int c = threadIdx.x; c < a.chunks; c += kThreads) {
    Chunk<T> g;
    g.w = dy[c];
    for (int j = 0; j < a.k; ++j) {
      const uint32_t r = static_cast<uint32_t>(a.row_map[t * a.k + j]);
      if (r < used)
        store_scaled<T>(g, a.w[t * a.k + j], static_cast<u32x4_t*>(a.d_o) + static_cast<int64_t>(r) * a.chunks + c);
    }
  }
}

template <class F>
void with_slots(int k, F f) {
  if (k == 1) f(std::integral_constant<int, 1>{});
  else if (k == 2) f(std::integral_constant<int, 2>{});
  else if (k <= 4) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

}  // namespace

size_t permute_workspace_bytes(int64_t T, int k, int E) {
  return one_launch(T, k) ? 0 : static_cast<size_t>((rank_chunks(T, k) + 1) * E) * sizeof(int32_t);
}

bool launch_permute(int64_t T, int row_bytes, int k, int E, int row_align, const void* x, int64_t x_pitch,
                    const int32_t* topk_idx, void* xp, int32_t* offsets, int32_t* row_map, int32_t* src_row, void* ws,
                    hipStream_t s) {
  if (T == 0) {
    launch_kernel("permute_rows", clear_offsets_kernel, dim3(1), dim3(kThreads), 0, s, offsets, E + 1);
    return launch_ok("permute_rows");
  }
  PermuteArgs a{T, row_bytes / 16, k, E, row_align, static_cast<const uint8_t*>(x), x_pitch, topk_idx,
                static_cast<uint8_t*>(xp), offsets, row_map, src_row, nullptr, nullptr, T, 0,
                pad_parts(row_align - 1, xp != nullptr ? row_bytes / 16 : 0, E,
                          one_launch(T, k) && T > kOneTokenAWorkgroup ? 128 : 512),
                streams((static_cast<double>(T) * k + static_cast<double>(E) * (row_align - 1)) * row_bytes)};
  const int pad_blocks = row_align > 1 ? E * a.pad_parts : 0;
  if (one_launch(T, k)) {
    auto few = [&](auto threads, auto tokens) {
      constexpr int THREADS = decltype(threads)::value, G = decltype(tokens)::value;
      a.token_blocks = (T + G - 1) / G;
      launch_kernel("permute_rows", permute_few_kernel<THREADS, G>,
                    dim3(static_cast<unsigned>(a.token_blocks + pad_blocks)), dim3(THREADS), 0, s, a);
    };
    if (T <= kOneTokenAWorkgroup) few(std::integral_constant<int, kThreads>{}, std::integral_constant<int, 1>{});
    else few(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
    return launch_ok("permute_rows");
  }
  const int64_t chunks = rank_chunks(T, k);
  int32_t* counts = static_cast<int32_t*>(ws);
  a.counts = counts;
  a.expert_count = counts + chunks * E;
  launch_kernel("permute_count", permute_count_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kRankChunk),
                count_lds_bytes(E), s, T * k, E, topk_idx, row_map, counts);
  if (!launch_ok("permute_count")) return false;
  int cols = 1;
  while (cols < E) cols *= 2;
  launch_kernel("permute_scan", permute_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, counts,
                static_cast<int>(chunks), E, cols, row_align, offsets, counts + chunks * E);
  if (!launch_ok("permute_scan")) return false;
  const bool lines = by_lines(T, k, a.chunks);
  auto rows = [&](auto team) {
    constexpr int TEAM = decltype(team)::value, kTeams = kThreads / TEAM;
    a.token_blocks = (T + kTeams - 1) / kTeams;
    launch_parts(a.token_blocks + pad_blocks, kThreads, [&](int64_t first, int64_t count) {
      a.first = first;
      launch_kernel("permute_rows", lines ? permute_rows_kernel<TEAM, (TEAM >= kWave)> : permute_rows_kernel<TEAM, false>,
                    dim3(static_cast<unsigned>(count)), dim3(kThreads), 0, s, a);
    });
  };
  // Lanes per token.  (16384 tokens in bf16 take 17 us with rows of 128, 36 with
  // 512, 86 with 1536.)
  if (a.chunks <= 16) rows(std::integral_constant<int, 16>{});
  else if (a.chunks <= 128) rows(std::integral_constant<int, kWave>{});
  else rows(std::integral_constant<int, kThreads>{});
  return launch_ok("permute_rows");
}

bool launch_gather_rows(int64_t T, int H, int k, int64_t rows, bool f32, const void* src, const int32_t* row_map,
                        const float* w, void* out, int64_t out_pitch, const char* name, hipStream_t s) {
  if (T == 0) return true;
  GatherArgs a{T, H / (f32 ? 4 : 8), k, 0, static_cast<uint32_t>(rows), src, row_map, w, out, out_pitch, 0};
  a.magic = static_cast<uint32_t>(((uint64_t{1} << 32) + a.chunks - 1) / a.chunks);
  const bool nt = streams(static_cast<double>(T) * k * H * (f32 ? 4 : 2));
  auto go = [&](auto elem, auto slots) {
    using Elem = decltype(elem);
    constexpr int K = decltype(slots)::value;
    launch_parts((T * a.chunks + kThreads - 1) / kThreads, kThreads, [&](int64_t first, int64_t count) {
      a.first = first;
      launch_kernel(name, nt ? gather_rows_kernel<Elem, K, true> : gather_rows_kernel<Elem, K, false>,
                    dim3(static_cast<unsigned>(count)), dim3(kThreads), 0, s, a);
    });
  };
  with_slots(k, [&](auto slots) {
    if (f32) go(float{}, slots);
    else go(uint16_t{}, slots);
  });
  return launch_ok(name);
}

bool launch_unpermute_bwd(int64_t T, int H, int k, int E, int64_t rows, bool f32, const void* dy, int64_t dy_pitch,
                          const void* o, const int32_t* row_map, const float* w, const int32_t* offsets,
                          const int32_t* src_row, void* d_o, float* dw, hipStream_t s) {
  if (T == 0) return true;
  UnpermuteBwdArgs a{T, H / (f32 ? 4 : 8), k, E, static_cast<uint32_t>(rows), dy, dy_pitch, o, row_map, w,
                     E > 0 ? offsets : nullptr, src_row, d_o, dw, UINT32_MAX, 0, 0, 1, false};
  const double row_bytes = 16.0 * a.chunks;
  auto go = [&](int64_t main_blocks, int64_t others, auto kernel) {
    a.main_blocks = main_blocks;
    launch_parts(main_blocks + others, kThreads, [&](int64_t first, int64_t count) {
      a.first = first;
      launch_kernel("unpermute_bwd", kernel, dim3(static_cast<unsigned>(count)), dim3(kThreads), 0, s, a);
    });
  };
  // Whatever the number of rows: where slots are not dispatched, padded groups may
  // fit a buffer of fewer rows than slots.  An expert's share of the rows beyond
  // the slots, or there of all rows, sets the number of workgroups alone.
  int pad_blocks = 0;
  if (d_o != nullptr && E > 0 && offsets != nullptr && src_row != nullptr) {
    a.pad_parts = pad_parts(std::min<int64_t>(127, ((rows > T * k ? rows - T * k : rows) + E - 1) / E), a.chunks, E);
    pad_blocks = E * a.pad_parts;
    a.pads_past = streams(rows * row_bytes);
  }
  // Both wanted of many wide rows: dp first, then do, so that reads and writes of
  // rows in token order do not alternate; dy is read twice, mostly from the
  // memory-side cache.  16384 tokens of 2048 202 us against 207 in one pass, 32768
  // 400 against 429, 16384 of 4096 393 against 437; 8192 of 2048 106 against 105, 4096
  // 58 against 54, 16384 of 1024 113 against 104.  Where few slots are dispatched dy
  // is much of the traffic and one pass takes less: 16384 of 2048 with a quarter of
  // the slots 67 us against 79, with half 114 against 117; 65536 279 against 372 and
  // 503 against 560; 16384 of 4096 135 against 161 and 252 against 243.  From five
  // eighths on two passes are as fast or faster but for 65536 (606 and 665).  The
  // number is known on the device: with fewer in use the first launch makes both
  // and the second, which ends at once, costs 5 us in 62 (16384 tokens).
  const bool apart = d_o != nullptr && dw != nullptr && a.chunks >= 256 && T * k * row_bytes >= 256.0 * 1024 * 1024;
  if (apart) a.apart = static_cast<uint32_t>(T * k / 8 * 5);
  auto scatter = [&] {
    const bool lines = by_lines(T, k, a.chunks);
    auto type = [&](auto elem) {
      using Elem = decltype(elem);
      go(T, pad_blocks, lines ? unpermute_bwd_scatter_kernel<Elem, true> : unpermute_bwd_scatter_kernel<Elem, false>);
    };
    if (f32) type(float{});
    else type(uint16_t{});
    return launch_ok("unpermute_bwd");
  };
  if (dw == nullptr) {
    a.apart = 0;
    return scatter();
  }
  // Four chunks a lane in flight where the row has as many: 16384 tokens of 128 37
  // us with a wave to an entry, 14 with 16 lanes; 256 39 and 24, 512 62 and 53; 640
  // 75 and with 32 lanes 66, 768 81 and 78, 1024 103 and 105.
  auto entries = [&](auto elem, auto lanes, auto nt) {
    constexpr int LANES = decltype(lanes)::value, kEntries = kThreads / LANES;
    go((T * k + kEntries - 1) / kEntries, apart ? 0 : pad_blocks,
       unpermute_bwd_entries_kernel<decltype(elem), LANES, decltype(nt)::value>);
  };
  auto shape = [&](auto elem, auto nt) {
    if (a.chunks <= 64) entries(elem, std::integral_constant<int, 16>{}, nt);
    else if (a.chunks < 128) entries(elem, std::integral_constant<int, 32>{}, nt);
    else entries(elem, std::integral_constant<int, kWave>{}, nt);
  };
  auto types = [&](auto nt) {
    if (f32) shape(float{}, nt);
    else shape(uint16_t{}, nt);
  };
  if (streams(T * k * row_bytes * (d_o != nullptr ? 2 : 1))) types(std::true_type{});
  else types(std::false_type{});
  if (!launch_ok("unpermute_bwd")) return false;
  return !apart || scatter();
}

}  // namespace w4a4
