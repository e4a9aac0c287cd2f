// The layer's pre-norm on gfx950: residual addition, RMS norm and the MX
// encoding of its output in one pass, its backward, and the MX encoding of
// bf16 rows alone.
//
//   s = rnd(x + r);  rstd = (mean_h s^2 + eps)^-1/2;  y = bf16(s rstd gamma);
//   codes, scales = MX(y)
//   n = s rstd;  dres = rstd (dy gamma - n mean_h(dy gamma n)) + dsum;
//   dgamma = sum_t dy n
//
// The codes are those of the bf16 y (not of the FP32 product), so that the
// fused call gives the bytes of the norm followed by the quantiser and the
// straight-through backward sees the operand that was quantised.
//
// The forward sums the squares in FP64 and multiplies by rstd as the sum of
// two floats, and y is rounded once: it is the bf16 nearest to the exact value.
// That costs no time beside HBM, and no row's squares overflow or underflow.
// Everything else is FP32.  Calls of many rows are bound by HBM: every tensor is
// read or written once.  The backward of few rows (kFewRows) reads dy and s a
// second time, from the L2, for dgamma; short calls are bound by latency.  16384 rows of 2048 in bf16 with FP8 codes take 43 us (5.4
// TB/s), with y and rstd 54 (5.6), the backward 48 (5.6); 4097 of 4096 with an
// FP32 residual 37 (5.0), 8191 of 5120 the backward 115 (5.1); the quantiser of
// 16384 rows of 4096 35 with FP8 (5.8), 32 with FP4 (5.2).  One row takes 2.6 us
// forward and 2.7 backward, one quantised row 2.7.

#include <algorithm>

#include "internal.h"
#include "mx_encode.h"

namespace w4a4 {
namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));

constexpr int kNormThreads = 256;
constexpr int kBwdThreads = 512;
constexpr int kFewRows = 512;
// Up to how many rows of 1024 < H <= 2048 a whole workgroup (forward) or half of
// one (backward) takes a row instead of one wave: H = 2048, FP8 codes: T = 1 2.6
// us against 4.5, T = 512 4.0 against 5.8, T = 2048 8.1 against 9.2, T = 3000 the
// same; backward: T = 1 2.7 against 3.3, T = 61 2.8 against 4.0, T = 256 3.5
// against 4.1, T = 512 5.7 against 4.7 (with dgamma; without it one wave takes a
// row at every T).
constexpr int kSpreadRows = 2048, kSpreadBwdRows = 256;

// Whether a call's loads are non-temporal: where it moves more than three
// quarters of the 256 MiB memory-side cache, its inputs cannot all still lie
// there, and loads that leave the cache alone are faster (16384 rows of 2048,
// forward with FP8 codes, 236 MB: 46.7 us against 49.0, backward, 268 MB: 50.8
// against 53.6); below, they would miss what the producer left (2000 rows of
// 8192, 115 MB: 28 against 22).
bool streams(double bytes) { return bytes > 0.75 * 256 * 1024 * 1024; }

// 8 consecutive elements as floats.  Stores are non-temporal (no output is
// read again by its call): 16384 rows of 2048 with all outputs 66 to 63 us,
// 2000 rows of 8192 38 to 25.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {   // bf16
  u32x4_t w;
  template <bool NT = false>
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (NT) w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
    else w = *reinterpret_cast<const u32x4_t*>(p);
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void zero() { w = u32x4_t{0u, 0u, 0u, 0u}; }
  // values rounded to bf16
  __device__ __forceinline__ void put(const float (&v)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = pack_bf16x2(v[2 * d], v[2 * d + 1]);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
  }
};
template <>
struct Vec8<float> {
  floatx4_t w[2];
  template <bool NT = false>
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (NT) w[h] = __builtin_nontemporal_load(reinterpret_cast<const floatx4_t*>(p) + h);
      else w[h] = reinterpret_cast<const floatx4_t*>(p)[h];
    }
  }
  __device__ __forceinline__ float get(int i) const { return w[i >> 2][i & 3]; }
  __device__ __forceinline__ void zero() { w[0] = w[1] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void put(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = v[i];
  }
  __device__ __forceinline__ void store(float* p) const {
    __builtin_nontemporal_store(w[0], reinterpret_cast<floatx4_t*>(p));
    __builtin_nontemporal_store(w[1], reinterpret_cast<floatx4_t*>(p) + 1);
  }
};

// Sum over a row of the lanes' chunk sums q, the same in each lane, in an order
// that depends on the row's length alone: a lane's chunks, then a wave's lanes
// by halves, then the waves.  TEAM > 64 meets in `slots` (LDS); a kernel that
// sums again takes two sets in turn, so that one barrier per sum is enough (a
// wave can be at most one sum ahead of a wave that still reads).
//
// 256 lanes with one chunk each are the spread form of 64 lanes with four
// chunks, for few rows: there each wave joins the four waves' chunks lane by
// lane first, in the order in which the lane of the narrow form adds its own, so
// that the two give the same bits.
template <int TEAM, int P>
constexpr bool kSpread = TEAM == 256 && P == 1;
template <int THREADS, int TEAM, int P>
constexpr int kSlots = kSpread<TEAM, P> ? THREADS : THREADS / kWave;

template <int TEAM, int P, typename T>
__device__ __forceinline__ T team_sum(const T (&q)[P], T* slots) {
  constexpr int kLanes = TEAM < kWave ? TEAM : kWave, kWaves = TEAM / kWave;
  const int wave = threadIdx.x / kWave;
  T v = q[0];
  if constexpr (kSpread<TEAM, P>) {
    slots[threadIdx.x] = v;
    __syncthreads();
    const T* mine = slots + threadIdx.x / TEAM * TEAM + threadIdx.x % kWave;
    v = mine[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += mine[w * kWave];
  } else {
#pragma unroll
    for (int p = 1; p < P; ++p) v += q[p];
  }
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if constexpr (TEAM > kWave && !kSpread<TEAM, P>) {
    const int first = wave / kWaves * kWaves;
    if (threadIdx.x % kWave == 0) slots[wave] = v;
    __syncthreads();
    v = slots[first];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += slots[first + w];
  }
  return v;
}

// Whether v lies halfway between two bf16 values.
__device__ __forceinline__ bool halfway(float v) { return (__float_as_uint(v) & 0xFFFFu) == 0x8000u; }

template <int P>
__device__ __forceinline__ void load_gamma(float (&g)[P][8], const void* gamma, bool gamma_f32, int lane, int team,
                                           int chunks) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = lane + p * team;
    if (c >= chunks) continue;
    if (gamma_f32) {
      Vec8<float> v;
      v.load(static_cast<const float*>(gamma) + c * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[p][i] = v.get(i);
    } else {
      Vec8<uint16_t> v;
      v.load(static_cast<const uint16_t*>(gamma) + c * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[p][i] = v.get(i);
    }
  }
}

// ------------------------------------------------------------------ forward
// TEAM lanes per row, lane l the 8-element chunks l, l + TEAM, ... (P of
// them): the row stays in registers between the sum of squares and the
// output.  One row per team and a workgroup per 256 / TEAM rows: workgroups
// that stride over the rows, loading the next row beside the current one's
// output, took 2 to 12% longer on large batches.
template <int TEAM, int P, typename RES, int FMT>
__global__ void __launch_bounds__(kNormThreads)
norm_fwd_kernel(NormFwdArgs a) {
  __shared__ double slots[kSlots<kNormThreads, TEAM, P>];
  const int lane = threadIdx.x % TEAM, chunks = a.H / 8;
  constexpr int kTeams = kNormThreads / TEAM;
  const RES* residual = static_cast<const RES*>(a.residual);
  RES* sum = static_cast<RES*>(a.sum);
  if (a.offsets != nullptr && a.first == 0 && blockIdx.x == 0 && threadIdx.x < 2)
    a.offsets[threadIdx.x] = threadIdx.x == 0 ? 0 : static_cast<int32_t>(a.T);
  const int64_t t = a.first + static_cast<int64_t>(blockIdx.x) * kTeams + threadIdx.x / TEAM;
  if (t >= a.T) return;   // TEAM > 64: the whole workgroup

  // every load of the row in flight before the first is used
  Vec8<uint16_t> x[P];
  Vec8<RES> s[P];
  auto load = [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = lane + p * TEAM;
      x[p].zero();
      s[p].zero();
      if (c < chunks) {
        x[p].template load<NT>(a.x + t * a.x_stride + c * 8);
        if (residual != nullptr) s[p].template load<NT>(residual + t * a.H + c * 8);
      }
    }
  };
  if (a.stream) load(std::true_type{});
  else load(std::false_type{});
  float g[P][8];
  load_gamma<P>(g, a.gamma, a.gamma_f32, lane, TEAM, chunks);
  double q[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = lane + p * TEAM;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = residual != nullptr ? x[p].get(i) + s[p].get(i) : x[p].get(i);
    s[p].put(v);
    if (sum != nullptr && c < chunks) s[p].store(sum + t * a.H + c * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double w = s[p].get(i);
      q[p] = i == 0 ? w * w : fma(w, w, q[p]);
    }
  }
  const double ss = team_sum<TEAM>(q, slots);
  const double r64 = 1.0 / sqrt(ss / a.H + static_cast<double>(a.eps));
  const float rstd = static_cast<float>(r64), rlow = static_cast<float>(r64 - static_cast<double>(rstd));
  if (a.rstd != nullptr && lane == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = lane + p * TEAM;
    if (c >= chunks) continue;
    // s (rstd + rlow) = n + low, and its product with gamma rounded once to
    // FP32.  Where that lands halfway between two bf16 values (1 of 2^16), it
    // moves one unit to the side on which the product lies, so that y is not
    // rounded twice.
    float v[8], n[8], low[8];
    bool tie = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = s[p].get(i);
      n[i] = x * rstd;
      low[i] = fmaf(x, rlow, fmaf(x, rstd, -n[i]));
      v[i] = fmaf(n[i], g[p][i], low[i] * g[p][i]);
      tie = tie || halfway(v[i]);
    }
    if (tie) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float rest = fmaf(low[i], g[p][i], fmaf(n[i], g[p][i], -v[i]));
        if (halfway(v[i]) && rest != 0.0f)
          v[i] = __uint_as_float(__float_as_uint(v[i]) + ((rest < 0.0f) == (v[i] < 0.0f) ? 1 : -1));
      }
    }
    Vec8<uint16_t> y;
    y.put(v);
    if (a.y != nullptr) y.store(a.y + t * a.H + c * 8);
    if constexpr (FMT != kMxNone) {   // H % 32 == 0: a quad's lanes are all here or all past the row
      uint32_t code[2];
      const uint32_t byte = mx_encode8<FMT>(y.w, code);
      mx_store8<FMT>(a.codes, a.scales, t * chunks + c, code, byte);
    }
  }
}

// ----------------------------------------------------------------- backward
// As the forward, 512 threads or 256; DG: each lane sums dy n of its columns over
// its rows in FP32, the workgroup's teams add theirs in LDS in team order and
// write one row of `part`, which dgamma_kernel adds in workgroup order.
//
// Up to kFewRows rows dgamma comes from the rows themselves instead, which lie
// in the L2 then: column_sums' workgroups follow the rows' in one launch and
// read them a second time.  Against partial rows and their sum, H = 2048, bf16:
// T = 512 4.7 against 8.5, T = 1024 8.1 against 9.3, T
// = 2048 16.6 against 11.9; H = 8192 in FP32: T = 512 17.3 against 17.6, T =
// 1024 31.0 against 27.7; H = 512: T = 512 4.1 against 5.9, T = 2048 11.7 against 6.0.
template <int THREADS, int TEAM, int P, typename RES, bool DG>
__device__ __forceinline__ void norm_bwd_rows(const NormBwdArgs& a, int block, int blocks) {
  extern __shared__ __attribute__((aligned(16))) float dg_lds[];   // DG: [teams][H]
  __shared__ float slots[2][kSlots<THREADS, TEAM, P>];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM, chunks = a.H / 8;
  constexpr int kTeams = THREADS / TEAM;
  const int64_t step = static_cast<int64_t>(blocks) * kTeams;
  const RES* s_in = static_cast<const RES*>(a.sum);
  const RES* dsum = static_cast<const RES*>(a.dsum);
  RES* dres = static_cast<RES*>(a.dres);
  float g[P][8], dg[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) g[p][i] = dg[p][i] = 0.0f;
  load_gamma<P>(g, a.gamma, a.gamma_f32, lane, TEAM, chunks);

  // TEAM > 64 has a barrier in its sum: every team of the workgroup runs the
  // same iterations, those past the last row without loads or stores
  int turn = 0;
  for (int64_t t = static_cast<int64_t>(block) * kTeams + team; t - team < a.T; t += step) {
    const bool live = t < a.T;
    const float rstd = live ? a.rstd[t] : 0.0f;
    Vec8<RES> s[P], ds[P];
    Vec8<uint16_t> dy[P];
    auto load = [&](auto nt) {
      constexpr bool NT = decltype(nt)::value;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = lane + p * TEAM;
        s[p].zero();
        ds[p].zero();
        dy[p].zero();
        if (live && c < chunks) {
          dy[p].template load<NT>(a.dy + t * a.H + c * 8);
          s[p].template load<NT>(s_in + t * a.H + c * 8);
          if (dsum != nullptr) ds[p].template load<NT>(dsum + t * a.H + c * 8);
        }
      }
    };
    if (a.stream) load(std::true_type{});
    else load(std::false_type{});
    float q[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      q[p] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = s[p].get(i) * rstd, d = dy[p].get(i);
        q[p] = fmaf(d * g[p][i], n, q[p]);
        if constexpr (DG) dg[p][i] = fmaf(d, n, dg[p][i]);
      }
    }
    const float inner = team_sum<TEAM>(q, slots[turn]) / static_cast<float>(a.H);
    turn ^= 1;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = lane + p * TEAM;
      if (!live || c >= chunks) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = s[p].get(i) * rstd;
        v[i] = fmaf(rstd, fmaf(dy[p].get(i), g[p][i], -(n * inner)), ds[p].get(i));
      }
      Vec8<RES> o;
      o.put(v);
      o.store(dres + t * a.H + c * 8);
      if (a.dx != nullptr) {
        Vec8<uint16_t> ox;
        ox.put(v);
        ox.store(a.dx + t * a.H + c * 8);
      }
    }
  }
  if constexpr (DG) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = lane + p * TEAM;
      if (c >= chunks) continue;
      floatx4_t* d = reinterpret_cast<floatx4_t*>(dg_lds + team * a.H + c * 8);
      d[0] = floatx4_t{dg[p][0], dg[p][1], dg[p][2], dg[p][3]};
      d[1] = floatx4_t{dg[p][4], dg[p][5], dg[p][6], dg[p][7]};
    }
    __syncthreads();
    float* out = a.part + static_cast<int64_t>(block) * a.H;
    for (int h = threadIdx.x; h < a.H; h += THREADS) {
      float v = dg_lds[h];
#pragma unroll
      for (int w = 1; w < kTeams; ++w) v += dg_lds[w * a.H + h];
      out[h] = v;
    }
  }
}

template <int THREADS, int TEAM, int P, typename RES, bool DG>
__global__ void __launch_bounds__(THREADS)
norm_bwd_kernel(NormBwdArgs a) {
  norm_bwd_rows<THREADS, TEAM, P, RES, DG>(a, blockIdx.x, gridDim.x);
}

// dgamma of 64 columns: lane l of eight takes the columns 8 l .. +7 of rows r,
// r + 64, ..., whose sums are added over a wave's eight r, then in wave order.
template <typename RES>
__device__ __forceinline__ void column_sums(const NormBwdArgs& a, int block) {
  __shared__ float sums[kBwdThreads / kWave][kWave];
  const int lane = threadIdx.x % 8, first = threadIdx.x / 8, wave = threadIdx.x / kWave;
  const int64_t c = static_cast<int64_t>(block) * kWave + lane * 8;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (c < a.H) {
#pragma unroll 4
    for (int64_t t = first; t < a.T; t += kBwdThreads / 8) {
      Vec8<uint16_t> dy;
      Vec8<RES> s;
      dy.load(a.dy + t * a.H + c);
      s.load(static_cast<const RES*>(a.sum) + t * a.H + c);
      const float rstd = a.rstd[t];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(dy.get(i), s.get(i) * rstd, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = 8; off < kWave; off <<= 1) v[i] += __shfl_xor(v[i], off, kWave);
    if (threadIdx.x % kWave < 8) sums[wave][lane * 8 + i] = v[i];
  }
  __syncthreads();
  const int64_t h = static_cast<int64_t>(block) * kWave + threadIdx.x;
  if (threadIdx.x < kWave && h < a.H) {
    float d = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kBwdThreads / kWave; ++w) d += sums[w][threadIdx.x];
    a.dgamma[h] = d;
  }
}

// Workgroups first, first + 1, ... of `rows` workgroups over rows and the
// column sums' behind them.
template <int TEAM, int P, typename RES>
__global__ void __launch_bounds__(kBwdThreads)
norm_bwd_few_kernel(NormBwdArgs a, int first, int rows) {
  const int block = blockIdx.x + first;
  if (block < rows) {
    norm_bwd_rows<kBwdThreads, TEAM, P, RES, false>(a, block, rows);
  } else {
    column_sums<RES>(a, block - rows);
  }
}

// dgamma[h] = sum of the G partial rows, wave w of a workgroup rows w, w +
// 16, ... of 64 columns, the waves' sums added in wave order.
constexpr int kDgThreads = 1024;
__global__ void __launch_bounds__(kDgThreads)
dgamma_kernel(const float* __restrict__ part, int G, int H, float* __restrict__ dgamma) {
  __shared__ float sums[kDgThreads];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int h = blockIdx.x * kWave + lane;
  float v = 0.0f;
  if (h < H) {
#pragma unroll 8
    for (int r = wave; r < G; r += kDgThreads / kWave) v += part[static_cast<int64_t>(r) * H + h];
  }
  sums[threadIdx.x] = v;
  __syncthreads();
  if (wave == 0 && h < H) {
#pragma unroll
    for (int w = 1; w < kDgThreads / kWave; ++w) v += sums[w * kWave + lane];
    dgamma[h] = v;
  }
}

__global__ void __launch_bounds__(kNormThreads)
zero_f32_kernel(float* p, int n) {
  const int i = blockIdx.x * kNormThreads + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// ------------------------------------------------------------ MX quantiser
// Output chunks are flat (K % 32 == 0: the code and scale index of a chunk
// does not depend on the row length); the input position moves by a fixed
// (rows, columns) step per iteration.
template <int FMT, bool NT>
__global__ void __launch_bounds__(kNormThreads)
quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t x_stride, int64_t total, int chunks, int64_t step_rows,
                     int step_cols, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int32_t* offsets,
                     int64_t T) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kNormThreads;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (offsets != nullptr && i < 2) offsets[i] = i == 0 ? 0 : static_cast<int32_t>(T);
  int64_t row = i / chunks;
  int col = static_cast<int>(i - row * chunks);
  for (; i < total; i += step) {   // total % 4 == 0: the lanes of a quad leave together
    Vec8<uint16_t> v;
    v.load<NT>(x + row * x_stride + col * 8);
    uint32_t code[2];
    const uint32_t byte = mx_encode8<FMT>(v.w, code);
    mx_store8<FMT>(codes, scales, i, code, byte);
    row += step_rows;
    col += step_cols;
    if (col >= chunks) {
      col -= chunks;
      ++row;
    }
  }
}

template <int TEAM, int P, typename RES, int FMT>
void launch_fwd_variant(const NormFwdArgs& a, hipStream_t s) {
  constexpr int kTeams = kNormThreads / TEAM;
  // a launch holds fewer than 2^32 threads: more rows take further launches
  constexpr int64_t kMost = int64_t{1} << 23;
  NormFwdArgs part = a;
  do {
    const int64_t blocks = std::min(kMost, std::max<int64_t>(1, (a.T - part.first + kTeams - 1) / kTeams));
    launch_kernel("add_rmsnorm", norm_fwd_kernel<TEAM, P, RES, FMT>, dim3(static_cast<unsigned>(blocks)),
                  dim3(kNormThreads), 0, s, part);
    part.first += blocks * kTeams;
  } while (part.first < a.T);
}

template <int TEAM, int P>
void launch_fwd_shape(const NormFwdArgs& a, bool res_f32, int format, hipStream_t s) {
  auto fmt = [&](auto res) {
    using RES = decltype(res);
    if (format == kMxFp8) launch_fwd_variant<TEAM, P, RES, kMxFp8>(a, s);
    else if (format == kMxFp4) launch_fwd_variant<TEAM, P, RES, kMxFp4>(a, s);
    else launch_fwd_variant<TEAM, P, RES, kMxNone>(a, s);
  };
  if (res_f32) fmt(float{});
  else fmt(uint16_t{});
}

// Lanes per row: a row's chunks fit its team's registers (P <= 4), and short
// rows share a wave.
int norm_team(int H) { return H <= 256 ? 16 : H <= 2048 ? 64 : 256; }

// Threads of the backward's workgroups: for wide rows one row each, two
// workgroups a CU, so that one loads beside the other's stores: 8191 rows of
// 5120 in FP32 115 us against 123, 16384 of 8192 in bf16 178 against 187; few
// of them are faster with half the partial sums (1000 of 8192 in bf16 18.9
// against 20.7, 2000 33.6 against 32.6).
int bwd_threads(int64_t T, int H) { return H > 4096 && T >= 2048 ? 256 : kBwdThreads; }

template <int THREADS, int TEAM, int P, typename RES, bool DG>
bool launch_bwd_variant(const NormBwdArgs& a, int blocks, hipStream_t s) {
  const uint32_t lds = DG ? static_cast<uint32_t>(THREADS / TEAM) * a.H * 4u : 0u;
  const auto kernel = norm_bwd_kernel<THREADS, TEAM, P, RES, DG>;
  if constexpr (DG) {
    static OncePerDevice limit;
    if (!set_lds(limit, kernel, THREADS * P * 32)) return launch_ok("add_rmsnorm_bwd") && false;
  }
  launch_kernel("add_rmsnorm_bwd", kernel, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), lds, s, a);
  return true;
}

template <int THREADS, int TEAM, int P>
bool launch_bwd_threads(const NormBwdArgs& a, bool res_f32, int blocks, hipStream_t s) {
  if (res_f32)
    return a.part ? launch_bwd_variant<THREADS, TEAM, P, float, true>(a, blocks, s)
                  : launch_bwd_variant<THREADS, TEAM, P, float, false>(a, blocks, s);
  return a.part ? launch_bwd_variant<THREADS, TEAM, P, uint16_t, true>(a, blocks, s)
                : launch_bwd_variant<THREADS, TEAM, P, uint16_t, false>(a, blocks, s);
}

// The column sums read dy and sum, which the rows may be written over: then
// they go first.
template <int TEAM, int P, typename RES>
bool launch_bwd_few(const NormBwdArgs& a, hipStream_t s) {
  constexpr int kTeams = kBwdThreads / TEAM;
  const int rows = static_cast<int>((a.T + kTeams - 1) / kTeams), columns = (a.H + kWave - 1) / kWave;
  auto launch = [&](int first, int blocks) {
    launch_kernel("add_rmsnorm_bwd", norm_bwd_few_kernel<TEAM, P, RES>, dim3(blocks), dim3(kBwdThreads), 0, s, a, first,
                  rows);
  };
  if (a.in_place) {
    launch(rows, columns);
    launch(0, rows);
  } else {
    launch(0, rows + columns);
  }
  return true;
}

template <int TEAM, int P>
bool launch_bwd_shape(const NormBwdArgs& a, bool res_f32, int blocks, hipStream_t s) {
  if (a.dgamma != nullptr && a.T <= kFewRows) {
    if constexpr (TEAM == 64 && P == 4)
      if (a.T <= kSpreadBwdRows)
        return res_f32 ? launch_bwd_few<256, 1, float>(a, s) : launch_bwd_few<256, 1, uint16_t>(a, s);
    return res_f32 ? launch_bwd_few<TEAM, P, float>(a, s) : launch_bwd_few<TEAM, P, uint16_t>(a, s);
  }
  if constexpr (TEAM == 256 && P == 4)
    if (bwd_threads(a.T, a.H) == TEAM) return launch_bwd_threads<TEAM, TEAM, P>(a, res_f32, blocks, s);
  return launch_bwd_threads<kBwdThreads, TEAM, P>(a, res_f32, blocks, s);
}

// Workgroups over rows, and rows of scratch that they take with dgamma: one a
// CU, two where the lanes of one hold too few bytes of their rows to cover the
// latency (one 16-byte chunk of each tensor, or two in the teams that wait at
// barriers) and there are two rounds of rows for two: 131072 rows of 512 in
// bf16 92 us against 113, of 2560 (16384 rows) 61 against 82, of 4096 88 against 101.  With
// wider rows two are slower (H = 2048 51 against 48, 5120 in FP32 126 against
// 123), and with few rows the second's partial sums cost more than it saves
// (1000 rows of 2560: 13.0 against 10.3).
int bwd_blocks(int64_t T, int H, bool res_f32) {
  const int threads = bwd_threads(T, H), teams = threads / norm_team(H);
  const int64_t need = (T + teams - 1) / teams;
  const bool narrow = !res_f32 && (H <= 128 || (H > 256 && H <= 512) || (H > 2048 && H <= 4096));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(need, threads == 256 || (narrow && need >= 1024) ? 512 : 256)));
}

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int H) {
  return T <= kFewRows ? 0 : static_cast<size_t>(bwd_blocks(T, H, false)) * H * 4;   // bf16 takes no fewer
}

bool launch_add_rmsnorm(const NormFwdArgs& args, bool res_f32, int format, hipStream_t s) {
  NormFwdArgs a = args;
  const int H = a.H, res = res_f32 ? 4 : 2;
  a.stream = streams(static_cast<double>(a.T) * H *
                     (2 + (a.residual ? res : 0) + (a.sum ? res : 0) + (a.y ? 2 : 0) + (a.codes ? 1 : 0)));
  if (H <= 128) launch_fwd_shape<16, 1>(a, res_f32, format, s);
  else if (H <= 256) launch_fwd_shape<16, 2>(a, res_f32, format, s);
  else if (H <= 512) launch_fwd_shape<64, 1>(a, res_f32, format, s);
  else if (H <= 1024) launch_fwd_shape<64, 2>(a, res_f32, format, s);
  else if (H <= 2048 && a.T <= kSpreadRows) launch_fwd_shape<256, 1>(a, res_f32, format, s);
  else if (H <= 2048) launch_fwd_shape<64, 4>(a, res_f32, format, s);
  else if (H <= 4096) launch_fwd_shape<256, 2>(a, res_f32, format, s);
  else if (H <= 8192) launch_fwd_shape<256, 4>(a, res_f32, format, s);
  else return false;
  return launch_ok("add_rmsnorm");
}

bool launch_add_rmsnorm_bwd(const NormBwdArgs& args, bool res_f32, hipStream_t s) {
  NormBwdArgs a = args;
  const int H = a.H, res = res_f32 ? 4 : 2;
  a.stream = streams(static_cast<double>(a.T) * H * (2 + 2 * res + (a.dsum ? res : 0) + (a.dx ? 2 : 0)));
  if (a.T == 0) {
    if (a.dgamma == nullptr) return true;
    launch_kernel("add_rmsnorm_dgamma", zero_f32_kernel, dim3((H + kNormThreads - 1) / kNormThreads),
                  dim3(kNormThreads), 0, s, a.dgamma, H);
    return launch_ok("add_rmsnorm_dgamma");
  }
  const int blocks = bwd_blocks(a.T, H, res_f32);
  bool ok = false;
  if (H <= 128) ok = launch_bwd_shape<16, 1>(a, res_f32, blocks, s);
  else if (H <= 256) ok = launch_bwd_shape<16, 2>(a, res_f32, blocks, s);
  else if (H <= 512) ok = launch_bwd_shape<64, 1>(a, res_f32, blocks, s);
  else if (H <= 1024) ok = launch_bwd_shape<64, 2>(a, res_f32, blocks, s);
  else if (H <= 2048) ok = launch_bwd_shape<64, 4>(a, res_f32, blocks, s);
  else if (H <= 4096) ok = launch_bwd_shape<256, 2>(a, res_f32, blocks, s);
  else if (H <= 8192) ok = launch_bwd_shape<256, 4>(a, res_f32, blocks, s);
  if (!ok || !launch_ok("add_rmsnorm_bwd")) return false;
  if (a.part == nullptr) return true;
  launch_kernel("add_rmsnorm_dgamma", dgamma_kernel, dim3((H + kWave - 1) / kWave), dim3(kDgThreads), 0, s,
                static_cast<const float*>(a.part), blocks, H, a.dgamma);
  return launch_ok("add_rmsnorm_dgamma");
}

bool launch_mx_quantize_rows(const uint16_t* x, int64_t x_stride, int64_t T, int K, int format, uint8_t* codes,
                             uint8_t* scales, int32_t* offsets, hipStream_t s) {
  const int chunks = K / 8;
  const int64_t total = T * chunks;
  const int64_t need = (total + kNormThreads - 1) / kNormThreads;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(need, static_cast<int64_t>(device_cu_count()) * 16));
  const int64_t step = blocks * kNormThreads;
  auto launch = [&](auto kernel) {
    launch_kernel("mx_quantize_rows", kernel, dim3(static_cast<unsigned>(blocks)), dim3(kNormThreads), 0, s, x,
                  x_stride, total, chunks, step / chunks, static_cast<int>(step % chunks), codes, scales, offsets, T);
  };
  if (format == kMxFp8)
    streams(T * (K * (3 + 1 / 32.0))) ? launch(&quantize_rows_kernel<kMxFp8, true>)
                                            : launch(&quantize_rows_kernel<kMxFp8, false>);
  else
    streams(T * (K * (2.5 + 1 / 32.0))) ? launch(&quantize_rows_kernel<kMxFp4, true>)
                                              : launch(&quantize_rows_kernel<kMxFp4, false>);
  return launch_ok("mx_quantize_rows");
}

}  // namespace w4a4
