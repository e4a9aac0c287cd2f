// SwiGLU with its input kept in 8 bits for the backward pass (gfx950):
//
//   s = sigmoid(gate);  a = bf16(gate s up);  codes, scales = MX(a)
//   checkpoint = MXFP8 of h = (gate, up), blocks of 32 along the row
//   dgate = bf16(da up s (1 + gate (1 - s)));  dup = bf16(da gate s)
//
// The checkpoint holds 33/32 bytes an element instead of h's two and stands for
// a as well, which the backward pass computes once more beside dh from the
// checkpoint's values (the operand of the next weight gradient).  The forward's
// a comes from the bf16 h itself.  Arithmetic is FP32 with the hardware's exp2
// and reciprocal, as in the expert path's epilogues, each result rounded once.
//
// Everything is element by element but the blocks' maxima, which a quad of
// lanes finds among itself: HBM binds the calls of many rows, latency those of
// few.

#include <algorithm>

#include "internal.h"
#include "launch_parts.h"
#include "mx_encode.h"

namespace w4a4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;                       // 8-element chunks of gate and up per lane
constexpr int kBlockChunks = kThreads * kUnroll;

// 2^X of the scale byte X + 127 (255, E8M0's NaN: NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}
__device__ __forceinline__ void mx_decode8(const u32x2_t& c, uint32_t byte, float (&v)[8]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const float scale = mx_scale(byte);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[d]), false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[d]), true);
    v[4 * d] = lo[0] * scale;
    v[4 * d + 1] = lo[1] * scale;
    v[4 * d + 2] = hi[0] * scale;
    v[4 * d + 3] = hi[1] * scale;
  }
}
__device__ __forceinline__ void unpack8(const u32x4_t& w, float (&v)[8]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    v[2 * d] = __uint_as_float(w[d] << 16);
    v[2 * d + 1] = __uint_as_float(w[d] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  u32x4_t w;
#pragma unroll
  for (int d = 0; d < 4; ++d) w[d] = pack_bf16x2(v[2 * d], v[2 * d + 1]);
  return w;
}

// The rows' chunks in flat order, kBlockChunks a workgroup: chunk u of this lane
// is chunk col[u] of row[u] (I / 8 a row); row[u] = T where there is none.
// I % 32 == 0 wherever blocks are encoded or read, so that a quad's lanes hold
// one block of one row.
struct Place {
  int64_t row[kUnroll];
  int col[kUnroll];
};
__device__ __forceinline__ bool place(const SwigluArgs& a, Place& p) {
  const int chunks = a.I / 8;
  const int64_t T = a.rows != nullptr ? min(a.T, static_cast<int64_t>(max(*a.rows, 0))) : a.T;
  const int64_t base = (a.first + blockIdx.x) * kBlockChunks;
  const int64_t row0 = base / chunks;
  if (row0 >= T) return false;
  const uint32_t col0 = static_cast<uint32_t>(base - row0 * chunks);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = col0 + u * kThreads + threadIdx.x;   // below chunks + kBlockChunks: magic divides exactly
    const uint32_t q = chunks > 1 ? __umulhi(i, a.magic) : i;
    const int64_t row = row0 + q;
    p.row[u] = row < T ? row : a.T;
    p.col[u] = static_cast<int>(i - q * chunks);
  }
  return true;
}

template <bool NT>
__device__ __forceinline__ u32x4_t load16(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
  else return *static_cast<const u32x4_t*>(p);
}

template <int FMT, bool CKPT>
__global__ void __launch_bounds__(kThreads)
swiglu_fwd_kernel(SwigluArgs a) {
  Place p;
  if (!place(a, p)) return;
  const int chunks = a.I / 8;
  u32x4_t g[kUnroll], v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    g[u] = v[u] = u32x4_t{0u, 0u, 0u, 0u};
    if (p.row[u] >= a.T) continue;
    const uint16_t* h = a.h + p.row[u] * a.h_stride + p.col[u] * 8;
    if (a.stream) {
      g[u] = load16<true>(h);
      v[u] = load16<true>(h + a.I);
    } else {
      g[u] = load16<false>(h);
      v[u] = load16<false>(h + a.I);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (p.row[u] >= a.T) continue;
    const int64_t at = p.row[u] * chunks + p.col[u];
    if constexpr (CKPT) {
      const int64_t hat = p.row[u] * 2 * chunks + p.col[u];
      uint32_t code[2];
      uint32_t byte = mx_encode8<kMxFp8>(g[u], code);
      mx_store8<kMxFp8>(a.h_codes, a.h_scales, hat, code, byte);
      byte = mx_encode8<kMxFp8>(v[u], code);
      mx_store8<kMxFp8>(a.h_codes, a.h_scales, hat + chunks, code, byte);
    }
    float gate[8], up[8], y[8];
    unpack8(g[u], gate);
    unpack8(v[u], up);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = gate[i] * sigmoid_fast(gate[i]) * up[i];
    const u32x4_t w = pack8(y);
    if (a.a != nullptr) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(a.a) + at);
    if constexpr (FMT != kMxNone) {
      uint32_t code[2];
      const uint32_t byte = mx_encode8<FMT>(w, code);
      mx_store8<FMT>(a.codes, a.scales, at, code, byte);
    }
  }
}

template <bool CKPT>
__global__ void __launch_bounds__(kThreads)
swiglu_bwd_kernel(SwigluArgs a) {
  Place p;
  if (!place(a, p)) return;
  const int chunks = a.I / 8;
  u32x4_t d[kUnroll], g[kUnroll], v[kUnroll];
  u32x2_t gc[kUnroll], vc[kUnroll];
  uint32_t gs[kUnroll], vs[kUnroll];
  auto load = [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (p.row[u] >= a.T) continue;
      if (a.da != nullptr) d[u] = load16<NT>(a.da + (p.row[u] * chunks + p.col[u]) * 8);
      if constexpr (CKPT) {
        const int64_t hat = p.row[u] * 2 * chunks + p.col[u];
        const u32x2_t* c = reinterpret_cast<const u32x2_t*>(a.h_codes) + hat;
        gc[u] = NT ? __builtin_nontemporal_load(c) : *c;
        vc[u] = NT ? __builtin_nontemporal_load(c + chunks) : c[chunks];
        gs[u] = a.h_scales[hat >> 2];
        vs[u] = a.h_scales[(hat + chunks) >> 2];
      } else {
        const uint16_t* h = a.h + p.row[u] * a.h_stride + p.col[u] * 8;
        g[u] = load16<NT>(h);
        v[u] = load16<NT>(h + a.I);
      }
    }
  };
  if (a.stream) load(std::true_type{});
  else load(std::false_type{});
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (p.row[u] >= a.T) continue;
    float gate[8], up[8], s[8], y[8];
    if constexpr (CKPT) {
      mx_decode8(gc[u], gs[u], gate);
      mx_decode8(vc[u], vs[u], up);
    } else {
      unpack8(g[u], gate);
      unpack8(v[u], up);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = sigmoid_fast(gate[i]);
    if (a.a != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = gate[i] * s[i] * up[i];
      __builtin_nontemporal_store(pack8(y), reinterpret_cast<u32x4_t*>(a.a) + p.row[u] * chunks + p.col[u]);
    }
    if (a.dh != nullptr) {
      float da[8], dg[8], du[8];
      unpack8(d[u], da);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dg[i] = da[i] * up[i] * s[i] * (1.0f + gate[i] * (1.0f - s[i]));
        du[i] = da[i] * gate[i] * s[i];
      }
      u32x4_t* dh = reinterpret_cast<u32x4_t*>(a.dh) + p.row[u] * 2 * chunks + p.col[u];
      __builtin_nontemporal_store(pack8(dg), dh);
      __builtin_nontemporal_store(pack8(du), dh + chunks);
    }
  }
}

// As the pre-norm: a call that moves more than three quarters of the 256 MiB
// memory-side cache loads past it.
bool streams(double bytes) { return bytes > 0.75 * 256 * 1024 * 1024; }

template <class F>
bool launch_chunks(SwigluArgs a, const char* name, hipStream_t s, F kernel) {
  const int chunks = a.I / 8;
  a.magic = static_cast<uint32_t>(((uint64_t{1} << 32) + chunks - 1) / chunks);
  const int64_t total = a.T * chunks;
  launch_parts((total + kBlockChunks - 1) / kBlockChunks, kThreads, [&](int64_t first, int64_t count) {
    a.first = first;
    launch_kernel(name, kernel, dim3(static_cast<unsigned>(count)), dim3(kThreads), 0, s, a);
  });
  return launch_ok(name);
}

}  // namespace

bool launch_swiglu_fwd(const SwigluArgs& args, int format, hipStream_t s) {
  if (args.T == 0) return true;
  SwigluArgs a = args;
  const bool ckpt = a.h_codes != nullptr;
  a.stream = streams(static_cast<double>(a.T) * a.I * (4 + (a.a ? 2 : 0) + (ckpt ? 2 : 0) + (a.codes ? 1 : 0)));
  auto go = [&](auto keep) {
    constexpr bool CKPT = decltype(keep)::value;
    if (format == kMxFp8) return launch_chunks(a, "swiglu_fwd", s, swiglu_fwd_kernel<kMxFp8, CKPT>);
    if (format == kMxFp4) return launch_chunks(a, "swiglu_fwd", s, swiglu_fwd_kernel<kMxFp4, CKPT>);
    return launch_chunks(a, "swiglu_fwd", s, swiglu_fwd_kernel<kMxNone, CKPT>);
  };
  return ckpt ? go(std::true_type{}) : go(std::false_type{});
}

bool launch_swiglu_bwd(const SwigluArgs& args, hipStream_t s) {
  if (args.T == 0) return true;
  SwigluArgs a = args;
  const bool ckpt = a.h_codes != nullptr;
  a.stream = streams(static_cast<double>(a.T) * a.I * ((ckpt ? 2 : 4) + (a.a ? 2 : 0) + (a.dh ? 6 : 0)));
  return ckpt ? launch_chunks(a, "swiglu_bwd", s, swiglu_bwd_kernel<true>)
              : launch_chunks(a, "swiglu_bwd", s, swiglu_bwd_kernel<false>);
}

}  // namespace w4a4
