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
// few.  131072 rows of 768 take 133 us with the checkpoint (6.1 TB/s; a linear
// copy reaches 6.5), 94 without, 160 backward (6.3); 5001 rows of 2048 16
// backward; 8 rows 2.1 on the device.

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "launch_parts.h"
#include "mx_encode.h"

namespace w4a4 {
namespace {

constexpr int kThreads = 256;

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

// The rows' 8-element chunks in flat order, one a lane (I / 8 a row; two a lane
// took 145 us against 142 for the forward below, four 152).  I % 32 == 0 wherever
// blocks are encoded or read, so that a quad's lanes hold one block of one row.
struct Place {
  int64_t row;
  int col;
};
__device__ __forceinline__ bool place(const SwigluArgs& a, Place& p) {
  const int chunks = a.I / 8;
  const int64_t T = a.rows != nullptr ? min(a.T, static_cast<int64_t>(max(*a.rows, 0))) : a.T;
  const int64_t base = (a.first + blockIdx.x) * kThreads, row0 = base / chunks;
  // below chunks + 256, where magic divides exactly
  const uint32_t i = static_cast<uint32_t>(base - row0 * chunks) + threadIdx.x;
  const uint32_t q = chunks > 1 ? __umulhi(i, a.magic) : i;
  p.row = row0 + q;
  p.col = static_cast<int>(i - q * chunks);
  return p.row < T;
}

template <bool NT>
__device__ __forceinline__ u32x4_t load16(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
  else return *static_cast<const u32x4_t*>(p);
}

// What becomes of h in the forward: nothing, or its checkpoint, stored past the
// caches where both halves of a row of codes are whole cache lines.
enum Keep { kDrop, kKeep, kKeepLines };

// The MXFP8 of 8 elements of h to the checkpoint.
template <Keep KEEP>
__device__ __forceinline__ void keep8(const SwigluArgs& a, const u32x4_t& v, int64_t chunk) {
  uint32_t code[2];
  const uint32_t byte = mx_encode8<kMxFp8>(v, code);
  mx_store8<kMxFp8, KEEP == kKeepLines>(a.h_codes, a.h_scales, chunk, code, byte);
}

// NT: loads past the caches (131072 rows of 768 with the checkpoint 134 us against
// 140, 8192 11.6 against 10.2; backward 160 against 165, 12.4 against 10.8).  It
// and the outputs of the backward pass are chosen outside the kernels: branches
// around single loads and stores took 142 us for 133, and 168 for 160 backward.
template <int FMT, Keep KEEP, bool NT>
__global__ void __launch_bounds__(kThreads)
swiglu_fwd_kernel(SwigluArgs a) {
  Place p;
  if (!place(a, p)) return;
  const int chunks = a.I / 8;
  const uint16_t* h = a.h + p.row * a.h_stride + p.col * 8;
  const u32x4_t g = load16<NT>(h), v = load16<NT>(h + a.I);
  const int64_t at = p.row * chunks + p.col;
  if constexpr (KEEP != kDrop) {
    const int64_t hat = p.row * 2 * chunks + p.col;
    keep8<KEEP>(a, g, hat);
    keep8<KEEP>(a, v, hat + chunks);
  }
  float gate[8], up[8], y[8];
  unpack8(g, gate);
  unpack8(v, up);
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

// DH, A: which outputs are wanted.
template <bool CKPT, bool DH, bool A, bool NT>
__global__ void __launch_bounds__(kThreads)
swiglu_bwd_kernel(SwigluArgs a) {
  Place p;
  if (!place(a, p)) return;
  const int chunks = a.I / 8;
  const int64_t at = p.row * chunks + p.col, hat = p.row * 2 * chunks + p.col;
  u32x4_t d;
  if constexpr (DH) d = load16<NT>(a.da + at * 8);
  float gate[8], up[8], s[8];
  if constexpr (CKPT) {
    const u32x2_t* c = reinterpret_cast<const u32x2_t*>(a.h_codes) + hat;
    const u32x2_t g = NT ? __builtin_nontemporal_load(c) : *c;
    const u32x2_t v = NT ? __builtin_nontemporal_load(c + chunks) : c[chunks];
    const uint32_t gs = a.h_scales[hat >> 2], vs = a.h_scales[(hat + chunks) >> 2];
    mx_decode8(g, gs, gate);
    mx_decode8(v, vs, up);
  } else {
    const uint16_t* h = a.h + p.row * a.h_stride + p.col * 8;
    const u32x4_t g = load16<NT>(h), v = load16<NT>(h + a.I);
    unpack8(g, gate);
    unpack8(v, up);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = sigmoid_fast(gate[i]);
  if constexpr (A) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = gate[i] * s[i] * up[i];
    __builtin_nontemporal_store(pack8(y), reinterpret_cast<u32x4_t*>(a.a) + at);
  }
  if constexpr (DH) {
    float da[8], dg[8], du[8];
    unpack8(d, da);
#pragma unroll
    for (int i = 0; i < 8; ++i) swiglu_grad(da[i], gate[i], up[i], s[i], dg[i], du[i]);
    u32x4_t* dh = reinterpret_cast<u32x4_t*>(a.dh) + hat;
    __builtin_nontemporal_store(pack8(dg), dh);
    __builtin_nontemporal_store(pack8(du), dh + chunks);
  }
}

template <class F>
bool launch_chunks(SwigluArgs a, const char* name, hipStream_t s, F kernel) {
  const int chunks = a.I / 8;
  a.magic = static_cast<uint32_t>(((uint64_t{1} << 32) + chunks - 1) / chunks);
  const int64_t total = a.T * chunks;
  launch_parts((total + kThreads - 1) / kThreads, kThreads, [&](int64_t first, int64_t count) {
    a.first = first;
    launch_kernel(name, kernel, dim3(static_cast<unsigned>(count)), dim3(kThreads), 0, s, a);
  });
  return launch_ok(name);
}

}  // namespace

bool launch_swiglu_fwd(const SwigluArgs& a, int format, hipStream_t s) {
  if (a.T == 0) return true;
  // The checkpoint is read again much later.  With lines that are written in two
  // parts (I = 96) stores past the caches took 18.5 us against 17.1, with whole
  // ones 137 against 142.
  const Keep keep = a.h_codes == nullptr ? kDrop : a.I % 128 == 0 ? kKeepLines : kKeep;
  const bool nt = streams(static_cast<double>(a.T) * a.I *
                          (4 + (a.a ? 2 : 0) + (keep != kDrop ? 2 : 0) + (a.codes ? 1 : 0)));
  auto go = [&](auto fmt, auto kept) {
    constexpr int FMT = decltype(fmt)::value;
    constexpr Keep KEEP = decltype(kept)::value;
    return nt ? launch_chunks(a, "swiglu_fwd", s, swiglu_fwd_kernel<FMT, KEEP, true>)
              : launch_chunks(a, "swiglu_fwd", s, swiglu_fwd_kernel<FMT, KEEP, false>);
  };
  auto with_format = [&](auto kept) {
    if (format == kMxFp8) return go(std::integral_constant<int, kMxFp8>{}, kept);
    if (format == kMxFp4) return go(std::integral_constant<int, kMxFp4>{}, kept);
    return go(std::integral_constant<int, kMxNone>{}, kept);
  };
  if (keep == kKeepLines) return with_format(std::integral_constant<Keep, kKeepLines>{});
  if (keep == kKeep) return with_format(std::integral_constant<Keep, kKeep>{});
  return with_format(std::integral_constant<Keep, kDrop>{});
}

bool launch_swiglu_bwd(const SwigluArgs& a, hipStream_t s) {
  if (a.T == 0) return true;
  const bool ckpt = a.h_codes != nullptr;
  const bool nt = streams(static_cast<double>(a.T) * a.I * ((ckpt ? 2 : 4) + (a.a ? 2 : 0) + (a.dh ? 6 : 0)));
  auto go = [&](auto kept, auto dh, auto out) {
    constexpr bool CKPT = decltype(kept)::value, DH = decltype(dh)::value, A = decltype(out)::value;
    return nt ? launch_chunks(a, "swiglu_bwd", s, swiglu_bwd_kernel<CKPT, DH, A, true>)
              : launch_chunks(a, "swiglu_bwd", s, swiglu_bwd_kernel<CKPT, DH, A, false>);
  };
  auto outputs = [&](auto kept) {
    if (a.a == nullptr) return go(kept, std::true_type{}, std::false_type{});
    if (a.dh == nullptr) return go(kept, std::false_type{}, std::true_type{});
    return go(kept, std::true_type{}, std::true_type{});
  };
  return ckpt ? outputs(std::true_type{}) : outputs(std::false_type{});
}

}  // namespace w4a4
