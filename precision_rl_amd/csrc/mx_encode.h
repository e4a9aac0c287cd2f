// Device encoders of MX blocks (OCP Microscaling Formats v1.0, section 6.3)
// in the lane layout of the row operators: a lane holds 8 consecutive bf16
// elements of a row (16 bytes), a block of 32 is a quad of lanes.
//   X = floor(log2 amax) - emax clamped to [-127, 127], scale byte X + 127,
//   elements x / 2^X rounded to nearest even, saturating (E4M3: emax 8, at
//   448; E2M1: emax 2, at 6); -0 keeps its sign.
// A block that holds an infinity or a NaN takes the scale byte 255 (E8M0's
// NaN) and zero codes, so that every product with it is NaN.
#pragma once

#include "device_common.h"

namespace w4a4 {

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));

enum MxFormat : int { kMxNone = -1, kMxFp4 = 0, kMxFp8 = 1 };

// Lane l's value from lane l ^ 1 / l ^ 2 of its quad (DPP quad_perm).
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true));
}

// Largest magnitude (bf16 bits) of the quad's 32 elements.  All four lanes of
// the quad must be active.
__device__ __forceinline__ uint32_t mx_block_amax(const u32x4_t& v) {
  u16x2_t m = __builtin_bit_cast(u16x2_t, v[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int d = 1; d < 4; ++d) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, v[d] & 0x7FFF7FFFu));
  uint32_t a = m[0] > m[1] ? m[0] : m[1];
  a = max(a, quad_xor1(a));
  return max(a, quad_xor2(a));
}

// The lane's codes of its block: two dwords (E4M3) or one (E2M1, in c[0]).
// Returns the block's scale byte.  From the exponent field eb of the block
// maximum, floor(log2 amax) = eb - 127, so the byte is max(eb - emax, 0);
// x 2^-X is exact in FP32 except where it underflows, far below the smallest
// midpoint of either grid.
template <int FMT>
__device__ __forceinline__ uint32_t mx_encode8(const u32x4_t& v, uint32_t (&c)[2]) {
  constexpr uint32_t kEmax = FMT == kMxFp8 ? 8u : 2u;
  const uint32_t eb = mx_block_amax(v) >> 7;
  const uint32_t byte = eb > kEmax ? eb - kEmax : 0u;
  const float inv = __uint_as_float((254u - byte) << 23);   // 2^-X
  c[0] = c[1] = 0u;
  if constexpr (FMT == kMxFp8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t half[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t w = v[2 * h + p];
        const float lo = __builtin_amdgcn_fmed3f(__uint_as_float(w << 16) * inv, -448.0f, 448.0f);
        const float hi = __builtin_amdgcn_fmed3f(__uint_as_float(w & 0xFFFF0000u) * inv, -448.0f, 448.0f);
        const s16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s16x2_t{0, 0}, lo, hi, 1.0f, false);
        half[p] = static_cast<uint32_t>(static_cast<uint16_t>(r[0]));
      }
      c[h] = half[0] | (half[1] << 16);
    }
  } else {
    uint32_t a = 0u;
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, __uint_as_float(v[0] << 16) * inv,
                                                 __uint_as_float(v[0] & 0xFFFF0000u) * inv, 1.0f, 0);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, __uint_as_float(v[1] << 16) * inv,
                                                 __uint_as_float(v[1] & 0xFFFF0000u) * inv, 1.0f, 1);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, __uint_as_float(v[2] << 16) * inv,
                                                 __uint_as_float(v[2] & 0xFFFF0000u) * inv, 1.0f, 2);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, __uint_as_float(v[3] << 16) * inv,
                                                 __uint_as_float(v[3] & 0xFFFF0000u) * inv, 1.0f, 3);
    c[0] = a;
  }
  if (eb == 255u) {
    c[0] = c[1] = 0u;
    return 255u;
  }
  return byte;
}

// Stores the lane's codes and, from the quad's first lane, the scale byte of
// the chunk with flat index `chunk` (8 elements each) of a dense [T, K] matrix.
template <int FMT>
__device__ __forceinline__ void mx_store8(uint8_t* codes, uint8_t* scales, int64_t chunk, const uint32_t (&c)[2],
                                          uint32_t byte) {
  if constexpr (FMT == kMxFp8)
    *reinterpret_cast<u32x2_t*>(codes + chunk * 8) = u32x2_t{c[0], c[1]};
  else
    *reinterpret_cast<uint32_t*>(codes + chunk * 4) = c[0];
  if ((chunk & 3) == 0) scales[chunk >> 2] = static_cast<uint8_t>(byte);
}

}  // namespace w4a4
