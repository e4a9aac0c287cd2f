// Device helpers shared by the HIP kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));   // scaled-MFMA operand (FP4 uses the low four)
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kWave = 64;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));

// Two floats -> packed bf16 bits (lo in the low half), round to nearest even:
// gfx950's v_cvt_pk_bf16_f32 (checked against the integer rounding on 2^24
// inputs, ties included).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{lo, hi}, bf16x2_t));
}

// float -> bf16 bits, round to nearest even.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  return static_cast<uint16_t>(pack_bf16x2(f, 0.0f));
}

// 1 / (1 + e^-x) from the hardware exp2 and reciprocal (each about 1 ulp);
// saturates to 0 / 1 without NaN for large |x|.  Used where the result is
// rounded to bf16 right after.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * 1.44269504088896341f));
}

// Gradients of a = gate s up, s = sigmoid(gate), for da.  Products from the bounded
// factor outwards: da up or da gate alone can pass the range where the result is
// 0 or moderate, and infinity times 0 is NaN.  s (1 + gate (1 - s)) reaches 1.0998,
// so dgate is made of its half: no product passes the range but where the result
// does.
__device__ __forceinline__ void swiglu_grad(float da, float gate, float up, float s, float& dgate, float& dup) {
  dgate = 2.0f * (da * (up * (s * (0.5f + gate * fmaf(-0.5f, s, 0.5f)))));
  dup = da * (gate * s);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    uint32_t o = __shfl_xor(v, off, kWave);
    v = o > v ? o : v;
  }
  return v;
}

}  // namespace w4a4
