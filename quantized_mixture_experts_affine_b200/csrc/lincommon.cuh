// Pieces shared by the linear kernels: code and token conversions to bf16
// pairs, the epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "ops.h"

namespace moeq {

// The activations use the fast exponential (relative |v| 2^-23 + 2^-22) and
// division; where their error is largest the value itself is smallest.
template <int ACT>
__device__ __forceinline__ float act1(float v) {
  if (ACT == MOEQ_ACT_SILU) return __fdividef(v, 1.0f + __expf(-v));
  if (ACT == MOEQ_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  if (ACT == MOEQ_ACT_GELU_TANH) {
    // 0.5 (1 + tanh(u)) = 1 / (1 + e^(-2u))
    const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
    return __fdividef(v, 1.0f + __expf(-2.0f * u));
  }
  if (ACT == MOEQ_ACT_RELU) return v > 0.0f ? v : (v != v ? v : 0.0f);
  if (ACT == MOEQ_ACT_SIGMOID) return __fdividef(1.0f, 1.0f + __expf(-v));
  return v;
}
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
#define MOEQ_ACT_CASE(A)                               \
  case A:                                              \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act1<A>(v[i]); \
    break;
  switch (act) {
    MOEQ_ACT_CASE(MOEQ_ACT_SILU)
    MOEQ_ACT_CASE(MOEQ_ACT_GELU)
    MOEQ_ACT_CASE(MOEQ_ACT_GELU_TANH)
    MOEQ_ACT_CASE(MOEQ_ACT_RELU)
    MOEQ_ACT_CASE(MOEQ_ACT_SIGMOID)
    default: break;
  }
#undef MOEQ_ACT_CASE
}
__device__ __forceinline__ float act_of(float v, int act) {
  float a[1] = {v};
  act_all(a, act);
  return a[0];
}

__device__ __forceinline__ float load_out(const void* p, int type, int64_t at) {
  return type == MOEQ_F32 ? reinterpret_cast<const float*>(p)[at]
                          : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void store_out(void* p, int type, int64_t at, float v) {
  if (type == MOEQ_F32) reinterpret_cast<float*>(p)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

// One output value: what it needs besides its sum, read ahead, and the rest.
struct Epilogue {
  float bias = 0.0f, mul = 1.0f, residual = 0.0f, x_scale = 1.0f;
  __device__ __forceinline__ void load(const moeq_linear_args& a, int64_t m, int o) {
    if (a.bias) bias = bf16_bits_to_float(a.bias[o]);
    if (a.mul) mul = load_out(a.mul, a.out_type, m * a.mul_stride + o);
    if (a.residual) residual = load_out(a.residual, a.out_type, m * a.residual_stride + o);
    if (a.x_type != MOEQ_BF16 && a.x_group == 0) x_scale = a.x_scales[m];
  }
  __device__ __forceinline__ void finish(const moeq_linear_args& a, int64_t m, int o,
                                         float v) const {
    v = act_of(v + bias, a.act);
    if (a.mul) v *= mul;
    store_out(a.y, a.out_type, m * a.y_stride + o, v + residual);
  }
};

// ------------------------------------------------------------------ code runs
// Words that hold a lane's C codes: its run may start inside a word when the
// width does not divide 32.
template <int BITS, int C>
struct Run {
  static constexpr int BITLEN = BITS * C;
  static constexpr int WORDS = BITLEN % 32 == 0 ? BITLEN / 32 : BITLEN / 32 + 1;
};

// Loads lane t's run of C codes of the span that starts at bit 4 C BITS sp of
// the row, in its first words from bit 0 on.  The words read lie in the span.
template <int BITS, int C>
__device__ __forceinline__ void load_run(const uint32_t* row, int sp, int t,
                                         uint32_t (&w)[Run<BITS, C>::WORDS]) {
  constexpr int BL = Run<BITS, C>::BITLEN, W = Run<BITS, C>::WORDS;
  if (BL % 32 == 0) {
    const uint32_t* p = row + (int64_t)sp * (4 * W) + t * W;
    if (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[W - 1] = v.w;
    } else if (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[W - 1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = p[i];
    }
    return;
  }
  const int bit = t * BL, first = bit >> 5, off = bit & 31;
  const uint32_t* p = row + (int64_t)sp * (4 * BL / 32) + first;
  const int last = 4 * BL / 32 - 1 - first;  // words of the span behind the first
  uint32_t raw[W + 1];
#pragma unroll
  for (int i = 0; i <= W; ++i) raw[i] = i <= last && 32 * i < off + BL ? p[i] : 0u;
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(raw[i], raw[i + 1], off);
}

// ------------------------------------------------------------------ bf16 pairs
// Four bytes (values 0..255, in order) as two bf16 pairs: 2^23 + c as fp32,
// minus 2^23; the upper half of an integer below 256 is its bf16.
__device__ __forceinline__ void bytes_to_bf16(uint32_t c, float bias, uint32_t& p0, uint32_t& p1) {
  const float f0 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7440u)) - bias;
  const float f1 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7441u)) - bias;
  const float f2 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7442u)) - bias;
  const float f3 = __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7443u)) - bias;
  p0 = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632u);
  p1 = __byte_perm(__float_as_uint(f2), __float_as_uint(f3), 0x7632u);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes below 128, two in the low bits of each half of c: 128 + q is a bf16
// with q in its mantissa.
__device__ __forceinline__ uint32_t low_to_bf16(uint32_t c) {
  return sub_bf16x2(c | 0x43004300u, 0x43004300u);
}

// Four E4M3 bytes as two bf16 pairs (exact).
__device__ __forceinline__ void e4m3_to_bf16(uint32_t c, uint32_t& p0, uint32_t& p1) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f16;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16) : "h"((uint16_t)(c >> (16 * h))));
    const __half2 v = *reinterpret_cast<const __half2*>(&f16);
    const float2 f = __half22float2(v);
    (h ? p1 : p0) = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632u);
  }
}

}  // namespace moeq
