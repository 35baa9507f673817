// Pieces shared by the tcgen05 linear kernels: row powers, the epilogue of an
// accumulator column, tensor maps.
#pragma once

#include <cuda.h>

#include "kernels.h"
#include "lincommon.cuh"
#include "tc.cuh"

namespace moeq {

constexpr int kBK = 64;  // columns per stage (128 bytes)

// tc::mbar_wait with the waiting out of line: these kernels run for a few
// microseconds, and fetching their instructions is much of that.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* status) {
  return tc::mbar_wait(bar, parity, status);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* status) {
  return tc::mbar_try_wait(bar, parity) || wait_on(bar, parity, status);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Power of two that brings a largest magnitude to [2^13, 2^14) (for tiny
// ones at most 2^126).
__device__ __forceinline__ int lift_of(float largest) {
  const int e = (int)(__float_as_uint(largest) >> 23) - 127;
  return largest > 0.0f ? min(13 - e, 126) : 0;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// The warp's index as a value the compiler knows to be the same in all lanes,
// and one lane of it: with both, a role's loop and its descriptors stay in
// uniform registers and the products are issued without branches.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// D (+)= A B^T as tc::mma_f16 and tc::mma_f16_pair, by the lane with `on`.
template <bool PAIR>
__device__ __forceinline__ void mma_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}

// 32 lanes x 16 columns of TMEM.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 lanes x 8 columns of TMEM.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// A warp's N tokens from m0 (nm of them real) of output column o: lane j's
// fx is token j's power.  mul and the residual are read together, before the
// stores that might overlap them, so that their latency is paid once.
// (Strides of at most 2^28 elements, kMaxStride: a row's address is one
// instruction.)  FULL: nm is N.
template <bool FULL = false, typename T, int N>
__device__ __forceinline__ void column(const void* p, int64_t stride, int64_t m0, int nm, int o,
                                       T (&r)[N]) {
  const char* c = reinterpret_cast<const char*>(reinterpret_cast<const T*>(p) + m0 * stride + o);
  const int step = (int)stride * (int)sizeof(T);
#pragma unroll
  for (int j = 0; j < N; ++j)
    r[j] = FULL || j < nm ? *reinterpret_cast<const T*>(c + (int64_t)step * j) : (T)0;
}
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ void as_out(float v, float* p) { *p = v; }
__device__ __forceinline__ void as_out(float v, uint16_t* p) {
  *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
}

// T: the type of y, mul and the residual (uint16_t: bf16 bits).  r: the
// residual's values, read ahead (unused without one).  (The two powers first:
// huge weights and tiny tokens make up for one another.)
template <typename T, int N, bool FULL = false>
__device__ __forceinline__ void finish_with(const moeq_linear_args& a, int64_t m0, int nm, int o,
                                            bool live, float fw, float bias, float fx,
                                            const uint32_t (&acc)[N], const T (&r)[N]) {
  float y[N];
#pragma unroll
  for (int j = 0; j < N; ++j)
    y[j] = __uint_as_float(acc[j]) * (fw * __shfl_sync(0xffffffffu, fx, j)) + bias;
  act_all(y, a.act);
  if (a.mul) {
    T f[N];
    column<FULL>(a.mul, a.mul_stride, m0, nm, o, f);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] *= as_float(f[j]);
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] += as_float(r[j]);
  }
  char* c = reinterpret_cast<char*>(reinterpret_cast<T*>(a.y) + m0 * a.y_stride + o);
  const int step = (int)a.y_stride * (int)sizeof(T);
  if (live) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (FULL || j < nm) as_out(y[j], reinterpret_cast<T*>(c + (int64_t)step * j));
  }
}
template <typename T, int N, bool FULL = false>
__device__ __forceinline__ void finish(const moeq_linear_args& a, int64_t m0, int nm, int o,
                                       bool live, float fw, float bias, float fx,
                                       const uint32_t (&acc)[N]) {
  T r[N];
  if (a.residual) column<FULL>(a.residual, a.residual_stride, m0, nm, o, r);
  finish_with<T, N, FULL>(a, m0, nm, o, live, fw, bias, fx, acc, r);
}

// [parts][rows][cols] fp16, boxes of 64 columns x `box` rows, 128-byte swizzle;
// what lies outside reads as zeros.
inline bool half_map(CUtensorMap* m, const __half* p, int cols, int64_t rows, int parts, int box) {
  auto fn = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(tensor_map_encoder());
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * 2 * rows};
  const cuuint32_t boxes[3] = {kBK, (cuuint32_t)box, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(p), dims, strides,
                  boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moeq
