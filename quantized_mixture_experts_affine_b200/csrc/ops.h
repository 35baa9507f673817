// Launchers of the routing, norm and linear operators (k_route.cu, k_norm.cu,
// k_linear.cu, k_lingemm.cu), called by ops_api.cu after its argument checks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moeq.h"

namespace moeq {

// Launches a kernel as the successor of whatever precedes it in the stream: its
// CTAs may be set up as soon as that one's have ended or let it (tc::grid_dep_launch),
// so every one of them waits (tc::grid_dep_wait) before it touches what the
// other may still write or read.  One call after the other, without a graph:
// 1 x 4096 x 4096 linear 8.6 -> 6.6 us, 64 x 4096 x 4096 14.3 -> 12.2, 16,068 x
// 128 routing 13.0 -> 11.2, 333 x 1000 norm 3.45 -> 3.0 (in a graph).
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 blocks, unsigned threads, size_t smem,
                         cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = blocks;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

cudaError_t launch_route_groups(const moeq_routing& r, const void* logits, int logit_type,
                                int64_t stride, const float* bias, int M, int32_t* idx, float* w,
                                cudaStream_t st);

cudaError_t launch_add_rmsnorm(const moeq_norm_args& n, int M, int H, cudaStream_t st);

// One matrix of a packed tensor and the operands around it, as the linear
// kernels read them.
struct LinArgs {
  const uint32_t* w;
  const uint16_t* scales;  // MX FP4: uint8 exponents
  const uint16_t* biases;
  int out_dim, in_dim, bits, G, mx;
  moeq_linear_args a;
  int M;
  int scales_wide;  // (k_linear.cu) a row's scales can be loaded four spans at a time
};

// Largest row stride of y, mul and the residual (elements).
constexpr int64_t kMaxStride = 1 << 28;

cudaError_t launch_linear_small(const LinArgs& l, cudaStream_t st);

// Many tokens: operand layout and product, over a workspace; *launches: how
// many kernels that took.
size_t linear_gemm_workspace(const moeq_qtensor& t, int M, int x_type, int out_type);
cudaError_t launch_linear_gemm(const LinArgs& l, void* ws, int* status, int* launches,
                               cudaStream_t st);
// Tiling of the product that unpacks the weights itself (tokens 0: its sums
// would be too long for the type of y) and the clocks that a call takes.
struct LinPlan {
  int tokens;      // of a tile
  int log2_split;  // CTAs that share a row's columns
  int tiles_m;
  double clocks;
};
LinPlan linear_fused_plan(int64_t M, int64_t in_dim, int64_t out_dim, int out_type);
// The product with the weights unpacked inside it, on tokens laid out
// in fp16 (fx, fw: the powers of two of token and weight rows; sb: scales and biases
// as fp16 pairs, [group][out_dim], times the weight row's power).
cudaError_t launch_linear_fused(const LinArgs& l, const __half* x16, const float* fx,
                                const float* fw, const uint32_t* sb, int* status,
                                cudaStream_t st);

}  // namespace moeq
