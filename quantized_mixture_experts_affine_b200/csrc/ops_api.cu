// Entry points of the routing, norm and linear operators and of the layer
// with such a router (include/moeq.h): argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "moeq.h"
#include "ops.h"

#define MOEQ_API extern "C" __attribute__((visibility("default")))

using namespace moeq;

namespace {

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t size_of(int type) { return type == MOEQ_F32 ? 4 : type == MOEQ_BF16 ? 2 : 1; }
bool finite(float v) { return v - v == 0.0f; }

moeq_status launched(cudaError_t e, int n = 1) {
  if (e != cudaSuccess) return MOEQ_ERR_CUDA;
  count_launches(n);
  return MOEQ_OK;
}

moeq_status check_routing(const moeq_routing* r) {
  if (!r) return MOEQ_ERR_INVALID_ARG;
  const int E = r->n_experts, K = r->top_k, G = r->n_groups;
  if (E <= 0 || K <= 0 || G <= 0 || r->topk_groups <= 0 || r->topk_groups > G)
    return MOEQ_ERR_INVALID_ARG;
  if (r->score != MOEQ_SCORE_SOFTMAX && r->score != MOEQ_SCORE_SIGMOID)
    return MOEQ_ERR_INVALID_ARG;
  if (r->group_top != 1 && r->group_top != 2) return MOEQ_ERR_INVALID_ARG;
  if (r->renorm != 0 && r->renorm != 1) return MOEQ_ERR_INVALID_ARG;
  if (!finite(r->router_scale) || !(r->router_scale > 0.0f) || !finite(r->routed_scale))
    return MOEQ_ERR_INVALID_ARG;
  if (E > kMaxE || K > kMaxK || G > 32) return MOEQ_ERR_UNSUPPORTED;
  if (E % G || K > E / G * r->topk_groups) return MOEQ_ERR_INVALID_ARG;
  return MOEQ_OK;
}

// Rows of `count` elements at p, `stride` apart, on their element's alignment.
moeq_status check_rows(const void* p, int type, int64_t stride, int64_t count) {
  if (stride < count) return MOEQ_ERR_INVALID_ARG;
  return on(p, size_of(type)) ? MOEQ_OK : MOEQ_ERR_ALIGNMENT;
}

bool float_type(int t) { return t == MOEQ_F32 || t == MOEQ_BF16; }

#define TRY(x)                         \
  do {                                 \
    const moeq_status s_ = (x);        \
    if (s_ != MOEQ_OK) return s_;      \
  } while (0)

moeq_status check_matrix(const moeq_qtensor* t, int32_t expert) {
  if (!t || expert < 0) return MOEQ_ERR_INVALID_ARG;
  TRY(tensor_check(t, (int64_t)expert + 1));
  if (expert > 0 && (t->expert_stride_w <= 0 || t->expert_stride_sb <= 0))
    return MOEQ_ERR_INVALID_ARG;
  return MOEQ_OK;
}

LinArgs lin_args(const moeq_qtensor& t, int expert, const moeq_linear_args& a, int M) {
  LinArgs l;
  l.w = t.w + (int64_t)expert * t.expert_stride_w;
  l.scales = scale_at(t, (int64_t)expert * t.expert_stride_sb);
  l.mx = t.format == MOEQ_FMT_MXFP4;
  l.biases = l.mx ? nullptr : t.biases + (int64_t)expert * t.expert_stride_sb;
  l.out_dim = t.out_dim;
  l.in_dim = t.in_dim;
  l.bits = t.bits;
  l.G = t.group_size;
  l.a = a;
  l.M = M;
  return l;
}

// The code products (k_linear.cu) take up to 16 tokens, and more while their
// CTAs (16 rows x 16 tokens each) are resident at once: one per SM, or two
// where y is fp32, which doubles the other path's products.  4096 columns:
// 512 rows, 64 tokens, fp32 (128 CTAs) 7.9 against 11.7 us; 128 tokens (256
// CTAs) 10.7 against 13.7; 1024 rows, 64 tokens, bf16 (256 CTAs) 12.8 against
// 10.4; 4096 rows, 16 tokens, bf16 11.0 against 11.3.
bool small_case(int64_t M, int64_t out_dim, int out_type) {
  return M <= 16 ||
         (M + 15) / 16 * ((out_dim + 15) / 16) <= (out_type == MOEQ_F32 ? 2 * 148 : 148);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

MOEQ_API moeq_status moeq_route_groups(const moeq_routing* r, const void* logits,
                                       int32_t logit_type, int64_t logit_stride,
                                       const float* bias, int32_t M, int32_t* idx, float* w,
                                       void* stream) {
  TRY(check_routing(r));
  if (M < 0) return MOEQ_ERR_INVALID_ARG;
  if (!float_type(logit_type)) return MOEQ_ERR_UNSUPPORTED;
  if (M == 0) return MOEQ_OK;
  if (!logits || !idx || !w) return MOEQ_ERR_INVALID_ARG;
  TRY(check_rows(logits, logit_type, logit_stride, r->n_experts));
  if (!on(bias, 4) || !on(idx, 4) || !on(w, 4)) return MOEQ_ERR_ALIGNMENT;
  return launched(launch_route_groups(*r, logits, logit_type, logit_stride, bias, M, idx, w,
                                      (cudaStream_t)stream));
}

MOEQ_API moeq_status moeq_add_rmsnorm(const moeq_norm_args* n, int32_t M, int32_t H,
                                      void* stream) {
  if (!n || M < 0 || H <= 0) return MOEQ_ERR_INVALID_ARG;
  if (H > 32768) return MOEQ_ERR_UNSUPPORTED;
  if (!finite(n->eps) || !(n->eps > 0.0f)) return MOEQ_ERR_INVALID_ARG;
  if (!float_type(n->x_type)) return MOEQ_ERR_UNSUPPORTED;
  if (M == 0) return MOEQ_OK;
  if (!n->x || !n->gamma || (!n->y && !n->q)) return MOEQ_ERR_INVALID_ARG;
  TRY(check_rows(n->x, n->x_type, n->x_stride, H));
  if (!on(n->gamma, 2)) return MOEQ_ERR_ALIGNMENT;
  if (n->residual) {
    if (!float_type(n->r_type)) return MOEQ_ERR_UNSUPPORTED;
    TRY(check_rows(n->residual, n->r_type, n->r_stride, H));
    if (n->r_out) TRY(check_rows(n->r_out, n->r_type, n->r_out_stride, H));
  } else if (n->r_out) {
    return MOEQ_ERR_INVALID_ARG;
  }
  if (n->y) TRY(check_rows(n->y, MOEQ_BF16, n->y_stride, H));
  if (n->q) {
    if (n->q_type != MOEQ_I8 && n->q_type != MOEQ_E4M3) return MOEQ_ERR_UNSUPPORTED;
    if (n->q_group != 0 && n->q_group != 128) return MOEQ_ERR_UNSUPPORTED;
    if (!n->q_scales) return MOEQ_ERR_INVALID_ARG;
    TRY(check_rows(n->q, n->q_type, n->q_stride, H));
    if (!on(n->q_scales, 4)) return MOEQ_ERR_ALIGNMENT;
  }
  return launched(launch_add_rmsnorm(*n, M, H, (cudaStream_t)stream));
}

MOEQ_API size_t moeq_linear_workspace_bytes(const moeq_qtensor* t, int32_t M, int32_t x_type,
                                            int32_t out_type) {
  const bool x8 = x_type == MOEQ_I8 || x_type == MOEQ_E4M3;
  if (check_matrix(t, 0) != MOEQ_OK || M <= 0 || small_case(M, t->out_dim, out_type) ||
      !(x8 || x_type == MOEQ_BF16) ||
      !float_type(out_type))
    return 0;
  return linear_gemm_workspace(*t, M, x_type, out_type);
}

MOEQ_API moeq_status moeq_linear(const moeq_qtensor* t, int32_t expert, const moeq_linear_args* a,
                                 int32_t M, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_matrix(t, expert));
  if (!a || M < 0) return MOEQ_ERR_INVALID_ARG;
  const bool x8 = a->x_type == MOEQ_I8 || a->x_type == MOEQ_E4M3;
  if (!x8 && a->x_type != MOEQ_BF16) return MOEQ_ERR_UNSUPPORTED;
  if (!float_type(a->out_type)) return MOEQ_ERR_UNSUPPORTED;
  if (a->act < MOEQ_ACT_NONE || a->act > MOEQ_ACT_SIGMOID) return MOEQ_ERR_INVALID_ARG;
  if (x8 && a->x_group != 0 && a->x_group != 128) return MOEQ_ERR_UNSUPPORTED;
  if (M == 0) return MOEQ_OK;
  if (!a->x || !a->y || (x8 && !a->x_scales)) return MOEQ_ERR_INVALID_ARG;
  TRY(check_rows(a->x, a->x_type, a->x_stride, t->in_dim));
  if (!on(a->x, 16) || (a->x_stride * (int64_t)size_of(a->x_type)) % 16) return MOEQ_ERR_ALIGNMENT;
  if (x8 && !on(a->x_scales, 4)) return MOEQ_ERR_ALIGNMENT;
  if (!on(a->bias, 2)) return MOEQ_ERR_ALIGNMENT;
  TRY(check_rows(a->y, a->out_type, a->y_stride, t->out_dim));
  if (a->mul) TRY(check_rows(a->mul, a->out_type, a->mul_stride, t->out_dim));
  if (a->residual) TRY(check_rows(a->residual, a->out_type, a->residual_stride, t->out_dim));
  if (a->y_stride > kMaxStride || (a->mul && a->mul_stride > kMaxStride) ||
      (a->residual && a->residual_stride > kMaxStride))
    return MOEQ_ERR_UNSUPPORTED;
  const size_t need = moeq_linear_workspace_bytes(t, M, a->x_type, a->out_type);
  if (need > 0) {
    if (!ws || ws_bytes < need) return MOEQ_ERR_WORKSPACE;
    if (!on(ws, 256)) return MOEQ_ERR_ALIGNMENT;
  }
  if (sm_count() <= 0) return MOEQ_ERR_CUDA;  // no current device to size launches for
  const LinArgs l = lin_args(*t, expert, *a, M);
  if (small_case(M, t->out_dim, a->out_type))
    return launched(launch_linear_small(l, (cudaStream_t)stream));
  int* status = device_status_word();
  if (!status) return MOEQ_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = launch_linear_gemm(l, ws, status, &launches, (cudaStream_t)stream);
  return launched(e, launches);
}

// ------------------------------------------------------------------ the layer with such a router
namespace {
struct RoutedWs {
  size_t logits, idx, w, rest, total;  // rest: the router's product, then the experts
};

bool routed_ws(const moeq_layer* L, int M, int mode, RoutedWs& o) {
  const size_t layer = moeq_workspace_bytes(L, M, mode);
  if (layer == 0) return false;
  const size_t lin = moeq_linear_workspace_bytes(&L->router, M, MOEQ_BF16, MOEQ_F32);
  o.logits = 0;
  o.idx = up256((size_t)M * L->n_experts * 4);
  o.w = o.idx + up256((size_t)M * L->top_k * 4);
  o.rest = o.w + up256((size_t)M * L->top_k * 4);
  o.total = o.rest + (layer > lin ? layer : lin);
  return true;
}
}  // namespace

MOEQ_API size_t moeq_routed_workspace_bytes(const moeq_layer* L, int32_t M, int32_t mode) {
  RoutedWs o;
  return routed_ws(L, M, mode, o) ? o.total : 0;
}

MOEQ_API moeq_status moeq_layer_forward_routed(const moeq_layer* L, const moeq_routing* r,
                                               const float* bias, const uint16_t* x, int32_t M,
                                               float* y, const float* residual, int32_t* idx_out,
                                               float* w_out, void* ws, size_t ws_bytes,
                                               int32_t mode, void* stream) {
  TRY(forward_arg_check(L, x, M, y, residual, mode, /*empty=*/true));
  TRY(check_routing(r));
  if (r->n_experts != L->n_experts || r->top_k != L->top_k) return MOEQ_ERR_INVALID_ARG;
  if (!on(bias, 4) || !on(idx_out, 4) || !on(w_out, 4)) return MOEQ_ERR_ALIGNMENT;
  if (M == 0) return MOEQ_OK;
  TRY(mode_check(L, M, mode));
  RoutedWs o;
  if (!routed_ws(L, M, mode, o)) return MOEQ_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < o.total) return MOEQ_ERR_WORKSPACE;
  if (!on(ws, 256)) return MOEQ_ERR_ALIGNMENT;
  char* base = (char*)ws;
  float* logits = (float*)(base + o.logits);
  int32_t* idx = idx_out ? idx_out : (int32_t*)(base + o.idx);
  float* w = w_out ? w_out : (float*)(base + o.w);
  moeq_linear_args a = {};
  a.x = x;
  a.x_type = MOEQ_BF16;
  a.x_stride = L->hidden;
  a.y = logits;
  a.out_type = MOEQ_F32;
  a.y_stride = L->n_experts;
  TRY(moeq_linear(&L->router, 0, &a, M, base + o.rest, o.total - o.rest, stream));
  TRY(moeq_route_groups(r, logits, MOEQ_F32, L->n_experts, bias, M, idx, w, stream));
  return moeq_expert_ffn(L, x, M, idx, w, residual, y, base + o.rest, o.total - o.rest, mode,
                         stream);
}
