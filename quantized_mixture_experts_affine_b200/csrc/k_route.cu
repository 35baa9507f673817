// Grouped top-k routing: softmax or sigmoid scores, a balance bias that only
// the selection sees, group-limited choice, renormalised weights.
//
// One warp per token.  The selection is exact: it gives what real arithmetic
// would.  Without a bias the experts are ordered by their logits.  With one
// (and for the sums of two that rank groups) the scores are taken in fp32
// first, with a bound on their error; only a row in which two candidates
// that decide something lie closer than that bound is done again in fp64.
// Near ties are rare (under 1 % of rows of 512 normal logits), so the row
// costs what the fp32 pass costs.
//
// Keys live in shared memory, four experts of a lane side by side, so that
// one code path serves 1 to 4096 experts and a pick rescans the winning
// lane's experts only.
#include "common.cuh"
#include "ops.h"
#include "route.cuh"

namespace moeq {
namespace {

struct RouteArgs {
  moeq_routing r;
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int64_t stride;
  int bf16;
  int M;
  int lanes_per_group;  // power of two
};

// Order-preserving keys.  0: dropped or taken; 1: an expert that is out (its
// logit is NaN or -inf) but may fill up; every other value is larger.
template <typename T>
struct Keys;
template <>
struct Keys<float> {
  using K = uint32_t;
  static __device__ __forceinline__ K of(float v) { return route_key(v); }
  static __device__ __forceinline__ float value(K k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
  }
  static __device__ __forceinline__ K max_of(K k) { return __reduce_max_sync(0xffffffffu, k); }
};
template <>
struct Keys<double> {
  using K = unsigned long long;
  static __device__ __forceinline__ K of(double v) {
    const K b = v == 0.0 ? 0ull : (K)__double_as_longlong(v);
    return (b >> 63) ? ~b : (b | (1ull << 63));
  }
  static __device__ __forceinline__ double value(K k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
  }
  static __device__ __forceinline__ K max_of(K k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo =
        __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((K)hi << 32) | lo;
  }
};

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

template <typename T>
__device__ __forceinline__ T warp_sum_t(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t row, int e) {
  return a.bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.logits)[row + e])
                : reinterpret_cast<const float*>(a.logits)[row + e];
}

__device__ __forceinline__ bool is_out(float l) { return !(l > -INFINITY); }

// Score of a logit: sigmoid, or the softmax's numerator relative to the
// row's largest logit.
template <typename T>
__device__ __forceinline__ T numerator(const moeq_routing& r, float l, float mx) {
  if (r.score == MOEQ_SCORE_SIGMOID) return (T)1 / ((T)1 + exp_of(-(T)r.router_scale * (T)l));
  return l == mx ? (T)1 : exp_of((T)r.router_scale * ((T)l - (T)mx));
}

// One pass over a token's row.  keys, raw: the warp's shared keys and fp32
// logits, a whole number of quads.  Returns false when fp32 cannot tell the
// selection (or hold the weights); nothing is written then.
template <typename T>
__device__ bool route_row(const RouteArgs& a, int m, typename Keys<T>::K* keys, float* raw) {
  using KT = Keys<T>;
  using K = typename KT::K;
  const moeq_routing& r = a.r;
  const int lane = threadIdx.x & 31;
  const int E = r.n_experts, nq = (E + 3) >> 2;
  const int64_t row = (int64_t)m * a.stride;
  const bool softmax = r.score == MOEQ_SCORE_SOFTMAX;
  const bool has_bias = a.bias != nullptr;
  const bool exact64 = sizeof(T) == 8;

  // ---- the row's logits, four neighbours per lane, kept as fp32 bits
  float mx = -INFINITY;
  {
    const size_t item = a.bf16 ? 2 : 4;
    const uintptr_t base = (uintptr_t)a.logits + (size_t)row * item;
    const bool vec = (base & (4 * item - 1)) == 0;
    for (int q = lane; q < nq; q += 32) {
      float l[4];
      if (vec && 4 * q + 4 <= E) {
        if (a.bf16) {
          const uint2 v = *reinterpret_cast<const uint2*>(base + (size_t)q * 8);
          l[0] = __uint_as_float(v.x << 16);
          l[1] = __uint_as_float(v.x & 0xFFFF0000u);
          l[2] = __uint_as_float(v.y << 16);
          l[3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(base + (size_t)q * 16);
          l[0] = v.x;
          l[1] = v.y;
          l[2] = v.z;
          l[3] = v.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) l[c] = 4 * q + c < E ? logit_at(a, row, 4 * q + c) : -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        raw[4 * q + c] = l[c];
        if (!is_out(l[c])) mx = fmaxf(mx, l[c]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }

  // ---- softmax normaliser (where a value of the scores themselves counts)
  T sum = (T)1;
  if (softmax && (has_bias || !r.renorm || (r.n_groups > 1 && r.group_top == 2))) {
    T z = (T)0;
    for (int q = lane; q < nq; q += 32)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float l = raw[4 * q + c];
        if (!is_out(l)) z += numerator<T>(r, l, mx);
      }
    sum = warp_sum_t(z);
  }
  // bound on the fp32 error of a score: a few roundings, the exponent's own
  // (|d| 2^-24, and e^-d d stays under 0.37) and the normaliser's additions
  // (nq / 8 + 5 of them in a row), all relative to the largest score
  T tol_s = (T)0;
  if (!exact64) {
    const T s_max = is_out(mx) ? (T)0 : numerator<T>(r, mx, mx) / (softmax ? sum : (T)1);
    tol_s = ((T)1.2e-6f + (softmax ? (T)6e-8f * (T)(nq / 8 + 12) : (T)0)) * s_max;
  }

  // ---- keys
  for (int q = lane; q < nq; q += 32) {
    K k[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = 4 * q + c;
      const float l = raw[e];
      if (e >= E) k[c] = 0;
      else if (is_out(l)) k[c] = 1;
      else if (!has_bias) k[c] = KT::of((T)l);
      else k[c] = KT::of(numerator<T>(r, l, mx) / sum + (T)a.bias[e]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) keys[4 * q + c] = k[c];
  }
  __syncwarp();

  bool sure = true;
  // ---- groups: the best topk_groups by their largest score, or the sum of
  // their two largest
  if (r.topk_groups < r.n_groups) {
    const int lpg = a.lanes_per_group, gs = E / r.n_groups;
    const int g = lane / lpg, sub = lane & (lpg - 1);
    K k1 = 0, k2 = 0;
    if (g < r.n_groups)
      for (int i = sub; i < gs; i += lpg) {
        const K k = keys[g * gs + i];
        if (k > k1) {
          k2 = k1;
          k1 = k;
        } else if (k > k2) {
          k2 = k;
        }
      }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
      const K p1 = __shfl_xor_sync(0xffffffffu, k1, o), p2 = __shfl_xor_sync(0xffffffffu, k2, o);
      const K lo = k1 < p1 ? k1 : p1, hi2 = k2 > p2 ? k2 : p2;
      k1 = k1 > p1 ? k1 : p1;
      k2 = lo > hi2 ? lo : hi2;
    }
    K gk = k1;
    T gv = (T)0;
    if (k1 > 1) {
      auto score = [&](K k) -> T {
        return has_bias ? KT::value(k) : numerator<T>(r, (float)KT::value(k), mx) / sum;
      };
      if (r.group_top == 2) {
        gv = score(k1) + (k2 > 1 ? score(k2) : (T)0);
        gk = KT::of(gv);
      } else if (has_bias) {
        gv = KT::value(k1);
      }
    }
    int rank = 0;
    for (int j = 0; j < r.n_groups; ++j) {
      const K kj = __shfl_sync(0xffffffffu, gk, j * lpg);
      rank += (kj > gk || (kj == gk && j < g)) ? 1 : 0;
    }
    const bool keep = g < r.n_groups && rank < r.topk_groups;
    const uint32_t kept = __ballot_sync(0xffffffffu, keep && sub == 0);
    if (!exact64 && (has_bias || r.group_top == 2)) {
      // the last kept and the first dropped group
      const bool in = g < r.n_groups && gk > 1;
      const K last = in && rank == r.topk_groups - 1 ? gk : 0;
      const K next = in && rank == r.topk_groups ? gk : 0;
      const K kl = KT::max_of(last), kn = KT::max_of(next);
      if (kl > 1 && kn > 1) {
        const T vl = KT::value(kl), vn = KT::value(kn);
        const T tol = (T)4 * tol_s + (T)4.8e-7f * (fabsf((float)vl) + fabsf((float)vn));
        if (!(vl - vn > tol)) sure = false;
      }
    }
    for (int q = lane; q < nq; q += 32)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = 4 * q + c;
        if (e < E && !((kept >> ((e / gs) * lpg)) & 1u)) keys[e] = 0;
      }
    __syncwarp();
  }

  // ---- the top_k largest keys, lower index first among equals
  K lk = 0;
  int li = kNoExpert;
  auto rescan = [&]() {
    lk = 0;
    li = kNoExpert;
    for (int q = lane; q < nq; q += 32)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const K k = keys[4 * q + c];
        if (k > lk) {
          lk = k;
          li = 4 * q + c;
        }
      }
  };
  rescan();
  K my_k = 0;
  int my_e = 0;
  for (int k = 0; k < r.top_k; ++k) {
    const K top = KT::max_of(lk);
    const int win =
        (int)__reduce_min_sync(0xffffffffu, (lk == top && li != kNoExpert) ? (uint32_t)li : 0x7fffffffu);
    if (li == win && win != kNoExpert) {
      keys[win] = 0;
      rescan();
    }
    if (lane == k) {
      my_k = top;
      my_e = win == kNoExpert ? 0 : win;
    }
  }
  const bool mine = lane < r.top_k;
  const bool valid = mine && my_k > 1;
  __syncwarp();

  // ---- doubt: neighbours in the order, and the last pick against the rest
  const float my_l = valid ? raw[my_e] : -INFINITY;
  if (!exact64 && has_bias) {
    const float v = valid ? (float)KT::value(my_k) : 0.0f;
    const float b = valid ? a.bias[my_e] : 0.0f;
    const float vn = __shfl_down_sync(0xffffffffu, v, 1);
    const float ln = __shfl_down_sync(0xffffffffu, my_l, 1);
    const float bn = __shfl_down_sync(0xffffffffu, b, 1);
    const bool next_valid = __shfl_down_sync(0xffffffffu, (int)valid, 1) && lane < 31;
    const float tol = 2.0f * (float)tol_s + 2.4e-7f * fabsf(v);
    if (valid && next_valid && lane + 1 < r.top_k && !(v - vn > tol) && !(my_l == ln && b == bn))
      sure = false;
    const int last = r.top_k - 1;
    const bool lv = __shfl_sync(0xffffffffu, (int)valid, last);
    const float v_last = __shfl_sync(0xffffffffu, v, last);
    const float l_last = __shfl_sync(0xffffffffu, my_l, last);
    const float b_last = __shfl_sync(0xffffffffu, b, last);
    const float tol_last = __shfl_sync(0xffffffffu, tol, last);
    // the largest key that is left decides whether any comes near
    if (lv && lk > 1 && !(v_last - (float)KT::value(lk) > tol_last)) {
      for (int q = lane; q < nq; q += 32)
        for (int c = 0; c < 4; ++c) {
          const int e = 4 * q + c;
          const K k = keys[e];
          if (k > 1 && !(v_last - (float)KT::value(k) > tol_last) &&
              !(raw[e] == l_last && a.bias[e] == b_last))
            sure = false;
        }
    }
  }

  // ---- weights
  const T p = valid ? numerator<T>(r, my_l, mx) : (T)0;
  T denom = sum;
  if (r.renorm) denom = warp_sum_t(p);
  if (!exact64 && r.renorm && denom < (T)1e-30f && __any_sync(0xffffffffu, valid)) sure = false;
  if (!exact64 && !__all_sync(0xffffffffu, sure)) return false;
  if (mine) {
    const int64_t at = (int64_t)m * r.top_k + lane;
    a.idx[at] = my_e;
    a.w[at] = denom > (T)0 ? (float)(p / denom * (T)r.routed_scale) : 0.0f;
  }
  return true;
}

__global__ void __launch_bounds__(256) k_route_groups(const __grid_constant__ RouteArgs a) {
  extern __shared__ uint64_t slots[];
  const int warp = threadIdx.x >> 5;
  const int m = blockIdx.x * (blockDim.x >> 5) + warp;
  if (m >= a.M) return;
  const int nq = (a.r.n_experts + 3) >> 2;
  uint64_t* mine = slots + (size_t)warp * (6 * nq);  // 4 nq keys of 8 bytes, 4 nq logits
  float* raw = reinterpret_cast<float*>(mine + 4 * nq);
  if (!route_row<float>(a, m, reinterpret_cast<uint32_t*>(mine), raw)) {
    __syncwarp();
    route_row<double>(a, m, reinterpret_cast<unsigned long long*>(mine), raw);
  }
}

}  // namespace

cudaError_t launch_route_groups(const moeq_routing& r, const void* logits, int logit_type,
                                int64_t stride, const float* bias, int M, int32_t* idx, float* w,
                                cudaStream_t st) {
  RouteArgs a;
  a.r = r;
  a.logits = logits;
  a.bias = bias;
  a.idx = idx;
  a.w = w;
  a.stride = stride;
  a.bf16 = logit_type == MOEQ_BF16;
  a.M = M;
  a.lanes_per_group = 1;
  while (a.lanes_per_group * 2 * r.n_groups <= 32) a.lanes_per_group *= 2;
  // 48 bytes per quad of experts and warp: 48 KB hold one row of 4096
  const int nq = (r.n_experts + 3) / 4;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  int warps = (M + sms - 1) / sms;  // few rows: spread over the SMs first
  if (warps > 8) warps = 8;
  while (warps > 1 && (size_t)warps * nq * 48 > 48 * 1024) --warps;
  k_route_groups<<<(M + warps - 1) / warps, warps * 32, (size_t)warps * nq * 48, st>>>(a);
  return cudaGetLastError();
}

}  // namespace moeq
