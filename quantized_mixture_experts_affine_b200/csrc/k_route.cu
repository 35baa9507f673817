// Grouped top-k routing: softmax or sigmoid scores, a balance bias that only
// the selection sees, group-limited choice, renormalised weights.
//
// The selection is exact: it gives what fp64 scores would.  Without a bias
// the experts are ordered by their logits.  With one (and for the sums of two
// that rank groups) the scores are taken in fp32 first, with a bound on their
// error; where two candidates that decide something lie closer than that, fp64
// decides: for picks among the few experts concerned, one per lane, for groups
// the whole row again.  Such rows are about 1 % of 512 normal logits.
//
// A row of up to 512 experts is held in registers by a warp, or with many rows
// by 8 or 16 lanes, groups padded to a power of two of quads (300 rows of 160 in
// 8 groups: 8.5 us in shared memory, 4.3 so); what is larger (k_route_any) lives
// in shared memory.  Few
// rows are bound by the chain of load, exponential and K picks (3.8 us for one
// row, 5.9 us for 2048 rows of 256 experts in 8 groups).  Many rows (16,068 of 128
// in 8 groups, top-8: 11.2 us; 15.4 us with picks that scanned 16 registers instead
// of a quad in shared memory, 24.3 us with a warp per row) take 423 warp
// instructions each, 6 us of issue at one a clock; the schedulers issue in 58 % of
// their clocks, the rest are the dependent steps of a pick (shuffles, shared
// memory) with six warps to hide them.
#include "common.cuh"
#include "ops.h"
#include "route.cuh"
#include "tc.cuh"

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
  int slot;             // 8-byte words of shared memory per warp
  // Registers path, with groups: quads laid out for one, a power of two, and
  // its experts (which may leave the last quads empty or end inside one).
  int group_quads, group_size;
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

// Where a row's largest score is below this, smaller ones leave fp32's normal
// range and what decides is taken in fp64.
constexpr float kTinyScore = 1e-30f;

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
  // bound on the fp32 error of a score, relative to the largest: a few roundings,
  // the exponential and the normaliser's additions (nq / 8 + 5 of them in a row);
  // a softmax's exponents d count from the largest (e^-d d stays under 0.37, the
  // normaliser's mean of d under ln 4096), a sigmoid's do not: where the largest
  // logit is below zero, all scores are off by its exponent's rounding
  T tol_s = (T)0;
  if (!exact64) {
    const T s_max = is_out(mx) ? (T)0 : numerator<T>(r, mx, mx) / (softmax ? sum : (T)1);
    const T far = softmax ? (T)6e-8f * (T)(nq / 8 + 12)
                          : (T)1.2e-7f * (T)fmaxf(0.0f, -r.router_scale * mx);
    tol_s = s_max < (T)kTinyScore ? (T)INFINITY : ((T)1.2e-6f + far) * s_max;
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

// ---- registers: up to 512 experts, counting what groups are padded with (GROUPS
// 2; 1: they are a power of two of whole quads)
// L lanes hold a row (a warp holds 32 / L rows): lane l of them the quads
// l + L j, experts 4 q .. 4 q + 3.  Same steps as route_row<float>; a group's
// members are neighbouring lanes, so its two largest keys come from a
// butterfly, and a pick rescans 4 NQ registers.  With L = 32 a doubt about
// the picks themselves is settled on the spot: the few experts concerned are
// scored in fp64, one per lane, and ranked again.

// 1 / (1 + e^-z) and e^d; the fast exponential and division are within 2 ulp,
// but for the exponent's rounding.  EXACT_EXP: the softmax's by expf, since beside
// a bias the normaliser's error counts (2048 x 256 in 8 groups: with the fast
// one's bound more rows are in doubt, 10.4 against 7.9 us).
template <bool EXACT_EXP>
__device__ __forceinline__ float fast_numerator(const moeq_routing& r, float l, float mx) {
  if (r.score == MOEQ_SCORE_SIGMOID) return __fdividef(1.0f, 1.0f + __expf(-r.router_scale * l));
  if (l == mx) return 1.0f;
  const float d = r.router_scale * (l - mx);
  return EXACT_EXP ? expf(d) : __expf(d);
}

// Keys<float>::of for what is not NaN (v + 0 makes one zero of both).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

template <int L>
__device__ __forceinline__ uint32_t seg_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L >> 1; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint32_t seg_min(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L >> 1; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The segment's bits of a ballot, from bit 0 on.
template <int L>
__device__ __forceinline__ uint32_t seg_ballot(bool p) {
  const uint32_t b = __ballot_sync(0xffffffffu, p);
  return L == 32 ? b : (b >> ((threadIdx.x & 31) & ~(L - 1))) & ((1u << (L & 31)) - 1u);
}

// Every lane of the warp calls it; m: its segment's token (store: whether to
// write it).  slots: 96 words of the warp's shared memory, then 4 NQ words for
// each lane.  Returns false
// in every lane of a segment whose row is not settled (nothing is written).
template <int L, int NQ, int GROUPS, bool BIAS>
__device__ __forceinline__ bool route_regs(const RouteArgs& a, int m, bool store,
                                           uint32_t* slots) {
  using KT = Keys<float>;
  const moeq_routing& r = a.r;
  const int lane = threadIdx.x & (L - 1), E = r.n_experts;
  const int64_t row = (int64_t)m * a.stride;
  const bool softmax = r.score == MOEQ_SCORE_SOFTMAX;
  // first expert of quad q, and how many it has
  auto quad = [&](int q, int& n) -> int {
    if (GROUPS == 2) {
      const int lg = 31 - __clz(a.group_quads), g = q >> lg, i = q & (a.group_quads - 1);
      n = g < r.n_groups ? a.group_size - 4 * i : 0;
      return g * a.group_size + 4 * i;
    }
    n = E - 4 * q;
    return 4 * q;
  };
  auto expert = [&](int place) -> int {  // of place 4 q + c
    int n;
    return GROUPS == 2 ? quad(place >> 2, n) + (place & 3) : place;
  };
  float l[NQ][4], b[NQ][4];
  {
    const size_t item = a.bf16 ? 2 : 4;
    const uintptr_t base = (uintptr_t)a.logits + (size_t)row * item;
    const bool even = GROUPS != 2 || (a.group_size & 3) == 0;
    const bool vec = even && (base & (4 * item - 1)) == 0,
               bvec = even && ((uintptr_t)a.bias & 15) == 0;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      int n;
      const int e0 = quad(lane + L * j, n);
#pragma unroll
      for (int c = 0; c < 4; ++c) l[j][c] = -INFINITY, b[j][c] = 0.0f;
      if (vec && n >= 4) {
        if (a.bf16) {
          const uint2 v = *reinterpret_cast<const uint2*>(base + (size_t)e0 * 2);
          l[j][0] = __uint_as_float(v.x << 16);
          l[j][1] = __uint_as_float(v.x & 0xFFFF0000u);
          l[j][2] = __uint_as_float(v.y << 16);
          l[j][3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(base + (size_t)e0 * 4);
          l[j][0] = v.x;
          l[j][1] = v.y;
          l[j][2] = v.z;
          l[j][3] = v.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < n) l[j][c] = logit_at(a, row, e0 + c);
      }
      if (BIAS) {
        if (bvec && n >= 4) {
          const float4 v = *reinterpret_cast<const float4*>(a.bias + e0);
          b[j][0] = v.x;
          b[j][1] = v.y;
          b[j][2] = v.z;
          b[j][3] = v.w;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < n) b[j][c] = a.bias[e0 + c];
        }
      }
    }
  }
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) mx = fmaxf(mx, l[j][c]);  // fmaxf passes over NaN
  mx = KT::value(seg_max<L>(KT::of(mx)));

  float sum = 1.0f;
  if (softmax && (BIAS || !r.renorm || (GROUPS && r.group_top == 2))) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (!is_out(l[j][c])) z += fast_numerator<BIAS>(r, l[j][c], mx);
    sum = seg_sum<L>(z);
  }
  const float inv = __fdividef(1.0f, sum);
  // Error of a score relative to the largest, in units of 2^-23 (1.2e-7).
  // Sigmoid: the exponential 2 + 1.18 |z| and half of |z| for its exponent's
  // rounding, times 1 - s; the sum and the division 3; above zero that is under 6,
  // below it 1.68 |z| of the largest logit come on top.  Softmax, x counted from the
  // largest: the exponential 2 + 1.18 x (expf: 2), its exponent's roundings x, all
  // that times e^-x, which is 2.1; the last rounding 0.5.  With a bias the
  // normaliser counts too: its terms 2 + x, whose mean is at most ln(E / sum) (an
  // entropy is at most ln E), half of its 4 NQ + 5 additions, and the division 2.
  const float s_max = is_out(mx) ? 0.0f : fast_numerator<BIAS>(r, mx, mx) * inv;
  float far = 0.0f;
  if (!softmax) far = 2.4e-7f * fmaxf(0.0f, -r.router_scale * mx);
  else if (BIAS) far = 1.2e-7f * __logf((float)E * 1.01f * inv) + 6e-8f * (4 * NQ + 7);
  const float tol_s = s_max < kTinyScore ? INFINITY : (7.2e-7f + far) * s_max;

  uint32_t k[NQ][4];
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    int n;
    quad(lane + L * j, n);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = BIAS ? fast_numerator<BIAS>(r, l[j][c], mx) * inv + b[j][c] : l[j][c];
      k[j][c] = c >= n ? 0u : is_out(l[j][c]) ? 1u : BIAS ? KT::of(v) : key_of(v);
    }
  }

  bool sure = true;
  if (GROUPS) {
    const int w = a.group_quads, lg = 31 - __clz(w);  // quads per group, a power of two
    uint32_t gk[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const uint32_t h0 = max(k[j][0], k[j][1]), l0 = min(k[j][0], k[j][1]);
      const uint32_t h1 = max(k[j][2], k[j][3]), l1 = min(k[j][2], k[j][3]);
      uint32_t k1 = max(h0, h1), k2 = max(min(h0, h1), max(l0, l1));
      for (int o = w >> 1; o > 0; o >>= 1) {
        const uint32_t p1 = __shfl_xor_sync(0xffffffffu, k1, o);
        const uint32_t p2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(min(k1, p1), max(k2, p2));
        k1 = max(k1, p1);
      }
      gk[j] = k1;
      if (r.group_top == 2 && k1 > 1) {
        const float v1 = BIAS ? KT::value(k1) : fast_numerator<BIAS>(r, KT::value(k1), mx) * inv;
        const float v2 = k2 <= 1 ? 0.0f
                         : BIAS  ? KT::value(k2)
                                 : fast_numerator<BIAS>(r, KT::value(k2), mx) * inv;
        gk[j] = KT::of(v1 + v2);
      }
    }
    // lane g: the key of group g (n_groups <= L)
    uint32_t mine = 0;
    const int at = lane << lg;  // its first quad
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const uint32_t v = __shfl_sync(0xffffffffu, gk[j], at & (L - 1), L);
      if (lane < r.n_groups && at / L == j) mine = v;
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < r.n_groups; ++g) {
      const uint32_t v = __shfl_sync(0xffffffffu, mine, g, L);
      rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    const bool in = lane < r.n_groups;
    const uint32_t kept = seg_ballot<L>(in && rank < r.topk_groups);
    if (BIAS || r.group_top == 2) {
      const uint32_t kl = seg_max<L>(in && rank == r.topk_groups - 1 ? mine : 0u);
      const uint32_t kn = seg_max<L>(in && rank == r.topk_groups ? mine : 0u);
      if (kl > 1 && kn > 1) {
        // two scores and three roundings on each side
        const float vl = KT::value(kl), vn = KT::value(kn);
        if (!(vl - vn > 4.0f * tol_s + 1.8e-7f * (fabsf(vl) + fabsf(vn)))) sure = false;
      }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j)
      if (!((kept >> (((lane + L * j) >> lg) & 31)) & 1u)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) k[j][c] = 0;
      }
  }

  // A lane keeps its quads' largest keys in registers and the keys themselves
  // in shared memory, where a pick clears one and looks at its quad again.
  uint32_t qk[NQ] = {}, lk = 0;
  int qi[NQ] = {}, li = kNoExpert;
  uint4* own = reinterpret_cast<uint4*>(slots + 96) + NQ * (threadIdx.x & 31);
  auto top_of = [](const uint4& v, uint32_t& k1, int& i1) {
    const bool a = v.y > v.x, b = v.w > v.z;
    const uint32_t ka = a ? v.y : v.x, kb = b ? v.w : v.z;
    const bool c = kb > ka;
    k1 = c ? kb : ka;
    i1 = c ? (b ? 3 : 2) : (a ? 1 : 0);
  };
  auto best = [&]() {
    lk = qk[0];
    li = qi[0];
#pragma unroll
    for (int j = 1; j < NQ; ++j)
      if (qk[j] > lk) {
        lk = qk[j];
        li = qi[j];
      }
    if (lk == 0) li = kNoExpert;
  };
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    const uint4 v = make_uint4(k[j][0], k[j][1], k[j][2], k[j][3]);
    own[j] = v;
    top_of(v, qk[j], qi[j]);
    qi[j] += 4 * (lane + L * j);
  }
  best();
  uint32_t my_k = 0;
  int my_e = 0;
#pragma unroll 1
  for (int i = 0; i < r.top_k; ++i) {
    const uint32_t top = seg_max<L>(lk);
    const int win = (int)seg_min<L>(lk == top ? (uint32_t)li : 0x7fffffffu);
    if (li == win && win != kNoExpert) {
      const int j0 = (win >> 2) / L;
      reinterpret_cast<uint32_t*>(own)[4 * j0 + (win & 3)] = 0u;
      uint32_t k1;
      int i1;
      top_of(own[j0], k1, i1);
      i1 += win & ~3;
#pragma unroll
      for (int j = 0; j < NQ; ++j)
        if (j == j0) {
          qk[j] = k1;
          qi[j] = i1;
        }
      best();
    }
    if (lane == i) {
      my_k = top;
      my_e = win == kNoExpert ? 0 : expert(win);
    }
  }
  const bool mine = lane < r.top_k;
  bool valid = mine && my_k > 1;
  // the picks' own logits: with a bias the key does not give them
  float my_l = -INFINITY, my_b = 0.0f;
  if (BIAS) {
    if (valid) {
      my_l = logit_at(a, row, my_e);
      my_b = a.bias[my_e];
    }
  } else if (valid) {
    my_l = KT::value(my_k);
  }

  if (BIAS) {
    const float v = valid ? KT::value(my_k) : 0.0f;
    const float vn = __shfl_down_sync(0xffffffffu, v, 1, L);
    const float ln = __shfl_down_sync(0xffffffffu, my_l, 1, L);
    const float bn = __shfl_down_sync(0xffffffffu, my_b, 1, L);
    const bool next_valid = __shfl_down_sync(0xffffffffu, (int)valid, 1, L) && lane < L - 1;
    const float tol = 2.0f * tol_s + 1.8e-7f * fabsf(v);
    bool doubt = valid && next_valid && !(v - vn > tol) && !(my_l == ln && my_b == bn);
    const int last = r.top_k - 1;
    const bool lv = __shfl_sync(0xffffffffu, (int)valid, last, L);
    const float border = __shfl_sync(0xffffffffu, v - tol, last, L);
    const float l_last = __shfl_sync(0xffffffffu, my_l, last, L);
    const float b_last = __shfl_sync(0xffffffffu, my_b, last, L);
    uint32_t near = 0;  // bit 4 j + c: an expert left that comes near the last pick
    if (lv && lk > 1 && !(KT::value(lk) < border)) {
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t left = reinterpret_cast<const uint32_t*>(own)[4 * j + c];
          if (left > 1 && !(KT::value(left) < border)) {
            near |= 1u << (4 * j + c);
            if (!(l[j][c] == l_last && b[j][c] == b_last)) doubt = true;
          }
        }
    }
    if (seg_ballot<L>(doubt)) {
      if (L < 32) {
        sure = false;
      } else if (__all_sync(0xffffffffu, sure)) {
        // candidates: the picks, and what comes near; one per lane
        const int count = __popc(near);
        int at = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int p = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += p;
        }
        const int n = r.top_k + __shfl_sync(0xffffffffu, at, 31);
        at += r.top_k - count;
        if (n > 32) {
          sure = false;
        } else {
          auto put = [&](int p, int e, float lg, float bi) {
            slots[p] = (uint32_t)e;
            slots[32 + p] = __float_as_uint(lg);
            slots[64 + p] = __float_as_uint(bi);
          };
          if (mine) put(lane, my_e, my_l, my_b);
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (near & (1u << (4 * j + c)))
                put(at++, expert(4 * (lane + L * j) + c), l[j][c], b[j][c]);
          double z = 1.0;
          if (softmax) {
            z = 0.0;
#pragma unroll 1
            for (int j = 0; j < NQ; ++j) {
              // (registers are not indexed: the row is read again)
              int n;
              const int e0 = quad(lane + L * j, n);
              for (int c = 0; c < 4; ++c) {
                const float le = c < n ? logit_at(a, row, e0 + c) : -INFINITY;
                if (!is_out(le)) z += numerator<double>(r, le, mx);
              }
            }
            z = warp_sum_t(z);
          }
          __syncwarp();
          const bool cand = lane < n;
          const int e = cand ? (int)slots[lane] : 0;
          const float le = cand ? __uint_as_float(slots[32 + lane]) : -INFINITY;
          const double v64 = is_out(le) ? -INFINITY
                                        : numerator<double>(r, le, mx) / z +
                                              (double)__uint_as_float(slots[64 + lane]);
          // (an expert that is out comes after one whose bias is -infinity)
          const int order = is_out(le) ? e + kMaxE : e;
          int rank = 0;
          for (int p = 0; p < n; ++p) {
            const double vp = __shfl_sync(0xffffffffu, v64, p);
            const int op = __shfl_sync(0xffffffffu, order, p);
            rank += (vp > v64 || (vp == v64 && op < order)) ? 1 : 0;
          }
          __syncwarp();
          if (cand) {
            slots[rank] = (uint32_t)e;
            slots[32 + rank] = __float_as_uint(le);
          }
          __syncwarp();
          if (mine) {
            my_e = (int)slots[lane];
            my_l = __uint_as_float(slots[32 + lane]);
            valid = !is_out(my_l);
          }
        }
      }
    }
  }

  const float p = valid ? numerator<float>(r, my_l, mx) : 0.0f;
  float denom = sum;
  if (r.renorm) denom = seg_sum<L>(p);
  const bool some = seg_ballot<L>(valid) != 0;
  if (r.renorm && some && denom < 1e-30f) sure = false;
  if (seg_ballot<L>(!sure)) return false;
  if (mine && store) {
    const int64_t at = (int64_t)m * r.top_k + lane;
    a.idx[at] = my_e;
    a.w[at] = denom > 0.0f ? p / denom * r.routed_scale : 0.0f;
  }
  return true;
}

__device__ __noinline__ void route_row64(const RouteArgs& a, int m, uint64_t* mine, float* raw) {
  __syncwarp();
  route_row<double>(a, m, reinterpret_cast<unsigned long long*>(mine), raw);
}

// A warp's slots: 4 nq keys of 8 bytes, then 4 nq logits.
__device__ __forceinline__ uint64_t* warp_slots(const RouteArgs& a, float*& raw) {
  extern __shared__ uint64_t slots[];
  const int nq = (a.r.n_experts + 3) >> 2;
  uint64_t* mine = slots + (size_t)(threadIdx.x >> 5) * a.slot;
  raw = reinterpret_cast<float*>(mine + 4 * nq);
  return mine;
}

// The rows a warp's segments could not settle, with all its lanes.
template <int NQ, int GROUPS, bool BIAS>
__device__ __noinline__ void route_again(const RouteArgs& a, int m, uint64_t* mine, float* raw) {
  if (!route_regs<32, NQ, GROUPS, BIAS>(a, m, true, reinterpret_cast<uint32_t*>(mine)))
    route_row64(a, m, mine, raw);
}

template <int L, int NQ, int GROUPS, bool BIAS>
__global__ void __launch_bounds__(256) k_route_regs(const __grid_constant__ RouteArgs a) {
  // (the next kernel's CTAs are not let in early: routing 16,068 rows again they
  // filled the SMs unevenly, 11.2 -> 13.1 us)
  tc::grid_dep_wait();
  constexpr int ROWS = 32 / L;
  const int lane = threadIdx.x & 31;
  const int64_t m0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * ROWS;
  if (m0 >= a.M) return;
  float* raw;
  uint64_t* mine = warp_slots(a, raw);
  const bool in = m0 + lane / L < a.M;
  const int m = in ? (int)m0 + lane / L : a.M - 1;
  const bool settled =
      route_regs<L, NQ, GROUPS, BIAS>(a, m, in, reinterpret_cast<uint32_t*>(mine));
  uint32_t left = __ballot_sync(0xffffffffu, !settled && in && lane % L == 0);
  if (L == 32) {
    if (left) route_row64(a, (int)m0, mine, raw);
    return;
  }
  constexpr int NQ32 = NQ * L / 32 > 0 ? NQ * L / 32 : 1;
  for (; left; left &= left - 1)
    route_again<NQ32, GROUPS, BIAS>(a, (int)m0 + (__ffs(left) - 1) / L, mine, raw);
}

// Any number of experts and groups of any size.
__global__ void __launch_bounds__(256) k_route_any(const __grid_constant__ RouteArgs a) {
  tc::grid_dep_wait();
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.M) return;
  const int m = (int)row;
  float* raw;
  uint64_t* mine = warp_slots(a, raw);
  if (!route_row<float>(a, m, reinterpret_cast<uint32_t*>(mine), raw)) route_row64(a, m, mine, raw);
}

template <int L, int NQ, int GROUPS>
cudaError_t run_regs(const RouteArgs& a, int blocks, int threads, size_t smem, cudaStream_t st) {
  auto* kernel = a.bias ? k_route_regs<L, NQ, GROUPS, true> : k_route_regs<L, NQ, GROUPS, false>;
  return launch_after(kernel, dim3(blocks), threads, smem, st, a);
}
template <int L, int NQ>
cudaError_t run_regs(const RouteArgs& a, int groups, int blocks, int threads, size_t smem,
                     cudaStream_t st) {
  if (groups == 0) return run_regs<L, NQ, 0>(a, blocks, threads, smem, st);
  if (groups == 1) return run_regs<L, NQ, 1>(a, blocks, threads, smem, st);
  return run_regs<L, NQ, 2>(a, blocks, threads, smem, st);
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
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // 1: groups that are a power of two of whole quads; 2: others, padded to that
  const int gs = r.n_experts / r.n_groups;
  int gq = 1;
  while (gq * 4 < gs) gq *= 2;
  const int groups = r.topk_groups == r.n_groups ? 0 : gs == 4 * gq ? 1 : 2;
  const int quads = (r.n_experts + 3) / 4, nq = groups == 2 ? r.n_groups * gq : quads;
  a.group_quads = gq;
  a.group_size = gs;
  const bool regs = nq <= 128 && !(groups && gq > 32);
  // Many rows of at most 128 (256) experts: four (two) rows share a warp, a
  // lane holds four quads; the picks sit one per lane.
  int lanes = 32;
  if (regs && M > sms * 16) {
    if (nq <= 32 && r.top_k <= 8 && !(groups && (gq > 8 || r.n_groups > 8))) lanes = 8;
    else if (nq <= 64 && r.top_k <= 16 && !(groups && (gq > 16 || r.n_groups > 16))) lanes = 16;
  }
  const int64_t rows = ((int64_t)M + 32 / lanes - 1) / (32 / lanes);  // warps
  // 48 bytes per quad of experts and warp (48 KB hold one row of 4096); in
  // registers 384 for a row's candidates and 64 per lane for its keys
  const size_t slot = regs && quads < 51 ? 384 + 32 * 64 : (size_t)quads * 48;
  a.slot = (int)(slot / 8);
  // few rows: spread over the SMs first
  int warps = (int)(rows > 8 * (int64_t)sms ? 8 : (rows + sms - 1) / sms);
  while (warps > 1 && warps * slot > 48 * 1024) --warps;
  const int blocks = (int)((rows + warps - 1) / warps), threads = warps * 32;
  const size_t smem = warps * slot;
  if (!regs) return launch_after(k_route_any, dim3(blocks), threads, smem, st, a);
  if (lanes == 8) return run_regs<8, 4>(a, groups, blocks, threads, smem, st);
  if (lanes == 16) return run_regs<16, 4>(a, groups, blocks, threads, smem, st);
  if (nq <= 32) return run_regs<32, 1>(a, groups, blocks, threads, smem, st);
  if (nq <= 64) return run_regs<32, 2>(a, groups, blocks, threads, smem, st);
  return run_regs<32, 4>(a, groups, blocks, threads, smem, st);
}

}  // namespace moeq
