// RMS norm of r = x + residual with the new residual stream, a bf16 output
// and an 8-bit output with scales, in one pass over the row.
//
// A CTA holds a row in registers (8-element vectors, 16-byte accesses), so
// x and the residual are read once and each output is written once: the
// kernel is bound by HBM, and by the two block reductions' latency for few
// rows.
//
// The codes do not depend on the norm's factor: with t = r gamma and
// a = max |t| over the row (or 128 columns), n / scale = t top / a, top = 127
// or 448.  They are the exact ones: r gamma is taken in fp32, and a value
// that comes within fp32's error of a rounding border (about one in 10^4)
// is rounded again from fp64, where r gamma (24 + 8 bits) is exact.
#include <cuda_fp8.h>

#include "common.cuh"
#include "ops.h"

namespace moeq {
namespace {

constexpr int kQGroup = 128;

struct NormArgs {
  moeq_norm_args n;
  int H, vecs;   // vecs: 8-element vectors of a row, the last one partial when H % 8
  int n_scales;  // scales per row
  // 16-byte accesses per operand (8 bytes for q) where pointer and stride allow
  bool vx, vr, vro, vg, vy, vq;
};

__device__ __forceinline__ void load8(const void* p, int type, int64_t at, int n, bool vec,
                                      float (&v)[8]) {
  if (vec && n == 8) {
    if (type == MOEQ_F32) {
      const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
      const float4 a = f[0], b = f[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (n <= 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < n)
      v[i] = type == MOEQ_F32 ? reinterpret_cast<const float*>(p)[at + i]
                              : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[at + i]);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void store8(void* p, int type, int64_t at, int n, bool vec,
                                       const float (&v)[8]) {
  if (vec && n == 8) {
    if (type == MOEQ_F32) {
      float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) =
          make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      if (type == MOEQ_F32) reinterpret_cast<float*>(p)[at + i] = v[i];
      else
        reinterpret_cast<__nv_bfloat16*>(p)[at + i] = __float2bfloat16_rn(v[i]);
    }
}

// Magnitude of t = r gamma exactly, as a key that orders like it: the fp32
// product's bits, then what its rounding left (fma), as an ordered integer.
// A NaN orders above infinity.
__device__ __forceinline__ unsigned long long mag_key(float r, float g) {
  const float t = r * g;
  float rest = __fmaf_rn(r, g, -t);
  rest = t < 0.0f ? -rest : rest;
  uint32_t b = __float_as_uint(rest == 0.0f ? 0.0f : rest);
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)(__float_as_uint(t) & 0x7FFFFFFFu) << 32) | b;
}
__device__ __forceinline__ double mag_value(unsigned long long k) {
  const uint32_t b = (uint32_t)k;
  const float rest = __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
  return (double)__uint_as_float((uint32_t)(k >> 32)) + (double)rest;
}

// Codes of one value from fp64 (the value next to a border, or tiny maxima).
__device__ __noinline__ uint32_t code_i8_64(float r, float g, double a) {
  const double v = (double)r * (double)g * 127.0 / a;
  return (uint32_t)(int)rint(fmin(fmax(v, -127.0), 127.0)) & 255u;
}
__device__ __noinline__ uint32_t code_e4m3_64(float r, float g, double a) {
  const double v = (double)r * (double)g * 448.0 / a;
  int e = (int)((__double_as_longlong(v) >> 52) & 2047) - 1023;
  if (e < -6) e = -6;
  const double step = __longlong_as_double((long long)(e - 3 + 1023) << 52);
  const float q = (float)(rint(v / step) * step);  // an e4m3 value: the conversion is exact
  return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// fp32 cannot hold top / a below this (and r gamma may have lost bits)
constexpr float kTinyMax = 1e-28f;

// The eight codes of a vector from values (r, g) of a group with maximum mk.
__device__ __forceinline__ uint2 codes8(int type, const float (&r)[8], const float (&g)[8],
                                        unsigned long long mk) {
  const float am = __uint_as_float((uint32_t)(mk >> 32));
  if (!(am < INFINITY)) return make_uint2(0u, 0u);
  const bool i8 = type == MOEQ_I8;
  const float f = __fdiv_rn(i8 ? 127.0f : 448.0f, am);
  float c[8];
  bool doubt[8], any = false;
  uint32_t out[2];
  if (i8) {
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = r[j] * g[j] * f;
      const float v = rintf(c[j]);
      q[j] = (uint32_t)__float2int_rn(v);
      // fp32's error of c: 4 roundings, 127 * 4 * 2^-24 < 3.1e-5
      doubt[j] = fabsf(fabsf(c[j] - v) - 0.5f) < 6e-5f;
      any |= doubt[j];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      out[h] = __byte_perm(__byte_perm(q[4 * h], q[4 * h + 1], 0x0040u),
                           __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0040u), 0x5410u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = r[j] * g[j] * f;
      // a border has the fraction bits below e4m3's three at exactly one half;
      // below 2^-6 (subnormal codes) fp64 decides
      const uint32_t low = __float_as_uint(c[j]) & 0xFFFFFu;
      doubt[j] = (low - 0x7FFF0u) <= 0x20u || (fabsf(c[j]) < 0.015625f && c[j] != 0.0f);
      any |= doubt[j];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(c[4 * h], c[4 * h + 1]),
                                                  __NV_SATFINITE, __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(c[4 * h + 2], c[4 * h + 3]),
                                                  __NV_SATFINITE, __NV_E4M3);
      out[h] = a | b << 16;
    }
  }
  const bool tiny = am < kTinyMax;
  if (any || tiny) {
    const double a64 = mag_value(mk);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (doubt[j] || tiny) {
        const uint32_t k = r[j] * g[j] == 0.0f ? 0u
                           : i8                ? code_i8_64(r[j], g[j], a64)
                                               : code_e4m3_64(r[j], g[j], a64);
        out[j / 4] = (out[j / 4] & ~(255u << (8 * (j & 3)))) | k << (8 * (j & 3));
      }
  }
  return make_uint2(out[0], out[1]);
}

// Largest |r gamma| of a thread's eight values as a key (see mag_key).  SHORT:
// r is a bf16, so r gamma is exact in fp32 and nothing is left over.
template <bool SHORT>
__device__ __forceinline__ unsigned long long max8(const float (&r)[8], const float (&g)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    top = max(top, __float_as_uint(r[j] * g[j]) & 0x7FFFFFFFu);  // a NaN is largest
  if (SHORT) return ((unsigned long long)top << 32) | 0x80000000u;
  unsigned long long key = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if ((__float_as_uint(r[j] * g[j]) & 0x7FFFFFFFu) == top) {
      const unsigned long long k = mag_key(r[j], g[j]);
      key = k > key ? k : key;
    }
  return key;
}

template <bool SHORT, int FIRST>
__device__ __forceinline__ unsigned long long max_lanes(unsigned long long k) {
  if (SHORT) {
    uint32_t t = (uint32_t)(k >> 32);
    if (FIRST == 16) {
      t = __reduce_max_sync(0xffffffffu, t);
    } else {
#pragma unroll
      for (int o = FIRST; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
    }
    return ((unsigned long long)t << 32) | 0x80000000u;
  }
#pragma unroll
  for (int o = FIRST; o > 0; o >>= 1) {
    const unsigned long long p = __shfl_xor_sync(0xffffffffu, k, o);
    k = p > k ? p : k;
  }
  return k;
}

// MAXT: threads of the largest block of this variant.
template <int NV, bool SHORT, int MAXT>
__global__ void __launch_bounds__(MAXT) k_add_rmsnorm(const __grid_constant__ NormArgs a) {
  __shared__ float red[32];
  __shared__ unsigned long long red_max[32];
  const moeq_norm_args& n = a.n;
  const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = T >> 5;
  const int64_t m = blockIdx.x;
  const bool whole = n.q && n.q_group == 0;
  float r[NV][8], g[NV][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * T;
    const int cnt = v < a.vecs ? min(8, a.H - 8 * v) : 0;
    load8(n.x, n.x_type, m * n.x_stride + 8 * v, cnt, a.vx, r[i]);
    if (n.residual) {
      float s[8];
      load8(n.residual, n.r_type, m * n.r_stride + 8 * v, cnt, a.vr, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] += s[j];
        // the norm is of the stream as it is stored
        if (n.r_type == MOEQ_BF16) r[i][j] = __bfloat162float(__float2bfloat16_rn(r[i][j]));
      }
    }
    load8(n.gamma, MOEQ_BF16, 8 * v, cnt, a.vg, g[i]);
  }
  unsigned long long row_max = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * T;
    const int cnt = v < a.vecs ? min(8, a.H - 8 * v) : 0;
    if (n.r_out && cnt > 0)
      store8(n.r_out, n.r_type, m * n.r_out_stride + 8 * v, cnt, a.vro, r[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __fmaf_rn(r[i][j], r[i][j], ss);
    if (whole) {
      const unsigned long long k = max8<SHORT>(r[i], g[i]);
      row_max = k > row_max ? k : row_max;
    }
  }
  ss = warp_sum(ss);
  if (whole) row_max = max_lanes<SHORT, 16>(row_max);
  if (lane == 0) {
    red[warp] = ss;
    red_max[warp] = row_max;
  }
  __syncthreads();
  ss = 0.0f;
  for (int i = 0; i < nw; ++i) {
    ss += red[i];
    row_max = red_max[i] > row_max ? red_max[i] : row_max;
  }
  const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)a.H) + n.eps));

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * T;
    const int cnt = v < a.vecs ? min(8, a.H - 8 * v) : 0;
    if (n.y && cnt > 0) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r[i][j] * inv * g[i][j];
      store8(n.y, MOEQ_BF16, m * n.y_stride + 8 * v, cnt, a.vy, o);
    }
    if (n.q) {
      // 16 neighbouring lanes hold 128 columns
      const unsigned long long mk =
          whole ? row_max : max_lanes<SHORT, 8>(max8<SHORT>(r[i], g[i]));
      if (cnt > 0) {
        if (whole ? v == 0 : (v & 15) == 0) {
          const float am = __uint_as_float((uint32_t)(mk >> 32));
          n.q_scales[m * a.n_scales + (whole ? 0 : v >> 4)] =
              am < INFINITY ? __fdiv_rn(am * inv, n.q_type == MOEQ_I8 ? 127.0f : 448.0f)
                            : __uint_as_float(0x7FC00000u);
        }
        const uint2 code = codes8(n.q_type, r[i], g[i], mk);
        uint8_t* q = reinterpret_cast<uint8_t*>(n.q) + m * n.q_stride + 8 * v;
        if (a.vq && cnt == 8) {
          *reinterpret_cast<uint2*>(q) = code;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < cnt) q[j] = (uint8_t)((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
        }
      }
    }
  }
}

template <bool SHORT>
void run(const NormArgs& a, int M, cudaStream_t st) {
  const int warps = (a.vecs + 31) / 32;
  if (warps <= 16) k_add_rmsnorm<1, SHORT, 512><<<M, warps * 32, 0, st>>>(a);
  else if (warps <= 32) k_add_rmsnorm<2, SHORT, 512><<<M, (warps + 1) / 2 * 32, 0, st>>>(a);
  else if (warps <= 64) k_add_rmsnorm<2, SHORT, 1024><<<M, (warps + 1) / 2 * 32, 0, st>>>(a);
  else k_add_rmsnorm<4, SHORT, 1024><<<M, (warps + 3) / 4 * 32, 0, st>>>(a);
}

bool wide(const void* p, int64_t stride, int item, int bytes) {
  return p && ((uintptr_t)p % bytes) == 0 && ((stride * item) % bytes) == 0;
}
int size_of(int type) { return type == MOEQ_F32 ? 4 : type == MOEQ_BF16 ? 2 : 1; }

}  // namespace

cudaError_t launch_add_rmsnorm(const moeq_norm_args& n, int M, int H, cudaStream_t st) {
  NormArgs a;
  a.n = n;
  a.H = H;
  a.vecs = (H + 7) / 8;
  a.n_scales = n.q_group ? (H + kQGroup - 1) / kQGroup : 1;
  a.vx = wide(n.x, n.x_stride, size_of(n.x_type), 16);
  a.vr = wide(n.residual, n.r_stride, size_of(n.r_type), 16);
  a.vro = wide(n.r_out, n.r_out_stride, size_of(n.r_type), 16);
  a.vg = wide(n.gamma, 0, 2, 16);
  a.vy = wide(n.y, n.y_stride, 2, 16);
  a.vq = wide(n.q, n.q_stride, 1, 8);
  // a bf16 stream: r gamma has 16 bits
  if ((n.residual ? n.r_type : n.x_type) == MOEQ_BF16) run<true>(a, M, st);
  else run<false>(a, M, st);
  return cudaGetLastError();
}

}  // namespace moeq
