// RMS norm of r = x + residual with the new residual stream, a bf16 output
// and an 8-bit output with scales, in one pass over the row.
//
// A CTA holds a row in registers (8-element vectors, 16-byte accesses; rows of
// other lengths and alignments one by one, neighbours across a warp: 848 x 4959
// 22.3 -> 12.5 us against eight neighbours per lane), so x and the residual are
// read once and each output is written once.  Few rows
// are bound by the trip to memory and the block reduction (1 x 4096: 3.1 us),
// many by HBM (16,068 x 4096, fp32 streams, e4m3 by 128: 124 us, the copy
// rate) or, on bf16 streams, nearly so (94 us, 4.9 TB/s, 75 % of it; the rest
// is instruction issue: taking the codes twice is 14 us of it).
//
// The codes do not depend on the norm's factor: with t = r gamma and
// a = max |t| over the row (or 128 columns), n / scale = t top / a, top = 127
// or 448.  They are the exact ones: they are taken in fp32 with the factor
// moved by its error bound either way, and where the two differ (about one
// value in 10^5) from fp64, where r gamma (24 + 8 bits) is exact.  Rows and groups
// whose products or squares leave fp32's range are done again (redo); half of the
// rows zero, 16,068 x 4096 bf16, cost 112 us.
#include <cuda_fp8.h>

#include "common.cuh"
#include "ops.h"
#include "tc.cuh"

namespace moeq {
namespace {

constexpr int kQGroup = 128;

struct NormArgs {
  moeq_norm_args n;
  int H, vecs;   // vecs: eights of a row's columns, the last one partial when H % 8
  int n_scales;  // scales per row
  float per_column;  // 1 / H
};

// Eight values of a row, in whole aligned vectors (n is 8 or 0), or (ANY) one by
// one, 32 apart, so that a warp's accesses are neighbours at any alignment: those
// below n, counted from the first.
template <bool ANY>
__device__ __forceinline__ void load8(const void* p, int type, int64_t at, int n, float (&v)[8]) {
  if (ANY) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = 32 * i >= n ? 0.0f
             : type == MOEQ_F32
                 ? reinterpret_cast<const float*>(p)[at + 32 * i]
                 : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[at + 32 * i]);
    return;
  }
  if (n <= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  } else if (type == MOEQ_F32) {
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
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool ANY>
__device__ __forceinline__ void store8(void* p, int type, int64_t at, int n, const float (&v)[8]) {
  if (ANY) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) {
        if (type == MOEQ_F32) reinterpret_cast<float*>(p)[at + 32 * i] = v[i];
        else reinterpret_cast<__nv_bfloat16*>(p)[at + 32 * i] = __float2bfloat16_rn(v[i]);
      }
  } else if (n > 0) {
    if (type == MOEQ_F32) {
      float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) =
          make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7]));
    }
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

// Code of one value t = r gamma (exact in fp64).
__device__ __forceinline__ uint32_t code64(bool i8, double t, double a) {
  if (t == 0.0) return 0u;
  const double v = t * (i8 ? 127.0 : 448.0) / a;
  if (i8) return (uint32_t)(int)rint(fmin(fmax(v, -127.0), 127.0)) & 255u;
  int e = (int)((__double_as_longlong(v) >> 52) & 2047) - 1023;
  if (e < -6) e = -6;
  const double step = __longlong_as_double((long long)(e - 3 + 1023) << 52);
  const float q = (float)(rint(v / step) * step);  // an e4m3 value: the conversion is exact
  return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// gamma's eight values from their bf16 pairs.
__device__ __forceinline__ void unpack8(const uint4& w, float (&g)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[2 * i] = __uint_as_float(u[i] << 16);
    g[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// `code` with the bytes that differ from `other` decided in fp64; a: the exact
// largest |r gamma|, of the first and the last four.  (Out of line: it is seldom
// called.)
__device__ __forceinline__ uint2 settle(bool i8, uint2 code, uint2 other, const float (&r)[8],
                                        const uint4& gp, const double (&a)[2]) {
  float g[8];
  unpack8(gp, g);
  uint32_t out[2] = {code.x, code.y};
  const uint32_t diff[2] = {code.x ^ other.x, code.y ^ other.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int sh = 8 * (j & 3);
    if ((diff[j / 4] >> sh) & 255u)
      out[j / 4] = (out[j / 4] & ~(255u << sh)) | code64(i8, (double)r[j] * (double)g[j], a[j / 4]) << sh;
  }
  return make_uint2(out[0], out[1]);
}
__device__ __noinline__ uint2 settle_one(bool i8, uint2 code, uint2 other, float r0, float r1,
                                         float r2, float r3, float r4, float r5, float r6,
                                         float r7, uint4 gp, double a) {
  return settle(i8, code, other, {r0, r1, r2, r3, r4, r5, r6, r7}, gp, {a, a});
}
__device__ __noinline__ uint2 settle_two(bool i8, uint2 code, uint2 other, float r0, float r1,
                                         float r2, float r3, float r4, float r5, float r6,
                                         float r7, uint4 gp, double a0, double a1) {
  return settle(i8, code, other, {r0, r1, r2, r3, r4, r5, r6, r7}, gp, {a0, a1});
}

// fp32 cannot hold top / a below the first (and r gamma may have lost bits); above
// the second the fast division gives 0, and products may have overflowed.  Rows and
// groups whose largest |r gamma| lies outside of them (zeros, infinities and NaN
// among them) are done again in fp64 (redo).
constexpr float kTinyMax = 1e-24f, kHugeMax = 4.2535296e37f;  // (2^125)
__device__ __forceinline__ bool is_odd(float a) { return !(a >= kTinyMax && a <= kHugeMax); }

// Eight codes of t f in fp32 (f0 for the first four).
__device__ __forceinline__ uint2 codes8(bool i8, const float (&t)[8], float f0, float f1) {
  uint32_t out[2];
  if (i8) {
    // t f + 1.5 2^23 rounds t f to the nearest whole number, in the low bits
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(__fmaf_rn(t[j], j < 4 ? f0 : f1, 12582912.0f));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      out[h] = __byte_perm(__byte_perm(q[4 * h], q[4 * h + 1], 0x0040u),
                           __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0040u), 0x5410u);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = h ? f1 : f0;
      asm("{\n\t.reg .b16 a, b;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b};\n\t}"
          : "=r"(out[h])
          : "f"(t[4 * h] * f), "f"(t[4 * h + 1] * f), "f"(t[4 * h + 2] * f),
            "f"(t[4 * h + 3] * f));
    }
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Largest |r gamma| of a thread's values from FIRST to LAST as a key (see mag_key).
template <int FIRST, int LAST>
__device__ __forceinline__ unsigned long long max_key(const float (&r)[8], const float (&g)[8]) {
  unsigned long long key = 0;
#pragma unroll
  for (int j = FIRST; j <= LAST; ++j) {
    const unsigned long long k = mag_key(r[j], g[j]);
    key = k > key ? k : key;
  }
  return key;
}

template <int FIRST>
__device__ __forceinline__ unsigned long long lanes_max(unsigned long long k) {
#pragma unroll
  for (int o = FIRST; o > 0; o >>= 1) {
    const unsigned long long p = __shfl_xor_sync(0xffffffffu, k, o);
    k = p > k ? p : k;
  }
  return k;
}
template <int FIRST>
__device__ __forceinline__ float lanes_max(float k) {
#pragma unroll
  for (int o = FIRST; o > 0; o >>= 1) k = max_nan(k, __shfl_xor_sync(0xffffffffu, k, o));
  return k;
}

// NV: vectors of a thread.  XT, RT: moeq_dtype of x and of the residual (RT
// kNone: there is none), for rows of whole, aligned vectors; kAny: any.
// MAXT: threads of the largest block.
constexpr int kAny = -1, kNone = -2;

// What fp32's range does not hold, done again: r is read from where it was written,
// or added up again.  Rows whose squares overflow (inv not above 0) are norm'd with
// the squares of r 2^-80.  Then the 8-bit output of the warp's columns, everything
// from fp64, which holds every product.  For such a row, and for rows with one
// scale, all threads of the block are here.
template <bool ANY>
__device__ __noinline__ void redo(const NormArgs& a, int nv, float inv, float* red,
                                  unsigned long long* red_key) {
  const moeq_norm_args& n = a.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int64_t m = blockIdx.x;
  const bool whole = n.q_group == 0, i8 = n.q_type == MOEQ_I8;
  // first column of vector i (see k_add_rmsnorm), its stream, its products, and their
  // largest from `first` to `last` as an ordered integer, NaN above all
  auto column = [&](int i) {
    return ANY ? 256 * (warp + i * nw) + lane : 256 * (warp * nv + i) + 8 * lane;
  };
  auto stream = [&](int i, float (&r)[8]) {
    const int c0 = column(i), cnt = a.H - c0;
    if (n.r_out) {
      load8<ANY>(n.r_out, n.r_type, m * n.r_out_stride + c0, cnt, r);
    } else {
      load8<ANY>(n.x, n.x_type, m * n.x_stride + c0, cnt, r);
      if (n.residual) {
        float s[8];
        load8<ANY>(n.residual, n.r_type, m * n.r_stride + c0, cnt, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] += s[j];
          if (n.r_type == MOEQ_BF16) r[j] = __bfloat162float(__float2bfloat16_rn(r[j]));
        }
      }
    }
  };
  auto products = [&](int i, double (&t)[8]) {
    float r[8], g[8];
    stream(i, r);
    load8<ANY>(n.gamma, MOEQ_BF16, column(i), a.H - column(i), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = (double)r[j] * (double)g[j];
  };
  auto largest = [](const double (&t)[8], int first, int last) {
    unsigned long long key = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned long long k = (unsigned long long)__double_as_longlong(fabs(t[j]));
      if (j >= first && j <= last && k > key) key = k;
    }
    return key;
  };
  if (!(inv > 0.0f)) {
    const float down = 8.27180613e-25f;  // 2^-80
    // (in k_add_rmsnorm's order, for one vector a thread and for two)
    const int sums = nv == 2 ? 2 * nw : nw;
    float part = 0.0f;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < nv; ++i) {
      float r[8], sum = 0.0f;
      stream(i, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __fmaf_rn(r[j] * down, r[j] * down, sum);
      part = warp_sum(sum) + (nv > 2 ? part : 0.0f);
      if (lane == 0) red[nv > 2 ? warp : ANY ? warp + i * nw : warp * nv + i] = part;
    }
    if (tid == 1)
      for (int i = sums; i & 3; ++i) red[i] = 0.0f;
    __syncthreads();
    float ss = 0.0f;
    for (int i = 0; i < sums; i += 4) ss += (red[i] + red[i + 1]) + (red[i + 2] + red[i + 3]);
    inv = rsqrtf(__fmaf_rn(ss, a.per_column, n.eps * down * down)) * down;
#pragma unroll 1
    for (int i = 0; n.y && i < nv; ++i) {
      const int c0 = column(i), cnt = a.H - c0;
      float r[8], g[8];
      stream(i, r);
      load8<ANY>(n.gamma, MOEQ_BF16, c0, cnt, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = r[j] * inv * g[j];
      store8<ANY>(n.y, MOEQ_BF16, m * n.y_stride + c0, cnt, g);
    }
  }
  if (!n.q) return;
  const double to_scale = (double)inv / (i8 ? 127.0 : 448.0);
  double t[8];
  unsigned long long row = 0;
  if (whole) {
#pragma unroll 1
    for (int i = 0; i < nv; ++i) {
      products(i, t);
      const unsigned long long k = largest(t, 0, 7);
      row = k > row ? k : row;
    }
    row = lanes_max<16>(row);
    __syncthreads();
    if (lane == 0) red_key[warp] = row;
    __syncthreads();
    for (int i = 0; i < nw; ++i) row = red_key[i] > row ? red_key[i] : row;
    if (row == 0) return;  // zeros: scale and codes are there
  }
#pragma unroll 1
  for (int i = 0; i < nv; ++i) {
    products(i, t);
    const int c0 = column(i), cnt = a.H - c0;
    unsigned long long key[2] = {row, row};  // of the first and the last four
    if (!whole) {
      key[0] = lanes_max<ANY ? 16 : 8>(largest(t, 0, ANY ? 3 : 7));
      key[1] = ANY ? lanes_max<16>(largest(t, 4, 7)) : key[0];
      if (__all_sync(0xffffffffu, (key[0] | key[1]) == 0)) continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const double top = __longlong_as_double((long long)key[h]);
      const bool finite = top < INFINITY;
      const float scale = finite ? (float)(top * to_scale) : __uint_as_float(0x7FC00000u);
      const int c = ANY ? c0 + 128 * h : c0;  // first of the four, in the row
      if (whole ? i + h + tid == 0 : (c & 127) == 0 && c < a.H && (ANY || h == 0))
        n.q_scales[m * a.n_scales + (whole ? 0 : c >> 7)] = scale;
#pragma unroll
      for (int j = 4 * h; j < 4 * h + 4; ++j) {
        const int at = ANY ? 32 * j : j;
        if (at < cnt)
          reinterpret_cast<uint8_t*>(n.q)[m * n.q_stride + c0 + at] =
              (uint8_t)(finite ? code64(i8, t[j], top) : 0u);
      }
    }
  }
}

// FULL: every thread has NV whole vectors.
template <int NV, int XT, int RT, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT) k_add_rmsnorm(const __grid_constant__ NormArgs a) {
  tc::grid_dep_wait();
  constexpr bool ANY = XT == kAny;
  __shared__ __align__(16) float red[32], red_max[32];
  __shared__ unsigned long long red_key[32];
  const moeq_norm_args& n = a.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int64_t m = blockIdx.x;
  const int xt = ANY ? n.x_type : XT, rt = ANY ? n.r_type : RT;
  const bool res = ANY ? n.residual != nullptr : RT != kNone;
  // r gamma of a bf16 stream (8 + 8 bits) is exact in fp32
  const bool exact = (res ? rt : xt) == MOEQ_BF16;
  const bool whole = n.q && n.q_group == 0, i8 = n.q_type == MOEQ_I8;
  // first column of a thread's vector i, and how many columns it has from there
  auto column = [&](int i) -> int {
    return ANY ? 256 * (warp + i * nw) + lane : 256 * (warp * NV + i) + 8 * lane;
  };
  auto count = [&](int i) -> int { return FULL ? 8 : a.H - column(i); };
  float r[NV][8];
  uint4 gp[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    load8<ANY>(n.x, xt, m * n.x_stride + column(i), count(i), r[i]);
  float s[NV][8];
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      load8<ANY>(n.residual, rt, m * n.r_stride + column(i), count(i), s[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    gp[i] = make_uint4(0u, 0u, 0u, 0u);
    if (ANY) {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = 32 * j < count(i) ? n.gamma[column(i) + 32 * j] : 0u;
      gp[i] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                         h[6] | h[7] << 16);
    } else if (count(i) > 0) {
      gp[i] = *reinterpret_cast<const uint4*>(n.gamma + column(i));
    }
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] += s[i][j];
      // the norm is of the stream as it is stored
      if (rt == MOEQ_BF16) {
        const uint4 p = make_uint4(bf16_pair(r[i][0], r[i][1]), bf16_pair(r[i][2], r[i][3]),
                                   bf16_pair(r[i][4], r[i][5]), bf16_pair(r[i][6], r[i][7]));
        unpack8(p, r[i]);
        if (!ANY) {
          if (n.r_out && count(i) > 0)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(n.r_out) + m * n.r_out_stride +
                                      column(i)) = p;
          continue;
        }
      }
      if (n.r_out) store8<ANY>(n.r_out, rt, m * n.r_out_stride + column(i), count(i), r[i]);
    }
  }
  // The squares are added up over 32 neighbouring vectors, then over those in pairs,
  // then over two pairs: the same whether a thread has one vector or two, so that a
  // row's norm does not change with the batch (see run).
  constexpr bool TWO = NV == 2;
  float ss = 0.0f, ss2 = 0.0f, row_max = 0.0f;
  unsigned long long row_key = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float& sum = TWO && i == 1 ? ss2 : ss;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __fmaf_rn(r[i][j], r[i][j], sum);
    if (whole) {
      float g[8];
      unpack8(gp[i], g);
      if (exact) {
#pragma unroll
        for (int j = 0; j < 8; ++j) row_max = max_nan(row_max, fabsf(r[i][j] * g[j]));
      } else {
        const unsigned long long k = max_key<0, 7>(r[i], g);
        row_key = k > row_key ? k : row_key;
      }
    }
  }
  if (TWO) {  // lanes below 16 add the first up, the others the second
    const float mine = lane & 16 ? ss2 : ss, other = lane & 16 ? ss : ss2;
    ss = mine + __shfl_xor_sync(0xffffffffu, other, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // the pair (ANY: another warp has the second's neighbour)
    if (!ANY || nw == 1) ss += __shfl_xor_sync(0xffffffffu, ss, 16);
  } else {
    ss = warp_sum(ss);
  }
  if (whole) {
    if (exact) row_max = lanes_max<16>(row_max);
    else row_key = lanes_max<16>(row_key);
  }
  if (nw > 1) {
    const int sums = TWO && ANY ? 2 * nw : nw;
    if (TWO && ANY && lane == 16) red[warp + nw] = ss;
    if (lane == 0) {
      red[warp] = ss;
      red_max[warp] = row_max;
      red_key[warp] = row_key;
    } else if (tid == 1) {  // (up to the next four)
      for (int i = sums; i & 3; ++i) red[i] = 0.0f;
      for (int i = nw; i & 3; ++i) red_max[i] = 0.0f;
    }
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < sums; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(red + i);
      if (TWO && !ANY) {
        ss += v.x + v.y;
        ss += v.z + v.w;
      } else {
        ss += (v.x + v.y) + (v.z + v.w);
      }
    }
    if (whole) {
      if (exact) {
        for (int i = 0; i < nw; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(red_max + i);
          row_max = max_nan(row_max, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
        }
      } else {
        for (int i = 0; i < nw; ++i) row_key = red_key[i] > row_key ? red_key[i] : row_key;
      }
    }
  }
  if (whole && !exact) row_max = __uint_as_float((uint32_t)(row_key >> 32));
  const float inv = rsqrtf(__fmaf_rn(ss, a.per_column, n.eps));
  const float top = i8 ? 127.0f : 448.0f, to_scale = inv * (i8 ? 1.0f / 127.0f : 1.0f / 448.0f);

  bool odd = whole && is_odd(row_max);  // (whole: there is an 8-bit output)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = column(i), cnt = count(i);
    float g[8];
    unpack8(gp[i], g);
    if (n.y) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r[i][j] * inv * g[j];
      store8<ANY>(n.y, MOEQ_BF16, m * n.y_stride + c0, cnt, o);
    }
    if (!n.q) continue;
    // The largest of the row, or of 128 columns: 16 neighbouring lanes hold them,
    // or (ANY) the warp its first and its last four values.
    float t[8], a0 = row_max;
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = r[i][j] * g[j];
    float a1 = a0;
    if (!whole) {
      a0 = a1 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (ANY && j >= 4) a1 = max_nan(a1, fabsf(t[j]));
        else a0 = max_nan(a0, fabsf(t[j]));
      }
      a0 = lanes_max<ANY ? 16 : 8>(a0);
      a1 = ANY ? lanes_max<16>(a1) : a0;
      odd |= cnt > 0 && (is_odd(a0) || (ANY && cnt > 128 && is_odd(a1)));
    }
    // t f is off by three roundings and the division's 2 ulp (2^-21 relative);
    // where moving it by 2^-20 either way changes a code, fp64 decides
    const float up = 1.0f + 9.5367431640625e-7f, down = 1.0f - 9.5367431640625e-7f;
    // (plus 2^-115, which only a tiny largest feels: the codes of zeros are zeros)
    const float least = 2.40741243e-35f;
    const float f0 = __fdividef(top, a0 + least), f1 = ANY ? __fdividef(top, a1 + least) : f0;
    uint2 code = codes8(i8, t, f0 * up, f1 * up);
    const uint2 other = codes8(i8, t, f0 * down, f1 * down);
    const bool doubt = code.x != other.x || code.y != other.y;
    if (ANY) {
      unsigned long long key0 = row_key, key1 = row_key;
      if (!exact && !whole && __any_sync(0xffffffffu, doubt)) {
        key0 = lanes_max<16>(max_key<0, 3>(r[i], g));
        key1 = lanes_max<16>(max_key<4, 7>(r[i], g));
      }
      if (doubt)
        code = settle_two(i8, code, other, r[i][0], r[i][1], r[i][2], r[i][3], r[i][4], r[i][5],
                          r[i][6], r[i][7], gp[i], exact ? (double)a0 : mag_value(key0),
                          exact ? (double)a1 : mag_value(key1));
    } else {
      unsigned long long key = row_key;
      if (!exact && !whole && __any_sync(0xffffffffu, doubt))
        key = lanes_max<8>(max_key<0, 7>(r[i], g));
      if (doubt)
        code = settle_one(i8, code, other, r[i][0], r[i][1], r[i][2], r[i][3], r[i][4], r[i][5],
                          r[i][6], r[i][7], gp[i], exact ? (double)a0 : mag_value(key));
    }
    float* scale = n.q_scales + m * a.n_scales;
    if (whole) {
      if (i == 0 && tid == 0) scale[0] = a0 * to_scale;
    } else if (ANY) {
      if (lane == 0 && cnt > 0) scale[c0 >> 7] = a0 * to_scale;
      if (lane == 0 && cnt > 128) scale[(c0 >> 7) + 1] = a1 * to_scale;
    } else if ((c0 & 127) == 0 && cnt > 0) {
      scale[c0 >> 7] = a0 * to_scale;
    }
    uint8_t* q = reinterpret_cast<uint8_t*>(n.q) + m * n.q_stride + c0;
    if (ANY) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (32 * j < cnt) q[32 * j] = (uint8_t)((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
    } else if (cnt > 0) {
      *reinterpret_cast<uint2*>(q) = code;
    }
  }
  // (inv is the same in all threads, a row odd in all or none, a group in all its lanes)
  if (__any_sync(0xffffffffu, odd || !(inv > 0.0f))) redo<ANY>(a, NV, inv, red, red_key);
}

template <int NV, int XT, int RT, int MAXT>
cudaError_t run_sized(const NormArgs& a, int M, int warps, cudaStream_t st) {
  if (XT != kAny && a.vecs == warps * 32 * NV)
    return launch_after(k_add_rmsnorm<NV, XT, RT, XT != kAny, MAXT>, dim3(M), warps * 32, 0, st, a);
  return launch_after(k_add_rmsnorm<NV, XT, RT, false, MAXT>, dim3(M), warps * 32, 0, st, a);
}

template <int XT, int RT>
cudaError_t run(const NormArgs& a, int M, int sms, cudaStream_t st) {
  const int warps = (a.vecs + 31) / 32;
  // Many rows: two vectors a thread, so that the reductions and addresses are
  // paid less often; few rows: as many threads as vectors, for the latency.
  if (warps <= 16 && M < 4 * sms) return run_sized<1, XT, RT, 512>(a, M, warps, st);
  if (warps <= 32) return run_sized<2, XT, RT, 512>(a, M, (warps + 1) / 2, st);
  return run_sized<4, XT, RT, 1024>(a, M, (warps + 3) / 4, st);
}

bool wide(const void* p, int64_t stride, int item, int bytes) {
  return ((uintptr_t)p % bytes) == 0 && ((stride * item) % bytes) == 0;
}
int size_of(int type) { return type == MOEQ_F32 ? 4 : type == MOEQ_BF16 ? 2 : 1; }

}  // namespace

cudaError_t launch_add_rmsnorm(const moeq_norm_args& n, int M, int H, cudaStream_t st) {
  NormArgs a;
  a.n = n;
  a.H = H;
  a.per_column = 1.0f / (float)H;
  a.vecs = (H + 7) / 8;
  a.n_scales = n.q_group ? (H + kQGroup - 1) / kQGroup : 1;
  const int sms = sm_count();
  const bool vec = H % 8 == 0 && wide(n.x, n.x_stride, size_of(n.x_type), 16) &&
                   wide(n.gamma, 0, 2, 16) &&
                   (!n.residual || wide(n.residual, n.r_stride, size_of(n.r_type), 16)) &&
                   (!n.r_out || wide(n.r_out, n.r_out_stride, size_of(n.r_type), 16)) &&
                   (!n.y || wide(n.y, n.y_stride, 2, 16)) && (!n.q || wide(n.q, n.q_stride, 1, 8));
  const bool xb = n.x_type == MOEQ_BF16, rb = n.r_type == MOEQ_BF16;
  if (!vec) return run<kAny, kAny>(a, M, sms, st);
  if (!n.residual && xb) return run<MOEQ_BF16, kNone>(a, M, sms, st);
  if (!n.residual) return run<MOEQ_F32, kNone>(a, M, sms, st);
  if (xb && rb) return run<MOEQ_BF16, MOEQ_BF16>(a, M, sms, st);
  if (xb) return run<MOEQ_BF16, MOEQ_F32>(a, M, sms, st);
  if (rb) return run<MOEQ_F32, MOEQ_BF16>(a, M, sms, st);
  return run<MOEQ_F32, MOEQ_F32>(a, M, sms, st);
}

}  // namespace moeq
