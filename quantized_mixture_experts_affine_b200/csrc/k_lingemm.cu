// Linear with many tokens: fp16 operands, tcgen05 products.
//
// Three launches.  Two, side by side, lay out the operands (k_lin_rows,
// k_lin_weights): token rows and weight rows as fp16, each row times a power
// of two that brings its largest magnitude to [2^13, 2^14), so that no bf16
// value is out of fp16's range; the powers are undone in the epilogue.  A
// token value of bf16 or 8 bits is exact in fp16 unless it lies 2^-28 below
// its row's largest; a weight is rounded once (relative 2^-11; y rounds by up
// to 2^-8 in bf16), and so is an 8-bit value times its scale where that changes
// along the row.  For an fp32 y the weights keep a second fp16 (22 bits),
// and so do tokens whose scales change along the row; the product is then the
// sum of the parts' products.
//
// The third (k_lin_gemm) is a persistent GEMM on CTA pairs (cta_group::2):
// D (256 rows of W) x (up to 256 tokens) per pair in TMEM, two accumulators,
// operands by TMA in the 128-byte swizzle.  A tile of 256 tokens needs 64
// bytes a clock and SM from L2, about what an SM gets; one of 128 needs 96 and
// ran at two thirds of the rate, so smaller tiles are taken only where they
// fill the waves better (tile_tokens below).  W's rows are D's rows, so a lane of
// the epilogue holds one output column o: bias and row power are one register,
// and a warp's accesses to y, mul and the residual are 32 neighbours at any
// alignment and stride.  The residual is read before the stores that might
// overlap it, 32 values at a time: read one by one it made the kernel 2.5
// times slower.
//
// Measured, 16,068 tokens, 4096 x 4096, 8-bit, bf16 y, residual: layout 36 us
// beside 16 us (16,068 x 4096 tokens are 263 MB), GEMM 342 to 366 us (1.5
// PFLOP/s), the call 416 us; under the power cap of a long loop 484 us.
// 2048 tokens, 2048 x 4096, MX FP4: 37 us, of which the GEMM 24 (144 tiles
// of 240 tokens: two waves of 74 pairs, nearly full).
#include "lingemm.cuh"

namespace moeq {
namespace {

constexpr int kTile = 128;  // rows of W per CTA (256 per pair)

// ------------------------------------------------------------------ operand layout
struct PrepArgs {
  LinArgs l;
  __half* x16;  // [x_parts][M][in_dim]
  float* fx;    // [M]
  __half* w16;  // [w_parts][out_dim][in_dim]
  float* fw;    // [out_dim]
  int x_parts, w_parts;
  int x_blocks;  // (k_lin_tokens) first blocks of the grid: tokens; the others: weights
  // For the product that unpacks the weights itself: rows padded with zeros
  // to x_row columns, eights of columns moved as its threads take them
  // (64 neighbours of 256 go to four blocks of 64), and with x_split each
  // eight in the order 0 4 1 5 2 6 3 7; and the weights' scales.
  int x_row, x_runs, x_split;
  uint32_t* sb;  // [group][out_dim]
};

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values as fp16 at p, and what that rounding left at p + part.
__device__ __forceinline__ void store_halves(__half* p, int64_t part, bool two,
                                             const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = half_pair(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
  if (!two) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    h[i] = half_pair(v[2 * i] - f.x, v[2 * i + 1] - f.y);
  }
  *reinterpret_cast<uint4*>(p + part) = make_uint4(h[0], h[1], h[2], h[3]);
}

__device__ __forceinline__ void load_x8(const void* row, int type, int c0, float (&v)[8]) {
  if (type == MOEQ_BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + c0);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    return;
  }
  const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(row) + c0);
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (type == MOEQ_I8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = (float)(int8_t)(u[i] >> (8 * j));
    } else {
      uint32_t p0, p1;
      e4m3_to_bf16(u[i], p0, p1);
      v[4 * i] = __uint_as_float(p0 << 16);
      v[4 * i + 1] = __uint_as_float(p0 & 0xFFFF0000u);
      v[4 * i + 2] = __uint_as_float(p1 << 16);
      v[4 * i + 3] = __uint_as_float(p1 & 0xFFFF0000u);
    }
  }
}

// Eight codes from column c0 (a multiple of 8) of a packed row, as loaded:
// the 8 * BITS bits of the run in two words.
template <int BITS>
__device__ __forceinline__ uint2 load_run8(const uint32_t* row, int c0) {
  if (BITS == 8) return *reinterpret_cast<const uint2*>(row + c0 / 4);
  if (BITS == 4) return make_uint2(row[c0 / 8], 0u);
  if (BITS == 2) return make_uint2(reinterpret_cast<const uint16_t*>(row)[c0 / 8], 0u);
  // 3, 5, 6 bits: the run starts on a byte and reaches into the next one or
  // two words only where it does not end before them
  const int bit = c0 * BITS, off = bit & 31, n = 8 * BITS;
  const uint32_t* p = row + (bit >> 5);
  const uint32_t a = p[0], b = off + n > 32 ? p[1] : 0u, c = off + n > 64 ? p[2] : 0u;
  return make_uint2(__funnelshift_r(a, b, off), __funnelshift_r(b, c, off));
}

// Their values times s plus b (MX FP4: element values times s).
template <int BITS, bool MX>
__device__ __forceinline__ void run8_values(uint2 w, float s, float b, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int bit = i * BITS;
    uint32_t q;
    if (BITS == 8 || bit + BITS <= 32) q = (bit < 32 ? w.x : w.y) >> (bit & 31);
    else if (bit >= 32) q = w.y >> (bit & 31);
    else q = __funnelshift_r(w.x, w.y, bit);
    q &= (1u << BITS) - 1u;
    if (MX) {
      // e2m1: exponent and mantissa at fp32's places, scaled by 2^126
      const float m = __uint_as_float((q & 7u) << 22) * __uint_as_float(0x7E800000u);
      v[i] = ((q & 8u) ? -m : m) * s;
    } else {
      v[i] = __fmaf_rn(__uint_as_float(0x4B000000u | q) - 8388608.0f, s, b);
    }
  }
}

// 1024 columns of a row of W by one warp, its loads all in flight at once.
constexpr int kPrepCols = 1024;
template <int BITS, bool MX, bool TWO>
__device__ __forceinline__ void prep_weights(const PrepArgs& p, int64_t o, int col0) {
  const LinArgs& l = p.l;
  const int lane = threadIdx.x & 31, K = l.in_dim;
  const int shift = l.G == 32 ? 5 : l.G == 64 ? 6 : 7, groups = K >> shift;
  const uint32_t* row = l.w + o * (K / 32 * BITS);
  const uint16_t* sc = l.scales + o * groups;
  const uint8_t* ex = reinterpret_cast<const uint8_t*>(l.scales) + o * groups;
  const uint16_t* bi = MX ? nullptr : l.biases + o * groups;
  constexpr int U = kPrepCols / 256;
  uint2 w[U];
  float s[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = min(col0 + lane * 8 + 256 * u, K - 8);
    w[u] = load_run8<BITS>(row, c);
    s[u] = MX ? mx_scale(ex[c >> shift]) : bf16_bits_to_float(sc[c >> shift]);
    b[u] = MX ? 0.0f : bf16_bits_to_float(bi[c >> shift]);
  }
  float largest = 0.0f;
#pragma unroll 2
  for (int g = lane; g < groups; g += 32)
    largest = fmaxf(largest, MX ? 6.0f * mx_scale(ex[g])
                                : fabsf(bf16_bits_to_float(sc[g])) * (float)((1u << BITS) - 1u) +
                                      fabsf(bf16_bits_to_float(bi[g])));
  const int k = lift_of(warp_max(largest));
  const float f = pow2(k);
  if (lane == 0 && col0 == 0) p.fw[o] = pow2(-k);
  __half* out = p.w16 + o * K;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = col0 + lane * 8 + 256 * u;
    if (c < K) {
      float v[8];
      run8_values<BITS, MX>(w[u], s[u] * f, b[u] * f, v);
      store_halves(out + c, (int64_t)l.out_dim * K, TWO, v);
    }
  }
}

// Eight halves (pairs of neighbours) in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 split_order(const uint4& h) {
  return make_uint4(__byte_perm(h.x, h.z, 0x5410u), __byte_perm(h.x, h.z, 0x7632u),
                    __byte_perm(h.y, h.w, 0x5410u), __byte_perm(h.y, h.w, 0x7632u));
}
// Where column c of a row goes in the layout of the product that unpacks the
// weights itself.
__device__ __forceinline__ int run_column(int c) {
  return (c & ~255) | (c & 0x30) << 2 | (c & 0xC0) >> 2 | (c & 8);
}

// A token row by one warp (many rows): the whole row in flight, up to
// 8 * 32 * RV columns of it in registers, longer ones read again.
constexpr int RV = 16;
__device__ __forceinline__ void prep_bf16_row(const PrepArgs& p, int64_t m) {
  const LinArgs& l = p.l;
  const int lane = threadIdx.x & 31, K = l.in_dim;
  const uint16_t* row = reinterpret_cast<const uint16_t*>(l.a.x) + m * l.a.x_stride + 8 * lane;
  __half* out = p.x16 + m * p.x_row + (p.x_runs ? run_column(8 * lane) : 8 * lane);
  uint4 v[RV];
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (8 * lane + 256 * i < K) v[i] = *reinterpret_cast<const uint4*>(row + 256 * i);
  }
  __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
  auto take = [&](uint32_t u) {
    u &= 0x7FFF7FFFu;
    top = __hmax2(top, *reinterpret_cast<const __nv_bfloat162*>(&u));
  };
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    if (256 * i >= K) break;
    take(v[i].x);
    take(v[i].y);
    take(v[i].z);
    take(v[i].w);
  }
  for (int c = 256 * RV; c + 8 * lane < K; c += 256) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + c);
    take(u.x);
    take(u.y);
    take(u.z);
    take(u.w);
  }
  const float2 t = __bfloat1622float2(top);
  const int k = lift_of(warp_max(fmaxf(t.x, t.y)));
  const float f = pow2(k);
  if (lane == 0) p.fx[m] = pow2(-k);
  auto pair = [&](uint32_t u) -> uint32_t {
    return half_pair(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f);
  };
  auto put = [&](int c, const uint4& u) {
    const uint4 h = make_uint4(pair(u.x), pair(u.y), pair(u.z), pair(u.w));
    *reinterpret_cast<uint4*>(out + c) = p.x_split ? split_order(h) : h;
  };
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    if (256 * i >= p.x_row) break;
    if (8 * lane + 256 * i < p.x_row) put(256 * i, v[i]);
  }
  for (int c = 256 * RV; c + 8 * lane < p.x_row; c += 256)
    put(c, c + 8 * lane < K ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u));
}

// The same for 8 bits: with a scale per row the values are fp16 values as they
// are; with one per 128 columns value times scale, lifted by the row's largest.
__device__ __forceinline__ void prep_8bit_row(const PrepArgs& p, int64_t m) {
  const LinArgs& l = p.l;
  const int lane = threadIdx.x & 31, K = l.in_dim;
  const bool i8 = l.a.x_type == MOEQ_I8, by128 = l.a.x_group == 128;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(l.a.x) + m * l.a.x_stride + 8 * lane;
  const float* xs = l.a.x_scales + m * (by128 ? (K + 127) / 128 : 1);
  __half* out = p.x16 + m * p.x_row + (p.x_runs ? run_column(8 * lane) : 8 * lane);
  const int64_t part = (int64_t)l.M * p.x_row;
  uint2 v[RV];
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    v[i] = make_uint2(0u, 0u);
    if (8 * lane + 256 * i < K) v[i] = *reinterpret_cast<const uint2*>(row + 256 * i);
  }
  auto values = [&](const uint2& w, float (&u)[8]) {
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (i8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[4 * h + j] = (float)(int8_t)(q[h] >> (8 * j));
      } else {
        uint32_t p0, p1;
        e4m3_to_bf16(q[h], p0, p1);
        u[4 * h] = __uint_as_float(p0 << 16);
        u[4 * h + 1] = __uint_as_float(p0 & 0xFFFF0000u);
        u[4 * h + 2] = __uint_as_float(p1 << 16);
        u[4 * h + 3] = __uint_as_float(p1 & 0xFFFF0000u);
      }
    }
  };
  auto scale = [&](int c) { return c + 8 * lane < K ? xs[(c + 8 * lane) >> 7] : 0.0f; };
  auto read = [&](int c) {
    return c + 8 * lane < K ? *reinterpret_cast<const uint2*>(row + c) : make_uint2(0u, 0u);
  };
  float f = 1.0f;
  if (by128) {
    float largest = 0.0f;
    auto take = [&](int c, const uint2& w) {
      float u[8], top = 0.0f;
      values(w, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(u[j]));
      largest = fmaxf(largest, top * fabsf(scale(c)));
    };
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      if (256 * i >= K) break;
      take(256 * i, v[i]);
    }
    for (int c = 256 * RV; c < K; c += 256) take(c, read(c));
    const int k = lift_of(warp_max(largest));
    f = pow2(k);
    if (lane == 0) p.fx[m] = pow2(-k);
  } else if (lane == 0) {
    p.fx[m] = xs[0];
  }
  auto put = [&](int c, const uint2& w) {
    float u[8];
    values(w, u);
    if (by128) {
      const float s = scale(c) * f;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] *= s;
    }
    if (p.x_split) {
      const float o[8] = {u[0], u[4], u[1], u[5], u[2], u[6], u[3], u[7]};
      store_halves(out + c, part, false, o);
    } else {
      store_halves(out + c, part, p.x_parts == 2, u);
    }
  };
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    if (256 * i >= p.x_row) break;
    if (8 * lane + 256 * i < p.x_row) put(256 * i, v[i]);
  }
  for (int c = 256 * RV; c + 8 * lane < p.x_row; c += 256) put(c, read(c));
}

// A token row by the whole CTA, in the layout of the product that unpacks the
// weights; up to 8 * NV values of a thread stay in registers between the maximum
// and the conversion, longer rows are read again (from L1).
constexpr int NV = 2;
__device__ __forceinline__ void prep_tokens(const PrepArgs& p, int64_t m) {
  __shared__ float red[32];
  const LinArgs& l = p.l;
  const int K = l.in_dim, T = blockDim.x, type = l.a.x_type;
  const char* row =
      reinterpret_cast<const char*>(l.a.x) + m * l.a.x_stride * (type == MOEQ_BF16 ? 2 : 1);
  const bool by128 = type != MOEQ_BF16 && l.a.x_group == 128;
  const float* xs = l.a.x_scales + m * (by128 ? (K + 127) / 128 : 1);
  __half* out = p.x16 + m * p.x_row;
  auto load = [&](int c, float (&v)[8]) {
    load_x8(row, type, c, v);
    if (by128) {
      const float s = xs[c >> 7];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
    }
  };
  float v[NV][8];
  float largest = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * ((int)threadIdx.x + i * T);
    if (c < K) load(c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (8 * ((int)threadIdx.x + i * T) < K) {
#pragma unroll
      for (int j = 0; j < 8; ++j) largest = fmaxf(largest, fabsf(v[i][j]));
    }
  const int rest = 8 * ((int)threadIdx.x + NV * T);
  for (int c = rest; c < K; c += 8 * T) {
    float u[8];
    load(c, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) largest = fmaxf(largest, fabsf(u[j]));
  }
  float f = 1.0f;
  if (type == MOEQ_BF16 || by128) {
    largest = warp_max(largest);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = largest;
    __syncthreads();
    for (int i = 0; i < T / 32; ++i) largest = fmaxf(largest, red[i]);
    const int k = lift_of(largest);
    f = pow2(k);
    if (threadIdx.x == 0) p.fx[m] = pow2(-k);
  } else if (threadIdx.x == 0) {
    // whole numbers and e4m3 values are fp16 values as they are
    p.fx[m] = xs[0];
  }
  auto put = [&](int c, float (&u)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] *= f;
    c = run_column(c);
    const float w[8] = {u[0], u[4], u[1], u[5], u[2], u[6], u[3], u[7]};
    if (p.x_split) store_halves(out + c, 0, false, w);
    else store_halves(out + c, 0, false, u);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * ((int)threadIdx.x + i * T);
    if (c < K) put(c, v[i]);
  }
  for (int c = rest; c < K; c += 8 * T) {
    float u[8];
    load(c, u);
    put(c, u);
  }
  for (int c = K + 8 * (int)threadIdx.x; c < p.x_row; c += 8 * T) {
    float u[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    put(c, u);
  }
}

// Token rows, one per warp.
__device__ __forceinline__ void prep_row(const PrepArgs& p, int64_t m) {
  if (m >= p.l.M) return;
  if (p.l.a.x_type == MOEQ_BF16) prep_bf16_row(p, m);
  else prep_8bit_row(p, m);
}
__global__ void __launch_bounds__(256) k_lin_rows(const __grid_constant__ PrepArgs p) {
  // (in this order: the weights' kernel writes what the last call's product reads)
  tc::grid_dep_wait();
  tc::grid_dep_launch();
  prep_row(p, (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5));
}

// Weights: 1024 columns of a row per warp.  Runs beside the tokens' kernel
// before it in the stream, and ends after it, so that what waits for this one
// has waited for both.
template <int BITS, bool MX, bool TWO>
__global__ void __launch_bounds__(256) k_lin_weights(const __grid_constant__ PrepArgs p) {
  tc::grid_dep_launch();
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int per_row = (p.l.in_dim + kPrepCols - 1) / kPrepCols;
  const int64_t o = i / per_row;
  if (o < p.l.out_dim) prep_weights<BITS, MX, TWO>(p, o, (int)(i - o * per_row) * kPrepCols);
  tc::grid_dep_wait();
}

// 2^-k of a weight row, by one warp.
__device__ __forceinline__ float row_lift(const LinArgs& l, int64_t o) {
  const int lane = threadIdx.x & 31, groups = l.in_dim / l.G;
  const uint16_t* sc = l.scales + o * groups;
  const uint8_t* ex = reinterpret_cast<const uint8_t*>(l.scales) + o * groups;
  const uint16_t* bi = l.biases + o * groups;
  const float qmax = (float)((1u << l.bits) - 1u);
  float largest = 0.0f;
#pragma unroll 2
  for (int g = lane; g < groups; g += 32)
    largest = fmaxf(largest, l.mx ? 6.0f * mx_scale(ex[g])
                                  : fabsf(bf16_bits_to_float(sc[g])) * qmax +
                                        fabsf(bf16_bits_to_float(bi[g])));
  return pow2(-lift_of(warp_max(largest)));
}

// Tokens as above, but of the weights the powers and scales only: eight rows
// per CTA, transposed through shared memory.
template <bool WARPS>
__global__ void __launch_bounds__(256) k_lin_tokens(const __grid_constant__ PrepArgs p) {
  // (in this order: the product reads weights before it waits)
  tc::grid_dep_wait();
  tc::grid_dep_launch();
  const LinArgs& l = p.l;
  if ((int)blockIdx.x < p.x_blocks) {
    if (WARPS) prep_row(p, (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5));
    else prep_tokens(p, blockIdx.x);
    return;
  }
  __shared__ uint32_t tile[32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, groups = l.in_dim / l.G;
  const int o0 = ((int)blockIdx.x - p.x_blocks) * 8;
  const int64_t o = min(o0 + warp, l.out_dim - 1);
  const float f = row_lift(l, o);                                         // 2^-k
  const float up = __uint_as_float((254u << 23) - __float_as_uint(f));  // 2^k
  if (lane == 0) p.fw[o] = f;
  const int g8 = threadIdx.x >> 3, r8 = threadIdx.x & 7;
  for (int g0 = 0; g0 < groups; g0 += 32) {
    const int64_t g = o * groups + min(g0 + lane, groups - 1);
    const float s = l.mx ? mx_scale(reinterpret_cast<const uint8_t*>(l.scales)[g])
                         : bf16_bits_to_float(l.scales[g]);
    tile[lane][warp] = half_pair(s * up, l.mx ? 0.0f : bf16_bits_to_float(l.biases[g]) * up);
    __syncthreads();
    if (g0 + g8 < groups && o0 + r8 < l.out_dim)
      p.sb[(int64_t)(g0 + g8) * l.out_dim + o0 + r8] = tile[g8][r8];
    __syncthreads();
  }
}

template <bool TWO>
cudaError_t run_weights(const PrepArgs& p, cudaStream_t st) {
  const int64_t warps = (int64_t)p.l.out_dim * ((p.l.in_dim + kPrepCols - 1) / kPrepCols);
  const unsigned b = (unsigned)((warps + 7) / 8);
  if (p.l.mx) return launch_after(k_lin_weights<4, true, TWO>, b, 256, 0, st, p);
  switch (p.l.bits) {
    case 2: return launch_after(k_lin_weights<2, false, TWO>, b, 256, 0, st, p);
    case 3: return launch_after(k_lin_weights<3, false, TWO>, b, 256, 0, st, p);
    case 4: return launch_after(k_lin_weights<4, false, TWO>, b, 256, 0, st, p);
    case 5: return launch_after(k_lin_weights<5, false, TWO>, b, 256, 0, st, p);
    case 6: return launch_after(k_lin_weights<6, false, TWO>, b, 256, 0, st, p);
    default: return launch_after(k_lin_weights<8, false, TWO>, b, 256, 0, st, p);
  }
}

// ------------------------------------------------------------------ GEMM
struct GemmArgs {
  CUtensorMap tm_w, tm_x;  // [part][row][column], boxes of 64 columns
  LinArgs l;
  const float* fx;
  const float* fw;
  int k_blocks;   // 64-column blocks of one product
  int products;   // 1: w x; 2: + (rest of w) x; 3: + w (rest of x)
  int tiles_o, tiles_m;
  int tokens;     // of a tile, a multiple of 16
  int* status;
};

constexpr int kMaxTokens = 256;  // of a tile

struct GemmSmem {
  static constexpr uint32_t A = kTile * 128, B = kMaxTokens / 2 * 128;
  static constexpr int STAGES = 6;
  static constexpr uint32_t BYTES = STAGES * (A + B) + 1024;
};

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, int x, int y,
                                                 int z, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}

// Warps 0: TMA, 1: MMA (rank 0), 2: TMEM; 4..19: epilogue.
//
// The tensor cores cut their sums off (towards zero): a chain of n products of
// 16 columns comes out about n 2^-27 too small.  A bf16 y does not show it;
// for an fp32 y (SUMS) the accumulator is read after every kChunk blocks and
// the parts are added in registers, rounded to nearest: the two accumulators
// then take turns within a tile too.  The products of the rests come first,
// while the accumulator is small and little is cut off: 202 x 1920 x 640, 4-bit,
// int8 by 128 columns, relative error 1.0e-6 with them last, 3.7e-7 so (the plain
// fp32 product 5.3e-7).
constexpr int kChunk = 8;
constexpr int kGemmThreads = 640;

template <bool SUMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_lin_gemm(const __grid_constant__ GemmArgs a) {
  using S = GemmSmem;
  const int BN = a.tokens;
  constexpr int ST = S::STAGES;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t full[ST], empty[ST], tmem_full[2], tmem_empty[2];
  __shared__ uint32_t tmem_holder;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const uint32_t base = (tc::smem_u32(dyn) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&tmem_full[i], 1);
      tc::mbar_init(&tmem_empty[i], 32);  // the epilogue warps of both CTAs
    }
    tc::fence_mbar_init();
  }
  if (warp == 2) {
    tc::tmem_alloc_pair(&tmem_holder, 2 * kMaxTokens);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_holder;
  tc::grid_dep_wait();

  const int unit0 = blockIdx.x >> 1, units = gridDim.x >> 1;
  const int items = a.tiles_o * a.tiles_m, KB = a.k_blocks;
  const int chunk = SUMS ? kChunk : KB;

  if (warp == 0) {
    uint32_t it = 0;
    for (int item = unit0; item < items; item += units) {
      const int o0 = item % a.tiles_o * (2 * kTile) + (int)rank * kTile;
      const int m0 = item / a.tiles_o * BN + (int)rank * (BN / 2);
      for (int k0 = 0; k0 < KB; k0 += chunk)
        for (int prod = a.products - 1; prod >= 0; --prod)
          for (int kb = k0; kb < min(k0 + chunk, KB); ++kb, ++it) {
            const uint32_t s = it % ST, ph = (it / ST) & 1u;
            if (!wait_bar(&empty[s], ph ^ 1u, a.status)) goto done;
            if (lane == 0) {
              const uint32_t bar = tc::mapa_shared(tc::smem_u32(&full[s]), 0);
              const uint32_t at = base + s * (S::A + S::B);
              if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], 2 * S::A + (uint32_t)BN * 128);
              tma_load_3d_pair(at, &a.tm_w, kb * kBK, o0, prod == 1 ? 1 : 0, bar);
              tma_load_3d_pair(at + S::A, &a.tm_x, kb * kBK, m0, prod == 2 ? 1 : 0, bar);
            }
            __syncwarp();
          }
    }
    // every release of this CTA's stages has landed before it may exit
    for (int j = 0; j < ST; ++j, ++it)
      if (!wait_bar(&empty[it % ST], ((it / ST) & 1u) ^ 1u, a.status)) goto done;
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = tc::idesc_f16_f32(2 * kTile, BN);
    const uint32_t on = elect_one();
    uint32_t it = 0, tile = 0;
    for (int item = unit0; item < items; item += units)
      for (int k0 = 0; k0 < KB; k0 += chunk, ++tile) {
        const uint32_t acc = tile & 1u;
        if (!wait_bar(&tmem_empty[acc], ((tile >> 1) & 1u) ^ 1u, a.status)) goto done;
        tc::tc_fence_after();
        const uint32_t d = tmem + acc * kMaxTokens;
        const int n = min(chunk, KB - k0) * a.products;
        for (int kb = 0; kb < n; ++kb, ++it) {
          const uint32_t s = it % ST;
          if (!wait_bar(&full[s], (it / ST) & 1u, a.status)) goto done;
          tc::tc_fence_after();
          const uint64_t da = tc::sw128_kmajor_desc(base + s * (S::A + S::B));
          const uint64_t db = tc::sw128_kmajor_desc(base + s * (S::A + S::B) + S::A);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma_if<true>(on, d, da + 2 * kk, db + 2 * kk, idesc, (kb | kk) != 0);
          if (on) tc::mma_commit_pair(&empty[s], 3);
          __syncwarp();
        }
        if (on) tc::mma_commit_pair(&tmem_full[acc], 3);
        __syncwarp();
      }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint32_t tile = 0;
    for (int item = unit0; item < items; item += units) {
      const int o = item % a.tiles_o * (2 * kTile) + (int)rank * kTile + q * 32 + lane;
      const int m0 = item / a.tiles_o * BN;
      const bool live = o < a.l.out_dim;
      const int oc = min(o, a.l.out_dim - 1);
      const float fw = a.fw[oc];
      const float bias = a.l.a.bias ? bf16_bits_to_float(a.l.a.bias[oc]) : 0.0f;
      // this warp's tokens: sixteen of every 64, from 16 `half` on
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * 16;
      // what the tile reads of mul goes to L2 under its products (2048 x 256 x 4096,
      // MX FP4, both: 37.5 -> 34.6 us; the residual is read a chunk ahead)
      if (a.l.a.mul) {
        constexpr int SIZE = SUMS ? 4 : 2;  // bytes; 32 columns are as many sectors
        const int col0 = item % a.tiles_o * (2 * kTile) + (int)rank * kTile + q * 32;
        for (int i = lane; i < kMaxTokens / 4; i += 32) {
          const int c = 16 * half + (i >> 4) * 64 + (i & 15);
          if (c >= BN || m0 + c >= a.l.M) break;
#pragma unroll
          for (int j = 0; j < SIZE; ++j)
            if (col0 + j * (32 / SIZE) < a.l.out_dim)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(
                  reinterpret_cast<const char*>(a.l.a.mul) +
                  ((int64_t)(m0 + c) * a.l.a.mul_stride + col0 + j * (32 / SIZE)) * SIZE));
        }
      }
      if (SUMS) {
        constexpr int CS = kMaxTokens / 4;
        uint32_t sum[CS];
#pragma unroll
        for (int j = 0; j < CS; ++j) sum[j] = 0u;
        for (int k0 = 0; k0 < KB; k0 += chunk, ++tile) {
          const uint32_t acc = tile & 1u;
          if (!wait_bar(&tmem_full[acc], (tile >> 1) & 1u, a.status)) goto done;
          tc::tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < CS; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(lanes + acc * kMaxTokens + 4 * c0, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              sum[c0 + j] = __float_as_uint(__uint_as_float(sum[c0 + j]) + __uint_as_float(v[j]));
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0)
            tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&tmem_empty[acc]), 0));
        }
#pragma unroll
        for (int c0 = 0; c0 < CS; c0 += 8) {
          const int c = 16 * half + (c0 >> 4) * 64 + (c0 & 8), m = m0 + c;
          const int nm = min(min(8, BN - c), a.l.M - m);
          if (nm <= 0) break;
          uint32_t v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = sum[c0 + j];
          const float fx = lane < nm ? a.fx[m + lane] : 0.0f;
          finish<float, 8>(a.l.a, m, nm, oc, live, fw, bias, fx, v);
        }
      } else {
        const uint32_t acc = tile & 1u;
        // What a chunk of sixteen reads from memory is asked for one chunk ahead,
        // the first before the sums are there.
        uint16_t res[16] = {};
        float fx = 0.0f;
        auto ahead = [&](int c) {
          const int m = m0 + c, nm = min(min(16, BN - c), a.l.M - m);
          if (nm <= 0) return;
          if (a.l.a.residual) {
            if (nm == 16) column<true>(a.l.a.residual, a.l.a.residual_stride, m, nm, oc, res);
            else column(a.l.a.residual, a.l.a.residual_stride, m, nm, oc, res);
          }
          fx = lane < nm ? a.fx[m + lane] : 0.0f;
        };
        ahead(16 * half);
        if (!wait_bar(&tmem_full[acc], (tile >> 1) & 1u, a.status)) goto done;
        tc::tc_fence_after();
        ++tile;
#pragma unroll 1
        for (int c = 16 * half; c < BN; c += 64) {
          const int m = m0 + c, nm = min(16, a.l.M - m);
          if (nm <= 0) break;
          uint32_t v[16];
          tmem_ld16(lanes + acc * kMaxTokens + c - 16 * half, v);
          uint16_t now[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) now[j] = res[j];
          const float fx_now = fx;
          ahead(c + 64);
          tc::tmem_wait_ld();
          if (nm == 16)
            finish_with<uint16_t, 16, true>(a.l.a, m, nm, oc, live, fw, bias, fx_now, v, now);
          else
            finish_with<uint16_t, 16>(a.l.a, m, nm, oc, live, fw, bias, fx_now, v, now);
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&tmem_empty[acc]), 0));
      }
    }
  }
done:
  tc::tc_fence_before();
  tc::cluster_sync();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, 2 * kMaxTokens);
  }
}

// Tokens of a tile: those whose waves take least.  A block of 64 columns costs
// a pair the bytes it brings, 128 rows of W and half the tokens per CTA, in
// proportion 256 + tokens; larger tiles bring fewer, smaller ones may fill the
// last wave better.
int tile_tokens(int64_t M, int64_t out_dim, int pairs) {
  const int64_t tiles_o = (out_dim + 2 * kTile - 1) / (2 * kTile);
  int best = kMaxTokens;
  int64_t least = INT64_MAX;
  for (int n = kMaxTokens; n >= 96; n -= 16) {
    const int64_t tiles = tiles_o * ((M + n - 1) / n);
    const int64_t cost = (tiles + pairs - 1) / pairs * (256 + n);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

// Whether the weights are unpacked inside the product (k_linfused.cu): for up to
// 256 tokens always (there it needs a small workspace only), beyond while its
// clocks are fewer than this way's.  These are a fit too, to the same calls (6 %
// off in the mean): the operands laid out, 1550 per million values; the waves'
// blocks, the epilogue of their tokens, and the first tile's latency per block.
// The choice so made is within 0.5 % of the better way in the mean, 10 % at worst.
// Inside against laid out first, 4-bit, residual: 4096 x 4096, bf16 y, 320 tokens
// 22.1 and 27.2 us, 480 tokens 28.5 and 28.6, 768 tokens 43.1 and 35.6; 512 x 2048,
// 1200 tokens 12.8 and 11.0; fp32 y, 15.7 and 17.8, 3000 tokens 34.4 and 30.5.
bool unpack_inside(int64_t M, int64_t in_dim, int64_t out_dim, int out_type) {
  const LinPlan plan = linear_fused_plan(M, in_dim, out_dim, out_type);
  if (plan.tokens == 0) return false;
  if (M <= 256) return true;
  const int64_t pairs = 74, n = tile_tokens(M, out_dim, (int)pairs);
  const int64_t tiles = (M + n - 1) / n * ((out_dim + 2 * kTile - 1) / (2 * kTile));
  const int64_t waves = (tiles + pairs - 1) / pairs, blocks = (in_dim + kBK - 1) / kBK;
  const bool two = out_type == MOEQ_F32;
  const int parts = two ? 2 : 1;
  const double clocks = (two ? 8300 : 9000) +
                        1550e-6 * (double)(in_dim * (out_dim * parts + M)) +
                        (two ? 0.6 : 0.5) * (double)(waves * blocks * (256 + n) * parts) +
                        (double)((two ? 99 : 49) * waves * n) + (double)((two ? 58 : 37) * blocks);
  return plan.clocks <= clocks;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Layout {
  size_t x16, fx, w16, fw, total;
};
Layout layout(int64_t M, int64_t K, int64_t O, int xp, int wp) {
  Layout o;
  o.x16 = 0;
  o.fx = o.x16 + up256((size_t)(M * K) * 2 * xp);
  o.w16 = o.fx + up256((size_t)M * 4);
  o.fw = o.w16 + up256((size_t)(O * K) * 2 * wp);
  o.total = o.fw + up256((size_t)O * 4);
  return o;
}
struct FusedLayout {
  size_t x16, fx, fw, sb, total;
};
FusedLayout fused_layout(int64_t M, int64_t K, int64_t O, int G) {
  FusedLayout o;
  o.x16 = 0;
  o.fx = o.x16 + up256((size_t)(M * ((K + 255) / 256 * 256)) * 2);
  o.fw = o.fx + up256((size_t)M * 4);
  o.sb = o.fw + up256((size_t)O * 4);
  o.total = o.sb + up256((size_t)(O * (K / G)) * 4);
  return o;
}
int x_parts_of(int x_type, int x_group, int out_type) {
  return out_type == MOEQ_F32 && x_type != MOEQ_BF16 && x_group == 128 ? 2 : 1;
}

template <bool SUMS>
cudaError_t run_gemm(GemmArgs& g, int sms, cudaStream_t st) {
  constexpr uint32_t bytes = GemmSmem::BYTES;
  cudaError_t e = cudaFuncSetAttribute(k_lin_gemm<SUMS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)g.tiles_o * g.tiles_m;
  const int64_t units = items < sms / 2 ? items : sms / 2;
  return launch_after(k_lin_gemm<SUMS>, (unsigned)(2 * units), kGemmThreads, bytes, st, g);
}

}  // namespace

size_t linear_gemm_workspace(const moeq_qtensor& t, int M, int x_type, int out_type) {
  // (an x of 8 bits with an fp32 y: by its x_group it takes either way)
  const int xp = x_parts_of(x_type, 128, out_type);
  const size_t fused = fused_layout(M, t.in_dim, t.out_dim, t.group_size).total;
  const size_t gemm =
      layout(M, t.in_dim, t.out_dim, xp, out_type == MOEQ_F32 ? 2 : 1).total;
  // beyond 256 tokens the choice may turn with M: room for both, so that a
  // workspace for many tokens serves fewer
  if (M <= 256 && xp == 1 && unpack_inside(M, t.in_dim, t.out_dim, out_type)) return fused;
  return fused > gemm ? fused : gemm;
}

cudaError_t launch_linear_gemm(const LinArgs& l, void* ws, int* status, int* launches,
                               cudaStream_t st) {
  *launches = 3;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  PrepArgs p;
  p.l = l;
  p.x_parts = x_parts_of(l.a.x_type, l.a.x_group, l.a.out_type);
  p.w_parts = l.a.out_type == MOEQ_F32 ? 2 : 1;
  const Layout lay = layout(l.M, l.in_dim, l.out_dim, p.x_parts, p.w_parts);
  char* base = (char*)ws;
  p.x16 = (__half*)(base + lay.x16);
  p.fx = (float*)(base + lay.fx);
  p.w16 = (__half*)(base + lay.w16);
  p.fw = (float*)(base + lay.fw);
  p.x_row = l.in_dim;
  p.x_blocks = p.x_runs = p.x_split = 0;
  if (unpack_inside(l.M, l.in_dim, l.out_dim, l.a.out_type) && p.x_parts == 1) {
    const FusedLayout fl = fused_layout(l.M, l.in_dim, l.out_dim, l.G);
    p.x16 = (__half*)(base + fl.x16);
    p.fx = (float*)(base + fl.fx);
    p.fw = (float*)(base + fl.fw);
    p.sb = (uint32_t*)(base + fl.sb);
    p.x_row = (l.in_dim + 255) / 256 * 256;
    p.x_runs = 1;
    p.x_split = l.bits == 2 || l.bits == 4;
    // a token row per CTA, for the latency, or per warp: 616 x 4480 x 128 13.2
    // against 14.3 us, 1868 x 384 x 960 17.7 against 12.3
    const bool warps = l.M > 1024;
    p.x_blocks = warps ? (l.M + 7) / 8 : l.M;
    *launches = 2;
    const cudaError_t e =
        launch_after(warps ? k_lin_tokens<true> : k_lin_tokens<false>,
                     (unsigned)(p.x_blocks + (l.out_dim + 7) / 8), 256, 0, st, p);
    return e != cudaSuccess ? e : launch_linear_fused(l, p.x16, p.fx, p.fw, p.sb, status, st);
  }
  GemmArgs g;
  const int bn = tile_tokens(l.M, l.out_dim, 74);
  g.tokens = bn;
  if (!half_map(&g.tm_w, p.w16, l.in_dim, l.out_dim, p.w_parts, kTile) ||
      !half_map(&g.tm_x, p.x16, l.in_dim, l.M, p.x_parts, bn / 2))
    return cudaErrorNotSupported;
  g.l = l;
  g.fx = p.fx;
  g.fw = p.fw;
  g.k_blocks = (l.in_dim + kBK - 1) / kBK;
  g.products = p.w_parts + p.x_parts - 1;
  g.tiles_o = (l.out_dim + 2 * kTile - 1) / (2 * kTile);
  g.tiles_m = (l.M + bn - 1) / bn;
  g.status = status;
  cudaError_t e = launch_after(
      k_lin_rows, (unsigned)(((int64_t)l.M + 7) / 8), 256, 0, st, p);
  if (e == cudaSuccess) e = p.w_parts == 2 ? run_weights<true>(p, st) : run_weights<false>(p, st);
  if (e != cudaSuccess) return e;
  return l.a.out_type == MOEQ_F32 ? run_gemm<true>(g, sms, st) : run_gemm<false>(g, sms, st);
}

}  // namespace moeq
