// Linear with few tokens: y = x W^T on the packed codes, exact products.
//
// A warp owns 16 MT rows of W and a run of columns; mma.m16n8k16 (bf16,
// fp32 sums) multiplies the codes, which bf16 holds exactly (integers to
// 255, or E2M1 values), with eight tokens at a time.  The codes go from
// global memory straight into the fragments: the order of the columns
// within a product is free as long as both operands share it, so lane t of
// a quad takes C neighbouring columns of a span of 4 C, which lies in one
// scale group.  Per span the sums of q x enter the total as
// s sum(q x) + b sum(x); sum(x) is one more product, with ones.
#include "lincommon.cuh"

namespace moeq {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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

// The run as bf16 pairs.  Pair order: widths of 2 and 4 bits (and MX) pair
// values i and i + 4 of each eight, the others neighbours.
template <int BITS>
constexpr bool kSplitPairs = BITS == 2 || BITS == 4;

template <int BITS, bool MX, int C>
__device__ __forceinline__ void to_pairs(const uint32_t (&w)[Run<BITS, C>::WORDS],
                                         uint32_t (&p)[C / 2]) {
  if (BITS == 4) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (MX) {
          // sign to bit 15, exponent and mantissa to the lowest exponent bits
          // and the highest mantissa bit: e2m1 / 2^126, then times 2^126
          const uint32_t s = (j == 3 ? w[i] : w[i] << (12 - 4 * j)) & 0x80008000u;
          const uint32_t v = (j == 0 ? w[i] << 6 : j == 1 ? w[i] << 2 : w[i] >> (4 * j - 6));
          const uint32_t b = s | (v & 0x01C001C0u);
          uint32_t d;
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(b), "r"(0x7E807E80u));
          p[4 * i + j] = d;
        } else {
          p[4 * i + j] = low_to_bf16((w[i] >> (4 * j)) & 0x000F000Fu);
        }
      }
  } else if (BITS == 2) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      // eight codes in 16 bits: the upper byte to the upper half
      const uint32_t u = __byte_perm(w[0], 0u, i == 0 ? 0x4140u : 0x4342u);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[4 * i + j] = low_to_bf16((u >> (2 * j)) & 0x00030003u);
    }
  } else if (BITS == 8) {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) bytes_to_bf16(w[i], 8388608.0f, p[2 * i], p[2 * i + 1]);
  } else {
    constexpr int W = Run<BITS, C>::WORDS;
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      const int bit = 4 * BITS * i, k = bit / 32, off = bit % 32;
      const uint32_t hi = k + 1 < W ? w[k + 1 < W ? k + 1 : 0] : 0u;
      const uint32_t c = Chunk<BITS>::spread4(__funnelshift_r(w[k], hi, off) &
                                              ((1u << (4 * BITS % 32)) - 1u));
      p[2 * i] = sub_bf16x2(__byte_perm(c, 0x43u, 0x4140u), 0x43004300u);
      p[2 * i + 1] = sub_bf16x2(__byte_perm(c, 0x43u, 0x4342u), 0x43004300u);
    }
  }
}

// C tokens values from column c0 as bf16 pairs in the codes' pair order.
template <int BITS, int C>
__device__ __forceinline__ void load_x(const void* row, int type, int64_t c0,
                                       uint32_t (&b)[C / 2]) {
  uint32_t x[C / 2];
  if (type == MOEQ_BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + c0);
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      const uint4 v = p[i];
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const uint2* p = reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(row) + c0);
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      const uint2 v = p[i];
      if (type == MOEQ_I8) {
        bytes_to_bf16(v.x ^ 0x80808080u, 8388736.0f, x[4 * i], x[4 * i + 1]);
        bytes_to_bf16(v.y ^ 0x80808080u, 8388736.0f, x[4 * i + 2], x[4 * i + 3]);
      } else {
        e4m3_to_bf16(v.x, x[4 * i], x[4 * i + 1]);
        e4m3_to_bf16(v.y, x[4 * i + 2], x[4 * i + 3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    if (kSplitPairs<BITS>) {
      b[4 * i] = __byte_perm(x[4 * i], x[4 * i + 2], 0x5410u);
      b[4 * i + 1] = __byte_perm(x[4 * i], x[4 * i + 2], 0x7632u);
      b[4 * i + 2] = __byte_perm(x[4 * i + 1], x[4 * i + 3], 0x5410u);
      b[4 * i + 3] = __byte_perm(x[4 * i + 1], x[4 * i + 3], 0x7632u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[4 * i + j] = x[4 * i + j];
    }
  }
}

// grid.x: blocks of 16 MT rows; grid.y: blocks of 8 NT tokens.  The eight
// warps split the spans; their sums are added in warp order.
template <int BITS, bool MX, int C, int MT, int NT>
__global__ void __launch_bounds__(kWarps * 32) k_linear_small(const __grid_constant__ LinArgs l) {
  constexpr int W = Run<BITS, C>::WORDS;
  constexpr int ROWS = 16 * MT, TOKS = 8 * NT;
  __shared__ float red[kWarps][ROWS][TOKS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int o0 = blockIdx.x * ROWS;
  const int64_t m0 = (int64_t)blockIdx.y * TOKS;
  const int spans = l.in_dim / (4 * C);
  const int sp0 = (int)((int64_t)spans * warp / kWarps);
  const int sp1 = (int)((int64_t)spans * (warp + 1) / kWarps);
  const int64_t words_per_row = (int64_t)l.in_dim * BITS / 32;
  const int groups = l.in_dim / l.G;

  const uint32_t* wrow[MT][2];
  const uint16_t* srow[MT][2];
  const uint16_t* brow[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = min(o0 + 16 * i + 8 * h + g, l.out_dim - 1);
      wrow[i][h] = l.w + r * words_per_row;
      srow[i][h] = MX ? reinterpret_cast<const uint16_t*>(
                            reinterpret_cast<const uint8_t*>(l.scales) + r * groups)
                      : l.scales + r * groups;
      brow[i][h] = MX ? nullptr : l.biases + r * groups;
    }
  const char* xrow[NT];
  const size_t item = l.a.x_type == MOEQ_BF16 ? 2 : 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t m = min(m0 + 8 * n + g, (int64_t)l.M - 1);
    xrow[n] = reinterpret_cast<const char*>(l.a.x) + m * l.a.x_stride * item;
  }
  const bool by128 = l.a.x_type != MOEQ_BF16 && l.a.x_group == 128;
  const int xsg = (l.in_dim + 127) / 128;

  float y[MT][NT][4] = {};
  for (int sp = sp0; sp < sp1; ++sp) {
    const int grp = sp * (4 * C) / l.G;
    float s[MT][2], b[MT][2];
    uint32_t a[MT][2][C / 2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[W];
        load_run<BITS, C>(wrow[i][h], sp, t, w);
        if (MX) {
          s[i][h] = mx_scale(reinterpret_cast<const uint8_t*>(srow[i][h])[grp]);
        } else {
          s[i][h] = bf16_bits_to_float(srow[i][h][grp]);
          b[i][h] = bf16_bits_to_float(brow[i][h][grp]);
        }
        to_pairs<BITS, MX, C>(w, a[i][h]);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t x[C / 2];
      load_x<BITS, C>(xrow[n], l.a.x_type, (int64_t)sp * (4 * C) + t * C, x);
      float xs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (!MX) {
        const uint32_t one = 0x3F803F80u;
#pragma unroll
        for (int j = 0; j < C / 4; ++j) mma_bf16(xs, one, one, one, one, x[2 * j], x[2 * j + 1]);
      }
      float f0 = 1.0f, f1 = 1.0f;
      if (by128) {
        const int64_t c = sp * (4 * C) / 128;
        const int64_t ma = min(m0 + 8 * n + 2 * t, (int64_t)l.M - 1);
        const int64_t mb = min(m0 + 8 * n + 2 * t + 1, (int64_t)l.M - 1);
        f0 = l.a.x_scales[ma * xsg + c];
        f1 = l.a.x_scales[mb * xsg + c];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < C / 4; ++j)
          mma_bf16(q, a[i][0][2 * j], a[i][1][2 * j], a[i][0][2 * j + 1], a[i][1][2 * j + 1],
                   x[2 * j], x[2 * j + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v = s[i][k >> 1] * q[k];
          if (!MX) v = __fmaf_rn(b[i][k >> 1], xs[k], v);
          y[i][n][k] = by128 ? __fmaf_rn(k & 1 ? f1 : f0, v, y[i][n][k]) : y[i][n][k] + v;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        red[warp][16 * i + 8 * (k >> 1) + g][8 * n + 2 * t + (k & 1)] = y[i][n][k];
  __syncthreads();
  for (int i = threadIdx.x; i < ROWS * TOKS; i += kWarps * 32) {
    const int row = i % ROWS, tok = i / ROWS;
    const int64_t m = m0 + tok;
    if (m >= l.M || o0 + row >= l.out_dim) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += red[k][row][tok];
    if (l.a.x_type != MOEQ_BF16 && l.a.x_group == 0) v *= l.a.x_scales[m];
    finish(l.a, m, o0 + row, v);
  }
}

template <int BITS, bool MX, int C>
cudaError_t run(const LinArgs& l, cudaStream_t st) {
  if (l.M <= 8) {
    const dim3 grid((l.out_dim + 15) / 16, 1);
    k_linear_small<BITS, MX, C, 1, 1><<<grid, kWarps * 32, 0, st>>>(l);
  } else {
    const dim3 grid((l.out_dim + 31) / 32, (l.M + 15) / 16);
    k_linear_small<BITS, MX, C, 2, 2><<<grid, kWarps * 32, 0, st>>>(l);
  }
  return cudaGetLastError();
}

// Spans of 64 columns lie in one group of 64 or 128, of 32 in one of 32.
template <int BITS>
cudaError_t run_bits(const LinArgs& l, cudaStream_t st) {
  return l.G == 32 ? run<BITS, false, 8>(l, st) : run<BITS, false, 16>(l, st);
}

}  // namespace

cudaError_t launch_linear_small(const LinArgs& l, cudaStream_t st) {
  if (l.mx) return run<4, true, 8>(l, st);
  switch (l.bits) {
    case 2: return run_bits<2>(l, st);
    case 3: return run_bits<3>(l, st);
    case 4: return run_bits<4>(l, st);
    case 5: return run_bits<5>(l, st);
    case 6: return run_bits<6>(l, st);
    default: return run_bits<8>(l, st);
  }
}

}  // namespace moeq
