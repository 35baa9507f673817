// Linear with few tokens: y = x W^T on the packed codes, exact products.
//
// A CTA owns 16 rows of W and all columns, a warp a run of them; mma.m16n8k16
// (bf16, fp32 sums) multiplies the codes, which bf16 holds exactly (integers to
// 255, or E2M1 values), with eight tokens at a time.  The codes go from global
// memory straight into the fragments: the order of the columns within a product
// is free as long as both operands share it, so lane t of a quad takes C
// neighbouring columns of a span of 4 C, which lies in one scale group.  Per
// span the sums of q x enter the total as s sum(q x) + b sum(x); sum(x) is one
// more product, with ones.
//
// mma.sync, not tcgen05: up to 16 tokens the products are a small part of the
// time, and fragments from registers need no shared-memory tiles, no token
// layout and no TMEM.  Bound by latency: two rounds of loads and products per
// warp.  One token 4096 x 4096, 4-bit: 6.5 us (1.5 TB/s; a launch is about 1.5
// of it); 8 tokens in int8, 1024 rows: 5.1 us; 64 tokens, 512 rows of 8 bits: 6.2.
#include "lincommon.cuh"
#include "tc.cuh"

namespace moeq {
namespace {

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// A lane's C token values from column c0, as loaded (8-bit: in the first words).
template <int C>
__device__ __forceinline__ void load_x(const char* row, bool bf16, int c0, uint32_t (&x)[C / 2]) {
  if (bf16) {
    const uint4* p = reinterpret_cast<const uint4*>(row + 2 * (int64_t)c0);
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      const uint4 v = p[i];
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const uint2* p = reinterpret_cast<const uint2*>(row + c0);
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      const uint2 v = p[i];
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  }
}

// The same as bf16 pairs in the codes' pair order.
template <int BITS, int C>
__device__ __forceinline__ void x_pairs(const uint32_t (&raw)[C / 2], int type,
                                        uint32_t (&b)[C / 2]) {
  uint32_t x[C / 2];
  if (type == MOEQ_BF16) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) x[i] = raw[i];
  } else if (type == MOEQ_I8) {
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      bytes_to_bf16(raw[i] ^ 0x80808080u, 8388736.0f, x[2 * i], x[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) e4m3_to_bf16(raw[i], x[2 * i], x[2 * i + 1]);
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

// The scales (or biases) of four spans from entry `at` on: four entries, or two
// where a group holds two spans (shift 1); MX FP4: four bytes.
template <bool MX>
__device__ __forceinline__ void four_scales(const uint16_t* p, int64_t at, int shift,
                                            uint32_t (&v)[2]) {
  v[1] = 0u;
  if (MX) {
    v[0] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p) + at);
  } else if (shift) {
    v[0] = *reinterpret_cast<const uint32_t*>(p + at);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p + at);
    v[0] = u.x;
    v[1] = u.y;
  }
}

// grid.x: blocks of 16 rows; grid.y: blocks of 8 NT tokens.  The warps split
// the spans; their sums are added in warp order.  A warp asks for everything
// of U spans before it uses the first, so that its run of a 4096-column row
// costs one trip to memory.
template <int BITS, bool MX, int C, int NT, int U, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) k_linear_small(const __grid_constant__ LinArgs l) {
  constexpr int W = Run<BITS, C>::WORDS;
  constexpr int TOKS = 8 * NT;
  __shared__ float red[WARPS][16][TOKS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int o0 = blockIdx.x * 16;
  const int64_t m0 = (int64_t)blockIdx.y * TOKS;
  const int spans = l.in_dim / (4 * C);
  // (whole fours of spans per warp: see below)
  const int fours = (spans + 3) >> 2;
  const int sp0 = 4 * (fours * warp / WARPS), sp1 = min(4 * (fours * (warp + 1) / WARPS), spans);
  const int64_t words_per_row = (int64_t)l.in_dim * BITS / 32;
  // spans per group: 1, or 2 (64-column spans in groups of 128)
  const int shift = l.G == 4 * C ? 0 : 1;
  const int groups = spans >> shift;
  // a row's scales of four spans in one load where they are aligned to that
  const bool wide = l.scales_wide;
  const bool bf16 = l.a.x_type == MOEQ_BF16;
  const bool by128 = !bf16 && l.a.x_group == 128;
  const int xsg = (l.in_dim + 127) / 128;

  const uint32_t* wrow[2];
  int64_t srow[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = min(o0 + 8 * h + g, l.out_dim - 1);
    wrow[h] = l.w + r * words_per_row;
    srow[h] = r * groups;
  }
  const char* xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t m = min(m0 + 8 * n + g, (int64_t)l.M - 1);
    xrow[n] = reinterpret_cast<const char*>(l.a.x) + m * l.a.x_stride * (bf16 ? 2 : 1);
  }

  // The run's codes go to L2 while the preceding kernel ends; what the epilogue
  // needs is asked for first: nothing later waits for DRAM.
  if (sp1 > sp0) {
    const char* p = reinterpret_cast<const char*>(wrow[t >> 1] + (int64_t)sp0 * (C * BITS / 8));
    const char* e = p + (int64_t)(sp1 - sp0) * (C * BITS / 2);
    for (const char* c = p + 128 * (t & 1); c < e; c += 256)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(c));
  }
  tc::grid_dep_wait();
  // (few CTAs: the next kernel's fit beside them; 5.3 -> 5.1 us for eight tokens)
  tc::grid_dep_launch();
  const int erow = threadIdx.x & 15, etok = threadIdx.x >> 4;
  const int64_t em = m0 + etok;
  const bool mine = threadIdx.x < 16 * TOKS && em < l.M && o0 + erow < l.out_dim;
  Epilogue ep;
  if (mine) ep.load(l.a, em, o0 + erow);

  float y[NT][4] = {};
#pragma unroll 1
  for (int base = sp0; base < sp1; base += U) {
    uint32_t w[U][2][W], x[U][NT][C / 2];
    uint32_t s[U][2], b[U][2];
    if (wide) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = srow[h] + ((base & ~3) >> shift);  // the four that holds base
        uint32_t sv[2], bv[2];
        four_scales<MX>(l.scales, at, shift, sv);
        if (!MX) four_scales<false>(l.biases, at, shift, bv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int e0 = (base & 3) + u;  // span within the four
          const int e = shift ? e0 >> 1 : e0;
          if (MX) {
            s[u][h] = (sv[0] >> (8 * e)) & 255u;
          } else {
            s[u][h] = __byte_perm(e & 2 ? sv[1] : sv[0], 0u, e & 1 ? 0x4432u : 0x4410u);
            b[u][h] = __byte_perm(e & 2 ? bv[1] : bv[0], 0u, e & 1 ? 0x4432u : 0x4410u);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int sp = min(base + u, sp1 - 1), grp = sp >> shift;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load_run<BITS, C>(wrow[h], sp, t, w[u][h]);
        if (wide) continue;
        if (MX) {
          s[u][h] = reinterpret_cast<const uint8_t*>(l.scales)[srow[h] + grp];
        } else {
          s[u][h] = l.scales[srow[h] + grp];
          b[u][h] = l.biases[srow[h] + grp];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) load_x<C>(xrow[n], bf16, sp * (4 * C) + t * C, x[u][n]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = base + u < sp1;  // (otherwise the last span again, times 0)
      uint32_t a[2][C / 2];
      float sf[2], bf[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        to_pairs<BITS, MX, C>(w[u][h], a[h]);
        sf[h] = !in ? 0.0f : MX ? mx_scale(s[u][h]) : __uint_as_float(s[u][h] << 16);
        bf[h] = !in || MX ? 0.0f : __uint_as_float(b[u][h] << 16);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t xb[C / 2];
        x_pairs<BITS, C>(x[u][n], l.a.x_type, xb);
        float q[4] = {0.0f, 0.0f, 0.0f, 0.0f}, xs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < C / 4; ++j) {
          mma_bf16(q, a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1], xb[2 * j],
                   xb[2 * j + 1]);
          if (!MX) {
            const uint32_t one = 0x3F803F80u;
            mma_bf16(xs, one, one, one, one, xb[2 * j], xb[2 * j + 1]);
          }
        }
        float f[2] = {1.0f, 1.0f};
        if (by128) {
          const int64_t c = (int64_t)min(base + u, sp1 - 1) * (4 * C) >> 7;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            f[i] = l.a.x_scales[min(m0 + 8 * n + 2 * t + i, (int64_t)l.M - 1) * xsg + c];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v = sf[k >> 1] * q[k];
          if (!MX) v = __fmaf_rn(bf[k >> 1], xs[k], v);
          y[n][k] = by128 ? __fmaf_rn(f[k & 1], v, y[n][k]) : y[n][k] + v;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) red[warp][8 * (k >> 1) + g][8 * n + 2 * t + (k & 1)] = y[n][k];
  __syncthreads();
  if (mine) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += red[k][erow][etok];
    if (!bf16 && !by128) v *= ep.x_scale;
    ep.finish(l.a, em, o0 + erow, v);
  }
}

template <int BITS, bool MX, int C, int WARPS>
cudaError_t run_warps(const LinArgs& l, int blocks, cudaStream_t st) {
  if (l.M <= 8)
    return launch_after(k_linear_small<BITS, MX, C, 1, 4, WARPS>, dim3(blocks), WARPS * 32, 0, st,
                        l);
  return launch_after(k_linear_small<BITS, MX, C, 2, 2, WARPS>, dim3(blocks, (l.M + 15) / 16),
                      WARPS * 32, 0, st, l);
}

// Sixteen warps a CTA (fewer spans for each) while one CTA per SM is all there
// are, eight when two have to share an SM.
template <int BITS, bool MX, int C>
cudaError_t run(const LinArgs& l, cudaStream_t st) {
  const int blocks = (l.out_dim + 15) / 16;
  const int64_t ctas = (int64_t)blocks * (l.M <= 8 ? 1 : (l.M + 15) / 16);
  return ctas <= sm_count() && l.in_dim / (4 * C) > 32 ? run_warps<BITS, MX, C, 16>(l, blocks, st)
                                                       : run_warps<BITS, MX, C, 8>(l, blocks, st);
}

// Spans of 64 columns lie in one group of 64 or 128, of 32 in one of 32.
template <int BITS>
cudaError_t run_bits(const LinArgs& l, cudaStream_t st) {
  return l.G == 32 ? run<BITS, false, 8>(l, st) : run<BITS, false, 16>(l, st);
}

}  // namespace

cudaError_t launch_linear_small(const LinArgs& args, cudaStream_t st) {
  LinArgs l = args;
  // four spans: 4 groups of 64 (of 32 with 32-column spans), 2 of 128
  const int entries = l.G == 128 ? 2 : 4, item = l.mx ? 1 : 2;
  l.scales_wide = (l.in_dim / l.G) % entries == 0 &&
                  ((uintptr_t)l.scales % (entries * item)) == 0 &&
                  (l.mx || ((uintptr_t)l.biases % (entries * item)) == 0);
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
