// Linear with a batch of tokens: weights unpacked inside a tcgen05 product.
//
// For some tens to hundreds of tokens a separate pass that writes W in fp16
// would cost more than the product.  Here a CTA owns 128 rows of W and a run of
// columns: eight warps unpack the codes of 64 columns at a time to fp16 in the
// 128-byte swizzle (one fused multiply-add each, a single rounding; for an fp32
// y a second tile holds what it left), TMA brings the tokens' 64 columns, and
// one thread issues D (128 rows of W) x (up to 256 tokens) in TMEM.  The tokens
// are fp16 rows with a power of two each, from k_lin_prep; the weights' power
// is taken per row and run from its scales and biases.
//
// The columns are split over a cluster of up to eight CTAs, so that few rows
// of W still fill the GPU; the partial sums meet through distributed shared
// memory, each CTA adding up, in rank order, and finishing its share of the
// tokens.  The weights of the run are pulled into L2 first, while the tokens'
// layout kernel still runs.
#include "lingemm.cuh"

namespace moeq {
namespace {

constexpr int kRows = 128;

struct FusedLinArgs {
  CUtensorMap tm_x;  // fp16 tokens, boxes of 64 columns x n rows
  LinArgs l;
  const float* fx;
  int n;        // tokens per CTA, a multiple of 16, at most 256
  int stages;
  int k_blocks;
  int* status;
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// The 32 codes in BITS words, as bytes in order (MX: 2 e2m1 + 12).
template <int BITS, bool MX>
__device__ __forceinline__ void to_bytes(const uint32_t (&w)[BITS], uint32_t (&c)[8]) {
  if (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = w[i < BITS ? i : 0];
  } else if (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e = w[i < BITS ? i : 0] & 0x0F0F0F0Fu;
      uint32_t o = (w[i < BITS ? i : 0] >> 4) & 0x0F0F0F0Fu;
      if (MX) {
        e = mx_q8(e);
        o = mx_q8(o);
      }
      c[2 * i] = __byte_perm(e, o, 0x5140u);
      c[2 * i + 1] = __byte_perm(e, o, 0x7362u);
    }
  } else if (BITS == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t v = (w[i / 4] >> (8 * (i & 3))) & 255u;
      const uint32_t x = (v | (v << 12)) & 0x000F000Fu;
      c[i] = (x | (x << 6)) & 0x03030303u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      constexpr int GB = 4 * BITS % 32;
      const int bit = 4 * BITS * i, k = bit / 32, off = bit % 32;
      const uint32_t hi = k + 1 < BITS ? w[k + 1 < BITS ? k + 1 : 0] : 0u;
      c[i] = Chunk<BITS>::spread4(__funnelshift_r(w[k], hi, off) & ((1u << GB) - 1u));
    }
  }
}

template <int BITS>
__device__ __forceinline__ void load32(const uint32_t* p, bool ok, uint32_t (&w)[BITS]) {
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0u;
  if (!ok) return;
  if (BITS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if (BITS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) w[i] = p[i];
  }
}

// Warps 0: TMA, 1: MMA, 2: TMEM; 4..11: weights, then the epilogue.
template <int BITS, bool MX, bool TWO>
__global__ void __launch_bounds__(384, 1) k_lin_fused(const __grid_constant__ FusedLinArgs a) {
  extern __shared__ uint8_t dyn[];
  constexpr int kMaxStages = 8;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tmem_full;
  __shared__ uint32_t tmem_holder;
  __shared__ float fws[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  uint32_t split;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
  const uint32_t base = (tc::smem_u32(dyn) + 1023u) & ~1023u;
  const int ST = a.stages, N = a.n;
  const uint32_t A1 = kRows * 128, A = TWO ? 2 * A1 : A1, STAGE = A + (uint32_t)N * 128;
  const LinArgs& l = a.l;
  const int o0 = (int)(blockIdx.x / split) * kRows;
  const int m0 = (int)blockIdx.y * N;
  const int kb0 = (int)((int64_t)a.k_blocks * rank / split);
  const int kb1 = (int)((int64_t)a.k_blocks * (rank + 1) / split);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1 + 8);
      tc::mbar_init(&empty[i], 1);
    }
    tc::mbar_init(&tmem_full, 1);
    tc::fence_mbar_init();
  }
  uint32_t cols = 32;
  while (cols < (uint32_t)N) cols *= 2;
  if (warp == 2) {
    tc::tmem_alloc(&tmem_holder, cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_holder;

  bool ok = true;
  if (warp == 0) {
    tc::grid_dep_wait();
    uint32_t s = 0, ph = 1;
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = tc::mbar_wait(&empty[s], ph, a.status);
      if (ok && lane == 0) {
        tc::mbar_arrive_expect_tx(&full[s], (uint32_t)N * 128);
        tc::tma_load_3d(base + s * STAGE + A, &a.tm_x, kb * kBK, m0, 0, &full[s]);
      }
      __syncwarp();
      if (++s == (uint32_t)ST) s = 0, ph ^= 1;
    }
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16_f32(kRows, N);
    uint32_t s = 0, ph = 0;
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = tc::mbar_wait(&full[s], ph, a.status);
      tc::tc_fence_after();
      if (ok && lane == 0) {
        const uint32_t at = base + s * STAGE;
#pragma unroll
        for (int h = 0; h < (TWO ? 2 : 1); ++h)
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            tc::mma_f16(tmem, tc::sw128_kmajor_desc(at + h * A1 + kk * 32),
                        tc::sw128_kmajor_desc(at + A + kk * 32), idesc,
                        (kb > kb0) || ((h | kk) != 0));
        tc::mma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == (uint32_t)ST) s = 0, ph ^= 1;
    }
    if (lane == 0) tc::mma_commit(&tmem_full);
    __syncwarp();
  } else if (warp >= 4) {
    const int t = threadIdx.x - 128, r = t >> 1, h = t & 1;
    const int64_t o = min(o0 + r, l.out_dim - 1);
    const uint32_t* row = l.w + o * ((int64_t)l.in_dim * BITS / 32);
    const int groups = l.in_dim / l.G, shift = l.G == 32 ? 5 : l.G == 64 ? 6 : 7;
    const uint16_t* sc = l.scales + o * groups;
    const uint8_t* ex = reinterpret_cast<const uint8_t*>(l.scales) + o * groups;
    const uint16_t* bi = MX ? nullptr : l.biases + o * groups;
    {
      // the run's codes into L2, a line per request
      const char* p = reinterpret_cast<const char*>(row + (int64_t)kb0 * 2 * BITS);
      const char* e = reinterpret_cast<const char*>(row) +
                      min((int64_t)kb1 * 8 * BITS, (int64_t)l.in_dim * BITS / 8);
      for (const char* c = p + 128 * h; c < e; c += 256)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(c));
    }
    // the run's largest magnitude
    const int g0 = (kb0 * kBK) >> shift, g1 = min((kb1 * kBK + l.G - 1) >> shift, groups);
    float largest = 0.0f;
    for (int g = g0 + h; g < g1; g += 2)
      largest = fmaxf(largest, MX ? finite_abs(6.0f * mx_scale(ex[g]))
                                  : finite_abs(fabsf(bf16_bits_to_float(sc[g])) *
                                                   (float)((1u << BITS) - 1u) +
                                               fabsf(bf16_bits_to_float(bi[g]))));
    largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
    const int k = lift_of(largest);
    const float f = pow2(k);
    if (h == 0) fws[r] = pow2(-k);

    constexpr int D = BITS == 8 ? 3 : 4;  // blocks of codes in flight
    uint32_t raw[D][BITS];
    float fs[D], fb[D];
    auto fetch = [&](int kb, int d) {
      const int c = kb * kBK + 32 * h;
      const bool in = kb < kb1 && c < l.in_dim;
      load32<BITS>(row + (int64_t)(c / 32) * BITS, in, raw[d]);
      const int g = in ? c >> shift : 0;
      fs[d] = MX ? mx_scale(ex[g]) * 0.5f : bf16_bits_to_float(sc[g]);
      fb[d] = MX ? -12.0f * fs[d] : bf16_bits_to_float(bi[g]);
      if (!in) fs[d] = fb[d] = 0.0f;
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(kb0 + d, d);
    uint32_t s = 0, ph = 1;
    for (int kb = kb0; kb < kb1 && ok; kb += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (kb + d >= kb1) break;
        ok = ok && tc::mbar_wait(&empty[s], ph, a.status);
        uint32_t c[8];
        to_bytes<BITS, MX>(raw[d], c);
        const float s32 = fs[d] * f, b32 = fb[d] * f;
        const uint32_t at = base + s * STAGE;
        if (ok) {
          if (TWO) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t q = c[2 * i + j / 2] >> (16 * (j & 1));
                const float w0 = __fmaf_rn((float)(q & 255u), s32, b32);
                const float w1 = __fmaf_rn((float)((q >> 8) & 255u), s32, b32);
                const __half2 p = __floats2half2_rn(w0, w1);
                const float2 b = __half22float2(p);
                const __half2 q2 = __floats2half2_rn(w0 - b.x, w1 - b.y);
                hi[j] = *reinterpret_cast<const uint32_t*>(&p);
                lo[j] = *reinterpret_cast<const uint32_t*>(&q2);
              }
              sts128(at + tc::sw128_offset(r, 4 * h + i), hi);
              sts128(at + A1 + tc::sw128_offset(r, 4 * h + i), lo);
            }
          } else {
            const __half2 s2 = __float2half2_rn(s32), b2 = __float2half2_rn(b32);
            const uint32_t su = *reinterpret_cast<const uint32_t*>(&s2);
            const uint32_t bu = *reinterpret_cast<const uint32_t*>(&b2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // 1024 + q is an fp16 with q in its mantissa
                const uint32_t q =
                    __byte_perm(c[2 * i + j / 2], 0x64646464u, (j & 1) ? 0x4342u : 0x4140u);
                v[j] = hfma2(hsub2(q, 0x64006400u), su, bu);
              }
              sts128(at + tc::sw128_offset(r, 4 * h + i), v);
            }
          }
        }
        fetch(kb + d + D, d);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full[s]);
        if (++s == (uint32_t)ST) s = 0, ph ^= 1;
      }
    }
  }

  // ---- epilogue: warp q + 4 j holds rows 32 q.., every second share of tokens
  const int q = warp & 3, half = (warp - 4) >> 2;
  const int o = o0 + q * 32 + lane;
  const bool live = o < l.out_dim;
  const int oc = min(o, l.out_dim - 1);
  if (warp >= 4) {
    tc::grid_dep_wait();  // the tokens' powers
    ok = tc::mbar_wait(&tmem_full, 0, a.status);
  }
  tc::tc_fence_after();
  __syncthreads();  // fws; every product has been waited for
  const float bias = live && l.a.bias ? bf16_bits_to_float(l.a.bias[oc]) : 0.0f;
  const float fw = warp >= 4 ? fws[q * 32 + lane] : 0.0f;
  if (split == 1) {
    if (warp >= 4 && ok)
      for (int c0 = half * 32; c0 < N; c0 += 64) {
        const int nm = min(min(32, N - c0), l.M - (m0 + c0));
        if (nm <= 0) break;
        uint32_t v[32];
        tc::tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
        const float fx = lane < nm ? a.fx[m0 + c0 + lane] : 0.0f;
        tc::tmem_wait_ld();
        if (l.a.out_type == MOEQ_F32)
          finish<float, 32>(l.a, m0 + c0, nm, oc, live, fw, bias, fx, v);
        else
          finish<uint16_t, 32>(l.a, m0 + c0, nm, oc, live, fw, bias, fx, v);
      }
  } else {
    // partial sums to shared memory, [token][row]
    float* part = reinterpret_cast<float*>(dyn + (base - tc::smem_u32(dyn)));
    if (warp >= 4 && ok)
      for (int c0 = half * 32; c0 < N; c0 += 64) {
        uint32_t v[32];
        tc::tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < N) part[(c0 + j) * kRows + q * 32 + lane] = __uint_as_float(v[j]) * fw;
      }
    tc::cluster_sync();
    if (warp >= 4) {
      const int n0 = (int)((uint32_t)N * rank / split), n1 = (int)((uint32_t)N * (rank + 1) / split);
      const uint32_t mine = base + (uint32_t)(q * 32 + lane) * 4;
      for (int c0 = n0 + half * 8; c0 < n1; c0 += 16) {
        const int nm = min(min(8, n1 - c0), l.M - (m0 + c0));
        if (nm <= 0) break;
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
        for (uint32_t p = 0; p < split; ++p) {
          const uint32_t from = tc::mapa_shared(mine, p);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < nm) sum[j] += ld_cluster(from + (uint32_t)(c0 + j) * (kRows * 4));
        }
        const float fx = lane < nm ? a.fx[m0 + c0 + lane] : 0.0f;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(sum[j]);
        if (l.a.out_type == MOEQ_F32)
          finish<float, 8>(l.a, m0 + c0, nm, oc, live, 1.0f, bias, fx, v);
        else
          finish<uint16_t, 8>(l.a, m0 + c0, nm, oc, live, 1.0f, bias, fx, v);
      }
    }
    tc::cluster_sync();  // a peer may still read this CTA's sums
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, cols);
  }
}

template <int BITS, bool MX, bool TWO>
cudaError_t run(const FusedLinArgs& a, int split, int tiles_o, int tiles_m, uint32_t bytes,
                cudaStream_t st) {
  auto* kernel = k_lin_fused<BITS, MX, TWO>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(tiles_o * split), (unsigned)tiles_m);
  c.blockDim = dim3(384);
  c.dynamicSmemBytes = bytes;
  c.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, kernel, a);
}

template <bool TWO>
cudaError_t run_format(const FusedLinArgs& a, int split, int to, int tm, uint32_t bytes,
                       cudaStream_t st) {
  if (a.l.mx) return run<4, true, TWO>(a, split, to, tm, bytes, st);
  switch (a.l.bits) {
    case 2: return run<2, false, TWO>(a, split, to, tm, bytes, st);
    case 3: return run<3, false, TWO>(a, split, to, tm, bytes, st);
    case 4: return run<4, false, TWO>(a, split, to, tm, bytes, st);
    case 5: return run<5, false, TWO>(a, split, to, tm, bytes, st);
    case 6: return run<6, false, TWO>(a, split, to, tm, bytes, st);
    default: return run<8, false, TWO>(a, split, to, tm, bytes, st);
  }
}

}  // namespace

cudaError_t launch_linear_fused(const LinArgs& l, const __half* x16, const float* fx, int* status,
                                cudaStream_t st) {
  const int sms = sm_count();
  FusedLinArgs a;
  a.l = l;
  a.fx = fx;
  a.status = status;
  const int tiles_m = (l.M + 255) / 256;
  a.n = ((l.M + tiles_m - 1) / tiles_m + 15) / 16 * 16;
  a.k_blocks = (l.in_dim + kBK - 1) / kBK;
  const int tiles_o = (l.out_dim + kRows - 1) / kRows;
  // as many CTAs as SMs, four blocks of columns each at least
  int split = 1;
  while (split < 8 && 2 * split * tiles_o * tiles_m <= sms && a.k_blocks >= 8 * split) split *= 2;
  const bool two = l.a.out_type == MOEQ_F32;
  const uint32_t stage = (two ? 2 : 1) * kRows * 128 + (uint32_t)a.n * 128;
  a.stages = (int)(200 * 1024 / stage);
  if (a.stages > 8) a.stages = 8;
  uint32_t bytes = (uint32_t)a.stages * stage;
  const uint32_t sums = (uint32_t)a.n * kRows * 4;  // fits: n is at most 256
  if (bytes < sums) bytes = sums;
  if (!half_map(&a.tm_x, x16, l.in_dim, l.M, 1, a.n)) return cudaErrorNotSupported;
  return two ? run_format<true>(a, split, tiles_o, tiles_m, bytes + 1024, st)
             : run_format<false>(a, split, tiles_o, tiles_m, bytes + 1024, st);
}

}  // namespace moeq
