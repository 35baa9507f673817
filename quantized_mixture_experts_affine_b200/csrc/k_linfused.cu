// Linear with a batch of tokens: weights unpacked inside a tcgen05 product.
//
// For some tens to hundreds of tokens a separate pass that writes W in fp16
// would cost more than the product.  Here a CTA owns 128 rows of W and a run of
// columns: sixteen warps unpack the codes to fp16 in the 128-byte swizzle (one
// fused multiply-add each, a single rounding; for an fp32 y a second tile holds
// what it left), TMA brings the tokens, and one thread issues D (128 rows of W)
// x (up to 256 tokens) in TMEM.  The tokens are fp16 rows with a power of two
// each, from k_lin_tokens, as are the weights' scales, times a power of their
// row.
//
// The columns are split over a cluster of up to eight CTAs, so that few rows
// of W still fill the GPU; each partial sum is pushed through distributed
// shared memory to the CTA that finishes its token, which adds the parts in
// rank order.  The weights of the run are pulled into L2 first, while the
// tokens' layout kernel still runs.
//
// What bounds it: under about 128 tokens the time around the loop (64 tokens,
// 4096 x 4096, 4-bit, bf16 y, 12.0 us, of which the layout's launch 2.5, the
// prologue 2, unpacking 4), above that the products (256 tokens 20.8 us, 480
// tokens 28.5 us, 0.57 PFLOP/s: the tile's operands and the unpacked weights
// together need 1.5 times an SM's shared-memory bandwidth, and one wave has no
// other tile to hide its ends behind).  fp32 y: 64 tokens 16.6 us, 256 tokens
// 26.7 us.  A thread takes 64 neighbouring codes, so its loads
// are wide and one or two scales serve them: with 16 codes and a scale from
// memory per block the loop was bound by the cache lines its loads touched
// (13.3 us).
#include <type_traits>

#include "lingemm.cuh"

namespace moeq {
namespace {

constexpr int kRows = 128;

struct FusedLinArgs {
  CUtensorMap tm_x;  // fp16 tokens, boxes of 64 columns x n rows
  LinArgs l;
  const float* fx;
  const float* fw;
  const uint32_t* sb;  // [group][out_dim] (s, b) as fp16, times the row's 2^k
  int n;        // tokens per CTA, a multiple of 16, at most 256
  int stages;
  int per;       // 64-column blocks of a stage
  int own_sums;  // the partial sums have a place behind the stages
  int k_runs;  // 256-column runs of a row, the last one padded
  int log2_split, log2_group, tmem_cols;
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// A thread's run: 64 neighbouring codes of a row, 2 BITS words.
template <int BITS>
struct Codes {
  static constexpr int W = 2 * BITS;
  uint32_t w[W];
  // half: the row ends after 32 codes (widths of 4 and 8 bits)
  __device__ __forceinline__ void load(const uint32_t* p, bool half) {
    if (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        if ((BITS == 4 || BITS == 8) && i >= W / 8 && half) break;
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint2 v = reinterpret_cast<const uint2*>(p)[i];
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
      }
    }
  }
  // Codes 4 i .. 4 i + 3 as bytes in order.
  __device__ __forceinline__ uint32_t bytes4(int i) const {
    if (BITS == 8) return w[i];
    const int bit = 4 * BITS * i, k = bit / 32, off = bit % 32;
    const uint32_t v = __funnelshift_r(w[k], k + 1 < W ? w[k + 1 < W ? k + 1 : 0] : 0u, off);
    if (BITS == 4) {
      const uint32_t x = (v & 0xFFu) | ((v & 0xFF00u) << 8);  // two codes per half
      return (x & 0x000F000Fu) | ((x & 0x00F000F0u) << 4);
    }
    if (BITS == 2) {
      const uint32_t x = (v & 0xFu) | ((v & 0xF0u) << 12);
      return (x & 0x00030003u) | ((x & 0x000C000Cu) << 6);
    }
    constexpr int GB = 4 * BITS % 32;
    return Chunk<BITS>::spread4(v & ((1u << GB) - 1u));
  }
};

// Codes 8 i .. 8 i + 7 of a run as fp16 values q s + b, one rounding, in the
// columns' order of the tokens' layout: widths of 2 and 4 bits pair columns j
// and j + 4, which lets one mask cut both out of a word (1024 + 2^k q is an
// fp16 with q in its mantissa), the others neighbours.
template <int BITS, bool MX>
__device__ __forceinline__ void halves8(const Codes<BITS>& c, int i, uint32_t s, uint32_t b,
                                        uint32_t (&v)[4]) {
  constexpr int W = Codes<BITS>::W;
  if (MX) {
    const uint32_t x = c.w[i < W ? i : 0];
    // sign, exponent and mantissa at fp16's places: e2m1 / 2^14, exactly
    v[0] = ((x << 12) & 0x80008000u) | ((x << 9) & 0x0E000E00u);
    v[1] = ((x << 8) & 0x80008000u) | ((x << 5) & 0x0E000E00u);
    v[2] = ((x << 4) & 0x80008000u) | ((x << 1) & 0x0E000E00u);
    v[3] = (x & 0x80008000u) | ((x >> 3) & 0x0E000E00u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = hmul2(hmul2(v[j], 0x74007400u), s);
    return;
  }
  uint32_t q[4];
  if (BITS == 4) {
    const uint32_t x = c.w[i < W ? i : 0], y = x >> 8;
    q[0] = hsub2((x & 0x000F000Fu) | 0x64006400u, 0x64006400u);
    q[1] = hfma2((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);  // / 16 - 64
    q[2] = hsub2((y & 0x000F000Fu) | 0x64006400u, 0x64006400u);
    q[3] = hfma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
  } else if (BITS == 2) {
    const uint32_t x = __byte_perm(c.w[i / 2 < W ? i / 2 : 0], 0u, (i & 1) ? 0x4342u : 0x4140u);
    q[0] = hsub2((x & 0x00030003u) | 0x64006400u, 0x64006400u);
    q[1] = hfma2((x & 0x000C000Cu) | 0x64006400u, 0x34003400u, 0xDC00DC00u);  // / 4 - 256
    q[2] = hfma2((x & 0x00300030u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
    q[3] = hfma2((x & 0x00C000C0u) | 0x64006400u, 0x24002400u, 0xCC00CC00u);  // / 64 - 16
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = hsub2(__byte_perm(c.bytes4(2 * i + j / 2), 0x64646464u, (j & 1) ? 0x4342u : 0x4140u),
                   0x64006400u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = hfma2(q[j], s, b);
}

// The same in fp32, as two fp16 each: the rounded value and what it left.
template <int BITS, bool MX>
__device__ __forceinline__ void halves8_two(const Codes<BITS>& codes, int i, float s, float b,
                                            uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  constexpr bool SPLIT = BITS == 4 || BITS == 2;
  uint32_t c[2] = {codes.bytes4(2 * i), codes.bytes4(2 * i + 1)};
  if (MX) {
    // 2 e2m1 + 12, times s / 2, less 6 s: exact
    c[0] = mx_q8(c[0]);
    c[1] = mx_q8(c[1]);
    b = -6.0f * s;
    s *= 0.5f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p0 = SPLIT ? j : 2 * j, p1 = SPLIT ? j + 4 : 2 * j + 1;
    // 2^23 + q is an fp32 with q in its mantissa
    const float q0 = __uint_as_float(__byte_perm(c[p0 / 4], 0x4B000000u, 0x7440u + (p0 & 3)));
    const float q1 = __uint_as_float(__byte_perm(c[p1 / 4], 0x4B000000u, 0x7440u + (p1 & 3)));
    const float w0 = __fmaf_rn(q0 - 8388608.0f, s, b), w1 = __fmaf_rn(q1 - 8388608.0f, s, b);
    const __half2 r = __floats2half2_rn(w0, w1);
    const float2 f = __half22float2(r);
    const __half2 d = __floats2half2_rn(w0 - f.x, w1 - f.y);
    hi[j] = *reinterpret_cast<const uint32_t*>(&r);
    lo[j] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

constexpr int kUnpackers = 16;  // warps
constexpr int kThreads = 128 + 32 * kUnpackers;

// Warps 0: TMA, 1: MMA, 2: TMEM; 4..19: weights, then the epilogue.
template <int BITS, bool MX, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) k_lin_fused(const __grid_constant__ FusedLinArgs a) {
  extern __shared__ uint8_t dyn[];
  constexpr int kMaxStages = 8;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tmem_full;
  __shared__ uint32_t tmem_holder;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const int lsplit = a.log2_split;
  const uint32_t base = (tc::smem_u32(dyn) + 1023u) & ~1023u;
  // a stage: `per` blocks of 64 columns, each a tile of weights (two for TWO)
  // and one of tokens
  const int ST = a.stages, N = a.n, per = a.per;
  constexpr uint32_t A1 = kRows * 128, A = TWO ? 2 * A1 : A1;
  const uint32_t BLOCK = A + (uint32_t)N * 128, STAGE = BLOCK * per;
  const LinArgs& l = a.l;
  const int o0 = (int)(blockIdx.x >> lsplit) * kRows;
  const int m0 = (int)blockIdx.y * N;
  const int kb0 = 4 * ((a.k_runs * (int)rank) >> lsplit);
  const int kb1 = 4 * ((a.k_runs * (int)(rank + 1)) >> lsplit);
  const int nt = N >> lsplit;  // tokens this CTA finishes, from n0
  const int n0 = m0 + (lsplit ? nt * (int)rank : 0);

  // ---- weights: of each 256 columns four threads per row take 64 neighbours,
  // 16 of them into each of the four 64-column blocks (the tokens' columns
  // are laid out to match), so that a thread's codes come in wide loads and
  // one or two scales serve all of them.  The first codes are asked for
  // before anything else.
  const int t = threadIdx.x - 128, r = t >> 2, part = t & 3;
  const int64_t wo = min(o0 + r, l.out_dim - 1);
  const int shift = a.log2_group;
  const uint32_t* row = l.w + wo * (l.in_dim / 32 * BITS) + part * Codes<BITS>::W;
  Codes<BITS> raw[2];
  auto fetch = [&](int kb, Codes<BITS>& c) {
    const int left = l.in_dim - (kb * kBK + 64 * part);
    if (kb < kb1 && left > 0) c.load(row + (kb >> 2) * (8 * BITS), left < 64);
  };
  if (warp >= 4) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
#pragma unroll
      for (int i = 0; i < Codes<BITS>::W; ++i) raw[d].w[i] = 0u;
      fetch(kb0 + 4 * d, raw[d]);
    }
    // the rest of the run, and what the epilogue reads, into L2
    const char* p = reinterpret_cast<const char*>(row + (kb0 >> 2) * (8 * BITS));
    const char* e = p + min((kb1 - kb0) * 8, (l.in_dim - kb0 * kBK) / 8 - 8 * part) * BITS;
#pragma unroll 1
    for (const char* c = p + 64 * BITS; c < e; c += 32 * BITS)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(c));
    const int size = l.a.out_type == MOEQ_F32 ? 4 : 2, col = o0 + part * (128 / size);
    if (l.a.residual && r < nt && n0 + r < l.M && col < l.out_dim)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          reinterpret_cast<const char*>(l.a.residual) +
          ((int64_t)(n0 + r) * l.a.residual_stride + col) * size));
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&full[i], 1 + kUnpackers);
      tc::mbar_init(&empty[i], 1);
    }
    tc::mbar_init(&tmem_full, 1);
    tc::fence_mbar_init();
  }
  const uint32_t cols = (uint32_t)a.tmem_cols;
  if (warp == 2) {
    tc::tmem_alloc(&tmem_holder, cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // (waited for before anything is written to another CTA: it runs by then)
  if (lsplit) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const uint32_t tmem = tmem_holder;

  bool ok = true;
  tc::grid_dep_wait();  // the tokens and all powers of two
  if (warp == 0) {
    uint32_t s = 0, ph = 1;
#pragma unroll 1
    for (int kb = kb0; kb < kb1 && ok; kb += per) {
      const int n = per;
      ok = wait_bar(&empty[s], ph, a.status);
      if (ok && lane == 0) {
        tc::mbar_arrive_expect_tx(&full[s], (uint32_t)(n * N) * 128);
#pragma unroll 1
        for (int i = 0; i < n; ++i)
          tc::tma_load_3d(base + s * STAGE + i * BLOCK + A, &a.tm_x, (kb + i) * kBK, m0, 0,
                          &full[s]);
      }
      __syncwarp();
      if (++s == (uint32_t)ST) s = 0, ph ^= 1;
    }
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_f16_f32(kRows, N), on = elect_one();
    uint32_t s = 0, ph = 0, more = 0;
#pragma unroll 1
    for (int kb = kb0; kb < kb1 && ok; kb += per) {
      const int n = per;
      ok = wait_bar(&full[s], ph, a.status);
      tc::tc_fence_after();
      if (!ok) break;
      uint32_t at = base + s * STAGE;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint64_t dw = tc::sw128_kmajor_desc(at), dx = tc::sw128_kmajor_desc(at + A);
#pragma unroll
        for (int p = 0; p < (TWO ? 2 : 1); ++p)
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            mma_if<false>(on, tmem + p * (uint32_t)N, dw + p * (A1 >> 4) + 2 * kk, dx + 2 * kk, idesc,
                          more | (kk != 0));
          }
        more = 1;
        at += BLOCK;
      }
      if (on) tc::mma_commit(&empty[s]);
      __syncwarp();
      if (++s == (uint32_t)ST) s = 0, ph ^= 1;
    }
    if (on) tc::mma_commit(&tmem_full);
    __syncwarp();
  } else if (warp >= 4) {
    const uint32_t o1 = tc::sw128_offset(r, 2 * part), o2 = tc::sw128_offset(r, 2 * part + 1);
    const uint32_t* sb = a.sb + wo;  // s and b of a group and row, times the row's 2^k
    auto scales = [&](int kb, uint32_t (&v)[2]) {
      const int col = kb * kBK + 64 * part;
      v[0] = v[1] = 0u;  // beyond the row: zeros
      if (kb < kb1 && col < l.in_dim) v[0] = sb[(int64_t)(col >> shift) * l.out_dim];
      // (the second half's own only for groups of 32: a copy would wait here)
      if (shift == 5 && kb < kb1 && col + 32 < l.in_dim)
        v[1] = sb[(int64_t)((col + 32) >> 5) * l.out_dim];
    };
    uint32_t sbw[2][2];
    scales(kb0, sbw[0]);
    scales(kb0 + 4, sbw[1]);
    uint32_t s = 0, ph = 1, at = base;
#pragma unroll 1
    for (int kb = kb0; kb < kb1 && ok; kb += 8) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int k4 = kb + 4 * d;
        if (k4 >= kb1 || !ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (blocks of a stage: 1, 2 or 4)
          if ((j & (per - 1)) == 0 && !wait_bar(&empty[s], ph, a.status)) {
            ok = false;
            break;
          }
          const uint32_t w = j >= 2 && shift == 5 ? sbw[d][1] : sbw[d][0];
          const uint32_t su = __byte_perm(w, 0u, 0x1010u), bu = __byte_perm(w, 0u, 0x3232u);
          if (TWO) {
            const __half2 h = *reinterpret_cast<const __half2*>(&w);
            const float2 f = __half22float2(h);
            uint32_t hi[4], lo[4];
            halves8_two<BITS, MX>(raw[d], 2 * j, f.x, f.y, hi, lo);
            sts128(at + o1, hi);
            sts128(at + A1 + o1, lo);
            halves8_two<BITS, MX>(raw[d], 2 * j + 1, f.x, f.y, hi, lo);
            sts128(at + o2, hi);
            sts128(at + A1 + o2, lo);
          } else {
            uint32_t v[4];
            halves8<BITS, MX>(raw[d], 2 * j, su, bu, v);
            sts128(at + o1, v);
            halves8<BITS, MX>(raw[d], 2 * j + 1, su, bu, v);
            sts128(at + o2, v);
          }
          at += BLOCK;
          if (((j + 1) & (per - 1)) == 0) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[s]);
            if (++s == (uint32_t)ST) s = 0, ph ^= 1;
            at = base + s * STAGE;
          }
        }
        fetch(k4 + 8, raw[d]);
        scales(k4 + 8, sbw[d]);
      }
    }
  }

  // ---- epilogue: warp 4 + q + 4 j holds rows 32 q.. of every fourth share of
  // the tokens
  const int q = warp & 3, share = (warp - 4) >> 2;
  const int o = o0 + q * 32 + lane;
  const bool live = o < l.out_dim;
  const int oc = min(o, l.out_dim - 1);
  const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
  const float bias = warp >= 4 && live && l.a.bias ? bf16_bits_to_float(l.a.bias[oc]) : 0.0f;
  const float fw = a.fw[oc];
  if (warp >= 4) ok = wait_bar(&tmem_full, 0, a.status) && ok;
  tc::tc_fence_after();
  // where a token's sums are added up
  const uint32_t sums = base + (a.own_sums ? (uint32_t)ST * STAGE : 0u);
  // Eight tokens at a time; what a chunk reads from memory is asked for one
  // chunk ahead, the first before the sums are exchanged.
  using T = typename std::conditional<TWO, float, uint16_t>::type;
  T res[8] = {};
  float fx = 0.0f;
  auto ahead = [&](int c0) {
    const int nm = min(min(8, nt - c0), l.M - (n0 + c0));
    if (warp < 4 || nm <= 0) return;
    if (l.a.residual) column(l.a.residual, l.a.residual_stride, n0 + c0, nm, oc, res);
    fx = lane < nm ? a.fx[n0 + c0 + lane] : 0.0f;
  };
  ahead(share * 8);
  if (lsplit) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // each partial sum goes to the rank that finishes its token:
    // [source rank][token of that rank][row].  Where the sums take the stages'
    // place every CTA has to be done with them.
    if (!a.own_sums) tc::cluster_sync();
    if (warp >= 4 && ok)
#pragma unroll 1
      for (int c0 = share * 16; c0 < N; c0 += 64) {
        uint32_t v[16];
        tmem_ld16(acc + c0, v);
        int dst = 0, tl = c0;
        while (tl >= nt) tl -= nt, ++dst;
        tc::tmem_wait_ld();
        if (TWO) {
          uint32_t u[16];
          tmem_ld16(acc + N + c0, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
        }
        const uint32_t to = sums + (uint32_t)(((int)rank * nt * kRows + q * 32 + lane) * 4);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          st_cluster(tc::mapa_shared(to, (uint32_t)dst) + (uint32_t)(tl * (kRows * 4)),
                     v[j]);
          if (++tl == nt) tl = 0, ++dst;
        }
      }
    tc::cluster_sync();
  }
  if (warp >= 4 && ok) {
    const uint32_t mine = sums + (uint32_t)(q * 32 + lane) * 4;
#pragma unroll 1
    for (int c0 = share * 8; c0 < nt; c0 += 32) {
      const int nm = min(min(8, nt - c0), l.M - (n0 + c0));
      if (nm <= 0) break;
      uint32_t v[8];
      if (lsplit) {
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
#pragma unroll 1
        for (int p = 0; p < 1 << lsplit; ++p)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < nm) sum[j] += lds_f32(mine + (uint32_t)((p * nt + c0 + j) * (kRows * 4)));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(sum[j]);
      } else {
        tmem_ld8(acc + c0, v);
        tc::tmem_wait_ld();
        if (TWO) {
          uint32_t u[8];
          tmem_ld8(acc + N + c0, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
        }
      }
      T now[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) now[j] = res[j];
      const float fx_now = fx;
      ahead(c0 + 32);
      finish_with<T, 8>(l.a, n0 + c0, nm, oc, live, fw, bias, fx_now, v, now);
    }
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
  c.blockDim = dim3(kThreads);
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

constexpr uint32_t kRoom = 224 * 1024;  // shared memory for stages and sums
uint32_t block_bytes(int n, bool two) { return (two ? 2 : 1) * kRows * 128 + (uint32_t)n * 128; }
// Whether the sums of n tokens have a place beside four blocks.
bool own_sums(int n, bool two) { return kRoom >= (uint32_t)n * kRows * 4 + 4 * block_bytes(n, two); }

}  // namespace

// Tiles and clusters of a call, and its clocks.
//
// As many CTAs as SMs, a run of columns each at least.  A cluster lies within
// one GPC: of four CTAs (one per SM) 33 fit at a time, of eight 15 (fewer where
// a GPU has other SMs switched off, so 32 and 14 here); one more and they take
// two waves (64 x 4096 x 2048: 16 tiles in clusters of eight 16.6 us, of four
// 11.7).  The tensor cores cut their sums off, about n 2^-27 for n products of
// 16 columns: for an fp32 y a CTA takes at most six runs (96 products; the
// rounding rests of the weights have an accumulator of their own).
//
// The clocks are fits to measured calls: a block of 64 columns takes 190 and 3.5
// a token, 470 at least for its unpacking (fp32 y: 750 and 4.2), the exchange of
// sums 2500 and 22 a token, 4000 more where it has to wait for the stages' place,
// an epilogue without it 12 a token, the rest 8500.  So 256 tokens are two tiles
// of 128 where the GPU has room (4096 x 2048: 20.2 -> 14.7 us; 2048 x 1024:
// 15.2 -> 9.5).  That fit is of up to 1024 tokens; the plan's clocks, which
// unpack_inside compares, are one of 320 to 8000 tokens, 128 to 4096 columns and
// 64 to 6000 rows (5 % off in the mean).
LinPlan linear_fused_plan(int64_t M, int64_t in_dim, int64_t out_dim, int out_type) {
  const int64_t tiles_o = (out_dim + kRows - 1) / kRows, runs = (in_dim + 255) / 256;
  const bool two = out_type == MOEQ_F32;
  const int fit[4] = {148, 74, 32, 14};
  LinPlan best = {0, 0, 0, 0.0};
  double least = 0.0;
  const int64_t first = (M + 255) / 256;
  for (int64_t tiles_m = first; tiles_m <= first + 3; ++tiles_m) {
    const int64_t n = ((M + tiles_m - 1) / tiles_m + 15) / 16 * 16;
    const int64_t tiles = (M + n - 1) / n * tiles_o;
    int l = 0;
    while (l < 3 && tiles <= fit[l + 1] && runs >= 2 << l) ++l;
    if (two)
      while (l < 3 && runs > 6 << l) ++l;
    if ((two && runs > 6 << l) || tiles_m > 65535) break;  // (tiles_m: the grid's limit)
    const double block = two ? 750 + 4.2 * n : n > 80 ? 190 + 3.5 * n : 470;
    const double waves = (double)((tiles + fit[l] - 1) / fit[l]);
    const double end = l ? 2500 + 22.0 * n + (own_sums((int)n, two) ? 0 : 4000) : 12.0 * n;
    const double clocks =
        8500 + waves * (4.0 * ((runs + (1 << l) - 1) >> l) * block + end);
    if (best.tokens == 0 || clocks < least) {
      least = clocks;
      const double blocks = waves * (4 * ((runs + (1 << l) - 1) >> l));
      const double nw = n * waves, nb = blocks * (n > 80 ? n : 80), laid = 1e-6 * (double)(M * in_dim);
      double c;
      if (two) c = 5200 + 1000 * laid + 1125 * blocks + nb + (l ? 76 * nw + 2300 * waves : 87 * nw);
      else if (l) c = 6000 + 1077 * laid + 570 * blocks + 0.83 * nb + 52 * nw + 2250 * waves;
      else c = 6000 + 1077 * laid + 570 * blocks + 0.83 * nb + 77 * nw;
      if (!two && l && !own_sums((int)n, two)) c += 2500 * waves;
      best = {(int)n, l, (int)((M + n - 1) / n), c};
    }
    if (n <= 64) break;
  }
  return best;
}

cudaError_t launch_linear_fused(const LinArgs& l, const __half* x16, const float* fx,
                                const float* fw, const uint32_t* sb, int* status,
                                cudaStream_t st) {
  FusedLinArgs a;
  a.l = l;
  a.fx = fx;
  a.fw = fw;
  a.sb = sb;
  a.status = status;
  const LinPlan plan = linear_fused_plan(l.M, l.in_dim, l.out_dim, l.a.out_type);
  a.n = plan.tokens;
  a.k_runs = (l.in_dim + 255) / 256;
  a.log2_split = plan.log2_split;
  const int split = 1 << plan.log2_split, tiles_m = plan.tiles_m;
  const int tiles_o = (l.out_dim + kRows - 1) / kRows;
  a.log2_group = l.G == 32 ? 5 : l.G == 64 ? 6 : 7;
  a.tmem_cols = 32;
  const bool two = l.a.out_type == MOEQ_F32;
  while (a.tmem_cols < a.n * (two ? 2 : 1)) a.tmem_cols *= 2;
  const uint32_t block = block_bytes(a.n, two);
  const uint32_t sums = split > 1 ? (uint32_t)a.n * kRows * 4 : 0u;
  // Two stages at least; as many blocks in each (up to four) as fit, so that
  // the waits and fences around a stage are paid seldom.
  a.own_sums = own_sums(a.n, two);
  const uint32_t left = kRoom - (a.own_sums ? sums : 0u);
  a.per = left >= 8 * block ? 4 : left >= 4 * block && a.n <= 192 ? 2 : 1;
  a.stages = (int)(left / (block * a.per));
  if (a.stages > 4) a.stages = 4;
  uint32_t bytes = (uint32_t)a.stages * a.per * block;
  if (a.own_sums) bytes += sums;
  else if (bytes < sums) bytes = sums;  // at most 128 KB
  if (!half_map(&a.tm_x, x16, 256 * a.k_runs, l.M, 1, a.n)) return cudaErrorNotSupported;
  return two ? run_format<true>(a, split, tiles_o, tiles_m, bytes + 1024, st)
             : run_format<false>(a, split, tiles_o, tiles_m, bytes + 1024, st);
}

}  // namespace moeq
