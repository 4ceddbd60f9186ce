// Device helpers of the dense operators (sm_100a): 16-bit conversions, the
// activations and their slopes, the E4M3 checkpoint format, tcgen05 MMAs on
// 16-bit operands by one CTA or a pair.
#pragma once

#include "common.cuh"
#include "dense.h"
#include "tc05.cuh"

namespace moe {

// --- 16-bit types (f16 = 0: bf16) ----------------------------------------------
// two floats -> one word, a in the low half; round to nearest even
MOE_DEV uint32_t pack16(int f16, float a, float b) {
  uint32_t r;
  if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
MOE_DEV void unpack16(int f16, uint32_t w, float& a, float& b) {
  if (f16) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = v.x;
    b = v.y;
  } else {
    a = bf16lo(w);
    b = bf16hi(w);
  }
}
MOE_DEV void unpack16x8(int f16, uint4 v, float* o) {
  unpack16(f16, v.x, o[0], o[1]);
  unpack16(f16, v.y, o[2], o[3]);
  unpack16(f16, v.z, o[4], o[5]);
  unpack16(f16, v.w, o[6], o[7]);
}
MOE_DEV uint4 pack16x8(int f16, const float* v) {
  return make_uint4(pack16(f16, v[0], v[1]), pack16(f16, v[2], v[3]), pack16(f16, v[4], v[5]),
                    pack16(f16, v[6], v[7]));
}

// --- activations -----------------------------------------------------------------
// The hardware exponential and quotient leave, over all 16-bit arguments within
// 13 of 0, f within 1.5e-7 |z| (silu) and 3.4e-7 |z| (gelu), slopes within 9e-7,
// and the far negative tail within 9e-7 (silu) and 3.6e-6 (gelu) of itself (its
// exponential's argument is rounded): far below half a step of the 16-bit
// outputs. silu and its slope are 0 below z = -87.3, where the divisor passes
// 2^126 and the true values are below 1e-36.

// The normal distribution function 0.5 erfc(-z / sqrt 2), e = exp(-z^2 / 2)
// given, without a branch: erfc(x) = t R(t) exp(-x^2) with t = 1 / (1 + 0.6 x)
// for x >= 0, R a polynomial fitted to erfc(x) exp(x^2) / t with evened-out
// relative errors at Chebyshev nodes of t; in fp32 t R is within 5.5e-7 of
// itself, the exponential comes on top. The slope's density shares it.
// erff, with its two branches taken by neighbouring lanes, made the gated
// epilogue of one wave of tiles cost more than its products.
MOE_DEV float normal_cdf(float z, float e) {
  const float t = __fdividef(1.0f, fmaf(0.6f * 0.70710678f, fabsf(z), 1.0f));
  float r = -0.092085987f;
  r = fmaf(r, t, 0.41196054f);
  r = fmaf(r, t, -0.64448047f);
  r = fmaf(r, t, 0.28379223f);
  r = fmaf(r, t, 0.073400266f);
  r = fmaf(r, t, 0.29160431f);
  r = fmaf(r, t, 0.33724868f);
  r = fmaf(r, t, 0.3385601f);
  const float tail = 0.5f * t * r * e;
  return z < 0.0f ? tail : 1.0f - tail;
}
MOE_DEV float normal_exp(float z) { return __expf(-0.5f * z * z); }
MOE_DEV float silu_gate(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
MOE_DEV float relu_keep(float z) { return z < 0.0f ? 0.0f : z; }      // keeps NaN

// v = f(v); the choice of f outside the loop, so that the elements overlap
template <int n>
MOE_DEV void fn_values(int fn, float (&v)[n]) {
  if (fn == MOE_FN_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = __fdividef(v[i], 1.0f + __expf(-v[i]));
  } else if (fn == MOE_FN_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] *= normal_cdf(v[i], normal_exp(v[i]));
  } else if (fn == MOE_FN_RELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = relu_keep(v[i]);
  }
}
// f = f(z) and s = f'(z): silu p (1 + z (1 - p)), gelu Phi(z) + z phi(z), relu 1 for z > 0
template <int n>
MOE_DEV void fn_slopes(int fn, const float (&z)[n], float (&f)[n], float (&s)[n]) {
  if (fn == MOE_FN_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float p = silu_gate(z[i]);
      f[i] = z[i] * p;
      s[i] = p * (1.0f + z[i] * (1.0f - p));
    }
  } else if (fn == MOE_FN_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float e = normal_exp(z[i]), p = normal_cdf(z[i], e);
      f[i] = z[i] * p;
      s[i] = fmaf(0.39894228f * z[i], e, p);
    }
  } else if (fn == MOE_FN_RELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      f[i] = relu_keep(z[i]);
      s[i] = z[i] > 0.0f ? 1.0f : (z[i] <= 0.0f ? 0.0f : z[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      f[i] = z[i];
      s[i] = 1.0f;
    }
  }
}

// --- E4M3 with one E8M0 scale per 32 elements ---------------------------------------
// Scale code of a block from its largest |x| as a bit pattern: the smallest
// power of two 2^X with |x| <= 448 * 2^X, so nothing saturates (448 = 1.75 *
// 2^8); 255 (NaN) when the block holds an infinity or a NaN.
MOE_DEV uint32_t e4m3_scale_code(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  if (e == 255) return 255u;
  const int c = e - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(0, c);
}
// 2^-X for code c = X + 127 (c = 255: 1, its block is NaN whatever the codes)
MOE_DEV float e4m3_inv_scale(uint32_t c) { return c == 255u ? 1.0f : pow2_f32(127 - (int)c); }
// two scaled floats -> two codes, a in the low byte; round to nearest even
MOE_DEV uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
MOE_DEV uint32_t e4m3_quad(const float* v, float inv) {
  return e4m3_pair(v[0] * inv, v[1] * inv) | (e4m3_pair(v[2] * inv, v[3] * inv) << 16);
}
// four codes -> four floats times `scale` (exact: E4M3 values are f16 values)
MOE_DEV void e4m3_unquad(uint32_t w, float scale, float* v) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x * scale;
  v[1] = a.y * scale;
  v[2] = b.x * scale;
  v[3] = b.y * scale;
}

namespace tc {

// kind::f16, fp32 accumulation; M rows over the CTAs of the group; a_mn / b_mn:
// the operand's M / N dimension is contiguous in shared memory instead of K
MOE_DEV uint32_t idesc_16(int f16, int M, int N, bool a_mn, bool b_mn) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 128-byte-swizzled tile whose 128-byte rows run along M or N, one row per k:
// 64-element column blocks `block_bytes` apart, 8-k groups 1024 bytes apart
MOE_DEV uint64_t desc_mn_sw128(uint32_t addr, uint32_t block_bytes) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(block_bytes >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
template <int kCg>
MOE_DEV void mma_16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCg == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
  }
}
template <int kCg>
MOE_DEV void alloc_cg(uint32_t* dst, uint32_t ncols) {
  if constexpr (kCg == 1) {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n"
                 ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
}
template <int kCg>
MOE_DEV void dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if constexpr (kCg == 1) tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}
// arrive on `bar` of every CTA of the group when this thread's MMAs are done
template <int kCg>
MOE_DEV void commit_cg(uint64_t* bar) {
  if constexpr (kCg == 1) commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
// shared::cluster address of `p` in the CTA of rank `rank`
MOE_DEV uint32_t mapa(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
MOE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// TMA load of a CTA pair: the bytes land in this CTA, the count on the barrier
// at shared::cluster address `bar` (the first CTA's)
MOE_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];\n"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
MOE_DEV void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// One lane of the warp, by elect.sync: the compiler then knows that the branch
// holds one thread, so the tcgen05 and TMA instructions in it take their
// operands from uniform registers. Behind `lane == 0` each was wrapped in a
// loop over the active lanes: a stage of four 256x256x16 MMAs cost 0.42 us,
// with elect.sync 0.37 us (256x128: 0.39 and 0.30).
MOE_DEV bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
MOE_DEV uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(t));
  return t;
}
// Bounded wait on phase `parity` of `bar` that gives up after about `limit_ns`
// or as soon as another role of the CTA has raised `*abort` (raising it
// itself on a timeout). kCluster: threads of another CTA arrive on `bar`.
constexpr uint32_t kSuspendNs = 1000000;   // a waiting thread sleeps this long at most before it looks again
template <bool kCluster = false>
MOE_DEV bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                          uint64_t limit_ns = 4000000000ull) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  while (true) {
    uint32_t done;
    if constexpr (kCluster)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(a), "r"(parity), "r"(kSuspendNs) : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(a), "r"(parity), "r"(kSuspendNs) : "memory");
    if (done) return true;
    if (*abort) return false;
    const uint64_t t = global_ns();
    if (t0 == 0) t0 = t;
    else if (t - t0 > limit_ns) break;
  }
  *abort = 1;
  return false;
}

// Before a CTA that gave up a wait may exit: its copies, `issued` stages in turn
// over a ring of nst, have landed (bounded; one thread)
MOE_DEV void drain_copies(uint64_t* full, int nst, long issued) {
  for (int i = 0; i < nst && i < issued; ++i)
    mbar_wait(&full[i], (uint32_t)((issued - 1 - i) / nst & 1), 1u << 14);
}

}  // namespace tc
}  // namespace moe
