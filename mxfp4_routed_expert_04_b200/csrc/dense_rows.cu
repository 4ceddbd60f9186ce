// Projections of few tokens (serving steps): y = f(x W^T + b) + r and the gated
// block's h, bound by the stream of the weights.
//
// A tile is 128 weight rows (the gated block: 64 gate and the same 64 up
// rows) and all tokens, on tcgen05 with the weights as the M side. The CTAs of
// a cluster each take a part of K, so that few rows still occupy every SM;
// each leaves its fp32 sums in its own shared memory, and after a cluster
// barrier every CTA adds its share of the outputs over the cluster's memories
// in rank order (the same bits every run) and finishes them. Two CTAs fit an
// SM: a following call's barriers, tensor memory and, where it may (`early`),
// first weights are there before this one ends.
#include "dense.cuh"

namespace moe {

namespace {

constexpr int kRowsMaxStages = dense_rows_max_stages();

MOE_DEV float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// sum over the cluster, in rank order, of 8 floats at byte offset `off` of `base`
MOE_DEV void cluster_sum8(const float* base, uint32_t off, int splits, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  for (int r = 0; r < splits; ++r) {
    const uint32_t p = tc::mapa(base, (uint32_t)r) + off;
    const float4 a = ld_cluster(p), b = ld_cluster(p + 16);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
}

// one 8-bit block of 32 columns held by four neighbouring lanes, 8 columns each
MOE_DEV void store_part8(const DenseGemmArgs& a, void* q, uint8_t* s, int row, int c, const float (&v)[8], bool on) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  if (!on) m = 0;
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t code = e4m3_scale_code(m);
  if (!on) return;
  codes8(a, q, row, c, v, e4m3_inv_scale(code));
  if (c % 32 == 0) s[(size_t)row * ((a.N + 31) / 32) + c / 32] = (uint8_t)code;
}

}  // namespace

template <int kEpi>
__global__ void __launch_bounds__(kRowsThreads, 2) k_dense_rows(const __grid_constant__ DenseRowsArgs p) {
  const DenseGemmArgs& a = p.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kRowsMaxStages], empty[kRowsMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  constexpr int kRows = kEpi == kEpiGlu ? 64 : 128;         // outputs of a tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tn = a.tile_n, nst = p.stages;
  const int stage_bytes = dense_rows_stage(tn);
  const int S = p.splits, rank = (int)blockIdx.x % S;
  const int n0 = (int)blockIdx.x / S * kRows;
  const int ks = (a.K + 63) / 64;
  const int j0 = (int)((long)ks * rank / S), j1 = (int)((long)ks * (rank + 1) / S);
  const uint32_t tcols = tn <= 32 ? 32u : tn <= 64 ? 64u : 128u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc_cg<1>(&tmem_slot, tcols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (tc::elect_one()) {
      auto load_w = [&](int s, int j) {
        uint8_t* st = smem + s * stage_bytes;
        mbar_expect_tx(&full[s], (uint32_t)stage_bytes);
        if (kEpi == kEpiGlu) {
          tc::tma_load_2d(st, &a.map_a[0], 64 * j, n0, &full[s]);
          tc::tma_load_2d(st + 8192, &a.map_a[1], 64 * j, n0, &full[s]);
        } else {
          tc::tma_load_2d(st, &a.map_a[0], 64 * j, n0, &full[s]);
        }
      };
      auto load_x = [&](int s, int j) {
        tc::tma_load_2d(smem + s * stage_bytes + 16384, &a.map_b[0], 64 * j, 0, &full[s]);
      };
      if (!p.early) pdl_wait();
      const int pre = min(nst, j1 - j0);
      for (int i = 0; i < pre; ++i) load_w(i, j0 + i);
      if (p.early) pdl_wait();
      for (int i = 0; i < pre; ++i) load_x(i, j0 + i);
      int s = pre == nst ? 0 : pre;
      uint32_t ph = pre == nst ? 1u : 0u;
      bool ok = true;
      for (int j = j0 + pre; j < j1; ++j) {
        if (!tc::wait_bounded(&empty[s], ph ^ 1u, abort)) { ok = false; break; }
        load_w(s, j);
        load_x(s, j);
        if (++s == nst) { s = 0; ph ^= 1u; }
      }
      if (!ok) {                        // let every issued copy land before the CTA can exit
        for (int i = 0; i < nst; ++i) mbar_wait(&full[i], i < s ? ph : ph ^ 1u, 1u << 14);
      }
    }
    __syncwarp();
    pdl_wait();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_16(a.f16, 128, tn, false, false);
      int s = 0;
      uint32_t ph = 0;
      for (int j = j0; j < j1; ++j) {
        if (!tc::wait_bounded(&full[s], ph, abort)) break;
        const uint32_t sa = smem_u32(smem + s * stage_bytes);
        const uint64_t da = tc::desc_sw128(sa), db = tc::desc_sw128(sa + 16384);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          tc::mma_16<1>(tbase, da + 2u * kb, db + 2u * kb, idesc, (j > j0 || kb > 0) ? 1u : 0u);
        tc::commit_cg<1>(&empty[s]);
        if (++s == nst) { s = 0; ph ^= 1u; }
      }
      tc::commit_cg<1>(&acc_full);      // also when it gave up: no MMA may run past the CTA's exit
    }
    __syncwarp();
    pdl_wait();
  } else {
    // ---------------- partial sums to shared memory (warps 2-5) ----------------
    pdl_wait();
  }
  pdl_trigger();
  // every thread: the sums are complete, the ring's last loads and MMAs are done
  tc::wait_bounded(&acc_full, 0, abort);
  tc::fence_after_sync();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);             // [tn][128], where the ring was
  if (warp >= 2 && !*abort) {
    const int wq = warp & 3;
    for (int c0 = 0; c0 < tn; c0 += 16) {
      uint32_t d[32];
      tc::ld_16cols(tbase + ((uint32_t)(32 * wq) << 16) + c0, d);
      tc::wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c0 + i) * 128 + 32 * wq + lane] = __uint_as_float(d[i]);
    }
  }
  tc::fence_before_sync();
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  // groups of 8 outputs, token by token; this CTA's share of the cluster's in
  // whole warps, so four lanes hold a 32-column block
  const int per = kRows / 8, groups = a.M * per;
  for (int b = 32 * (rank * (kRowsThreads / 32) + warp); b < groups; b += S * kRowsThreads) {
    const int i = b + lane, t = i / per, m = 8 * (i - t * per);
    const bool on = i < groups && n0 + m < a.N;
    const int tt = min(t, a.M - 1);
    float v[8];
    cluster_sum8(part, (uint32_t)((tt * 128 + m) * 4), S, v);
    if (kEpi == kEpiGlu) {
      float u[8];
      cluster_sum8(part, (uint32_t)((tt * 128 + 64 + m) * 4), S, u);
      if (a.g && a.saved8) {
        store_part8(a, a.g, a.g_s, t, n0 + m, v, on);
        store_part8(a, a.u, a.u_s, t, n0 + m, u, on);
      }
      if (on) glu8(a, t, n0 + m, v, u);
    } else {
      if (on) linear8(a, 0, t, n0 + m, v);
    }
  }
  if (threadIdx.x == 0 && *abort) atomicOr(a.status, kStatusWaitTimeout);
  if (S > 1) tc::cluster_sync();        // the other CTAs read this one's sums
  else __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, tcols);
  }
}

template __global__ void k_dense_rows<kEpiLinear>(const __grid_constant__ DenseRowsArgs);
template __global__ void k_dense_rows<kEpiGlu>(const __grid_constant__ DenseRowsArgs);

}  // namespace moe
