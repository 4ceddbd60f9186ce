// Tiled GEMM of the dense operators on tcgen05 (kind::f16, fp32 accumulation
// in tensor memory): the projections, and every product of the backward passes.
//
//   D[m, n] = sum_k A[m, k] B[n, k]
//
// Each operand may have its contraction dimension contiguous (K-major: the
// tokens and weights of a forward product) or its other one (MN-major: the
// weights of dX = dZ W, both operands of dW = dZ^T X), so no operand is ever
// transposed in memory: a stage holds 64 k of either, in 128-byte rows with
// the 128-byte swizzle, and the descriptors say which way they run. Rows,
// columns and k past a matrix read as zeros (the tensor maps' fill) and are
// not stored.
//
// kCg = 2: a pair of CTAs (cluster) shares a tile of 256 rows. Each loads its
// own 128 rows of A and half of B; the first CTA's MMAs read both halves of B
// from both shared memories, so B crosses shared memory once per 256 rows and
// the ring holds more k.
//
// Roles: warp 0 loads by TMA, warp 1 issues the MMAs, warps 2-9 run the
// epilogue out of one accumulator buffer while the next tile fills the other.
// Every wait is bounded; a wait that gives up raises the CTA's abort flag and
// the status word.
#include "dense.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;                       // two per 32-row quarter of the accumulator
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxStages = 10;
constexpr int kATile = 128 * 128;                  // 128 rows x 64 elements of 16 bits
constexpr int kRing = 225 * 1024;
constexpr int kGroupM = 8;                         // row tiles that share their column tiles in L2

struct Tile {
  int seg, m0, n0;
};

}  // namespace

// the 32 accumulator columns at col of row `row`
MOE_DEV void epi_linear(const DenseGemmArgs& a, int seg, int row, int col, const uint32_t (&d)[32]) {
  if (row >= a.M) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + 8 * j >= a.N) break;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(d[8 * j + i]);
    linear8(a, seg, row, col + 8 * j, v);
  }
}

// one row's 32 values as one block of an 8-bit checkpoint (columns past N are zeros)
MOE_DEV void store_block8(const DenseGemmArgs& a, void* q, uint8_t* s, int row, int col, const uint32_t (&d)[32]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, d[i] & 0x7FFFFFFFu);
  const uint32_t code = e4m3_scale_code(m);
  const float inv = e4m3_inv_scale(code);
  s[(size_t)row * ((a.N + 31) / 32) + col / 32] = (uint8_t)code;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + 8 * j >= a.N) break;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(d[8 * j + i]);
    codes8(a, q, row, col + 8 * j, v, inv);
  }
}

MOE_DEV void epi_glu(const DenseGemmArgs& a, int row, int col, const uint32_t (&g)[32], const uint32_t (&u)[32]) {
  if (row >= a.M || col >= a.N) return;
  if (a.g && a.saved8) {
    store_block8(a, a.g, a.g_s, row, col, g);
    store_block8(a, a.u, a.u_s, row, col, u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + 8 * j >= a.N) break;
    float gv[8], uv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gv[i] = __uint_as_float(g[8 * j + i]);
      uv[i] = __uint_as_float(u[8 * j + i]);
    }
    glu8(a, row, col + 8 * j, gv, uv);
  }
}

MOE_DEV void epi_dglu(const DenseGemmArgs& a, int row, int col, const uint32_t (&d)[32]) {
  if (row >= a.M || col >= a.N) return;
  float gs = 1.0f, us = 1.0f;
  if (a.saved8) {
    const size_t so = (size_t)row * ((a.N + 31) / 32) + col / 32;
    gs = e8m0_to_f32(a.g_s[so]);
    us = e8m0_to_f32(a.u_s[so]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = col + 8 * j;
    if (c >= a.N) break;
    const size_t o = (size_t)row * a.N + c;
    float gv[8], uv[8], dg[8], du[8], h[8];
    if (a.saved8) {
      const uint2 gq = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.g) + o));
      const uint2 uq = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.u) + o));
      e4m3_unquad(gq.x, gs, gv);
      e4m3_unquad(gq.y, gs, gv + 4);
      e4m3_unquad(uq.x, us, uv);
      e4m3_unquad(uq.y, us, uv + 4);
    } else {
      unpack16x8(a.f16, ldg16(static_cast<const uint16_t*>(a.g) + o), gv);
      unpack16x8(a.f16, ldg16(static_cast<const uint16_t*>(a.u) + o), uv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float dh = __uint_as_float(d[8 * j + i]);
      float f, s;
      fn_slope(a.fn, gv[i], f, s);
      dg[i] = dh * uv[i] * s;
      du[i] = dh * f;
      h[i] = f * uv[i];
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[0]) + o) = pack16x8(a.f16, dg);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[1]) + o) = pack16x8(a.f16, du);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.pre) + o) = pack16x8(a.f16, h);
  }
}

template <int kEpi, bool kAMn, bool kBMn, int kCg>
__global__ void __launch_bounds__(kThreads, 1) k_dense_gemm(const __grid_constant__ DenseGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kCg == 1 ? 0u : tc::cluster_rank();
  const int tn = a.tile_n, bn = tn / kCg;                   // B rows of a tile, of this CTA
  const int cols = kEpi == kEpiGlu ? tn / 2 : tn;           // output columns of a tile
  const int stage_bytes = kATile + bn * 128;
  const int nst = min(kMaxStages, kRing / stage_bytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps * kCg);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
    tc::prefetch_map(&a.map_a[0]);
    tc::prefetch_map(&a.map_b[0]);
  }
  if (warp == 1) tc::alloc_cg<kCg>(&tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  if (kCg > 1) tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int mt1 = (a.M + 128 * kCg - 1) / (128 * kCg);      // row tiles of a segment
  const int mt = mt1 * a.m_segs, nt = (a.N + cols - 1) / cols;
  const int tiles = mt * nt;
  const int ks1 = (a.K + 63) / 64, ks = ks1 * a.k_segs;
  const int first = (int)blockIdx.x / kCg, step = (int)gridDim.x / kCg;
  // groups of kGroupM row tiles; in a group the row tiles of one column tile follow each other
  auto tile_of = [&](int q) {
    const int per = kGroupM * nt;
    const int grp = q / per, r = q - grp * per;
    const int gm = min(kGroupM, mt - grp * kGroupM);
    const int n = r / gm, m = grp * kGroupM + r - n * gm;
    Tile t;
    t.seg = m / mt1;
    t.m0 = (m - t.seg * mt1) * 128 * kCg + 128 * (int)rank;
    t.n0 = n * cols;
    return t;
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (tc::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      long issued = 0;
      bool ok = true;
      for (int q = first; q < tiles && ok; q += step) {
        const Tile t = tile_of(q);
        for (int j = 0; j < ks; ++j) {
          if (!tc::wait_bounded(&empty[s], ph ^ 1u, abort)) { ok = false; break; }
          uint8_t* sa = smem + s * stage_bytes;
          uint8_t* sb = sa + kATile;
          const int kseg = j >= ks1 ? 1 : 0;
          const int k0 = (j - kseg * ks1) * 64;
          const CUtensorMap* ma = &a.map_a[a.m_segs > 1 ? t.seg : kseg];
          const CUtensorMap* mb = &a.map_b[kseg];
          if (rank == 0) mbar_expect_tx(&full[s], (uint32_t)(stage_bytes * kCg));
          auto load = [&](uint8_t* dst, const CUtensorMap* m, int x, int y) {
            if (kCg == 1) tc::tma_load_2d(dst, m, x, y, &full[s]);
            else tc::tma_load_2d_pair(dst, m, x, y, tc::mapa(&full[s], 0));
          };
          if (kAMn) {
            load(sa, ma, t.m0, k0);
            load(sa + 8192, ma, t.m0 + 64, k0);
          } else {
            load(sa, ma, k0, t.m0);
          }
          if (kEpi == kEpiGlu) {
            if (kCg == 1) {
              load(sb, &a.map_b[0], k0, t.n0);
              load(sb + cols * 128, &a.map_b[1], k0, t.n0);
            } else {
              load(sb, &a.map_b[rank], k0, t.n0);
            }
          } else if (kBMn) {
            for (int i = 0; i < bn / 64; ++i) load(sb + i * 8192, mb, t.n0 + (int)rank * bn + 64 * i, k0);
          } else {
            load(sb, mb, k0, t.n0 + (int)rank * bn);
          }
          ++issued;
          if (++s == nst) { s = 0; ph ^= 1u; }
        }
      }
      // every stage handed back: no arrival of the pair's MMAs is left to come
      for (int i = 0; i < nst && ok; ++i) {
        ok = tc::wait_bounded(&empty[s], ph ^ 1u, abort);
        if (++s == nst) { s = 0; ph ^= 1u; }
      }
      if (!ok && rank == 0) {           // let every issued copy land before the CTA can exit
        for (int i = 0; i < nst && i < issued; ++i) {
          const long last = (issued - 1 - i) / nst;           // last use of stage i
          mbar_wait(&full[i], (uint32_t)(last & 1), 1u << 14);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // the whole loop in one elected thread
    if (rank == 0 && tc::elect_one()) {
      const uint32_t idesc = tc::idesc_16(a.f16, 128 * kCg, tn, kAMn, kBMn);
      constexpr uint32_t a_step = kAMn ? 2048 >> 4 : 32 >> 4, b_step = kBMn ? 2048 >> 4 : 32 >> 4;
      int s = 0, n_it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int q = first; q < tiles && ok; q += step, ++n_it) {
        const int buf = n_it & 1;
        const uint32_t acc_ph = (uint32_t)((n_it >> 1) & 1);
        if (!tc::wait_bounded<(kCg > 1)>(&acc_empty[buf], acc_ph ^ 1u, abort)) break;
        tc::fence_after_sync();
        const uint32_t d = tbase + 256u * buf;
        for (int j = 0; j < ks; ++j) {
          if (!tc::wait_bounded(&full[s], ph, abort)) { ok = false; break; }
          const uint32_t sa = smem_u32(smem + s * stage_bytes), sb = sa + kATile;
          const uint64_t da = kAMn ? tc::desc_mn_sw128(sa, 8192) : tc::desc_sw128(sa);
          const uint64_t db = kBMn ? tc::desc_mn_sw128(sb, 8192) : tc::desc_sw128(sb);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)                    // K = 16 per MMA
            tc::mma_16<kCg>(d, da + kb * a_step, db + kb * b_step, idesc, (j > 0 || kb > 0) ? 1u : 0u);
          tc::commit_cg<kCg>(&empty[s]);
          if (j == ks - 1) tc::commit_cg<kCg>(&acc_full[buf]);
          if (++s == nst) { s = 0; ph ^= 1u; }
        }
      }
      if (*abort) {                     // no MMA may run past the CTA's exit
        tc::commit_cg<kCg>(&drain);
        mbar_wait(&drain, 0);
      }
    }
    __syncwarp();
  } else {
    // ---------------- epilogue (warps 2-9) ----------------
    // two warps share a quarter's 32 rows: 32-column chunks in turn
    const int wq = warp & 3, cfirst = 32 * ((warp - 2) >> 2);
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    int n_it = 0;
    for (int q = first; q < tiles; q += step, ++n_it) {
      const Tile t = tile_of(q);
      const int buf = n_it & 1;
      const bool ok = tc::wait_bounded(&acc_full[buf], (uint32_t)((n_it >> 1) & 1), abort);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc::fence_after_sync();
      const uint32_t dcol = tbase + lane_off + 256u * buf;
      const int row = t.m0 + 32 * wq + lane;
      auto release = [&]() {            // accumulators read: the MMA may reuse them
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (kCg == 1) tc::mbar_arrive(&acc_empty[buf]);
          else tc::arrive_cluster(tc::mapa(&acc_empty[buf], 0));
        }
      };
      if (cfirst >= cols) release();
      for (int c0 = cfirst; c0 < cols; c0 += 64) {
        uint32_t d[32], u[32];
        tc::ld_32cols(dcol + c0, d);
        if (kEpi == kEpiGlu) tc::ld_32cols(dcol + cols + c0, u);
        tc::wait_ld();
        if (c0 + 64 >= cols) release();
        if (kEpi == kEpiGlu) epi_glu(a, row, t.n0 + c0, d, u);
        else if (kEpi == kEpiDGlu) epi_dglu(a, row, t.n0 + c0, d);
        else epi_linear(a, t.seg, row, t.n0 + c0, d);
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) atomicOr(a.status, kStatusWaitTimeout);
  if (kCg > 1) tc::cluster_sync();      // the pair's MMAs read both CTAs' memory
  if (warp == 1) {
    tc::fence_after_sync();
    tc::dealloc_cg<kCg>(tbase, 512);
  }
}

template __global__ void k_dense_gemm<kEpiLinear, false, false, 1>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, false, true, 1>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, true, true, 1>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, false, false, 1>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiDGlu, false, true, 1>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, false, false, 2>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, false, true, 2>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, true, true, 2>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, false, false, 2>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiDGlu, false, true, 2>(const __grid_constant__ DenseGemmArgs);

size_t dense_gemm_smem_bytes() { return kRing + 1024; }
int dense_gemm_threads() { return kThreads; }

}  // namespace moe
