// Projections of few tokens (serving steps): y = f(x W^T + b) + r and the gated
// block's h, bound by the stream of the weights; and of few tokens' gradients
// dX = dZ W and the block's hidden gradient (kWMn: the weights' output
// dimension is the contiguous one).
//
// A tile is 128 weight rows (the gated block: 64 gate and the same 64 up
// rows) and all tokens, on tcgen05 with the weights as the M side. The CTAs of
// a cluster each take a part of K, so that few rows still occupy every SM.
// Their fp32 sums are added in rank order (the same bits every run), in one of
// two ways. Up to kRowsPush tokens every CTA writes its sums into the shared
// memory of the CTA that finishes the outputs, and one cluster barrier later
// they are there. The remote stores of more tokens take longer than the round
// trip they save: there each CTA keeps its sums, over its ring, and each
// fetches its share of the outputs from all (one token of 7168 -> 2048: 6.6 us
// pushed, 7.9 fetched; 16 tokens of 2048 -> 7168: 10.0 and 8.8). Two CTAs fit
// an SM: a following call's barriers, tensor memory and, where it may
// (`early`), first weights are there before this one ends.
#include "dense.cuh"

namespace moe {

namespace {

MOE_DEV void st_cluster4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};\n"
               ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
MOE_DEV float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
MOE_DEV void add_parts(const float4 (&q)[kRowsSplits], int splits, float (&v)[4]) {
  v[0] = q[0].x; v[1] = q[0].y; v[2] = q[0].z; v[3] = q[0].w;
#pragma unroll
  for (int r = 1; r < kRowsSplits; ++r) {
    if (r < splits) {
      v[0] += q[r].x; v[1] += q[r].y; v[2] += q[r].z; v[3] += q[r].w;
    }
  }
}
// sum in rank order, all loads first: of pushed parts `stride` float4 apart
MOE_DEV void sum_pushed(const float4* p, int splits, int stride, float (&v)[4]) {
  float4 q[kRowsSplits];
#pragma unroll
  for (int r = 0; r < kRowsSplits; ++r)
    if (r < splits) q[r] = p[r * stride];
  add_parts(q, splits, v);
}
// and of kept parts, at byte offset `off` of every CTA's `base`
MOE_DEV void sum_kept(const float* base, uint32_t off, int splits, float (&v)[4]) {
  float4 q[kRowsSplits];
#pragma unroll
  for (int r = 0; r < kRowsSplits; ++r)
    if (r < splits) q[r] = ld_cluster4(tc::mapa(base, (uint32_t)r) + off);
  add_parts(q, splits, v);
}
MOE_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
MOE_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

MOE_DEV float load16(int f16, const void* base, size_t off) {
  const uint32_t w = static_cast<const uint16_t*>(base)[off];
  float a, b;
  unpack16(f16, w, a, b);
  return a;
}
MOE_DEV void store16(void* base, size_t off, int f16, float v) {
  static_cast<uint16_t*>(base)[off] = (uint16_t)(pack16(f16, v, v) & 0xFFFFu);
}

// a block of an 8-bit checkpoint, one column a lane (zero past N)
MOE_DEV void store_lanes8(const DenseGemmArgs& a, void* q, uint8_t* s, int row, int c, float v, bool on, int lane) {
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
  const uint32_t code = e4m3_scale_code(m);
  if (!on) return;
  static_cast<uint8_t*>(q)[(size_t)row * a.p[0].N + c] = (uint8_t)(e4m3_pair(v * e4m3_inv_scale(code), 0.0f) & 0xFFu);
  if (lane == 0) s[(size_t)row * ((a.p[0].N + 31) / 32) + c / 32] = (uint8_t)code;
}
// one held by eight neighbouring lanes, 4 columns each
MOE_DEV void store_quads8(const DenseGemmArgs& a, void* q, uint8_t* s, int row, int c, const float (&v)[4], bool on) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  if (!on) m = 0;
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  const uint32_t code = e4m3_scale_code(m);
  if (!on) return;
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(q) + (size_t)row * a.p[0].N + c) = e4m3_quad(v, e4m3_inv_scale(code));
  if (c % 32 == 0) s[(size_t)row * ((a.p[0].N + 31) / 32) + c / 32] = (uint8_t)code;
}
MOE_DEV uint2 load4(const void* base, size_t off) {
  return *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + off);
}
MOE_DEV void store4(void* base, size_t off, int f16, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + off) =
      make_uint2(pack16(f16, v[0], v[1]), pack16(f16, v[2], v[3]));
}
MOE_DEV void add4(int f16, uint2 w, float (&v)[4]) {
  float t[4];
  unpack16(f16, w.x, t[0], t[1]);
  unpack16(f16, w.y, t[2], t[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += t[i];
}

// g or u as the forward pass saved them: 4 columns, or one
MOE_DEV void saved4(const DenseGemmArgs& a, const void* q, const uint8_t* s, int row, int c, float (&v)[4]) {
  const size_t o = (size_t)row * a.p[0].N + c;
  if (a.saved8) {
    e4m3_unquad(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(q) + o),
                e8m0_to_f32(s[(size_t)row * ((a.p[0].N + 31) / 32) + c / 32]), v);
  } else {
    const uint2 w = load4(q, o);
    unpack16(a.f16, w.x, v[0], v[1]);
    unpack16(a.f16, w.y, v[2], v[3]);
  }
}
MOE_DEV float saved1(const DenseGemmArgs& a, const void* q, const uint8_t* s, int row, int c) {
  const size_t o = (size_t)row * a.p[0].N + c;
  if (!a.saved8) return load16(a.f16, q, o);
  float v[4];
  e4m3_unquad(static_cast<const uint8_t*>(q)[o], e8m0_to_f32(s[(size_t)row * ((a.p[0].N + 31) / 32) + c / 32]), v);
  return v[0];
}

// Kept sums: groups of 4 outputs, token by token, this CTA's share of the
// cluster's in whole warps, so eight lanes hold a 32-column block.
template <int kEpi>
MOE_DEV void finish_kept(const DenseGemmArgs& a, const float* part, int n0, int rank, int S, int warp, int lane) {
  constexpr int kPer = (kEpi == kEpiGlu ? 64 : 128) / 4;
  const int groups = a.p[0].M * kPer;
  for (int b = 32 * (rank * (kRowsThreads / 32) + warp); b < groups; b += S * kRowsThreads) {
    const int i = b + lane, t = i / kPer, m = 4 * (i - t * kPer), c = n0 + m;
    const bool on = i < groups && c < a.p[0].N;
    const uint32_t off = on ? (uint32_t)((t * 128 + m) * 4) : 0u;
    const size_t o = (size_t)t * a.p[0].N + c;
    float v[4];
    if (kEpi == kEpiDGlu) {
      float g[4], u[4], f[4], d[4];
      if (on) {
        saved4(a, a.g, a.g_s, t, c, g);
        saved4(a, a.u, a.u_s, t, c, u);
      }
      sum_kept(part, off, S, v);
      if (on) {
        fn_slopes(a.fn, g, f, d);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[k] *= v[k] * u[k];          // dg
          v[k] *= f[k];                 // du
          u[k] *= f[k];                 // h
        }
        store4(a.p[0].out[0], o, a.f16, d);
        store4(a.p[0].out[1], o, a.f16, v);
        store4(a.pre, o, a.f16, u);
      }
    } else if (kEpi == kEpiGlu) {
      float u[4];
      sum_kept(part, off, S, v);
      sum_kept(part, off + 256, S, u);          // the up rows, 64 further on
      if (a.g && a.saved8) {
        store_quads8(a, a.g, a.g_s, t, c, v, on);
        store_quads8(a, a.u, a.u_s, t, c, u, on);
      }
      if (on) {
        if (a.g && !a.saved8) {
          store4(a.g, o, a.f16, v);
          store4(a.u, o, a.f16, u);
        }
        fn_values(a.fn, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= u[k];
        store4(a.p[0].out[0], o, a.f16, v);
      }
    } else {
      uint2 bias = make_uint2(0u, 0u), res = bias;
      if (on && a.bias) bias = load4(a.bias, (size_t)c);
      if (on && a.residual) res = load4(a.residual, (size_t)t * a.ldr + c);
      sum_kept(part, off, S, v);
      if (on) {
        if (a.bias) add4(a.f16, bias, v);
        if (a.pre) store4(a.pre, o, a.f16, v);
        fn_values(a.fn, v);
        if (a.residual) add4(a.f16, res, v);
        const size_t y = (size_t)t * a.p[0].ldo + c;
        if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.p[0].out[0]) + y) = make_float4(v[0], v[1], v[2], v[3]);
        else store4(a.p[0].out[0], y, a.f16, v);
      }
    }
  }
}

}  // namespace

template <int kEpi, bool kWMn, bool kPieces>
__global__ void __launch_bounds__(kRowsThreads, 2) k_dense_rows(const __grid_constant__ DenseRowsArgs p) {
  const DenseGemmArgs& a = p.g;
  const DenseProblem& b = a.p[0];
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kDenseRowsStages], empty[kDenseRowsStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, issued;
  volatile int* abort = &abort_flag;
  constexpr int kRows = kEpi == kEpiGlu ? 64 : 128;         // outputs of a tile
  constexpr int kPer = kRows / 32;                          // units of 4 tokens
  constexpr int kUnit = kEpi == kEpiGlu ? 64 : 32;          // rows (of 4 tokens) of a unit's part: gate, up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tn = a.tile_n, nst = p.stages;
  const int stage_bytes = dense_rows_stage(tn);
  const int S = p.splits, rank = (int)blockIdx.x % S;
  const int n0 = (int)blockIdx.x / S * kRows;
  const int ks1 = (b.K + 63) / 64, ks = ks1 * b.k_segs;
  const int j0 = (int)((long)ks * rank / S), j1 = (int)((long)ks * (rank + 1) / S);
  const uint32_t acols = tn <= 32 ? 32u : 64u;              // columns of an accumulator
  const uint32_t tcols = kPieces ? 2u * acols : acols;
  const int pieces = kPieces ? pieces_of(j1 - j0) : 1;
  // pushed: units of 4 tokens x 32 rows, [unit slot][rank][kUnit] of 4 tokens of a
  // row, behind the ring; kept: floats [token][128 rows], over it
  const bool push = b.M <= kRowsPush;
  float4* parts = reinterpret_cast<float4*>(smem + (push ? nst * stage_bytes : 0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc_cg<1>(&tmem_slot, tcols);
  tc::fence_before_sync();
  __syncthreads();
  cluster_arrive();                     // this CTA runs: its memory may be written
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;
  const int wq = warp & 3;              // warps 2-5: which 32 of the 128 rows
  const uint32_t row0 = tbase + ((uint32_t)(32 * wq) << 16);
  float sum[kPieces ? kRowsTokens : 1]; // kPieces: this lane's row, all tokens
  bool whole = true;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (tc::elect_one()) {
      auto load_w = [&](int s, int j) {
        uint8_t* st = smem + s * stage_bytes;
        const int seg = j >= ks1 ? 1 : 0, k0 = 64 * (j - seg * ks1);
        mbar_expect_tx(&full[s], (uint32_t)stage_bytes);
        if (kEpi == kEpiGlu) {
          tc::tma_load_2d(st, &b.map_a[0], k0, n0, &full[s]);
          tc::tma_load_2d(st + 8192, &b.map_a[1], k0, n0, &full[s]);
        } else if (kWMn) {
          tc::tma_load_2d(st, &b.map_a[seg], n0, k0, &full[s]);
          tc::tma_load_2d(st + 8192, &b.map_a[seg], n0 + 64, k0, &full[s]);
        } else {
          tc::tma_load_2d(st, &b.map_a[0], k0, n0, &full[s]);
        }
      };
      auto load_x = [&](int s, int j) {
        const int seg = j >= ks1 ? 1 : 0;
        tc::tma_load_2d(smem + s * stage_bytes + 16384, &b.map_b[seg], 64 * (j - seg * ks1), 0, &full[s]);
      };
      if (!p.early) pdl_wait();
      const int pre = min(nst, j1 - j0);
      for (int i = 0; i < pre; ++i) load_w(i, j0 + i);
      if (p.early) pdl_wait();
      for (int i = 0; i < pre; ++i) load_x(i, j0 + i);
      int s = pre == nst ? 0 : pre;
      uint32_t ph = pre == nst ? 1u : 0u;
      int j = j0 + pre;
      for (; j < j1; ++j) {
        if (!tc::wait_bounded(&empty[s], ph ^ 1u, abort)) break;
        load_w(s, j);
        load_x(s, j);
        if (++s == nst) { s = 0; ph ^= 1u; }
      }
      issued = j - j0;
    }
    __syncwarp();
    pdl_wait();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    pdl_wait();                         // its bounded waits begin when the tokens can arrive
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_16(a.f16, 128, tn, kWMn, false);
      constexpr uint32_t w_step = kWMn ? 2048 >> 4 : 32 >> 4;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; i < pieces && ok; ++i) {
        const int buf = i & 1;
        const int b0 = kPieces ? j0 + (j1 - j0) * i / pieces : j0, b1 = kPieces ? j0 + (j1 - j0) * (i + 1) / pieces : j1;
        if (kPieces) {
          ok = tc::wait_bounded(&acc_empty[buf], (uint32_t)((i >> 1) & 1) ^ 1u, abort);
          tc::fence_after_sync();
        }
        const uint32_t d = tbase + acols * (uint32_t)buf;
        for (int j = b0; j < b1 && ok; ++j) {
          if (!tc::wait_bounded(&full[s], ph, abort)) { ok = false; break; }
          const uint32_t sa = smem_u32(smem + s * stage_bytes);
          const uint64_t da = kWMn ? tc::desc_mn_sw128(sa, 8192) : tc::desc_sw128(sa), db = tc::desc_sw128(sa + 16384);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
            tc::mma_16<1>(d, da + kb * w_step, db + 2u * kb, idesc, (j > b0 || kb > 0) ? 1u : 0u);
          tc::commit_cg<1>(&empty[s]);
          if (++s == nst) { s = 0; ph ^= 1u; }
        }
        tc::commit_cg<1>(&acc_full[buf]);
      }
      tc::commit_cg<1>(&drain);
    }
    __syncwarp();
  } else {
    // ---------------- sums (warps 2-5; to shared memory further down) ----------------
    pdl_wait();
    if constexpr (kPieces) {
      // The pieces as they come, in order. In front of the cluster barrier: the
      // MMAs wait for these warps, and warps 0 and 1 come to it behind the MMAs.
      pdl_trigger();
      for (int i = 0; i < pieces && whole; ++i) {
        whole = __all_sync(0xFFFFFFFFu, tc::wait_bounded(&acc_full[i & 1], (uint32_t)((i >> 1) & 1), abort));
        if (!whole) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < kRowsTokens / 16; ++c) {
          if (16 * c < b.M) {
            uint32_t d[32];
            tc::ld_16cols(row0 + acols * (uint32_t)(i & 1) + 16 * c, d);
            tc::wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[16 * c + k] = __uint_as_float(d[k]) + (i ? sum[16 * c + k] : 0.0f);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[i & 1]);
      }
    }
  }
  pdl_trigger();
  cluster_wait();
  if (warp >= 2) {
    const uint32_t at = (uint32_t)(rank * kUnit + (kEpi == kEpiGlu ? 32 * (wq >> 1) : 0) + lane) * 16u;
    int slot = 0, owner = wq & (kPer - 1);          // of unit kPer * (token / 4) + this warp's rows
    // this lane's row and tokens c0.. of the finished sums, to where they are added up
    auto give = [&](int c0, const uint32_t* d) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        if (c0 + i < b.M) {
          if (push) {
            while (owner >= S) { owner -= S; ++slot; }
            st_cluster4(tc::mapa(parts, (uint32_t)owner) + (uint32_t)(slot * S * kUnit * 16) + at, d + i);
            owner += kPer;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts32(smem_u32(parts) + (uint32_t)(((c0 + i + k) * 128 + 32 * wq + lane) * 4), d[i + k]);
          }
        }
      }
    };
    if constexpr (kPieces) {
      if (whole) {
#pragma unroll
        for (int c = 0; c < kRowsTokens / 16; ++c) {
          if (16 * c < b.M) {
            uint32_t d[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) d[k] = __float_as_uint(sum[16 * c + k]);
            give(16 * c, d);
          }
        }
      }
    } else {
      const bool ok = tc::wait_bounded(&acc_full[0], 0, abort);
      if (__all_sync(0xFFFFFFFFu, ok)) {  // the sums are complete
        tc::fence_after_sync();
        for (int c0 = 0; c0 < b.M; c0 += 16) {
          uint32_t d[32];
          tc::ld_16cols(row0 + c0, d);
          tc::wait_ld();
          give(c0, d);
        }
      }
    }
  }
  if (warp == 1) mbar_wait(&drain, 0);  // no MMA runs past the CTA's exit, also when a wait gave up
  __syncwarp();
  tc::fence_before_sync();
  cluster_arrive();
  // pushed: this CTA's units (unit u is CTA u % S's), one a warp and turn; the
  // first one's inputs before the wait
  const int units = push ? (b.M + 3) / 4 * kPer : 0;
  const int first = rank + S * warp, step = S * (kRowsThreads / 32);
  auto inputs = [&](int u, float& bias, float (&res)[4]) {
    const int t = u / kPer * 4, c = n0 + 32 * (u % kPer) + lane;
    const bool on = kEpi == kEpiLinear && u < units && c < b.N;
    bias = on && a.bias ? load16(a.f16, a.bias, (size_t)c) : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      res[k] = on && a.residual && t + k < b.M ? load16(a.f16, a.residual, (size_t)(t + k) * a.ldr + c) : 0.0f;
  };
  float bias, res[4];
  inputs(first, bias, res);
  cluster_wait();
  if (!push) finish_kept<kEpi>(a, reinterpret_cast<const float*>(parts), n0, rank, S, warp, lane);
  for (int u = first; u < units; u += step) {
    const int t = u / kPer * 4, c = n0 + 32 * (u % kPer) + lane;
    const float4* part = parts + (size_t)(u / S) * S * kUnit + lane;
    float v[4], up[4];
    sum_pushed(part, S, kUnit, v);
    if (kEpi == kEpiGlu) sum_pushed(part + 32, S, kUnit, up);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t + k >= b.M) break;                      // the same in every lane
      const bool on = c < b.N;
      const size_t o = (size_t)(t + k) * b.N + c;
      if (kEpi == kEpiDGlu) {
        if (on) {
          const float g[1] = {saved1(a, a.g, a.g_s, t + k, c)};
          const float u = saved1(a, a.u, a.u_s, t + k, c);
          float f[1], d[1];
          fn_slopes(a.fn, g, f, d);
          store16(b.out[0], o, a.f16, v[k] * u * d[0]);
          store16(b.out[1], o, a.f16, v[k] * f[0]);
          store16(a.pre, o, a.f16, f[0] * u);
        }
      } else if (kEpi == kEpiGlu) {
        if (a.g && a.saved8) {
          store_lanes8(a, a.g, a.g_s, t + k, c, v[k], on, lane);
          store_lanes8(a, a.u, a.u_s, t + k, c, up[k], on, lane);
        }
        if (on) {
          if (a.g && !a.saved8) {
            store16(a.g, o, a.f16, v[k]);
            store16(a.u, o, a.f16, up[k]);
          }
          float h[1] = {v[k]};
          fn_values(a.fn, h);
          store16(b.out[0], o, a.f16, h[0] * up[k]);
        }
      } else {
        float z[1] = {v[k] + bias};
        if (on && a.pre) store16(a.pre, o, a.f16, z[0]);
        fn_values(a.fn, z);
        const float y = z[0] + res[k];
        if (on) {
          if (a.out_f32) static_cast<float*>(b.out[0])[(size_t)(t + k) * b.ldo + c] = y;
          else store16(b.out[0], (size_t)(t + k) * b.ldo + c, a.f16, y);
        }
      }
    }
    if (kEpi == kEpiLinear) inputs(u + step, bias, res);
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort) {
    atomicOr(a.status, kStatusWaitTimeout);
    tc::drain_copies(full, nst, issued);
  }
  __syncwarp();
  if (!push) {                          // the other CTAs fetch this one's sums
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, tcols);
  }
}

template __global__ void k_dense_rows<kEpiLinear, false, false>(const __grid_constant__ DenseRowsArgs);
template __global__ void k_dense_rows<kEpiGlu, false, false>(const __grid_constant__ DenseRowsArgs);
template __global__ void k_dense_rows<kEpiGlu, false, true>(const __grid_constant__ DenseRowsArgs);
template __global__ void k_dense_rows<kEpiLinear, true, false>(const __grid_constant__ DenseRowsArgs);
template __global__ void k_dense_rows<kEpiDGlu, true, false>(const __grid_constant__ DenseRowsArgs);

}  // namespace moe
