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
// Every wait on a barrier in shared memory is bounded; one that gives up raises
// the CTA's abort flag and the status word, and the CTA's own copies and MMAs
// are waited for before it exits. (Cluster barriers and the allocation of tensor
// memory have no bound: every CTA comes to them, whether it gave up or not.)
#include <type_traits>

#include "dense.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;                       // two per 32-row quarter of the accumulator
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxStages = 10;
constexpr int kATile = 128 * 128;                  // 128 rows x 64 elements of 16 bits
constexpr int kRing = 192 * 1024;
constexpr int kGroupM = 8;                         // row tiles that share their column tiles in L2

struct Tile {
  int prob, seg, m0, n0;
};
// f(a_mn, b_mn) as compile-time constants: the directions that the launches use
template <int kEpi, typename F>
MOE_DEV void by_direction(const DenseProblem& p, F&& f) {
  using K = std::false_type;
  using MN = std::true_type;
  if constexpr (kEpi == kEpiGlu) f(K(), K());
  else if constexpr (kEpi == kEpiDGlu) f(K(), MN());
  else if (p.a_mn) f(MN(), MN());
  else if (p.b_mn) f(K(), MN());
  else f(K(), K());
}
// 64-k stages of a tile, its contraction segments one after the other
MOE_DEV int stages_of(const DenseProblem& p) { return (p.K + 63) / 64 * p.k_segs; }

}  // namespace

// --- epilogue of one warp: 32 rows x 32 columns at a time ------------------------
// A lane holds one row of the accumulator, but global rows are read and
// written with neighbouring lanes on neighbouring 16 bytes (8 rows x 64 bytes
// an instruction, whole sectors), and change hands in the warp's 4 KB of
// shared memory: two buffers of 32 rows x 64 bytes, or one of 32 x 128. The
// inputs of the next 32 columns are on their way while these are worked on
// (with each lane on its own row and no look-ahead, 4096 x 8192 x 2048 with a
// bias and a residual took 147 us, without them 106).
struct EpiPos {
  int row, col;             // first row and column of the 32 x 32 block
  int M, N;                 // the problem's extents
};
struct EpiIn {
  uint4 a[4], b[4];         // kEpiLinear: residual, bias; kEpiDGlu: g, u
  float sa, sb;             // kEpiDGlu: scales of this lane's row (8-bit)
};

// shared address of 16-byte chunk c of row r, rows of 64 (c < 4) or 128 (c < 8)
// bytes: both ways round without bank conflicts
MOE_DEV uint32_t stage64(uint32_t buf, int r, int c) { return buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }
MOE_DEV uint32_t stage128(uint32_t buf, int r, int c) { return buf + r * 128 + ((c ^ (r & 7)) << 4); }
// 8-byte chunk c of row r, rows of 32 bytes
MOE_DEV uint32_t stage32(uint32_t buf, int r, int c) { return buf + r * 32 + ((c ^ ((r >> 2) & 3)) << 3); }
MOE_DEV uint2 lds8b(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
MOE_DEV void sts8b(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};\n" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// this lane's pieces of the block's rows in global memory: row 8 i + lane / 4, columns 8 (lane % 4)..
MOE_DEV bool piece(const DenseGemmArgs& a, const EpiPos& e, int i, int lane, int& r, int& c) {
  r = e.row + 8 * i + (lane >> 2);
  c = e.col + 8 * (lane & 3);
  return r < e.M && c < e.N;
}
MOE_DEV void fetch16(const DenseGemmArgs& a, const EpiPos& e, const void* base, int64_t ld, int lane, uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int r, c;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (piece(a, e, i, lane, r, c))
      v[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + (size_t)r * ld + c);
  }
}
MOE_DEV void fetch8(const DenseGemmArgs& a, const EpiPos& e, const void* base, int lane, uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int r, c;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (piece(a, e, i, lane, r, c)) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + (size_t)r * e.N + c));
      v[i].x = w.x;
      v[i].y = w.y;
    }
  }
}
// pieces -> buffer
MOE_DEV void pieces_to_stage(uint32_t buf, int lane, const uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sts16(stage64(buf, 8 * i + (lane >> 2), lane & 3), v[i]);
}
MOE_DEV void pieces8_to_stage(uint32_t buf, int lane, const uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sts8b(stage32(buf, 8 * i + (lane >> 2), lane & 3), make_uint2(v[i].x, v[i].y));
}
// buffer (this lane's row in it, rounded to 16 bits) -> global rows
MOE_DEV void row_to_stage(uint32_t buf, int lane, int f16, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) sts16(stage64(buf, lane, j), pack16x8(f16, v + 8 * j));
}
MOE_DEV void flush16(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, void* base, int64_t ld) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int r, c;
    if (piece(a, e, i, lane, r, c))
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + (size_t)r * ld + c) =
          lds16(stage64(buf, 8 * i + (lane >> 2), lane & 3));
  }
}
MOE_DEV void put16(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, const float (&v)[32], void* base,
                   int64_t ld) {
  __syncwarp();
  row_to_stage(buf, lane, a.f16, v);
  __syncwarp();
  flush16(a, e, buf, lane, base, ld);
}
MOE_DEV void put32(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, const float (&v)[32], void* base,
                   int64_t ld) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts16(stage128(buf, lane, j), make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                             __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = e.col + 4 * (lane & 7);
    if (e.row + r < e.M && c < e.N)
      *reinterpret_cast<uint4*>(static_cast<float*>(base) + (size_t)(e.row + r) * ld + c) =
          lds16(stage128(buf, r, lane & 7));
  }
}
// this lane's row as one block of an 8-bit checkpoint (columns past N are zeros)
MOE_DEV void put8(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, const float (&v)[32], void* q,
                  uint8_t* s) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t code = e4m3_scale_code(m);
  const float inv = e4m3_inv_scale(code);
  if (e.row + lane < e.M && e.col < e.N) s[(size_t)(e.row + lane) * ((e.N + 31) / 32) + e.col / 32] = (uint8_t)code;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    sts8b(stage32(buf, lane, j), make_uint2(e4m3_quad(v + 8 * j, inv), e4m3_quad(v + 8 * j + 4, inv)));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int r, c;
    if (piece(a, e, i, lane, r, c))
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(q) + (size_t)r * e.N + c) =
          lds8b(stage32(buf, 8 * i + (lane >> 2), lane & 3));
  }
}

MOE_DEV void floats(const uint32_t (&d)[32], float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(d[i]);
}

template <int kEpi>
MOE_DEV void epi_fetch(const DenseGemmArgs& a, const EpiPos& e, int lane, EpiIn& in) {
  if (kEpi == kEpiLinear) {
    if (a.residual) fetch16(a, e, a.residual, a.ldr, lane, in.a);
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        in.b[j] = e.col + 8 * j < e.N ? ldg16(static_cast<const uint16_t*>(a.bias) + e.col + 8 * j)
                                      : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (kEpi == kEpiDGlu) {
    if (a.saved8) {
      fetch8(a, e, a.g, lane, in.a);
      fetch8(a, e, a.u, lane, in.b);
      in.sa = in.sb = 0.0f;
      if (e.row + lane < e.M && e.col < e.N) {
        const size_t so = (size_t)(e.row + lane) * ((e.N + 31) / 32) + e.col / 32;
        in.sa = e8m0_to_f32(__ldg(a.g_s + so));
        in.sb = e8m0_to_f32(__ldg(a.u_s + so));
      }
    } else {
      fetch16(a, e, a.g, e.N, lane, in.a);
      fetch16(a, e, a.u, e.N, lane, in.b);
    }
  }
}

MOE_DEV void epi_linear(const DenseGemmArgs& a, const DenseProblem& p, int seg, const EpiPos& e, uint32_t buf, int lane, const EpiIn& in,
                        float (&v)[32]) {
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float t[8];
      unpack16x8(a.f16, in.b[j], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * j + i] += t[i];
    }
  }
  if (a.pre) put16(a, e, buf, lane, v, a.pre, e.N);
  fn_values(a.fn, v);
  if (a.residual) {
    __syncwarp();
    pieces_to_stage(buf, lane, in.a);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float t[8];
      unpack16x8(a.f16, lds16(stage64(buf, lane, j)), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * j + i] += t[i];
    }
  }
  if (a.out_f32) put32(a, e, buf, lane, v, p.out[seg], p.ldo);
  else put16(a, e, buf, lane, v, p.out[seg], p.ldo);
}

MOE_DEV void epi_glu(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, float (&g)[32], float (&u)[32]) {
  if (a.g) {
    if (a.saved8) {
      put8(a, e, buf, lane, g, a.g, a.g_s);
      put8(a, e, buf + 2048, lane, u, a.u, a.u_s);
    } else {
      put16(a, e, buf, lane, g, a.g, e.N);
      put16(a, e, buf + 2048, lane, u, a.u, e.N);
    }
  }
  fn_values(a.fn, g);
#pragma unroll
  for (int i = 0; i < 32; ++i) g[i] *= u[i];
  put16(a, e, buf, lane, g, a.p[0].out[0], e.N);
}

MOE_DEV void epi_dglu(const DenseGemmArgs& a, const EpiPos& e, uint32_t buf, int lane, const EpiIn& in,
                      float (&dh)[32]) {
  const uint32_t ga = buf, ua = buf + 2048;
  __syncwarp();
  if (a.saved8) {
    pieces8_to_stage(ga, lane, in.a);
    pieces8_to_stage(ua, lane, in.b);
  } else {
    pieces_to_stage(ga, lane, in.a);
    pieces_to_stage(ua, lane, in.b);
  }
  __syncwarp();
  uint4 gq[4], uq[4], hq[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float g[8], u[8], f[8], s[8], x[8], y[8], h[8];
    if (a.saved8) {
      const uint2 p = lds8b(stage32(ga, lane, j)), q = lds8b(stage32(ua, lane, j));
      e4m3_unquad(p.x, in.sa, g);
      e4m3_unquad(p.y, in.sa, g + 4);
      e4m3_unquad(q.x, in.sb, u);
      e4m3_unquad(q.y, in.sb, u + 4);
    } else {
      unpack16x8(a.f16, lds16(stage64(ga, lane, j)), g);
      unpack16x8(a.f16, lds16(stage64(ua, lane, j)), u);
    }
    fn_slopes(a.fn, g, f, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = dh[8 * j + i] * u[i] * s[i];
      y[i] = dh[8 * j + i] * f[i];
      h[i] = f[i] * u[i];
    }
    gq[j] = pack16x8(a.f16, x);
    uq[j] = pack16x8(a.f16, y);
    hq[j] = pack16x8(a.f16, h);
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sts16(stage64(ga, lane, j), gq[j]);
    sts16(stage64(ua, lane, j), uq[j]);
  }
  __syncwarp();
  flush16(a, e, ga, lane, a.p[0].out[0], e.N);
  flush16(a, e, ua, lane, a.p[0].out[1], e.N);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) sts16(stage64(ga, lane, j), hq[j]);
  __syncwarp();
  flush16(a, e, ga, lane, a.pre, e.N);
}

template <int kEpi, int kCg, bool kPieces>
__global__ void __launch_bounds__(kThreads, 1) k_dense_gemm(const __grid_constant__ DenseGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ long issued;
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
    for (int i = 0; i < a.problems; ++i) {
      tc::prefetch_map(&a.p[i].map_a[0]);
      tc::prefetch_map(&a.p[i].map_b[0]);
    }
  }
  if (warp == 1) tc::alloc_cg<kCg>(&tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  if (kCg > 1) tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;
  pdl_wait();
  pdl_trigger();

  // this CTA's (pair's) tiles
  const int slot = (int)blockIdx.x / kCg, slots = (int)gridDim.x / kCg;
  int q0 = slot, q1 = a.tiles, dq = slots;
  if (a.balanced) {
    long total = 0;
    for (int i = 0; i < a.problems; ++i) {
      const int end = i + 1 < a.problems ? a.p[i + 1].first : a.tiles;
      total += (long)(end - a.p[i].first) * stages_of(a.p[i]);
    }
    auto start = [&](int s) {           // the first tile whose stages begin at or after share s
      long w = (total * s + slots - 1) / slots;
      for (int i = 0; i < a.problems; ++i) {
        const int end = i + 1 < a.problems ? a.p[i + 1].first : a.tiles, ks = stages_of(a.p[i]);
        const long all = (long)(end - a.p[i].first) * ks;
        if (w < all) return a.p[i].first + (int)((w + ks - 1) / ks);
        w -= all;
      }
      return a.tiles;
    };
    q0 = start(slot);
    q1 = start(slot + 1);
    dq = 1;
  }
  // groups of kGroupM row tiles; in a group the row tiles of one column tile follow each other
  auto tile_of = [&](int q) {
    Tile t;
    t.prob = 0;
    while (t.prob + 1 < a.problems && q >= a.p[t.prob + 1].first) ++t.prob;
    const DenseProblem& p = a.p[t.prob];
    q -= p.first;
    const int mt1 = (p.M + 128 * kCg - 1) / (128 * kCg), mt = mt1 * p.m_segs, nt = (p.N + cols - 1) / cols;
    const int per = kGroupM * nt;
    const int grp = q / per, r = q - grp * per;
    const int gm = min(kGroupM, mt - grp * kGroupM);
    const int n = r / gm, m = grp * kGroupM + r - n * gm;
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
      long n = 0;
      bool ok = true;
      for (int q = q0; q < q1 && ok; q += dq) {
        const Tile t = tile_of(q);
        const DenseProblem& p = a.p[t.prob];
        const int ks1 = (p.K + 63) / 64, ks = ks1 * p.k_segs;
        auto fill = [&](auto a_mn, auto b_mn) {       // by direction, so the loop has no branches
          for (int j = 0; j < ks; ++j) {
            if (!tc::wait_bounded(&empty[s], ph ^ 1u, abort)) { ok = false; break; }
            uint8_t* sa = smem + s * stage_bytes;
            uint8_t* sb = sa + kATile;
            const int kseg = j >= ks1 ? 1 : 0;
            const int k0 = (j - kseg * ks1) * 64;
            const CUtensorMap* ma = &p.map_a[p.m_segs > 1 ? t.seg : kseg];
            const CUtensorMap* mb = &p.map_b[kseg];
            if (rank == 0) mbar_expect_tx(&full[s], (uint32_t)(stage_bytes * kCg));
            auto load = [&](uint8_t* dst, const CUtensorMap* m, int x, int y) {
              if (kCg == 1) tc::tma_load_2d(dst, m, x, y, &full[s]);
              else tc::tma_load_2d_pair(dst, m, x, y, tc::mapa(&full[s], 0));
            };
            if constexpr (a_mn) {
              load(sa, ma, t.m0, k0);
              load(sa + 8192, ma, t.m0 + 64, k0);
            } else {
              load(sa, ma, k0, t.m0);
            }
            if constexpr (kEpi == kEpiGlu) {
              if (kCg == 1) {
                load(sb, &p.map_b[0], k0, t.n0);
                load(sb + cols * 128, &p.map_b[1], k0, t.n0);
              } else {
                load(sb, &p.map_b[rank], k0, t.n0);
              }
            } else if constexpr (b_mn) {
              for (int i = 0; i < bn / 64; ++i) load(sb + i * 8192, mb, t.n0 + (int)rank * bn + 64 * i, k0);
            } else {
              load(sb, mb, k0, t.n0 + (int)rank * bn);
            }
            ++n;
            if (++s == nst) { s = 0; ph ^= 1u; }
          }
        };
        by_direction<kEpi>(p, fill);
      }
      issued = n;
      // every stage handed back: no arrival of the pair's MMAs is left to come
      for (int i = 0; i < nst && ok; ++i) {
        ok = tc::wait_bounded(&empty[s], ph ^ 1u, abort);
        if (++s == nst) { s = 0; ph ^= 1u; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // the whole loop in one elected thread
    if (rank == 0 && tc::elect_one()) {
      int s = 0, n_it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int q = q0; q < q1 && ok; q += dq) {
        const DenseProblem& p = a.p[tile_of(q).prob];
        const int ks = stages_of(p);
        auto issue = [&](auto a_mn, auto b_mn) {
          const uint32_t idesc = tc::idesc_16(a.f16, 128 * kCg, tn, a_mn, b_mn);
          constexpr uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
          const int pieces = kPieces ? pieces_of(ks) : 1;
          for (int i = 0; i < pieces && ok; ++i, ++n_it) {
            const int buf = n_it & 1;
            const int j0 = kPieces ? ks * i / pieces : 0, j1 = kPieces ? ks * (i + 1) / pieces : ks;
            if (!tc::wait_bounded<(kCg > 1)>(&acc_empty[buf], (uint32_t)((n_it >> 1) & 1) ^ 1u, abort)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const uint32_t d = tbase + 256u * buf;
            for (int j = j0; j < j1; ++j) {
              if (!tc::wait_bounded(&full[s], ph, abort)) { ok = false; break; }
              const uint32_t sa = smem_u32(smem + s * stage_bytes), sb = sa + kATile;
              const uint64_t da = a_mn ? tc::desc_mn_sw128(sa, 8192) : tc::desc_sw128(sa);
              const uint64_t db = b_mn ? tc::desc_mn_sw128(sb, 8192) : tc::desc_sw128(sb);
#pragma unroll
              for (int kb = 0; kb < 4; ++kb)                  // K = 16 per MMA
                tc::mma_16<kCg>(d, da + kb * a_step, db + kb * b_step, idesc, (j > j0 || kb > 0) ? 1u : 0u);
              tc::commit_cg<kCg>(&empty[s]);
              if (j == j1 - 1) tc::commit_cg<kCg>(&acc_full[buf]);
              if (++s == nst) { s = 0; ph ^= 1u; }
            }
          }
        };
        by_direction<kEpi>(p, issue);
      }
      tc::commit_cg<kCg>(&drain);
    }
    __syncwarp();
    // no MMA runs past the CTA's exit, also when a wait gave up (the pair's second
    // CTA looks when its epilogue is through, not all the while)
    if (rank == 0) mbar_wait(&drain, 0);
  } else {
    // ---------------- epilogue (warps 2-9) ----------------
    // two warps share a quarter's 32 rows: 32-column chunks in turn
    const int wq = warp & 3, cfirst = 32 * ((warp - 2) >> 2);
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    const uint32_t stage = smem_u32(smem + kRing) + 4096u * (uint32_t)(warp - 2);
    int n_it = 0;
    // the accumulators of turn n_it are complete; they are handed back by release()
    auto ready = [&]() {
      const bool ok = tc::wait_bounded(&acc_full[n_it & 1], (uint32_t)((n_it >> 1) & 1), abort);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      tc::fence_after_sync();
      return true;
    };
    auto release = [&]() {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (kCg == 1) tc::mbar_arrive(&acc_empty[n_it & 1]);
        else tc::arrive_cluster(tc::mapa(&acc_empty[n_it & 1], 0));
      }
    };
    bool ok = true;
    for (int q = q0; q < q1 && ok; q += dq) {
      const Tile t = tile_of(q);
      const DenseProblem& p = a.p[t.prob];
      EpiPos e = {t.m0 + 32 * wq, t.n0 + cfirst, p.M, p.N};
      if constexpr (kPieces) {
        // this warp's columns, at most two blocks of 32, added up over the pieces
        float g[2][32], u[2][32];
        const int pieces = pieces_of(stages_of(p));
        for (int i = 0; i < pieces; ++i, ++n_it) {
          if (!(ok = ready())) break;
          const uint32_t dcol = tbase + lane_off + 256u * (n_it & 1);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int c0 = cfirst + 64 * c;
            if (c0 < cols) {
              uint32_t d[32], d2[32];
              tc::ld_32cols(dcol + c0, d);
              tc::ld_32cols(dcol + cols + c0, d2);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                g[c][k] = __uint_as_float(d[k]) + (i ? g[c][k] : 0.0f);
                u[c][k] = __uint_as_float(d2[k]) + (i ? u[c][k] : 0.0f);
              }
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (cfirst + 64 * c < cols) epi_glu(a, e, stage, lane, g[c], u[c]);
          e.col += 64;
        }
      } else {
        EpiIn in;
        if (cfirst < cols) epi_fetch<kEpi>(a, e, lane, in);
        if (!(ok = ready())) break;
        const uint32_t dcol = tbase + lane_off + 256u * (n_it & 1);
        if (cfirst >= cols) release();
        for (int c0 = cfirst; c0 < cols; c0 += 64) {
          uint32_t d[32], d2[32];
          tc::ld_32cols(dcol + c0, d);
          if (kEpi == kEpiGlu) tc::ld_32cols(dcol + cols + c0, d2);
          const EpiIn now = in;
          const EpiPos at = e;
          e.col += 64;
          if (kEpi != kEpiGlu && c0 + 64 < cols) epi_fetch<kEpi>(a, e, lane, in);
          tc::wait_ld();
          if (c0 + 64 >= cols) release();
          float v[32];
          floats(d, v);
          if (kEpi == kEpiGlu) {
            float u[32];
            floats(d2, u);
            epi_glu(a, at, stage, lane, v, u);
          } else if (kEpi == kEpiDGlu) {
            epi_dglu(a, at, stage, lane, now, v);
          } else {
            epi_linear(a, p, t.seg, at, stage, lane, now, v);
          }
        }
        ++n_it;
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) {
    atomicOr(a.status, kStatusWaitTimeout);
    // the second CTA's copies count on the first one's barriers: it gives its own
    // time to land by a barrier that nothing completes
    if (rank == 0) tc::drain_copies(full, nst, issued);
    else mbar_wait(&full[0], 0, 1u << 8);
  }
  if (rank != 0 && warp == 1) mbar_wait(&drain, 0);
  __syncwarp();
  if (kCg > 1) tc::cluster_sync();      // the pair's MMAs read both CTAs' memory
  if (warp == 1) {
    tc::fence_after_sync();
    tc::dealloc_cg<kCg>(tbase, 512);
  }
}

// --- small products ----------------------------------------------------------------
// One tile of 128 rows a cluster, whose CTAs divide its stages: for a product
// that leaves SMs idle in k_dense_gemm although its few tiles are long. Two
// CTAs fit an SM where there are more than SMs, so a CTA's start and epilogue
// run under its neighbour's products. The CTAs keep their fp32 sums in their
// own shared memory, over the ring; behind a cluster barrier the 32 x 32 blocks
// of the tile go to the cluster's warps, which add the CTAs' parts in rank
// order (the same bits every run) and run the epilogue above.
namespace {

constexpr int kSplitWarps = 4;                     // epilogue warps: two CTAs' registers fit an SM
constexpr int kSplitThreads = 64 + 32 * kSplitWarps;

MOE_DEV float4 ld_cluster16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// byte offset of 16-byte chunk c of row r in the sums [128][tn] (no bank conflicts down a column)
MOE_DEV uint32_t sum_at(int r, int c, int tn) { return (uint32_t)(r * tn * 4 + ((c ^ (r & 7)) << 4)); }
// the cluster's sums of a block (rows r0.., columns col..) in the epilogue's
// layout, one row a lane. Neighbouring lanes fetch neighbouring chunks (a lane
// on its own row made 32 requests of each load) and rows change hands in `buf`.
MOE_DEV void sum_block(const uint8_t* sums, int splits, int r0, int col, int tn, uint32_t buf, int lane,
                       float (&v)[32]) {
  const int r = lane >> 3, c = lane & 7;
  float4 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = 0; k < splits; ++k) {
    const uint32_t base = tc::mapa(sums, (uint32_t)k);
    float4 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ld_cluster16(base + sum_at(r0 + 4 * i + r, col / 4 + c, tn));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i].x += q[i].x;
      t[i].y += q[i].y;
      t[i].z += q[i].z;
      t[i].w += q[i].w;
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    sts16(stage128(buf, 4 * i + r, c), make_uint4(__float_as_uint(t[i].x), __float_as_uint(t[i].y),
                                                  __float_as_uint(t[i].z), __float_as_uint(t[i].w)));
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 w = lds16(stage128(buf, lane, j));
    v[4 * j] = __uint_as_float(w.x);
    v[4 * j + 1] = __uint_as_float(w.y);
    v[4 * j + 2] = __uint_as_float(w.z);
    v[4 * j + 3] = __uint_as_float(w.w);
  }
}

}  // namespace

template <int kEpi>
__global__ void __launch_bounds__(kSplitThreads, 2) k_dense_split(const __grid_constant__ DenseGemmArgs a, int splits, int nst) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kSplitStages], empty[kSplitStages], acc_full, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, issued;
  volatile int* abort = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tn = a.tile_n, cols = kEpi == kEpiGlu ? tn / 2 : tn;
  const int stage_bytes = kATile + tn * 128;
  const int rank = (int)blockIdx.x % splits, q = (int)blockIdx.x / splits;

  // the tile: column tiles of a row tile follow each other
  const DenseProblem& p = a.p[0];
  const int mt1 = (p.M + 127) / 128, nt = (p.N + cols - 1) / cols;
  const int m = q / nt, seg = m / mt1;
  const int m0 = (m - seg * mt1) * 128, n0 = (q - m * nt) * cols;
  const int ks1 = (p.K + 63) / 64, ks = ks1 * p.k_segs;
  const int j0 = (int)((long)ks * rank / splits), j1 = (int)((long)ks * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
    tc::prefetch_map(&p.map_a[p.m_segs > 1 ? seg : 0]);
    tc::prefetch_map(&p.map_b[0]);
  }
  if (warp == 1) tc::alloc_cg<1>(&tmem_slot, tn <= 64 ? 64u : 128u);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (tc::elect_one()) {
      int s = 0, n = 0;
      uint32_t ph = 0;
      auto fill = [&](auto a_mn, auto b_mn) {
        for (int j = j0; j < j1; ++j) {
          if (!tc::wait_bounded(&empty[s], ph ^ 1u, abort)) break;
          uint8_t* sa = smem + s * stage_bytes;
          uint8_t* sb = sa + kATile;
          const int kseg = j >= ks1 ? 1 : 0, k0 = (j - kseg * ks1) * 64;
          const CUtensorMap* ma = &p.map_a[p.m_segs > 1 ? seg : kseg];
          const CUtensorMap* mb = &p.map_b[kseg];
          mbar_expect_tx(&full[s], (uint32_t)stage_bytes);
          if constexpr (a_mn) {
            tc::tma_load_2d(sa, ma, m0, k0, &full[s]);
            tc::tma_load_2d(sa + 8192, ma, m0 + 64, k0, &full[s]);
          } else {
            tc::tma_load_2d(sa, ma, k0, m0, &full[s]);
          }
          if constexpr (kEpi == kEpiGlu) {
            tc::tma_load_2d(sb, &p.map_b[0], k0, n0, &full[s]);
            tc::tma_load_2d(sb + cols * 128, &p.map_b[1], k0, n0, &full[s]);
          } else if constexpr (b_mn) {
            for (int i = 0; i < tn / 64; ++i) tc::tma_load_2d(sb + i * 8192, mb, n0 + 64 * i, k0, &full[s]);
          } else {
            tc::tma_load_2d(sb, mb, k0, n0, &full[s]);
          }
          ++n;
          if (++s == nst) { s = 0; ph ^= 1u; }
        }
      };
      by_direction<kEpi>(p, fill);
      issued = n;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (tc::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      auto issue = [&](auto a_mn, auto b_mn) {
        const uint32_t idesc = tc::idesc_16(a.f16, 128, tn, a_mn, b_mn);
        constexpr uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
        for (int j = j0; j < j1; ++j) {
          if (!tc::wait_bounded(&full[s], ph, abort)) break;
          const uint32_t sa = smem_u32(smem + s * stage_bytes), sb = sa + kATile;
          const uint64_t da = a_mn ? tc::desc_mn_sw128(sa, 8192) : tc::desc_sw128(sa);
          const uint64_t db = b_mn ? tc::desc_mn_sw128(sb, 8192) : tc::desc_sw128(sb);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
            tc::mma_16<1>(tbase, da + kb * a_step, db + kb * b_step, idesc, (j > j0 || kb > 0) ? 1u : 0u);
          tc::commit_cg<1>(&empty[s]);
          if (++s == nst) { s = 0; ph ^= 1u; }
        }
      };
      by_direction<kEpi>(p, issue);
      tc::commit_cg<1>(&acc_full);
      tc::commit_cg<1>(&drain);
    }
    __syncwarp();
    mbar_wait(&drain, 0);               // no MMA runs past the CTA's exit, also when a wait gave up
  } else {
    // ---------------- this CTA's sums, over the ring (warps 2-5) ----------------
    const int wq = warp & 3;
    const bool ok = tc::wait_bounded(&acc_full, 0, abort);
    if (__all_sync(0xFFFFFFFFu, ok)) {
      tc::fence_after_sync();
      for (int c0 = 0; c0 < tn; c0 += 32) {
        uint32_t d[32];
        tc::ld_32cols(tbase + ((uint32_t)(32 * wq) << 16) + c0, d);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sts16(smem_u32(smem) + sum_at(32 * wq + lane, c0 / 4 + j, tn),
                make_uint4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]));
      }
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  tc::cluster_sync();
  if (warp >= 2) {
    // ---------------- the tile's 32 x 32 blocks, dealt to the cluster's warps ----------------
    const uint32_t stage = smem_u32(smem + 128 * tn * 4) + 4096u * (uint32_t)(warp - 2);
    const int blocks = 4 * (cols / 32);
    for (int b = rank + splits * (warp - 2); b < blocks; b += splits * kSplitWarps) {
      const int r0 = 32 * (b & 3), c0 = 32 * (b >> 2);
      const EpiPos e = {m0 + r0, n0 + c0, p.M, p.N};
      if (e.row >= p.M || e.col >= p.N) continue;
      EpiIn in;
      epi_fetch<kEpi>(a, e, lane, in);
      float v[32];
      sum_block(smem, splits, r0, c0, tn, stage, lane, v);
      if constexpr (kEpi == kEpiGlu) {
        float u[32];
        sum_block(smem, splits, r0, cols + c0, tn, stage, lane, u);
        epi_glu(a, e, stage, lane, v, u);
      } else if constexpr (kEpi == kEpiDGlu) {
        epi_dglu(a, e, stage, lane, in, v);
      } else {
        epi_linear(a, p, seg, e, stage, lane, in, v);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort) {
    atomicOr(a.status, kStatusWaitTimeout);
    tc::drain_copies(full, nst, issued);
  }
  __syncwarp();
  tc::cluster_sync();                   // the other CTAs read this one's sums
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, tn <= 64 ? 64u : 128u);
  }
}

template __global__ void k_dense_split<kEpiLinear>(const __grid_constant__ DenseGemmArgs, int, int);
template __global__ void k_dense_split<kEpiGlu>(const __grid_constant__ DenseGemmArgs, int, int);
template __global__ void k_dense_split<kEpiDGlu>(const __grid_constant__ DenseGemmArgs, int, int);
int dense_split_threads() { return kSplitThreads; }

template __global__ void k_dense_gemm<kEpiLinear, 1, false>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, 1, false>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, 1, true>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiDGlu, 1, false>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiLinear, 2, false>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, 2, false>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiGlu, 2, true>(const __grid_constant__ DenseGemmArgs);
template __global__ void k_dense_gemm<kEpiDGlu, 2, false>(const __grid_constant__ DenseGemmArgs);

size_t dense_gemm_smem_bytes() { return kRing + 4096 * kEpiWarps + 1024; }
int dense_gemm_threads() { return kThreads; }

}  // namespace moe
