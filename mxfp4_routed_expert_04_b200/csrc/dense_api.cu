// C ABI of the dense operators: validation, workspace plan, launch order.
// Declared in include/moe_mxfp4.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>
#include <utility>

#include "../../include/moe_mxfp4.h"
#include "dense.h"
#include "kernels.h"

namespace {

moe_status fail(moe_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return moe::record_error(s, msg);
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
char* at(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

#define NEED(p)                                                                         \
  do {                                                                                  \
    if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);                       \
    if (!aligned16(p)) return fail(MOE_ERR_ALIGNMENT, "%s is not 16-byte aligned", #p); \
  } while (0)
#define MAYBE(p)                                                                        \
  do {                                                                                  \
    if (!aligned16(p)) return fail(MOE_ERR_ALIGNMENT, "%s is not 16-byte aligned", #p); \
  } while (0)
#define TRY(e)                         \
  do {                                 \
    const moe_status s_ = (e);         \
    if (s_ != MOE_OK) return s_;       \
  } while (0)

constexpr size_t kStatusBytes = 256;
constexpr long kSmallWeights = 1 << 18;

moe_status check_width(const char* name, int v) {
  if (v < 8 || v > 65536 || v % 8 != 0)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s=%d is not a multiple of 8 in [8, 65536]", name, v);
  return MOE_OK;
}
moe_status check_common(int T, int fn, int dtype, int out_f32) {
  if (T < 1 || T > 65536) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d outside [1, 65536]", T);
  if (fn < MOE_FN_NONE || fn > MOE_FN_RELU) return fail(MOE_ERR_INVALID_ARG, "fn %d is not a moe_fn", fn);
  if (dtype != MOE_BF16 && dtype != MOE_F16) return fail(MOE_ERR_INVALID_ARG, "dtype %d is not a moe_dtype", dtype);
  if (out_f32 != 0 && out_f32 != 1) return fail(MOE_ERR_INVALID_ARG, "out_f32 %d is not 0 or 1", out_f32);
  return MOE_OK;
}
// a row pitch (0: packed) into *out
moe_status check_pitch(const char* name, int64_t ld, int cols, int64_t* out) {
  if (ld == 0) ld = cols;
  if (ld < cols || ld % 8 != 0 || ld >= ((int64_t)1 << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s=%lld is not a multiple of 8 in [%d, 2^31)", name, (long long)ld, cols);
  *out = ld;
  return MOE_OK;
}
moe_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned16(ws)) return fail(MOE_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, need);
  return MOE_OK;
}

moe_status launched(cudaError_t e, const char* what) {
  const cudaError_t last = cudaGetLastError();
  if (e == cudaSuccess) e = last;
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MOE_OK;
}

// --- overlap ------------------------------------------------------------------
// A buffer as the bytes that a call touches: rows of `width` bytes, `pitch` apart.
struct Span {
  const char* name;
  uintptr_t p;
  size_t rows, width, pitch;
};
// whether they share a byte, exactly (slices of one buffer, side by side, do not)
bool overlap(Span a, Span b) {
  if (b.p < a.p) std::swap(a, b);
  if (b.p >= a.p + (a.rows - 1) * a.pitch + a.width) return false;
  size_t i = (b.p - a.p) / a.pitch, j = 0;
  if (a.pitch == b.pitch) {             // b's rows start in the same place of each of a's
    const size_t d = b.p - a.p - i * a.pitch;
    return d < a.width || d + b.width > a.pitch;
  }
  while (i < a.rows && j < b.rows) {    // both in order of address
    const uintptr_t x = a.p + i * a.pitch, y = b.p + j * b.pitch;
    if (x < y + b.width && y < x + a.width) return true;
    if (x < y) ++i;
    else ++j;
  }
  return false;
}
// The buffers of a call. CTAs write their outputs while others still read, so an
// output may share no byte with what the call reads, nor with another output.
class Spans {
 public:
  void in(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t bytes) {
    add(in_, n_in_, name, p, rows, cols, ld, bytes);
  }
  void out(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t bytes) {
    add(out_, n_out_, name, p, rows, cols, ld, bytes);
  }
  // an input that the first output may lie on
  void free_in(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t bytes) {
    add(free_, n_free_, name, p, rows, cols, ld, bytes);
  }
  moe_status check() const {
    for (int o = 0; o < n_out_; ++o) {
      for (int k = o + 1; k < n_out_; ++k) TRY(pair(out_[o], out_[k]));
      for (int k = 0; k < n_in_; ++k) TRY(pair(out_[o], in_[k]));
      for (int k = 0; k < n_free_ && o > 0; ++k) TRY(pair(out_[o], free_[k]));
    }
    return MOE_OK;
  }

 private:
  static constexpr int kMost = 10;      // the inputs of moe_ffn_backward from 8 bits
  Span in_[kMost], out_[kMost], free_[2];
  int n_in_ = 0, n_out_ = 0, n_free_ = 0;

  static void add(Span* to, int& n, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld,
                  size_t bytes) {
    if (!p) return;
    if (ld == cols || rows == 1) {      // packed: one row
      cols *= rows;
      ld = cols;
      rows = 1;
    }
    to[n++] = {name, reinterpret_cast<uintptr_t>(p), (size_t)rows, (size_t)cols * bytes, (size_t)ld * bytes};
  }
  static moe_status pair(const Span& a, const Span& b) {
    if (overlap(a, b)) return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
    return MOE_OK;
  }
};

// --- plans --------------------------------------------------------------------

struct LinearPlan {
  int T, N, K, fn, f16, out_f32;
  int64_t ldx, ldy, ldr;
  int dz_rows, dz_chunks;       // row chunks of the bias gradient's partial sums
  size_t off_dz, off_part, total;
};
// rows of a bias-gradient chunk: all of few tokens (no second kernel), else at
// most 128 chunks of at least 16 rows
int dz_chunk_rows(int T) { return T <= 64 ? T : std::max(16, (T + 127) / 128); }

moe_status make_plan(const moe_linear_dims* d, LinearPlan& p) {
  if (!d) return fail(MOE_ERR_INVALID_ARG, "dims is NULL");
  TRY(check_common(d->T, d->fn, d->dtype, d->out_f32));
  TRY(check_width("N", d->N));
  TRY(check_width("K", d->K));
  p.T = d->T; p.N = d->N; p.K = d->K; p.fn = d->fn; p.f16 = d->dtype; p.out_f32 = d->out_f32;
  TRY(check_pitch("ldx", d->ldx, d->K, &p.ldx));
  TRY(check_pitch("ldy", d->ldy, d->N, &p.ldy));
  TRY(check_pitch("ldr", d->ldr, d->N, &p.ldr));
  p.dz_rows = dz_chunk_rows(p.T);
  p.dz_chunks = (p.T + p.dz_rows - 1) / p.dz_rows;
  size_t o = kStatusBytes;
  p.off_dz = o;
  o = align_up(o + (p.fn ? (size_t)p.T * p.N * 2 : 0), 256);
  p.off_part = o;
  o = align_up(o + (size_t)p.dz_chunks * p.N * 4, 256);
  p.total = o;
  return MOE_OK;
}

struct FfnPlan {
  int T, H, I, fn, f16, save, out_f32;
  int64_t ldx, ldy, ldr;
  size_t off_h, off_dg, off_du, off_x, total;
};

moe_status make_plan(const moe_ffn_dims* d, FfnPlan& p) {
  if (!d) return fail(MOE_ERR_INVALID_ARG, "dims is NULL");
  TRY(check_common(d->T, d->fn, d->dtype, d->out_f32));
  TRY(check_width("H", d->H));
  TRY(check_width("I", d->I));
  if (d->save < MOE_SAVE_NONE || d->save > MOE_SAVE_8)
    return fail(MOE_ERR_INVALID_ARG, "save %d is not a moe_save", d->save);
  if (d->reserved != 0) return fail(MOE_ERR_INVALID_ARG, "reserved is not 0");
  p.T = d->T; p.H = d->H; p.I = d->I; p.fn = d->fn; p.f16 = d->dtype; p.save = d->save; p.out_f32 = d->out_f32;
  TRY(check_pitch("ldx", d->ldx, d->H, &p.ldx));
  TRY(check_pitch("ldy", d->ldy, d->H, &p.ldy));
  TRY(check_pitch("ldr", d->ldr, d->H, &p.ldr));
  const size_t hidden = align_up((size_t)p.T * p.I * 2, 256);
  size_t o = kStatusBytes;
  p.off_h = o;
  o += hidden;
  p.off_dg = o;
  if (p.save != MOE_SAVE_NONE) o += hidden;
  p.off_du = o;
  if (p.save != MOE_SAVE_NONE) o += hidden;
  p.off_x = o;
  if (p.save == MOE_SAVE_8) o += align_up((size_t)p.T * p.H * 2, 256);
  p.total = o;
  return MOE_OK;
}

// --- device ----------------------------------------------------------------------

struct Device {
  bool ready = false;
  int num_sms = 0;
  // clusters of s CTAs that run at once with an SM for each CTA (the SMs of a GPC
  // are not a multiple of every s: 45 of 3, 33 of 4, 15 of 8). The occupancy
  // query counts one CTA an SM for kernels with tensor memory whatever they
  // take; where memory and registers leave room for two, two run (seen from
  // their SM numbers and times), so twice as many clusters.
  int clusters[moe::kMaxSplits + 1] = {};
};
std::mutex g_mu;
Device g_dev[64];

template <int kEpi>
cudaError_t allow_split() {
  return cudaFuncSetAttribute(moe::k_dense_split<kEpi>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              moe::kSplitRingAlone + 1024);
}
template <int kEpi, bool kPieces = false>
cudaError_t allow_smem() {
  const int bytes = (int)moe::dense_gemm_smem_bytes();
  const cudaError_t e = cudaFuncSetAttribute(moe::k_dense_gemm<kEpi, 1, kPieces>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(moe::k_dense_gemm<kEpi, 2, kPieces>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int kEpi, bool kWMn, bool kPieces = false>
cudaError_t allow_rows() {
  return cudaFuncSetAttribute(moe::k_dense_rows<kEpi, kWMn, kPieces>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)moe::dense_rows_smem_bytes());
}
template <typename K>
cudaError_t resident(K kernel, int threads, size_t smem, int (&out)[moe::kMaxSplits + 1]) {
  for (int s = 2; s <= moe::kMaxSplits; ++s) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = s;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&out[s], kernel, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

moe_status device(const Device** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(MOE_ERR_CUDA, "cudaGetDevice failed");
  std::lock_guard<std::mutex> lk(g_mu);
  Device& s = g_dev[dev];
  if (!s.ready) {
    cudaError_t e = cudaDeviceGetAttribute(&s.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = allow_smem<moe::kEpiLinear>();
    if (e == cudaSuccess) e = allow_smem<moe::kEpiGlu>();
    if (e == cudaSuccess) e = allow_split<moe::kEpiLinear>();
    if (e == cudaSuccess) e = allow_split<moe::kEpiGlu>();
    if (e == cudaSuccess) e = allow_split<moe::kEpiDGlu>();
    if (e == cudaSuccess) e = allow_smem<moe::kEpiGlu, true>();
    if (e == cudaSuccess) e = allow_smem<moe::kEpiDGlu>();
    if (e == cudaSuccess) e = allow_rows<moe::kEpiLinear, false>();
    if (e == cudaSuccess) e = allow_rows<moe::kEpiGlu, false>();
    if (e == cudaSuccess) e = allow_rows<moe::kEpiGlu, false, true>();
    if (e == cudaSuccess) e = allow_rows<moe::kEpiLinear, true>();
    if (e == cudaSuccess) e = allow_rows<moe::kEpiDGlu, true>();
    if (e == cudaSuccess)
      e = resident(moe::k_dense_split<moe::kEpiLinear>, moe::dense_split_threads(), moe::kSplitRingAlone + 1024,
                   s.clusters);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "device setup: %s", cudaGetErrorString(e));
    s.ready = true;
  }
  *out = &s;
  return MOE_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// 16-bit matrix [rows, cols] with row pitch ld, read in boxes of box_rows rows
// x 64 elements with the 128-byte swizzle
moe_status map16(CUtensorMap* m, const void* base, int f16, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                 const char* what) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "tensor map for %s: CUresult %d", what, (int)r);
  return MOE_OK;
}

// Launch with programmatic stream serialization (every kernel waits in
// pdl_wait() before it touches memory) and clusters of `cg` CTAs.
template <typename... KArgs, typename... Args>
moe_status launch(const char* what, void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int cg,
                  cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cg;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cg > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, args...), what);
}

// --- products ----------------------------------------------------------------------

// An operand: a packed or pitched row-major matrix
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
};

// A launch of products: collected first, then given a tile and enqueued.
struct Launch {
  moe::DenseGemmArgs g;
  Mat a[moe::kDenseProblems][2], b[moe::kDenseProblems][2];
  int na[moe::kDenseProblems], nb[moe::kDenseProblems];

  Launch(int f16, void* ws) {
    memset(&g, 0, sizeof(g));
    g.f16 = f16;
    g.status = static_cast<int32_t*>(ws);
  }
  moe::DenseProblem& add(int M, int N, int K, bool a_mn, const Mat* am, int an, bool b_mn, const Mat* bm, int bn) {
    const int i = g.problems++;
    moe::DenseProblem& p = g.p[i];
    p.M = M; p.N = N; p.K = K;
    p.k_segs = 1; p.m_segs = 1;
    p.a_mn = a_mn; p.b_mn = b_mn;
    na[i] = an;
    nb[i] = bn;
    for (int k = 0; k < an; ++k) a[i][k] = am[k];
    for (int k = 0; k < bn; ++k) b[i][k] = bm[k];
    return p;
  }
  // problem i as a launch of its own
  Launch only(int i) const {
    Launch l = *this;
    l.g.problems = 0;
    l.copy(*this, i);
    return l;
  }
  void take(const Launch& one) { copy(one, 0); }

 private:
  void copy(const Launch& from, int i) {
    const int to = g.problems++;
    g.p[to] = from.g.p[i];
    na[to] = from.na[i];
    nb[to] = from.nb[i];
    for (int k = 0; k < 2; ++k) {
      a[to][k] = from.a[i][k];
      b[to][k] = from.b[i][k];
    }
  }
};

// Tile of a launch: a pair's 256 rows or one CTA's 128, and the columns, from
// the time of a wave of tiles in a long product. That time grows with the
// columns (MMAs) and with a constant (the A rows every tile loads): measured at
// 4096 x 4096 x 8192, pairs of 256 / 192 / 160 / 128 columns 188 / 189 / 197 /
// 213 us, single CTAs of 256 / 192 / 128 columns 218 / 223 / 257 us, which the
// two lines below fit within 5%. MN-major B comes in boxes of 64 columns per CTA.
// A pair also starts and ends later than a CTA: products of one wave are faster
// on single CTAs up to about 25 stages (728 x 160 x 488: 6.0 us, pairs 6.7; at 128
// stages 29 and 25).
constexpr long kPairCost = 125000;
struct TileChoice {
  int cg, n;
};
long tiles_of(const moe::DenseProblem& p, int cg, int cols) {
  return p.m_segs * (long)((p.M + 128 * cg - 1) / (128 * cg)) * ((p.N + cols - 1) / cols);
}
long stages_of(const moe::DenseProblem& p) { return (p.K + 63) / 64 * (long)p.k_segs; }
TileChoice pick_tile(const Device& dv, const moe::DenseGemmArgs& g, bool glu) {
  TileChoice best = {1, 64};
  long best_cost = -1;
  int rows = 0, longest = 0;
  bool b_mn = false;
  for (int i = 0; i < g.problems; ++i) {
    rows = std::max(rows, g.p[i].M);
    longest = std::max<int>(longest, (int)stages_of(g.p[i]));
    b_mn |= g.p[i].b_mn != 0;
  }
  for (int cg = rows > 128 ? 2 : 1; cg >= 1; --cg) {
    for (int n = 256; n >= 64; n -= 32) {
      if (b_mn && n % (64 * cg) != 0) continue;
      if (glu && n % 64 != 0) continue;
      const long slots = dv.num_sms / cg;
      long work = 0, tiles = 0;
      for (int i = 0; i < g.problems; ++i) {
        const long t = tiles_of(g.p[i], cg, glu ? n / 2 : n);
        tiles += t;
        work += t * stages_of(g.p[i]);
      }
      // stages of the fullest slot: whole waves of one product; of several, an
      // even share and the tile that ends it
      const long stages = g.problems == 1 ? (tiles + slots - 1) / slots * longest
                                          : std::max<long>(longest, (work + slots - 1) / slots + longest / 2);
      const long cost = cg == 2 ? stages * 100L * (n + 100) + kPairCost : stages * 107L * (n + 136);
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best = {cg, n};
      }
    }
  }
  return best;
}

// Tensor maps and tile numbers of a launch's products for tile `t`; returns the tiles.
moe_status place(Launch& l, const TileChoice& t, bool glu, long* tiles, const char* what) {
  moe::DenseGemmArgs& g = l.g;
  g.tile_n = t.n;
  *tiles = 0;
  for (int i = 0; i < g.problems; ++i) {
    moe::DenseProblem& p = g.p[i];
    p.first = (int)*tiles;
    *tiles += tiles_of(p, t.cg, glu ? t.n / 2 : t.n);
    for (int k = 0; k < l.na[i]; ++k) {
      const Mat& m = l.a[i][k];
      TRY(map16(&p.map_a[k], m.p, g.f16, m.rows, m.cols, m.ld, p.a_mn ? 64 : 128, what));
    }
    for (int k = 0; k < l.nb[i]; ++k) {
      const Mat& m = l.b[i][k];
      TRY(map16(&p.map_b[k], m.p, g.f16, m.rows, m.cols, m.ld, p.b_mn ? 64 : glu ? t.n / 2 : t.n / t.cg, what));
    }
  }
  g.tiles = (int)*tiles;
  return MOE_OK;
}

// A product whose tiles leave SMs idle and are long: one tile a cluster, its K
// divided (k_dense_split). Times in us, fitted to both kernels at 18 shapes
// from 80 x 1024 x 1024 to 2048 x 512 x 4096 (within 15%): the tiled kernel
// takes 4.5 and 0.24 a stage; a cluster 5, 0.22 or 0.25 (64 or 128 columns) a
// stage, 1.7 times that with two CTAs on an SM, and 0.4 for each CTA and 64
// columns that are added up. (100 x 2048 x 8192: 36 us tiled, 13.5 in clusters
// of 4; 512 x 512 x 8192: 31 and 14.)
struct SplitChoice {
  int n, splits;            // splits 0: the tiled kernel
};
SplitChoice pick_split(const Device& dv, const Launch& one, bool glu, bool grads, int longest_piece) {
  SplitChoice best = {0, 0};
  const moe::DenseProblem& p = one.g.p[0];
  const TileChoice t = pick_tile(dv, one.g, glu);
  if (tiles_of(p, t.cg, glu ? t.n / 2 : t.n) > dv.num_sms / t.cg) return best;    // more than a wave
  const long ks = stages_of(p);
  double best_us = 4.5 + 0.24 * ks;
  if (grads) best_us *= 0.75;           // gradients share a launch otherwise, which is worth about a quarter
  for (int n = 64; n <= 128; n *= 2) {
    const long tiles = tiles_of(p, 1, glu ? n / 2 : n);
    for (int s = 2; s <= moe::kMaxSplits && 2 * s <= ks; ++s) {
      if (tiles > 2 * dv.clusters[s] || (ks + s - 1) / s > longest_piece) continue;
      const double stage = (n == 64 ? 0.22 : 0.25) * (tiles > dv.clusters[s] ? 1.7 : 1.0);
      const double us = 5.0 + stage * ((ks + s - 1) / s) + 0.4 * s * (n / 64);
      if (us < best_us) {
        best_us = us;
        best = {n, s};
      }
    }
  }
  return best;
}
template <int kEpi>
moe_status split(const Device& dv, Launch& l, const SplitChoice& c, cudaStream_t st, const char* what) {
  long tiles = 0;
  TRY(place(l, {1, c.n}, kEpi == moe::kEpiGlu, &tiles, what));
  // up to one CTA an SM: the ring takes the SM's memory, also so that clusters
  // that start under the previous kernel do not gather, two CTAs an SM, on the
  // SMs it leaves idle (a block's input gradient behind its hidden gradient at
  // T = 777: 26 us, 15 by itself)
  const int ring = tiles <= dv.clusters[c.splits] ? moe::kSplitRingAlone : moe::kSplitRingShared;
  const int stages = std::min(moe::kSplitStages, ring / (128 * 128 + c.n * 128));
  return launch(what, moe::k_dense_split<kEpi>, dim3((unsigned)(tiles * c.splits)), moe::dense_split_threads(),
                (size_t)ring + 1024, c.splits, st, l.g, c.splits, stages);
}

// Few tokens: the weights' rows over clusters that split K, down to two stages
// of 64 k a CTA while there are fewer CTAs than SMs, four beyond (24 x 1024 ->
// 1024: 3.9 us with 8 splits, 4.3 with 4; 24 x 1024 -> 4096: 6.4 with 8, 4.9
// with 4). Above 32 tokens a K below 512 leaves nothing to split, and the tiled
// kernel is faster (64 x 256 -> 256: 4.2 us and 5.9).
bool few_tokens(int T, int K) { return T <= moe::kRowsTokens && (T <= 32 || K >= 512); }
template <int kEpi, bool kWMn = false>
moe_status rows(const Device& dv, const Launch& l, bool early, cudaStream_t st, const char* what) {
  constexpr bool glu = kEpi == moe::kEpiGlu;
  moe::DenseRowsArgs r;
  r.g = l.g;
  r.early = early;
  moe::DenseProblem& p = r.g.p[0];
  r.g.tile_n = (p.M + 15) / 16 * 16;
  for (int i = 0; i < l.na[0]; ++i) {
    const Mat& x = l.a[0][i];
    TRY(map16(&p.map_b[i], x.p, r.g.f16, x.rows, x.cols, x.ld, r.g.tile_n, what));
  }
  for (int i = 0; i < l.nb[0]; ++i) {
    const Mat& w = l.b[0][i];
    TRY(map16(&p.map_a[i], w.p, r.g.f16, w.rows, w.cols, w.ld, glu || kWMn ? 64 : 128, what));
  }
  const int tile = glu ? 64 : 128, tiles = (p.N + tile - 1) / tile, ks = (int)stages_of(p);
  r.splits = std::max(std::min(dv.num_sms / tiles, ks / 2), std::min(7 * dv.num_sms / 4 / tiles, ks / 4));
  r.splits = std::max(1, std::min(moe::kRowsSplits, r.splits));
  r.stages = moe::dense_rows_stages(p.M, r.g.tile_n);
  auto kernel = moe::k_dense_rows<kEpi, kWMn, false>;
  if constexpr (glu) {
    if (r.g.saved8 && (ks + r.splits - 1) / r.splits > moe::kPieceStages) kernel = moe::k_dense_rows<kEpi, kWMn, true>;
  }
  return launch(what, kernel, dim3((unsigned)(tiles * r.splits)), moe::kRowsThreads, moe::dense_rows_smem_bytes(),
                r.splits, st, r);
}

template <int kEpi, bool kPieces = false>
moe_status enqueue(const Device& dv, Launch& l, cudaStream_t st, const char* what) {
  constexpr bool glu = kEpi == moe::kEpiGlu;
  // whether a product is split goes by itself alone, so its results do not
  // depend on which others are asked for
  Launch rest = l;
  rest.g.problems = 0;
  for (int i = 0; i < l.g.problems; ++i) {
    Launch one = l.only(i);
    const moe::DenseProblem& p = one.g.p[0];
    // dX and the hidden gradient of few tokens; a small dX stays in the launch
    // that dW needs (22 tokens of 232 <- 1584: 11.7 us apart, 13.8 together; 6 of
    // 192 <- 248: 9.2 and 7.7)
    if constexpr (!glu) {
      const bool large = kEpi == moe::kEpiDGlu || (long)p.K * p.k_segs * p.N >= kSmallWeights;
      if (p.b_mn && !p.a_mn && large && few_tokens(p.M, p.K * p.k_segs)) {
        TRY((rows<kEpi, true>(dv, one, false, st, what)));
        continue;
      }
    }
    const SplitChoice c = pick_split(dv, one, glu, kEpi == moe::kEpiLinear && p.b_mn, kPieces ? moe::kPieceStages : 1 << 30);
    if (c.splits) TRY(split<kEpi>(dv, one, c, st, what));
    else rest.take(one);
  }
  if (rest.g.problems == 0) return MOE_OK;
  moe::DenseGemmArgs& g = rest.g;
  const TileChoice t = pick_tile(dv, g, glu);
  const long slots = dv.num_sms / t.cg;
  long tiles = 0;
  for (int i = 0; i < g.problems; ++i) tiles += tiles_of(g.p[i], t.cg, glu ? t.n / 2 : t.n);
  // Several products go in one launch, in equal shares of their stages, while
  // they are a few waves together; longer ones keep their own launches, whose
  // neighbouring tiles share operands in L2 (gradients at T = 777, 1000 x 1352:
  // 63 us in three launches, 49 in one; at 4096, 8192 x 2048: 682 and 691).
  const bool together = g.problems == 1 || tiles < 4 * slots;
  for (int i = 0; i < (together ? 1 : g.problems); ++i) {
    Launch part = together ? rest : rest.only(i);
    const TileChoice pt = together ? t : pick_tile(dv, part.g, glu);
    TRY(place(part, pt, glu, &tiles, what));
    part.g.balanced = part.g.problems > 1;
    const int ctas = (int)std::min<long>(tiles, dv.num_sms / pt.cg) * pt.cg;
    TRY(launch(what, pt.cg == 2 ? moe::k_dense_gemm<kEpi, 2, kPieces> : moe::k_dense_gemm<kEpi, 1, kPieces>,
               dim3((unsigned)ctas), moe::dense_gemm_threads(), moe::dense_gemm_smem_bytes(), pt.cg, st, part.g));
  }
  return MOE_OK;
}

// y[T, N] = f(x W^T + bias) + residual
moe_status project(const Device& dv, int T, int N, int K, int f16, int fn, int out_f32, const void* x, int64_t ldx,
                   const void* w, const void* bias, const void* residual, int64_t ldr, void* y, int64_t ldy,
                   void* pre, void* ws, cudaStream_t st, const char* what, bool early = false) {
  Launch l(f16, ws);
  const Mat a = {x, T, K, ldx}, b = {w, N, K, K};
  moe::DenseProblem& p = l.add(T, N, K, false, &a, 1, false, &b, 1);
  p.out[0] = y; p.ldo = ldy;
  l.g.fn = fn; l.g.out_f32 = out_f32; l.g.bias = bias; l.g.residual = residual; l.g.ldr = ldr; l.g.pre = pre;
  return few_tokens(T, K) ? rows<moe::kEpiLinear>(dv, l, early, st, what)
                               : enqueue<moe::kEpiLinear>(dv, l, st, what);
}

// dx[T, K] = sum_s dz_s[T, N] W_s[N, K]
void add_input_grad(Launch& l, int T, int N, int K, const Mat* dz, const Mat* w, int segs, void* dx, int64_t lddx) {
  moe::DenseProblem& p = l.add(T, K, N, false, dz, segs, true, w, segs);
  p.k_segs = segs; p.out[0] = dx; p.ldo = lddx;
}

// dw_s[N, K] = dz_s[T, N]^T x[T, K]
void add_weight_grad(Launch& l, int T, int N, int K, const Mat* dz, int segs, const Mat& x, void* dw0, void* dw1) {
  moe::DenseProblem& p = l.add(N, K, T, true, dz, segs, true, &x, 1);
  p.m_segs = segs; p.out[0] = dw0; p.out[1] = dw1; p.ldo = K;
}

moe_status ckpt8(const Device& dv, bool pack, int f16, int64_t rows, int cols, const void* src, void* dst, int64_t ld,
                 uint8_t* q, uint8_t* s, cudaStream_t st) {
  moe::Ckpt8Args c;
  c.src = src; c.dst = dst; c.q = q; c.s = s; c.rows = rows; c.ld = ld; c.cols = cols; c.f16 = f16;
  const int groups = (cols + 31) / 32 * 4;
  for (c.width = 4; c.width < groups && c.width < moe::kCkptThreads;) c.width *= 2;
  const int64_t high = (int64_t)moe::kCkptThreads / c.width * moe::kCkptRows;
  const dim3 grid((unsigned)((rows + high - 1) / high), (unsigned)((groups + c.width - 1) / c.width));
  return launch(pack ? "checkpoint pack" : "checkpoint unpack", pack ? moe::k_ckpt8_pack : moe::k_ckpt8_unpack, grid,
                moe::kCkptThreads, 0, 1, st, c);
}

moe_status check_ckpt8(int32_t dtype, int64_t rows, int32_t cols, const void* x, int64_t* ld, const void* q,
                       const void* s, const char* name) {
  if (dtype != MOE_BF16 && dtype != MOE_F16) return fail(MOE_ERR_INVALID_ARG, "dtype %d is not a moe_dtype", dtype);
  if (rows < 1 || rows > 0x7FFFFFFF)
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "rows=%lld outside [1, 2^31 - 1]", (long long)rows);
  TRY(check_width("cols", cols));
  TRY(check_pitch("ld", *ld, cols, ld));
  if (!x) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(x)) return fail(MOE_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  NEED(q);
  NEED(s);
  return MOE_OK;
}

// the saved buffers that `save` asks for
moe_status check_saved(const FfnPlan& p, const moe_ffn_saved* saved) {
  if (p.save == MOE_SAVE_NONE) {
    if (saved) return fail(MOE_ERR_INVALID_ARG, "saved is not NULL, but save is MOE_SAVE_NONE");
    return MOE_OK;
  }
  if (!saved) return fail(MOE_ERR_INVALID_ARG, "saved is NULL");
  NEED(saved->g);
  NEED(saved->u);
  if (p.save == MOE_SAVE_8) {
    NEED(saved->g_s);
    NEED(saved->u_s);
    if (!saved->x_q != !saved->x_s)
      return fail(MOE_ERR_INVALID_ARG, "saved->x_q and saved->x_s: both or neither");
    MAYBE(saved->x_q);
    MAYBE(saved->x_s);
  } else if (saved->g_s || saved->u_s || saved->x_q || saved->x_s) {
    return fail(MOE_ERR_INVALID_ARG, "saved scales or x codes with MOE_SAVE_16");
  }
  return MOE_OK;
}

}  // namespace

// ===========================================================================
// C ABI
// ===========================================================================
extern "C" {

moe_status moe_dense_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  TRY(check_ws(ws, ws_bytes, kStatusBytes));
  const cudaError_t e = cudaMemsetAsync(ws, 0, kStatusBytes, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "status clear: %s", cudaGetErrorString(e));
  return MOE_OK;
}

size_t moe_linear_workspace_size(const moe_linear_dims* dims) {
  LinearPlan p;
  return make_plan(dims, p) == MOE_OK ? p.total : 0;
}

size_t moe_ffn_workspace_size(const moe_ffn_dims* dims) {
  FfnPlan p;
  return make_plan(dims, p) == MOE_OK ? p.total : 0;
}

moe_status moe_linear(const moe_linear_dims* dims, const void* x, const void* w, const void* bias,
                      const void* residual, void* y, void* pre, void* ws, size_t ws_bytes, void* stream) {
  LinearPlan p;
  TRY(make_plan(dims, p));
  NEED(x);
  NEED(w);
  NEED(y);
  MAYBE(bias);
  MAYBE(residual);
  MAYBE(pre);
  if (y == residual && (p.out_f32 || p.ldy != p.ldr))
    return fail(MOE_ERR_INVALID_ARG, "y is the residual, but not of its type and pitch");
  TRY(check_ws(ws, ws_bytes, p.total));
  Spans b;
  b.out("y", y, p.T, p.N, p.ldy, p.out_f32 ? 4 : 2);
  b.out("pre", pre, p.T, p.N, p.N, 2);
  b.out("the workspace", ws, 1, (int64_t)p.total, (int64_t)p.total, 1);
  b.in("x", x, p.T, p.K, p.ldx, 2);
  b.in("w", w, p.N, p.K, p.K, 2);
  b.in("bias", bias, 1, p.N, p.N, 2);
  if (residual == y) b.free_in("residual", residual, p.T, p.N, p.ldr, 2);
  else b.in("residual", residual, p.T, p.N, p.ldr, 2);
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  return project(*dv, p.T, p.N, p.K, p.f16, p.fn, p.out_f32, x, p.ldx, w, bias, residual, p.ldr, y, p.ldy, pre, ws,
                 (cudaStream_t)stream, "projection");
}

moe_status moe_linear_backward(const moe_linear_dims* dims, const void* dy, const void* x, const void* w,
                               const void* pre, void* dx, void* dw, void* dbias,
                               void* ws, size_t ws_bytes, void* stream) {
  LinearPlan p;
  TRY(make_plan(dims, p));
  NEED(dy);
  if (!dx && !dw && !dbias) return fail(MOE_ERR_INVALID_ARG, "dx, dw and dbias are all NULL");
  if (dx) NEED(w);
  if (dw) NEED(x);
  if (p.fn) NEED(pre);
  if (!p.fn && pre) return fail(MOE_ERR_INVALID_ARG, "pre is not NULL, but fn is MOE_FN_NONE");
  MAYBE(dx);
  MAYBE(dw);
  MAYBE(dbias);
  TRY(check_ws(ws, ws_bytes, p.total));
  const size_t ob = p.out_f32 ? 4 : 2;
  Spans b;
  b.out("dx", dx, p.T, p.K, p.ldx, ob);
  b.out("dw", dw, p.N, p.K, p.K, ob);
  b.out("dbias", dbias, 1, p.N, p.N, ob);
  b.out("the workspace", ws, 1, (int64_t)p.total, (int64_t)p.total, 1);
  b.in("dy", dy, p.T, p.N, p.ldy, 2);
  b.in("pre", pre, p.T, p.N, p.N, 2);
  if (dx) b.in("w", w, p.N, p.K, p.K, 2);
  if (dw) b.in("x", x, p.T, p.K, p.ldx, 2);
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  cudaStream_t st = (cudaStream_t)stream;
  Mat dz = {dy, p.T, p.N, p.ldy};
  if (p.fn || dbias) {
    moe::DzArgs z;
    z.dy = dy; z.pre = pre; z.lddy = p.ldy;
    z.dz = p.fn && (dx || dw) ? at(ws, p.off_dz) : nullptr;
    const bool one = p.dz_chunks == 1;
    z.part = dbias && !one ? reinterpret_cast<float*>(at(ws, p.off_part)) : nullptr;
    z.db = one ? dbias : nullptr;
    z.out_f32 = p.out_f32;
    z.T = p.T; z.N = p.N; z.rows = p.dz_rows; z.f16 = p.f16; z.fn = p.fn;
    TRY(launch("activation gradient", moe::k_dz,
               dim3((unsigned)((p.N + moe::kDzCols - 1) / moe::kDzCols), (unsigned)p.dz_chunks), moe::kDzThreads, 0, 1,
               st, z));
    if (z.part)
      TRY(launch("bias gradient", moe::k_colsum, dim3((unsigned)((p.N + 31) / 32)), 256, 0, 1, st,
                 (const float*)z.part, p.dz_chunks, p.N, p.f16, p.out_f32, dbias));
    if (z.dz) dz = {z.dz, p.T, p.N, p.N};
  }
  if (!dx && !dw) return MOE_OK;
  Launch l(p.f16, ws);
  l.g.out_f32 = p.out_f32;
  const Mat wm = {w, p.N, p.K, p.K}, xm = {x, p.T, p.K, p.ldx};
  if (dx) add_input_grad(l, p.T, p.N, p.K, &dz, &wm, 1, dx, p.ldx);
  if (dw) add_weight_grad(l, p.T, p.N, p.K, &dz, 1, xm, dw, nullptr);
  return enqueue<moe::kEpiLinear>(*dv, l, st, "projection gradients");
}

moe_status moe_ffn(const moe_ffn_dims* dims, const void* x, const void* wg, const void* wu, const void* wd,
                   const void* residual, void* y, const moe_ffn_saved* saved,
                   void* ws, size_t ws_bytes, void* stream) {
  FfnPlan p;
  TRY(make_plan(dims, p));
  NEED(x);
  NEED(wg);
  NEED(wu);
  NEED(wd);
  NEED(y);
  MAYBE(residual);
  if (y == residual && (p.out_f32 || p.ldy != p.ldr))
    return fail(MOE_ERR_INVALID_ARG, "y is the residual, but not of its type and pitch");
  TRY(check_saved(p, saved));
  TRY(check_ws(ws, ws_bytes, p.total));
  const int64_t nh = (p.H + 31) / 32, ni = (p.I + 31) / 32;
  Spans b;
  b.out("y", y, p.T, p.H, p.ldy, p.out_f32 ? 4 : 2);
  if (saved) {
    const size_t sb = p.save == MOE_SAVE_8 ? 1 : 2;
    b.out("saved->g", saved->g, p.T, p.I, p.I, sb);
    b.out("saved->u", saved->u, p.T, p.I, p.I, sb);
    b.out("saved->g_s", saved->g_s, p.T, ni, ni, 1);
    b.out("saved->u_s", saved->u_s, p.T, ni, ni, 1);
    b.out("saved->x_q", saved->x_q, p.T, p.H, p.H, 1);
    b.out("saved->x_s", saved->x_s, p.T, nh, nh, 1);
  }
  b.out("the workspace", ws, 1, (int64_t)p.total, (int64_t)p.total, 1);
  b.free_in("x", x, p.T, p.H, p.ldx, 2);        // the down projection writes y behind the last read of x
  b.in("wg", wg, p.I, p.H, p.H, 2);
  b.in("wu", wu, p.I, p.H, p.H, 2);
  b.in("wd", wd, p.H, p.I, p.I, 2);
  if (residual == y) b.free_in("residual", residual, p.T, p.H, p.ldr, 2);
  else b.in("residual", residual, p.T, p.H, p.ldr, 2);
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  cudaStream_t st = (cudaStream_t)stream;
  void* h = at(ws, p.off_h);
  Launch l(p.f16, ws);
  const Mat xm = {x, p.T, p.H, p.ldx};
  const Mat wm[2] = {{wg, p.I, p.H, p.H}, {wu, p.I, p.H, p.H}};
  moe::DenseProblem& gu = l.add(p.T, p.I, p.H, false, &xm, 1, false, wm, 2);
  gu.out[0] = h; gu.ldo = p.I;
  l.g.fn = p.fn;
  if (saved) {
    l.g.g = saved->g; l.g.u = saved->u; l.g.g_s = saved->g_s; l.g.u_s = saved->u_s;
    l.g.saved8 = p.save == MOE_SAVE_8;
  }
  const char* what = "gate/up projection";
  if (few_tokens(p.T, p.H)) TRY(rows<moe::kEpiGlu>(*dv, l, false, st, what));
  else if (l.g.saved8) TRY((enqueue<moe::kEpiGlu, true>(*dv, l, st, what)));
  else TRY(enqueue<moe::kEpiGlu>(*dv, l, st, what));
  if (saved && saved->x_q)
    TRY(ckpt8(*dv, true, p.f16, p.T, p.H, x, nullptr, p.ldx, saved->x_q, saved->x_s, st));
  return project(*dv, p.T, p.H, p.I, p.f16, MOE_FN_NONE, p.out_f32, h, p.I, wd, nullptr, residual, p.ldr, y, p.ldy,
                 nullptr, ws, st, "down projection", true);
}

moe_status moe_ffn_backward(const moe_ffn_dims* dims, const void* dy, const void* x, const void* wg,
                            const void* wu, const void* wd, const moe_ffn_saved* saved, void* dx, void* dwg,
                            void* dwu, void* dwd, void* ws, size_t ws_bytes, void* stream) {
  FfnPlan p;
  TRY(make_plan(dims, p));
  if (p.save == MOE_SAVE_NONE) return fail(MOE_ERR_INVALID_ARG, "save is MOE_SAVE_NONE: nothing to go back from");
  NEED(dy);
  NEED(wd);
  if (!dwg != !dwu) return fail(MOE_ERR_INVALID_ARG, "dwg and dwu: both or neither");
  if (!dx && !dwg && !dwd) return fail(MOE_ERR_INVALID_ARG, "dx, dwg, dwu and dwd are all NULL");
  if (dx) {
    NEED(wg);
    NEED(wu);
  }
  MAYBE(x);
  MAYBE(dx);
  MAYBE(dwg);
  MAYBE(dwu);
  MAYBE(dwd);
  TRY(check_saved(p, saved));
  if (dwg && !x && !saved->x_q)
    return fail(MOE_ERR_INVALID_ARG, "x is NULL and saved holds no x_q: the weight gradients need one");
  TRY(check_ws(ws, ws_bytes, p.total));
  const int64_t nh = (p.H + 31) / 32, ni = (p.I + 31) / 32;
  const size_t ob = p.out_f32 ? 4 : 2, sb = p.save == MOE_SAVE_8 ? 1 : 2;
  Spans b;
  b.out("dx", dx, p.T, p.H, p.ldx, ob);
  b.out("dwg", dwg, p.I, p.H, p.H, ob);
  b.out("dwu", dwu, p.I, p.H, p.H, ob);
  b.out("dwd", dwd, p.H, p.I, p.I, ob);
  b.out("the workspace", ws, 1, (int64_t)p.total, (int64_t)p.total, 1);
  b.in("dy", dy, p.T, p.H, p.ldy, 2);
  b.in("wd", wd, p.H, p.I, p.I, 2);
  if (dx) {
    b.in("wg", wg, p.I, p.H, p.H, 2);
    b.in("wu", wu, p.I, p.H, p.H, 2);
  }
  b.in("saved->g", saved->g, p.T, p.I, p.I, sb);
  b.in("saved->u", saved->u, p.T, p.I, p.I, sb);
  b.in("saved->g_s", saved->g_s, p.T, ni, ni, 1);
  b.in("saved->u_s", saved->u_s, p.T, ni, ni, 1);
  if (dwg && x) b.in("x", x, p.T, p.H, p.ldx, 2);
  if (dwg && !x) {
    b.in("saved->x_q", saved->x_q, p.T, p.H, p.H, 1);
    b.in("saved->x_s", saved->x_s, p.T, nh, nh, 1);
  }
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  cudaStream_t st = (cudaStream_t)stream;
  const Mat dym = {dy, p.T, p.H, p.ldy};
  Mat xm = {x, p.T, p.H, p.ldx};
  if (dwg && !x) {
    TRY(ckpt8(*dv, false, p.f16, p.T, p.H, nullptr, at(ws, p.off_x), p.H, saved->x_q, saved->x_s, st));
    xm = {at(ws, p.off_x), p.T, p.H, p.H};
  }
  void *dg = at(ws, p.off_dg), *du = at(ws, p.off_du), *h = at(ws, p.off_h);
  Launch hidden(p.f16, ws);
  const Mat wdm = {wd, p.H, p.I, p.I};
  moe::DenseProblem& dh = hidden.add(p.T, p.I, p.H, false, &dym, 1, true, &wdm, 1);
  dh.out[0] = dg; dh.out[1] = du; dh.ldo = p.I;
  hidden.g.fn = p.fn; hidden.g.saved8 = p.save == MOE_SAVE_8; hidden.g.pre = h;
  hidden.g.g = saved->g; hidden.g.u = saved->u; hidden.g.g_s = saved->g_s; hidden.g.u_s = saved->u_s;
  TRY(enqueue<moe::kEpiDGlu>(*dv, hidden, st, "hidden gradient"));
  // the three products that read it, in one launch
  Launch l(p.f16, ws);
  l.g.out_f32 = p.out_f32;
  const Mat dgu[2] = {{dg, p.T, p.I, p.I}, {du, p.T, p.I, p.I}};
  const Mat wm[2] = {{wg, p.I, p.H, p.H}, {wu, p.I, p.H, p.H}}, hm = {h, p.T, p.I, p.I};
  if (dx) add_input_grad(l, p.T, p.I, p.H, dgu, wm, 2, dx, p.ldx);
  if (dwg) add_weight_grad(l, p.T, p.I, p.H, dgu, 2, xm, dwg, dwu);
  if (dwd) add_weight_grad(l, p.T, p.H, p.I, &dym, 1, hm, dwd, nullptr);
  return enqueue<moe::kEpiLinear>(*dv, l, st, "block gradients");
}

moe_status moe_ckpt8_pack(int32_t dtype, int64_t rows, int32_t cols, const void* src, int64_t ld,
                          uint8_t* q, uint8_t* s, void* stream) {
  TRY(check_ckpt8(dtype, rows, cols, src, &ld, q, s, "src"));
  Spans b;
  b.out("q", q, rows, cols, cols, 1);
  b.out("s", s, rows, (cols + 31) / 32, (cols + 31) / 32, 1);
  b.in("src", src, rows, cols, ld, 2);
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  return ckpt8(*dv, true, dtype, rows, cols, src, nullptr, ld, q, s, (cudaStream_t)stream);
}

moe_status moe_ckpt8_unpack(int32_t dtype, int64_t rows, int32_t cols, const uint8_t* q, const uint8_t* s,
                            void* dst, int64_t ld, void* stream) {
  TRY(check_ckpt8(dtype, rows, cols, dst, &ld, q, s, "dst"));
  Spans b;
  b.out("dst", dst, rows, cols, ld, 2);
  b.in("q", q, rows, cols, cols, 1);
  b.in("s", s, rows, (cols + 31) / 32, (cols + 31) / 32, 1);
  TRY(b.check());
  const Device* dv;
  TRY(device(&dv));
  return ckpt8(*dv, false, dtype, rows, cols, nullptr, dst, ld, const_cast<uint8_t*>(q), const_cast<uint8_t*>(s),
               (cudaStream_t)stream);
}

}  // extern "C"
