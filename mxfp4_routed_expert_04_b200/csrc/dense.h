// Internal interfaces of the dense operators: the projection with a fused
// epilogue (moe_linear), the gated feed-forward block (moe_ffn), their backward
// passes and the 8-bit activation checkpoints.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_mxfp4.h"

namespace moe {


// --- tiled GEMM (dense_gemm.cu) -----------------------------------------------
// D[M, N] = sum over segments of A_s B_s with the epilogue of `kEpi`. What goes
// into the next product (h, dg, du; dz of k_dz) is rounded to 16 bits, since
// kind::f16 takes no more; each as a sum of two would double that product's
// MMAs. (In bf16 outputs are then off by 2.2e-3 to 2.4e-3, root mean square,
// their own rounding alone is 1.66e-3.)
enum DenseEpi {
  kEpiLinear = 0,   // y = f(D + bias) + residual (and the f argument, for the backward pass)
  kEpiGlu = 1,      // D holds gate and up columns side by side: h = f(g) * u (and g, u saved)
  kEpiDGlu = 2,     // D = dh: dg = dh u f'(g), du = dh f(g), h = f(g) u
};

// One product. a_mn / b_mn: the operand's M / N dimension is contiguous in
// memory, not its contraction dimension.
struct DenseProblem {
  // A and B of the contraction segments (dX of the gated block: dG Wg + dU Wu),
  // or A of the row segments (dWg and dWu share B), or B of the gate and up halves
  CUtensorMap map_a[2], map_b[2];
  void* out[2];             // kEpiLinear: per row segment; kEpiGlu: h; kEpiDGlu: dg, du
  int64_t ldo;
  int M, N, K;              // rows of one row segment, output columns (h columns for kEpiGlu), contraction
  int k_segs;               // contraction segments (1 or 2)
  int m_segs;               // row segments (1 or 2), each M rows with its own A and output
  int a_mn, b_mn;
  int first;                // its first tile in the launch
};
constexpr int kDenseProblems = 3;
struct DenseGemmArgs {
  DenseProblem p[kDenseProblems];   // products of one launch (the epilogue's inputs below are the first one's)
  int problems, tiles;      // tiles of all
  int balanced;             // CTAs (pairs) take consecutive tiles of equal work instead of every n-th tile
  int tile_n;               // columns of a tile (accumulator columns), a multiple of 32 up to 256
  int f16;                  // 16-bit type: 0 bf16, 1 f16
  int fn;                   // moe_fn
  int out_f32;              // out[] in fp32 instead of the 16-bit type
  int saved8;               // kEpiGlu writes / kEpiDGlu reads g and u as 8-bit checkpoints
  const void* bias;         // [N] 16-bit or NULL
  const void* residual;     // [M, ldr] 16-bit or NULL
  int64_t ldr;              // row pitch in elements
  void* pre;                // kEpiLinear: D + bias [M, N] 16-bit or NULL; kEpiDGlu: h
  void* g;                  // kEpiGlu out (or NULL) / kEpiDGlu in: [M, N] 16-bit, or E4M3 codes
  void* u;
  uint8_t* g_s;             // E8M0 scales [M, ceil(N/32)] of the codes
  uint8_t* u_s;
  int32_t* status;
};

// Longest sum, in stages of 64 k, in front of an 8-bit checkpoint (K = 1024). A
// tensor-core sum is cut off towards zero at every step of 16 k and loses about
// 1.5e-8 of itself each time (random signs; measured 7.8e-6 at K = 8192, fp32
// FMAs 0). In 16-bit outputs that is nothing, but an 8-bit checkpoint moves a
// value that lies so close to a border of its grid by a whole step: 3.3e-4 of
// the codes in one piece of K = 8192, 8e-5 in pieces of 2048. (Sums of one sign
// lose more: at K = 65536 one code in 100 in one piece, in pieces none beyond
// the error of 64 steps.) kPieces: the stages of a tile, or of a CTA's part of
// one, go in pieces of at most this many, each with an accumulator of its own,
// added up in registers (32 tokens through a block of 8192 / 8192: 76.0 us in
// pieces, 75.8 in one; 64 through 8192 / 18432: 156.8 and 156.2).
constexpr int kPieceStages = 16;
constexpr int pieces_of(int stages) { return (stages + kPieceStages - 1) / kPieceStages; }

template <int kEpi, int kCg, bool kPieces>
__global__ void k_dense_gemm(const __grid_constant__ DenseGemmArgs a);
// one small product: a tile of 128 rows and 64 or 128 columns per cluster of `splits` (2 to 8) CTAs
template <int kEpi>
__global__ void k_dense_split(const __grid_constant__ DenseGemmArgs a, int splits, int stages);
constexpr int kMaxSplits = 8, kSplitStages = 8;
constexpr int kSplitRingShared = 108 * 1024, kSplitRingAlone = 196 * 1024;   // two CTAs an SM, one
int dense_split_threads();
size_t dense_gemm_smem_bytes();
int dense_gemm_threads();

// --- few tokens (dense_rows.cu) -------------------------------------------------
// Problem 0 with the sides exchanged: the weights are the MMA's 128 rows (map_a;
// kEpiGlu: 64 gate and 64 up rows), the tokens its columns (map_b[0], tile_n = T rounded up to 16). A cluster of
// `splits` CTAs divides K and adds its partial sums through shared memory.
// M, N, K as above (M tokens, N outputs); early: the weights are not written
// by the previous kernel of the stream and may be loaded before it ends.
struct DenseRowsArgs {
  DenseGemmArgs g;
  int splits, stages, early;
};
constexpr int kRowsSplits = 8;          // most CTAs of a cluster
constexpr int kRowsTokens = 64;         // most tokens of this kernel
constexpr int kRowsThreads = 192;
constexpr int kRowsMemory = 110 * 1024; // two CTAs of an SM, so the next call starts under this one
constexpr int dense_rows_stage(int tile_n) { return 128 * 128 + tile_n * 128; }
// The partial sums: 512 bytes a token, in units of 4 tokens and of 512 (gated:
// 1024) bytes; pushed ones up to a unit more for each CTA of the cluster, behind
// the ring; kept ones over it.
constexpr int kRowsPush = 8;
constexpr int dense_rows_stages(int T, int tile_n) {
  return (kRowsMemory - (T > kRowsPush ? 0 : 512 * (T + 3) + 1024 * (kRowsSplits - 1))) / dense_rows_stage(tile_n);
}
static_assert(512 * kRowsTokens <= dense_rows_stage(16) * 2, "kept sums fit the ring's first two stages");
constexpr int kDenseRowsStages = dense_rows_stages(16, 16);
constexpr size_t dense_rows_smem_bytes() { return kRowsMemory + 1024; }
template <int kEpi, bool kWMn, bool kPieces>
__global__ void k_dense_rows(const __grid_constant__ DenseRowsArgs a);

// --- element kernels (dense_elem.cu) ------------------------------------------
// dz = dy * f'(pre) rounded to 16 bits (dz NULL: not written; pre NULL: f' = 1)
// and, per chunk of `rows` rows, the column sums of the unrounded dz
struct DzArgs {
  const void* dy;
  const void* pre;
  void* dz;
  float* part;              // [chunks, N] or NULL
  void* db;                 // a single chunk: the sums themselves [N], or NULL
  int T, N, rows, f16, fn, out_f32;
  int64_t lddy;
};
__global__ void k_dz(DzArgs a);
constexpr int kDzCols = 256, kDzThreads = 256;
// out[n] = sum over chunks, in order
__global__ void k_colsum(const float* part, int chunks, int N, int f16, int out_f32, void* out);

// 16-bit rows -> E4M3 codes with one E8M0 scale per 32 elements of a row, and back
struct Ckpt8Args {
  const void* src;
  void* dst;
  uint8_t* q;
  uint8_t* s;
  int64_t rows, ld;         // ld: row pitch of the 16-bit side, in elements
  int cols, f16;
  int width;                // 8-element groups of a block's row, a power of two in [4, kCkptThreads]
};
__global__ void k_ckpt8_pack(Ckpt8Args a);
__global__ void k_ckpt8_unpack(Ckpt8Args a);
constexpr int kCkptThreads = 256, kCkptRows = 4;    // threads of a block; rows of a thread

}  // namespace moe
