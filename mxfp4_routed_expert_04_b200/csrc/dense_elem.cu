// Element kernels of the dense operators: the activation's slope with the bias
// gradient's column sums, and the 8-bit activation checkpoints. All are bound
// by HBM, so each thread has several 16-byte loads in flight before it works.
#include "dense.cuh"

namespace moe {

MOE_DEV void store_sum(int f16, int out_f32, void* out, int c, float s) {
  if (out_f32) static_cast<float*>(out)[c] = s;
  else static_cast<uint16_t*>(out)[c] = (uint16_t)(pack16(f16, s, s) & 0xFFFFu);
}

// block: 32 column groups of 8 (256 columns) x 8 row lanes; grid: column
// blocks x row chunks. The column sums are added per row lane in row order,
// then over the 8 lanes in order, then (k_colsum; not for a single chunk) over
// the chunks in order: the same bits every run.
__global__ void __launch_bounds__(kDzThreads, 4) k_dz(DzArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][kDzCols];
  constexpr int kAhead = 2;               // rows a thread loads before it works
  const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * kDzCols + 8 * cg;
  const int r0 = (int)blockIdx.y * a.rows, r1 = min(a.T, r0 + a.rows);
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  if (col < a.N) {
    for (int r = r0 + rl; r < r1; r += 8 * kAhead) {
      uint4 y[kAhead], p[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (r + 8 * k < r1) y[k] = ldg16(static_cast<const uint16_t*>(a.dy) + (size_t)(r + 8 * k) * a.lddy + col);
      if (a.pre) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (r + 8 * k < r1) p[k] = ldg16(static_cast<const uint16_t*>(a.pre) + (size_t)(r + 8 * k) * a.N + col);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (r + 8 * k >= r1) break;
        float v[8];
        unpack16x8(a.f16, y[k], v);
        if (a.pre) {
          float z[8], f[8], d[8];
          unpack16x8(a.f16, p[k], z);
          fn_slopes(a.fn, z, f, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= d[i];
        }
        if (a.dz)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dz) + (size_t)(r + 8 * k) * a.N + col) =
              pack16x8(a.f16, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
      }
    }
  }
  if (!a.part && !a.db) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rl][8 * cg + i] = sum[i];
  __syncthreads();
  const int c = (int)blockIdx.x * kDzCols + threadIdx.x;
  if (c < a.N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    if (a.db) store_sum(a.f16, a.out_f32, a.db, c, s);
    else a.part[(size_t)blockIdx.y * a.N + c] = s;
  }
}

// block: 32 columns x 8 lanes over the chunks (lane l takes chunks l, l + 8, ..)
__global__ void __launch_bounds__(256) k_colsum(const float* part, int chunks, int N, int f16, int out_f32, void* out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int c = (int)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < N) {
#pragma unroll 8
    for (int i = l; i < chunks; i += 8) s += part[(size_t)i * N + c];
  }
  red[l][lane] = s;
  __syncthreads();
  if (l != 0 || c >= N) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += red[i][lane];
  store_sum(f16, out_f32, out, c, s);
}

namespace {

// Groups of 8 elements. A block is `width` groups wide (a power of two, so the
// four lanes of a scale's 32 elements are neighbours) and kCkptThreads / width
// rows high; a thread keeps its column and takes kAhead rows, all loaded before
// it works, so no index is divided (with a division per group the kernels were
// bound by instructions: 4096 x 8192 packed in 24 us).
constexpr int kAhead = kCkptRows;

struct Place {
  int64_t row;              // first row; the next ones `high` further on
  int group, high;
};
MOE_DEV Place place_of(const Ckpt8Args& a) {
  Place p;
  p.high = kCkptThreads / a.width;
  p.row = (int64_t)blockIdx.x * (p.high * kAhead) + threadIdx.x / a.width;
  p.group = (int)(blockIdx.y * a.width + (threadIdx.x & (a.width - 1)));
  return p;
}
MOE_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_pack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32;
  const Place p = place_of(a);
  const bool in_row = 8 * p.group < a.cols;
  uint4 w[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t r = p.row + k * p.high;
    w[k] = make_uint4(0u, 0u, 0u, 0u);
    if (in_row && r < a.rows) w[k] = ldg_stream(static_cast<const uint16_t*>(a.src) + r * a.ld + 8 * p.group);
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    // the largest magnitude as a 16-bit pattern: they grow with it, NaN above all
    uint32_t m = max_u16x2(max_u16x2(w[k].x & 0x7FFF7FFFu, w[k].y & 0x7FFF7FFFu),
                           max_u16x2(w[k].z & 0x7FFF7FFFu, w[k].w & 0x7FFF7FFFu));
    m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float top, unused;
    unpack16(a.f16, max(m & 0xFFFFu, m >> 16), top, unused);
    const uint32_t code = e4m3_scale_code(__float_as_uint(top));
    const float inv = e4m3_inv_scale(code);
    float v[8];
    unpack16x8(a.f16, w[k], v);
    const int64_t r = p.row + k * p.high;
    if (!in_row || r >= a.rows) continue;
    *reinterpret_cast<uint2*>(a.q + r * a.cols + 8 * p.group) = make_uint2(e4m3_quad(v, inv), e4m3_quad(v + 4, inv));
    if ((p.group & 3) == 0) a.s[r * nb + p.group / 4] = (uint8_t)code;
  }
}

__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_unpack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32;
  const Place p = place_of(a);
  if (8 * p.group >= a.cols) return;
  uint2 w[kAhead];
  uint32_t code[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t r = p.row + k * p.high;
    w[k] = make_uint2(0u, 0u);
    code[k] = 0u;
    if (r < a.rows) {
      w[k] = __ldg(reinterpret_cast<const uint2*>(a.q + r * a.cols + 8 * p.group));
      code[k] = __ldg(a.s + r * nb + p.group / 4);
    }
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t r = p.row + k * p.high;
    if (r >= a.rows) break;
    const float s = e8m0_to_f32(code[k]);
    float v[8];
    e4m3_unquad(w[k].x, s, v);
    e4m3_unquad(w[k].y, s, v + 4);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst) + r * a.ld + 8 * p.group) = pack16x8(a.f16, v);
  }
}

}  // namespace moe
