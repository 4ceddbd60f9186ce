// Element kernels of the dense operators: the activation's slope with the bias
// gradient's column sums, and the 8-bit activation checkpoints. All are bound
// by HBM, so each thread has several 16-byte loads in flight before it works.
#include "dense.cuh"

namespace moe {

// block: 32 column groups of 8 (256 columns) x 8 row lanes; grid: column
// blocks x row chunks. The column sums are added per row lane in row order,
// then over the 8 lanes in order, then (k_colsum) over the chunks in order:
// the same bits every run.
__global__ void __launch_bounds__(kDzThreads) k_dz(DzArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][kDzCols];
  constexpr int kAhead = 4;               // rows a thread loads before it works
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
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rl][8 * cg + i] = sum[i];
  __syncthreads();
  const int c = (int)blockIdx.x * kDzCols + threadIdx.x;
  if (c < a.N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    a.part[(size_t)blockIdx.y * a.N + c] = s;
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
  if (out_f32) static_cast<float*>(out)[c] = s;
  else static_cast<uint16_t*>(out)[c] = (uint16_t)(pack16(f16, s, s) & 0xFFFFu);
}

namespace {

// Element groups of 8, rows padded to whole blocks of 4 groups: group i of a
// span of kSpan belongs to thread i % kCkptThreads, so neighbouring lanes hold
// neighbouring 16 bytes and four lanes a block.
constexpr int kSpan = kCkptSpan, kPerThread = kSpan / kCkptThreads;

struct Place {
  int64_t row;
  int group;                // group of the row
  bool on;
};
// place of group i of the span that starts at group g0 of row row0
MOE_DEV Place place_of(const Ckpt8Args& a, int64_t row0, int g0, int i, int per_row) {
  const int g = g0 + i, dr = g / per_row;
  Place p;
  p.row = row0 + dr;
  p.group = g - dr * per_row;
  p.on = p.row < a.rows && 8 * p.group < a.cols;
  return p;
}

}  // namespace

__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_pack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32, per_row = 4 * nb;
  const int64_t total = a.rows * per_row;
  for (int64_t base = (int64_t)blockIdx.x * kSpan; base < total; base += (int64_t)gridDim.x * kSpan) {
    const int64_t row0 = base / per_row;
    const int g0 = (int)(base - row0 * per_row);
    Place p[kPerThread];
    uint4 w[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      p[k] = place_of(a, row0, g0, threadIdx.x + k * kCkptThreads, per_row);
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (p[k].on) w[k] = ldg_stream(static_cast<const uint16_t*>(a.src) + p[k].row * a.ld + 8 * p[k].group);
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      float v[8];
      unpack16x8(a.f16, w[k], v);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t code = e4m3_scale_code(m);
      const float inv = e4m3_inv_scale(code);
      if (!p[k].on) continue;
      *reinterpret_cast<uint2*>(a.q + p[k].row * a.cols + 8 * p[k].group) =
          make_uint2(e4m3_quad(v, inv), e4m3_quad(v + 4, inv));
      if ((p[k].group & 3) == 0) a.s[p[k].row * nb + p[k].group / 4] = (uint8_t)code;
    }
  }
}

__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_unpack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32, per_row = 4 * nb;
  const int64_t total = a.rows * per_row;
  for (int64_t base = (int64_t)blockIdx.x * kSpan; base < total; base += (int64_t)gridDim.x * kSpan) {
    const int64_t row0 = base / per_row;
    const int g0 = (int)(base - row0 * per_row);
    Place p[kPerThread];
    uint2 w[kPerThread];
    uint32_t code[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      p[k] = place_of(a, row0, g0, threadIdx.x + k * kCkptThreads, per_row);
      w[k] = make_uint2(0u, 0u);
      code[k] = 0u;
      if (p[k].on) {
        w[k] = __ldg(reinterpret_cast<const uint2*>(a.q + p[k].row * a.cols + 8 * p[k].group));
        code[k] = __ldg(a.s + p[k].row * nb + p[k].group / 4);
      }
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (!p[k].on) continue;
      const float s = e8m0_to_f32(code[k]);
      float v[8];
      e4m3_unquad(w[k].x, s, v);
      e4m3_unquad(w[k].y, s, v + 4);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst) + p[k].row * a.ld + 8 * p[k].group) =
          pack16x8(a.f16, v);
    }
  }
}

}  // namespace moe
