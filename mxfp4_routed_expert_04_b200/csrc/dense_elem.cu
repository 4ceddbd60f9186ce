// Element kernels of the dense operators: the activation's slope with the bias
// gradient's column sums, and the 8-bit activation checkpoints.
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
  const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * kDzCols + 8 * cg;
  const int r0 = (int)blockIdx.y * a.rows, r1 = min(a.T, r0 + a.rows);
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  if (col < a.N) {
    for (int r = r0 + rl; r < r1; r += 8) {
      float v[8];
      unpack16x8(a.f16, ldg16(static_cast<const uint16_t*>(a.dy) + (size_t)r * a.lddy + col), v);
      if (a.pre) {
        float z[8];
        unpack16x8(a.f16, ldg16(static_cast<const uint16_t*>(a.pre) + (size_t)r * a.N + col), z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, d;
          fn_slope(a.fn, z[i], f, d);
          v[i] *= d;
        }
      }
      if (a.dz)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dz) + (size_t)r * a.N + col) = pack16x8(a.f16, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
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

__global__ void k_colsum(const float* part, int chunks, int N, int f16, int out_f32, void* out) {
  pdl_wait();
  pdl_trigger();
  const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  if (c >= N) return;
  float s = 0.0f;
  for (int i = 0; i < chunks; ++i) s += part[(size_t)i * N + c];
  if (out_f32) static_cast<float*>(out)[c] = s;
  else static_cast<uint16_t*>(out)[c] = (uint16_t)(pack16(f16, s, s) & 0xFFFFu);
}

// one thread per block of 32 elements (64 bytes in, 32 + 1 out)
__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_pack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32;
  const int64_t total = a.rows * nb;
  for (int64_t i = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kCkptThreads) {
    const int64_t row = i / nb;
    const int col = (int)(i - row * nb) * 32;
    const uint16_t* p = static_cast<const uint16_t*>(a.src) + row * a.ld + col;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (col + 8 * j < a.cols) unpack16x8(a.f16, ldg16(p + 8 * j), v + 8 * j);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * j + k] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[8 * j + k]) & 0x7FFFFFFFu);
    }
    const uint32_t code = e4m3_scale_code(m);
    const float inv = e4m3_inv_scale(code);
    a.s[i] = (uint8_t)code;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + 8 * j < a.cols)
        *reinterpret_cast<uint2*>(a.q + row * a.cols + col + 8 * j) =
            make_uint2(e4m3_quad(v + 8 * j, inv), e4m3_quad(v + 8 * j + 4, inv));
  }
}

__global__ void __launch_bounds__(kCkptThreads) k_ckpt8_unpack(Ckpt8Args a) {
  pdl_wait();
  pdl_trigger();
  const int nb = (a.cols + 31) / 32, n8 = a.cols / 8;
  const int64_t total = a.rows * n8;
  for (int64_t i = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kCkptThreads) {
    const int64_t row = i / n8;
    const int col = (int)(i - row * n8) * 8;
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.cols + col));
    const float s = e8m0_to_f32(__ldg(a.s + row * nb + col / 32));
    float v[8];
    e4m3_unquad(q.x, s, v);
    e4m3_unquad(q.y, s, v + 4);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst) + row * a.ld + col) = pack16x8(a.f16, v);
  }
}

}  // namespace moe
