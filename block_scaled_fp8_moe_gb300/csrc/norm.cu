// Residual addition, RMS norm and MXFP8 quantisation of rows in one pass over them.
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

// A row lies in the registers of `tpr` threads, VPT groups of 8 values each, thread t those t, t + tpr, ... tpr is a multiple
// of 32, or for rows of up to 256 values a power of two below it; a block has blockDim / tpr rows. Bound: HBM, 9.03 bytes a
// value (32768 x 4096: 172 us, 7.03 TB/s); from 48 rows of 4096 down the 2.2 us of a launch.
template <int VPT>
__global__ void add_rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* __restrict__ weight, float eps, uint4* sum,
                                   uint4* y, uint2* __restrict__ q, uint8_t* __restrict__ s, int rows, int vecs, int tpr) {
  __shared__ float part[32];
  pdl_trigger();
  const int in_block = threadIdx.x / tpr, t = threadIdx.x - in_block * tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + in_block;
  const bool live = row < rows;
  pdl_wait();
  uint4 a[VPT], b[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * tpr;
    const bool in = live && c < vecs;
    a[i] = in ? x[row * vecs + c] : make_uint4(0, 0, 0, 0);
    b[i] = in && residual ? residual[row * vecs + c] : make_uint4(0, 0, 0, 0);
  }
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * tpr;
    const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][2 * j] = bf16_lo(wa[j]);
      h[i][2 * j + 1] = bf16_hi(wa[j]);
      if (residual) {
        h[i][2 * j] += bf16_lo(wb[j]);
        h[i][2 * j + 1] += bf16_hi(wb[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    if (sum && live && c < vecs)
      sum[row * vecs + c] = make_uint4(bf16x2(h[i][0], h[i][1]), bf16x2(h[i][2], h[i][3]), bf16x2(h[i][4], h[i][5]),
                                       bf16x2(h[i][6], h[i][7]));
  }
  for (int d = min(tpr, 32) / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (tpr > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < tpr / 32; ++i) ss += part[in_block * (tpr / 32) + i];
  }
  const float r = 1.f / sqrtf(ss / (float)(vecs * 8) + eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * tpr;
    const bool in = live && c < vecs;
    const uint4 w = in ? __ldg(weight + c) : make_uint4(0, 0, 0, 0);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
    float f[8], m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = bf16x2(h[i][2 * j] * r * bf16_lo(ww[j]), h[i][2 * j + 1] * r * bf16_hi(ww[j]));
      f[2 * j] = bf16_lo(o[j]);
      f[2 * j + 1] = bf16_hi(o[j]);
      m = fmaxf(m, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
    }
    if (y && in) y[row * vecs + c] = make_uint4(o[0], o[1], o[2], o[3]);
    if (!q) continue;
    // 4 lanes hold a block of 32 values (vecs and tpr are multiples of 4)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int se = e4m3_scale_exp_bf16(__float_as_uint(m) >> 16);
    const float sc = pow2_neg(se);
    if (in) {
      q[row * vecs + c] = make_uint2(e4m3x2(f[0] * sc, f[1] * sc) | (e4m3x2(f[2] * sc, f[3] * sc) << 16),
                                     e4m3x2(f[4] * sc, f[5] * sc) | (e4m3x2(f[6] * sc, f[7] * sc) << 16));
      if ((c & 3) == 0) s[(row * vecs + c) >> 2] = (uint8_t)(se + 127);
    }
  }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_add_rmsnorm_mxfp8(int32_t rows, int32_t cols, const uint16_t* x, const uint16_t* residual,
                                     const uint16_t* weight, float eps, uint16_t* sum, uint16_t* y, uint8_t* q,
                                     uint8_t* s, void* stream) {
  if (rows < 0 || cols <= 0 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (cols % 32 || cols > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !weight || (!q) != (!s) || (!sum && !y && !q)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)x, (const void*)residual, (const void*)weight, (const void*)sum, (const void*)y})
    if (reinterpret_cast<uintptr_t>(p) & 15) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(q) & 7) return MOE_ERR_INVALID_ARG;
  const int vecs = cols / 8;
  // Threads of a row and their groups of 8: whatever leaves the fewest threads without values (with 1024 threads of two groups
  // each, rows of 8224 went at 3.9 TB/s), two groups where that is even. At most 512 threads: rows of 16384 took 1024 of two
  // groups 234 us for 8000 rows, 512 of four take 170.
  int vpt = 1, tpr = 4;
  while (tpr < vecs && tpr < 32) tpr *= 2;
  if (vecs > 32) {
    int least = 1 << 30;
    for (int v : {2, 1, 3, 4}) {
      const int t = (vecs + 32 * v - 1) / (32 * v) * 32;
      if (t <= 512 && t * v - vecs < least) least = t * v - vecs, vpt = v, tpr = t;
    }
  }
  const int per = tpr < 256 ? 256 / tpr : 1;
  auto kern = vpt == 1 ? add_rmsnorm_kernel<1> : vpt == 2 ? add_rmsnorm_kernel<2> : vpt == 3 ? add_rmsnorm_kernel<3>
                                                                                           : add_rmsnorm_kernel<4>;
  return launch_pdl(kern, dim3((unsigned)((rows + (long long)per - 1) / per)), dim3(tpr * per), 0,
                    static_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(x),
                    reinterpret_cast<const uint4*>(residual), reinterpret_cast<const uint4*>(weight), eps,
                    reinterpret_cast<uint4*>(sum), reinterpret_cast<uint4*>(y), reinterpret_cast<uint2*>(q), s, (int)rows, vecs,
                    tpr);
}
