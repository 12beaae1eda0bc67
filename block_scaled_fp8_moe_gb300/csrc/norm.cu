// Residual addition, RMS norm and MXFP8 quantisation of rows in one pass over them.
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

// TPR threads hold one row in registers, VPT groups of 8 values each; a block holds ROWS rows.
template <int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
add_rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* __restrict__ weight, float eps, uint4* sum,
                   uint4* y, uint2* __restrict__ q, uint8_t* __restrict__ s, int rows, int vecs) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  constexpr int WARPS = TPR / 32;
  __shared__ float part[ROWS * WARPS];
  pdl_trigger();
  const int t = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
  const bool live = row < rows;
  pdl_wait();
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * TPR;
    const bool in = live && c < vecs;
    const uint4 a = in ? x[row * vecs + c] : make_uint4(0, 0, 0, 0);
    const uint4 b = in && residual ? residual[row * vecs + c] : make_uint4(0, 0, 0, 0);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
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
    if (sum && in)
      sum[row * vecs + c] = make_uint4(bf16x2(h[i][0], h[i][1]), bf16x2(h[i][2], h[i][3]), bf16x2(h[i][4], h[i][5]),
                                       bf16x2(h[i][6], h[i][7]));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (WARPS > 1) {
    if ((t & 31) == 0) part[threadIdx.x / 32] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) ss += part[threadIdx.x / TPR * WARPS + i];
  }
  const float r = 1.f / sqrtf(ss / (float)(vecs * 8) + eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * TPR;
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
    // 4 lanes hold a block of 32 values (vecs is a multiple of 4)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int se = e4m3_scale_exp(m);
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
  auto go = [&](auto kern, int tpr) {
    const int per = tpr < 256 ? 256 / tpr : 1;
    return launch_pdl(kern, dim3((rows + per - 1) / per), dim3(tpr < 256 ? 256 : tpr), 0,
                      static_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(x),
                      reinterpret_cast<const uint4*>(residual), reinterpret_cast<const uint4*>(weight), eps,
                      reinterpret_cast<uint4*>(sum), reinterpret_cast<uint4*>(y), reinterpret_cast<uint2*>(q), s,
                      (int)rows, vecs);
  };
  if (vecs <= 64) return go(add_rmsnorm_kernel<32, 2>, 32);
  if (vecs <= 128) return go(add_rmsnorm_kernel<64, 2>, 64);
  if (vecs <= 256) return go(add_rmsnorm_kernel<128, 2>, 128);
  if (vecs <= 512) return go(add_rmsnorm_kernel<256, 2>, 256);
  if (vecs <= 1024) return go(add_rmsnorm_kernel<512, 2>, 512);
  return go(add_rmsnorm_kernel<1024, 2>, 1024);
}
