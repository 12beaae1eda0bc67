// New tokens' keys and values into the paged cache, copied (bf16) or quantised (MXFP8).
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

// One thread per 8 values (16 bytes in); 4 neighbouring lanes hold one block of 32.
template <bool MX>
__global__ void __launch_bounds__(256)
kv_append_kernel(moe_kv_cache c, int T, const uint16_t* __restrict__ k, long long k_stride,
                 const uint16_t* __restrict__ v, long long v_stride, const int32_t* __restrict__ slots,
                 uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int per_head = c.D / 8, per_tok = c.Hkv * per_head;
  const long long total = 2LL * T * per_tok;     // of every token: its keys, then its values
  const long long n_slots = (long long)c.pages * c.page_size;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long tk = i / per_tok;
    const int e = (int)(i - tk * per_tok);
    const long long t = tk >> 1;
    const bool is_v = tk & 1;
    const int slot = __ldg(slots + t);
    const int h = e / per_head, d8 = e % per_head;
    const uint4 a = *reinterpret_cast<const uint4*>((is_v ? v + t * v_stride : k + t * k_stride) + e * 8);
    const bool in = slot >= 0 && slot < n_slots;
    if (!in && slot != -1 && e == 0 && !is_v) atomicCAS(status, 0u, (uint32_t)DEV_BAD_INPUT);
    const long long row = in ? ((long long)(slot / c.page_size) * c.Hkv + h) * c.page_size + slot % c.page_size : 0;
    if (!MX) {
      if (in) reinterpret_cast<uint4*>(is_v ? c.v : c.k)[row * per_head + d8] = a;
    } else {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
      float f[8], m = 0.f;
      bool finite = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
        finite = finite && (w[j] & 0x7F80u) != 0x7F80u && (w[j] & 0x7F800000u) != 0x7F800000u;
      }
      // total is a multiple of 4 and so is the first index of a group: a group's lanes are all here
      const unsigned group = 0xFu << (threadIdx.x & 28);
      finite = __all_sync(group, finite);
      m = fmaxf(m, __shfl_xor_sync(group, m, 1));
      m = fmaxf(m, __shfl_xor_sync(group, m, 2));
      const int se = e4m3_scale_exp(m);
      const float sc = finite ? pow2_neg(se) : 0.f;
      if (in) {
        uint2 codes = make_uint2(0, 0);
        if (finite)
          codes = make_uint2(e4m3x2(f[0] * sc, f[1] * sc) | (e4m3x2(f[2] * sc, f[3] * sc) << 16),
                             e4m3x2(f[4] * sc, f[5] * sc) | (e4m3x2(f[6] * sc, f[7] * sc) << 16));
        reinterpret_cast<uint2*>(is_v ? c.v : c.k)[row * per_head + d8] = codes;
        if ((d8 & 3) == 0) (is_v ? c.v_s : c.k_s)[row * (c.D / 32) + d8 / 4] = finite ? (uint8_t)(se + 127) : 255;
      }
    }
  }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_kv_append(const moe_kv_cache* cache, int32_t T, const uint16_t* k, int64_t k_stride,
                             const uint16_t* v, int64_t v_stride, const int32_t* slots, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!cache || T < 0) return MOE_ERR_INVALID_ARG;
  if (!kv_cache_ok(cache)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!status_ws_ok(ws, ws_bytes)) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  const int64_t row = (int64_t)cache->Hkv * cache->D;
  if (!k || !v || !slots || !kv_cache_pointers_ok(cache) || k_stride < row || v_stride < row || k_stride % 8 ||
      v_stride % 8)
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slots) & 3) return MOE_ERR_INVALID_ARG;
  const long long total = 2LL * T * row / 8;
  const int blocks = (int)std::min<long long>((total + 255) / 256, (long long)num_sms() * 8);
  auto kern = cache->format == MOE_KV_MXFP8 ? kv_append_kernel<true> : kv_append_kernel<false>;
  return launch_pdl(kern, dim3(blocks), dim3(256), 0, static_cast<cudaStream_t>(stream), *cache, (int)T, k,
                    (long long)k_stride, v, (long long)v_stride, slots, static_cast<uint32_t*>(ws));
}
