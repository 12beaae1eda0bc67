// New tokens' keys and values into the paged cache, copied (bf16) or quantised (MXFP8, MXFP4).
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 2;

// A thread has 8 values (16 bytes) of `kAppendUnroll` tokens at a time, all loaded before any is written; 4 neighbouring lanes
// have one block of 32. `group` threads (a power of two, up to a block) share a token, its keys first, then its values.
// Bound: HBM, 4 bytes a value in bf16, 3.03 in MXFP8 and 2.53 in MXFP4. Two tokens at a time: with four, 48 tokens took 2.5 us in
// MXFP8 instead of 1.6, with one, 20011 tokens 31.6 us instead of 28.
template <int FMT>
__global__ void __launch_bounds__(kAppendThreads, 8)
kv_append_kernel(const moe_kv_cache c, int T, const uint16_t* __restrict__ k, long long k_stride,
                 const uint16_t* __restrict__ v, long long v_stride, const int32_t* __restrict__ slots, int group_log2,
                 int page_log2, uint32_t* status) {
  constexpr int U = kAppendUnroll;
  constexpr bool MX4 = FMT == MOE_KV_MXFP4;
  pdl_trigger();
  pdl_wait();
  const int head_log2 = c.D == 128 ? 4 : 3, per_tok = c.Hkv << head_log2;     // 16-byte parts of a head, of a token's keys
  const int tokens = kAppendThreads >> group_log2;                           // of a block at a time
  const int t0 = blockIdx.x * (tokens * U) + (threadIdx.x >> group_log2);
  const long long n_slots = (long long)c.pages << page_log2;
  // groups of less than a token's parts go through them in turns; every lane goes along (the shuffles need it)
  for (int e0 = 0; e0 < 2 * per_tok; e0 += 1 << group_log2) {
    const int e = e0 + (threadIdx.x & ((1 << group_log2) - 1));
    const bool part = e < 2 * per_tok, is_v = e >= per_tok;
    const int x = is_v ? e - per_tok : e, h = x >> head_log2, d8 = x & ((1 << head_log2) - 1);
    const uint16_t* src = (is_v ? v : k) + x * 8;
    const long long stride = is_v ? v_stride : k_stride;
    uint4 a[U];
    int slot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * tokens;
      const bool there = part && t < T;
      slot[u] = there ? __ldg(slots + t) : -1;
      a[u] = there ? __ldcs(reinterpret_cast<const uint4*>(src + t * stride)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = slot[u] >= 0 && slot[u] < n_slots;
      if (!in && slot[u] != -1 && e == 0) atomicCAS(status, 0u, (uint32_t)DEV_BAD_INPUT);
      const long long page = in ? slot[u] >> page_log2 : 0;
      const long long row = ((page * c.Hkv + h) << page_log2) + (in ? slot[u] & (c.page_size - 1) : 0);
      if (FMT == MOE_KV_BF16) {
        if (in) reinterpret_cast<uint4*>(is_v ? c.v : c.k)[(row << head_log2) + d8] = a[u];
      } else {
        // the largest magnitude by its bits: what is not finite lies above all else
        const uint32_t w[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        const unsigned four = 0xFu << (threadIdx.x & 28);
        m2 = __vmaxu2(m2, __shfl_xor_sync(four, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(four, m2, 2));
        const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        const bool finite = m < 0x7F80u;
        const int se = MX4 ? e2m1_scale_exp(__uint_as_float(m << 16)) : e4m3_scale_exp_bf16(m);
        const float sc = pow2_neg(se);
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
        // a row's scale bytes in one word: bytes of the lanes 4, 8 and 12 behind the row's first
        uint32_t sb = finite ? (uint32_t)(se + 127) : 255u;
        sb |= __shfl_down_sync(0xffffffffu, sb, 4) << 8;
        sb |= __shfl_down_sync(0xffffffffu, sb, 8) << 16;
        if (in) {
          if constexpr (MX4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= sc;
            reinterpret_cast<uint32_t*>(is_v ? c.v : c.k)[(row << head_log2) + d8] = finite ? e2m1x8(f) : 0u;
          } else {
            uint2 codes = make_uint2(0, 0);
            if (finite)
              codes = make_uint2(e4m3x2(f[0] * sc, f[1] * sc) | (e4m3x2(f[2] * sc, f[3] * sc) << 16),
                                 e4m3x2(f[4] * sc, f[5] * sc) | (e4m3x2(f[6] * sc, f[7] * sc) << 16));
            reinterpret_cast<uint2*>(is_v ? c.v : c.k)[(row << head_log2) + d8] = codes;
          }
          uint8_t* scales = (is_v ? c.v_s : c.k_s) + (row << (head_log2 - 2));
          if (d8 == 0) {
            if (head_log2 == 4) *reinterpret_cast<uint32_t*>(scales) = sb;
            else *reinterpret_cast<uint16_t*>(scales) = (uint16_t)sb;
          }
        }
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
  int group_log2 = 4, page_log2 = 3;
  while ((1 << group_log2) < 2 * row / 8 && (1 << group_log2) < kAppendThreads) ++group_log2;
  while ((1 << page_log2) < cache->page_size) ++page_log2;
  const int per_block = (kAppendThreads >> group_log2) * kAppendUnroll;
  auto kern = cache->format == MOE_KV_MXFP8   ? kv_append_kernel<MOE_KV_MXFP8>
              : cache->format == MOE_KV_MXFP4 ? kv_append_kernel<MOE_KV_MXFP4>
                                              : kv_append_kernel<MOE_KV_BF16>;
  return launch_pdl(kern, dim3((unsigned)((T + (long long)per_block - 1) / per_block)), dim3(kAppendThreads), 0,
                    static_cast<cudaStream_t>(stream), *cache, (int)T, k, (long long)k_stride, v, (long long)v_stride, slots,
                    group_log2, page_log2, static_cast<uint32_t*>(ws));
}
