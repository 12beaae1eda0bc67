// Attention of a few new rows of every sequence over the paged cache.
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kRowWarps = 8;

struct PagedArgs {
  moe_attention a;
  moe_kv_cache c;
  int rows, max_len, table_width;
  const uint16_t* q;
  long long q_stride;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* out;
  uint32_t* status;
};

// One block per (head, row, sequence), its warps over the keys.
template <int D, bool MX>
__global__ void __launch_bounds__(kRowWarps * 32) paged_rows_kernel(const PagedArgs p) {
  constexpr int N = D / 32;
  __shared__ float sm[kRowWarps], sl[kRowWarps], so[kRowWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.x, r = blockIdx.y % p.rows, hk = h / (p.a.Hq / p.a.Hkv);
  const long long b = blockIdx.y / p.rows;
  int len = p.lens[b];
  if (len < 0 || len > p.max_len) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
    len = 0;
  }
  const Visible see(len == 0 ? -1 : len - p.rows + r, p.a.window, p.a.sinks);
  LaneRow<D> q;
  q.load_bf16(p.q + (b * p.rows + r) * p.q_stride + (long long)h * D, lane);
  float m = -INFINITY, l = 0.f, o[N] = {};
  attend_row<D>(q, see, warp, kRowWarps, p.a.scale * 1.4426950408889634f, m, l, o,
                [&](int j, LaneRow<D>& k, LaneRow<D>& v) {
                  const int page = p.table[b * p.table_width + j / p.c.page_size];
                  if (page < 0 || page >= p.c.pages) {
                    if (lane == 0) atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
                    return false;
                  }
                  const long long row = ((long long)page * p.c.Hkv + hk) * p.c.page_size + j % p.c.page_size;
                  if (MX) {
                    k.load_mxfp8(static_cast<const uint8_t*>(p.c.k) + row * D, p.c.k_s + row * N, lane);
                    v.load_mxfp8(static_cast<const uint8_t*>(p.c.v) + row * D, p.c.v_s + row * N, lane);
                  } else {
                    k.load_bf16(static_cast<const uint16_t*>(p.c.k) + row * D, lane);
                    v.load_bf16(static_cast<const uint16_t*>(p.c.v) + row * D, lane);
                  }
                  return true;
                });
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) so[warp][lane * N + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, tl = 0.f, to = 0.f;
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < kRowWarps; ++w) {
      const float f = exp2f(sm[w] - (top == -INFINITY ? 0.f : top));
      tl += sl[w] * f;
      to += so[w][threadIdx.x] * f;
    }
    reinterpret_cast<__nv_bfloat16*>(p.out)[((b * p.rows + r) * p.a.Hq + h) * D + threadIdx.x] =
        __float2bfloat16_rn(tl == 0.f ? 0.f : to / tl);
  }
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_paged_attention_workspace_bytes(const moe_attention* a, int32_t rows, int32_t max_len) {
  if (!attention_ok(a) || rows < 1 || rows > 64 || max_len < 0) return 0;
  return 256;
}

extern "C" int moe_paged_attention(const moe_attention* a, const moe_kv_cache* cache, int32_t rows, int32_t max_len,
                                   const uint16_t* q, int64_t q_stride, const int32_t* block_table,
                                   int32_t table_width, const int32_t* seq_lens, uint16_t* out, void* ws,
                                   size_t ws_bytes, void* stream) {
  if (!a || !cache) return MOE_ERR_INVALID_ARG;
  if (!attention_ok(a) || !kv_cache_ok(cache) || rows < 1 || rows > 64) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (cache->Hkv != a->Hkv || cache->D != a->D) return MOE_ERR_INVALID_ARG;
  if (max_len < 0 || table_width < 0 || max_len > (int64_t)table_width * cache->page_size) return MOE_ERR_INVALID_ARG;
  if (!status_ws_ok(ws, ws_bytes) || ws_bytes < moe_paged_attention_workspace_bytes(a, rows, max_len))
    return MOE_ERR_WORKSPACE;
  if (a->B == 0) return MOE_OK;
  if (!q || !block_table || !seq_lens || !out || !kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (q_stride < (int64_t)a->Hq * a->D || q_stride % 8) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens)) & 3) return MOE_ERR_INVALID_ARG;
  if ((int64_t)a->B * rows > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
  const PagedArgs p{*a, *cache, rows, max_len, table_width, q, q_stride, block_table, seq_lens, out,
                    static_cast<uint32_t*>(ws)};
  const bool mx = cache->format == MOE_KV_MXFP8;
  auto kern = a->D == 64 ? (mx ? paged_rows_kernel<64, true> : paged_rows_kernel<64, false>)
                         : (mx ? paged_rows_kernel<128, true> : paged_rows_kernel<128, false>);
  kern<<<dim3(a->Hq, a->B * rows), kRowWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}
