// Attention of whole prompts, packed one behind the other.
#include <cuda_runtime.h>

#include "attention.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

struct PrefillArgs {
  moe_attention a;
  int Tq, Tk;
  const uint16_t* q;
  long long q_stride;
  const uint16_t* k;
  long long k_stride;
  const uint16_t* v;
  long long v_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  uint32_t* status;
};

struct Span {
  int q0, qn, k0, kn;   // a sequence's first query row and their number, its first key and theirs
};

// Sequence b's rows; empty (and recorded) where its entries break the rule.
__device__ __forceinline__ Span span_of(const PrefillArgs& p, int b) {
  Span s;
  s.q0 = p.cu_q[b];
  s.qn = p.cu_q[b + 1] - s.q0;
  s.k0 = p.cu_k[b];
  s.kn = p.cu_k[b + 1] - s.k0;
  if (s.q0 < 0 || s.qn < 0 || s.q0 > p.Tq - s.qn || s.k0 < 0 || s.kn < 0 || s.k0 > p.Tk - s.kn ||
      (b == 0 && (s.q0 || s.k0))) {
    atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
    s.qn = s.kn = 0;
  }
  return s;
}

// One warp per (row, head): the row's sequence by a walk over cu_q.
template <int D>
__global__ void __launch_bounds__(256) prefill_rows_kernel(const PrefillArgs p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x % 32, h = blockIdx.y, hk = h / (p.a.Hq / p.a.Hkv);
  const int t = blockIdx.x * 8 + threadIdx.x / 32;
  Span s{0, 0, 0, 0};
  for (int b = 0; b < p.a.B; ++b) {
    s = span_of(p, b);
    if (t >= s.q0 && t < s.q0 + s.qn) break;
    s.qn = 0;
  }
  if (s.qn == 0) return;
  const Visible see(s.kn - s.qn + t - s.q0, p.a.window, p.a.sinks);
  LaneRow<D> q;
  q.load_bf16(p.q + (long long)t * p.q_stride + (long long)h * D, lane);
  float m = -INFINITY, l = 0.f, o[N] = {};
  attend_row<D>(q, see, 0, 1, p.a.scale * 1.4426950408889634f, m, l, o, [&](int j, LaneRow<D>& k, LaneRow<D>& v) {
    k.load_bf16(p.k + (long long)(s.k0 + j) * p.k_stride + (long long)hk * D, lane);
    v.load_bf16(p.v + (long long)(s.k0 + j) * p.v_stride + (long long)hk * D, lane);
    return true;
  });
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + ((long long)t * p.a.Hq + h) * D + lane * N);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) out[i] = bf16x2(l == 0.f ? 0.f : o[2 * i] * inv, l == 0.f ? 0.f : o[2 * i + 1] * inv);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_prefill_attention(const moe_attention* a, int32_t Tq, int32_t Tk, const uint16_t* q,
                                     int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                     int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, uint16_t* out,
                                     void* ws, size_t ws_bytes, void* stream) {
  if (!a || Tq < 0 || Tk < 0) return MOE_ERR_INVALID_ARG;
  if (!attention_ok(a)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!status_ws_ok(ws, ws_bytes)) return MOE_ERR_WORKSPACE;
  if (a->B == 0 || Tq == 0) return MOE_OK;
  if (!q || !cu_q || !out || (Tk && (!k || !v))) return MOE_ERR_INVALID_ARG;
  const int64_t qr = (int64_t)a->Hq * a->D, kr = (int64_t)a->Hkv * a->D;
  if (q_stride < qr || k_stride < kr || v_stride < kr || (q_stride | k_stride | v_stride) % 8) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3) return MOE_ERR_INVALID_ARG;
  const PrefillArgs p{*a, Tq, Tk, q, q_stride, k, k_stride, v, v_stride, cu_q, cu_k ? cu_k : cu_q, out,
                      static_cast<uint32_t*>(ws)};
  auto kern = a->D == 64 ? prefill_rows_kernel<64> : prefill_rows_kernel<128>;
  kern<<<dim3((Tq + 7) / 8, a->Hq), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}
