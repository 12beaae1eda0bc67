// What the attention kernels share: argument checks, which keys a row sees, and what values that are not finite add to a
// row.
#pragma once
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "ptx.cuh"

namespace moe {

inline bool attention_ok(const moe_attention* a) {
  return a && a->B >= 0 && a->Hq > 0 && a->Hkv > 0 && a->Hq % a->Hkv == 0 && (a->D == 64 || a->D == 128) &&
         a->Hq <= 65535 && a->B <= (1 << 24) && a->window >= 0 && a->sinks >= 0 && std::isfinite(a->scale);
}

inline bool kv_cache_ok(const moe_kv_cache* c) {
  return c && c->pages > 0 && c->Hkv > 0 && (c->D == 64 || c->D == 128) && c->page_size >= 8 && c->page_size <= 256 &&
         (c->page_size & (c->page_size - 1)) == 0 && (c->format == MOE_KV_BF16 || c->format == MOE_KV_MXFP8 || c->format == MOE_KV_MXFP4) &&
         (int64_t)c->pages * c->Hkv < ((int64_t)1 << 31) / c->page_size;
}

inline bool kv_cache_pointers_ok(const moe_kv_cache* c) {
  const bool mx = c->format != MOE_KV_BF16;
  if (!c->k || !c->v || (mx && (!c->k_s || !c->v_s))) return false;
  uintptr_t any = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v);
  if (mx) any |= reinterpret_cast<uintptr_t>(c->k_s) | reinterpret_cast<uintptr_t>(c->v_s);
  return (any & 127) == 0;
}

inline bool status_ws_ok(void* ws, size_t ws_bytes) {
  return ws && !(reinterpret_cast<uintptr_t>(ws) & 255) && ws_bytes >= 256;
}

// The load of each block that is told to wait for more bytes than come (none below zero), by moe_selftest_attention_hold.
int held_load();

// The keys that the row at position p sees are [0, low) and [first, p + 1), low <= first; none for p < 0.
struct Visible {
  int low, first, end;
  __device__ __forceinline__ Visible(int p, int window, int sinks) {
    end = p + 1;
    first = (window && p >= window) ? p + 1 - window : 0;
    low = min(sinks, first);
  }
  __device__ __forceinline__ bool sees(int j) const { return j < end && (j >= first || j < low); }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two bf16, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^(b - 127) of a UE8M0 byte in fp32 (b = 0 is the subnormal 2^-127, b = 255 is NaN).
__device__ __forceinline__ float ue8m0(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

// One E4M3 code in fp32, the format's NaN codes aside.
__device__ __forceinline__ float e4m3(uint32_t c) {
  // sign, exponent and fraction moved into fp32's places give the value times 2^(7 - 127), subnormals too
  return __uint_as_float(((c & 0x80u) << 24) | ((c & 0x7Fu) << 20)) * __uint_as_float((127u + 120u) << 23);
}

// One E2M1 code in fp32.
__device__ __forceinline__ float e2m1(uint32_t c) {
  // as above: exponent and fraction moved into fp32's places give the value times 2^(1 - 127)
  return __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * __uint_as_float((127u + 126u) << 23);
}

// A lane's part of a row of D values: the values lane * D/32 ... in fp32.
template <int D>
struct LaneRow {
  static constexpr int N = D / 32;
  float f[N];
  __device__ __forceinline__ void load_bf16(const uint16_t* row, int lane) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + lane * N + 2 * i);
      f[2 * i] = bf16_lo(w);
      f[2 * i + 1] = bf16_hi(w);
    }
  }
  __device__ __forceinline__ void load_mxfp8(const uint8_t* row, const uint8_t* scales, int lane) {
    const float sc = ue8m0(scales[lane * N / 32]);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = e4m3(row[lane * N + i]) * sc;
  }
  __device__ __forceinline__ void load_mxfp4(const uint8_t* row, const uint8_t* scales, int lane) {
    const float sc = ue8m0(scales[lane * N / 32]);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = e2m1((row[(lane * N + i) / 2] >> (4 * (i & 1))) & 15u) * sc;
  }
};

// The keys of an item that have a value that is not finite and that the product was kept from, because some row of the item
// does not see them: 128 keys a step, a bit each. Only steps at an edge of the mask are looked over. An item of n <= 256
// neighbouring rows has at most 7: steps that hold the end of some rows' keys (n + 126 places for its first key), the
// beginning of their window (n + 126), the end of the first tokens (one).
constexpr int kBadSteps = 8;
struct BadKeys {
  int some;
  int j0[kBadSteps];                    // a step's first key, or -1; used from the first on
  uint32_t keys[kBadSteps][4];
  __device__ __forceinline__ void clear(int lane) {      // by a warp
    if (lane < kBadSteps) j0[lane] = -1;
    (&keys[0][0])[lane] = 0;
    if (lane == 0) some = 0;
  }
  __device__ __forceinline__ void add(int j) {           // by any thread
    for (int s = 0; s < kBadSteps; ++s) {
      const int was = atomicCAS(&j0[s], -1, j & ~127);
      if (was != -1 && was != (j & ~127)) continue;
      atomicOr(&keys[s][(j & 127) / 32], 1u << (j & 31));
      *const_cast<volatile int*>(&some) = 1;
      return;
    }
  }
  template <class F>
  __device__ __forceinline__ void each(const F& f) const {
    for (int s = 0; s < kBadSteps && j0[s] >= 0; ++s)
      for (int w = 0; w < 4; ++w)
        for (uint32_t m = keys[s][w]; m; m &= m - 1) f(j0[s] + 32 * w + __ffs(m) - 1);
  }
};
static_assert(sizeof(BadKeys::keys) == 32 * 4, "a word a lane");

// What those keys add to one row's result, by one warp, its lanes spread over D: values that are not finite, times a weight
// that is above zero, however small, or zero for a score of minus infinity; which size it has does not matter to them. All
// else that the keys have is in the result already. `load(j, k, v)` fetches a key, `add(i, x)` adds x to the result's i-th
// column of the lane. The cost goes with the keys that are listed, not with the row's length.
template <int D, class Load, class Add>
__device__ __forceinline__ void add_not_finite(const BadKeys& bad, const LaneRow<D>& q, const Visible& see, float scale,
                                               const Load& load, const Add& add) {
  constexpr int N = D / 32;
  float acc[N] = {};
  uint32_t hit = 0;
  bad.each([&](int j) {
    if (!see.sees(j)) return;
    LaneRow<D> k, v;
    load(j, k, v);
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < N; ++d) s = fmaf(q.f[d], k.f[d], s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float p = s * scale == -INFINITY ? 0.f : 1.f;
#pragma unroll
    for (int d = 0; d < N; ++d)
      if (!isfinite(v.f[d])) acc[d] += p * v.f[d], hit |= 1u << d;
  });
#pragma unroll
  for (int d = 0; d < N; ++d)
    if ((hit >> d) & 1u) add(d, acc[d]);
}

}  // namespace moe
