// Rotary positions: heads of queries and keys turned by their tokens' positions, alone (moe_rope) or on the way into the paged
// cache (moe_rope_kv_append).
//
// Pair i of a head, (a, b), goes to (a cos t - b sin t, a sin t + b cos t) with t = position * w_i. An angle is needed modulo
// one turn only, so w_i is held as the 64-bit integer 2^64 w_i / 2 pi: its product with the position, modulo 2^64, is the
// fraction of the turn, off by less than 2^-33 of one for any 32-bit position (fp32 angles would be off by 0.06 rad at a
// million); in fp32, from where the cosine takes it, by 2^-26.
//
// Bound: HBM, 4 bytes a value turned; what is stored adds 2, 1.03 or 0.53 a value and 2 read. Cosines and sines are worked out
// once for all heads of a token, left in shared memory, and held by every thread for its own places in a head. All of a head that
// a warp writes it has read before, so rows may be turned where they are.
//
// 20011 tokens of 32 heads over 8 of 128 into a bf16 cache: 84 us, 5.8 TB/s. 16384 tokens of 16 and 16 heads of 80, turned back: 36 us,
// 4.7 TB/s. 3061 tokens into an MXFP4 cache: 19 us, 3.5 TB/s, the quantisation's arithmetic. With a chunk a lane and the other half
// from another lane, cosines by every warp, these take 147, 55 and 29 us. 6 tokens: 2.4 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kRopeWarps = 8;
constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxT = 1 << 30;
constexpr int kNoCache = -1;

struct RopeArgs {
  int half, axes;                       // pairs; positions of a token
  int back;                             // the other way round
  float factor;
  const uint64_t* turns;
  const uint8_t* axis;
  int T, D, lanes;                      // lanes of a head
  int Hq, Hk, Hv;                       // heads turned into q_out, into k_out and the cache, stored as they are
  int groups;                           // heads of a token in groups of a warp's width
  int tokens;                           // tokens of a block
  int per, parts;                       // the general kernel's: groups of a warp; warps of a token
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* pos;
  long long pos_stride;
  uint16_t* q_out;
  uint16_t* k_out;
  long long qo_stride, ko_stride;
  moe_kv_cache c;
  int page_log2;
  const int32_t* slots;
  uint32_t* status;
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint16_t* p) {
  if constexpr (N == 4) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N]) {
  if constexpr (N == 4) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 2) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *static_cast<uint32_t*>(p) = w[0];
}

// A lane's VEC values, which are 1/4 (1/8) of a block, in the cache's MX format: the block's scale byte, and the codes. All lanes of
// the warp call this.
template <int VEC, int FMT, int N>
__device__ __forceinline__ uint32_t mx_codes(const float (&f)[VEC], uint32_t (&w)[N]) {
  static_assert(N == (FMT == MOE_KV_MXFP8 ? VEC / 4 : 1), "words of codes");
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < VEC; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);    // what is not finite lies above all else
#pragma unroll
  for (int d = 1; d < 32 / VEC; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool finite = m < 0x7F800000u;
  const uint32_t byte = FMT == MOE_KV_MXFP8 ? mx_scale_byte<8, 0x600000u>(m) : mx_scale_byte<2, 0x400000u>(m);
  const float sc = __uint_as_float((254u - byte) << 23);
  float x[8] = {};
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = f[e] * sc;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (FMT == MOE_KV_MXFP8) w[i] = e4m3x2(x[4 * i], x[4 * i + 1]) | e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16;
    else w[i] = e2m1x8(x);
    if (!finite) w[i] = 0;
  }
  return finite ? byte : 255u;
}

// VEC values of a row that go into the cache, from value d0 on; `row` counts the cache's rows of D values. All lanes of the warp
// call this; `mine`: this lane's are stored.
template <int VEC, int FMT>
__device__ __forceinline__ void store_kv(const RopeArgs& a, const float (&f)[VEC], const uint32_t (&o)[VEC / 2], bool mine,
                                         bool is_v, long long row, int d0) {
  uint8_t* data = static_cast<uint8_t*>(is_v ? a.c.v : a.c.k);
  if constexpr (FMT == MOE_KV_BF16) {
    if (mine) store_words(reinterpret_cast<uint16_t*>(data) + row * a.D + d0, o);
  } else {
    uint32_t w[FMT == MOE_KV_MXFP8 ? VEC / 4 : 1];
    const uint32_t byte = mx_codes<VEC, FMT>(f, w);
    if (!mine) return;
    if constexpr (FMT == MOE_KV_MXFP8) store_words(data + row * a.D + d0, w);
    else if constexpr (VEC == 8) *reinterpret_cast<uint32_t*>(data + (row * a.D + d0) / 2) = w[0];
    else *reinterpret_cast<uint16_t*>(data + (row * a.D + d0) / 2) = (uint16_t)w[0];
    if (d0 % 32 == 0) (is_v ? a.c.v_s : a.c.k_s)[(row * a.D + d0) / 32] = (uint8_t)byte;
  }
}

// The cosine and sine of pair i of token t.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int t, int i) {
  const int x = a.axis ? min((int)a.axis[i], a.axes - 1) : 0;
  uint64_t n = (uint64_t)(long long)a.pos[x * a.pos_stride + t] * a.turns[i];
  if (a.back) n = 0 - n;
  float s, c;
  sincospif((float)(int32_t)((n + 0x80000000u) >> 32) * 0x1p-31f, &s, &c);    // the fraction in half turns, from -1 to 1
  return make_float2(c * a.factor, s * a.factor);
}

// Where a token is stored: its row in head 0 of its page, or -1.
__device__ __forceinline__ long long kv_row(const RopeArgs& a, int t, bool report) {
  const int slot = a.slots[t];
  const bool in = slot >= 0 && slot < (long long)a.c.pages << a.page_log2;
  if (!in && slot != -1 && report) atomicCAS(a.status, 0u, (uint32_t)DEV_BAD_INPUT);
  return in ? (((long long)(slot >> a.page_log2) * a.c.Hkv) << a.page_log2) + (slot & (a.c.page_size - 1)) : -1;
}

// Head u of a token's q, k and v, as they are read.
__device__ __forceinline__ const uint16_t* row_of(const RopeArgs& a, int t, int u) {
  return u < a.Hq        ? a.q + t * a.q_stride + u * a.D
         : u < a.Hq + a.Hk ? a.k + t * a.k_stride + (u - a.Hq) * a.D
                           : a.v + t * a.v_stride + (u - a.Hq - a.Hk) * a.D;
}

// A thread has two chunks of 8 values of a head, which are the halves of 8 pairs, or 4 pairs each (PAIRS: neighbours), or two that
// are copied; D / 16 threads a head. So no value passes from lane to lane. A block takes `tokens` tokens (1, 2, 4 or 8): its threads
// work out their cosines and sines together, while the first heads are on their way, and its warps share the tokens' heads.
template <bool PAIRS, int FMT>
__global__ void __launch_bounds__(kRopeWarps * 32, FMT == kNoCache || FMT == MOE_KV_BF16 ? 4 : 3)
rope_paired_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int U = 2;                  // groups of heads under way; 1 and 3 are slower or the same, and so are other numbers of blocks
  __shared__ float2 turn[kRopeWarps][kRopeMaxD / 2];    // by token of the block
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int share = kRopeWarps / a.tokens, mine = warp / share;          // warps of a token
  const int t = min((int)blockIdx.x * a.tokens + mine, a.T - 1);
  const bool there = blockIdx.x * (long long)a.tokens + mine < a.T;
  const int heads = 32 / a.lanes, in_warp = lane / a.lanes, l = lane - in_warp * a.lanes;
  const int n = a.half / 8, tail = a.lanes - n;         // lanes of what is turned, of what is not
  const bool turned = l < n;
  const int d0 = 8 * (turned ? l : n + l), d1 = d0 + 8 * (turned ? n : tail);
  const int units = in_warp < heads && there ? a.Hq + a.Hk + a.Hv : 0;

  uint32_t x[U][2][4];
  auto fetch = [&](int g0) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = (g0 + j * share) * heads + in_warp;
      if (u < units) {
        const uint16_t* row = row_of(a, t, u);
        load_words(x[j][0], row + d0);
        load_words(x[j][1], row + d1);
      }
    }
  };
  int g0 = warp - mine * share;
  fetch(g0);
  for (int i = threadIdx.x; i < a.tokens * a.half; i += kRopeWarps * 32) {
    const int k = i / a.half, at = blockIdx.x * a.tokens + k;
    if (at < a.T) turn[k][i - k * a.half] = turn_of(a, at, i - k * a.half);
  }
  long long row0 = -1;
  if constexpr (FMT != kNoCache) {
    if (there) row0 = kv_row(a, t, lane == 0 && warp == mine * share);
  }
  __syncthreads();
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // of neighbours, chunk d0 has pairs d0 / 2 to d0 / 2 + 3, and d1 the other four
    const float2 cs = turned ? turn[mine][PAIRS ? (e < 4 ? d0 / 2 + e : d1 / 2 + e - 4) : d0 + e] : make_float2(1.f, 0.f);
    c[e] = cs.x, s[e] = cs.y;
  }

  for (; g0 < a.groups; g0 += U * share) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g0 + j * share >= a.groups) break;
      const int u = (g0 + j * share) * heads + in_warp;
      const bool is_q = u < min(a.Hq, units), is_k = !is_q && u < min(a.Hq + a.Hk, units), is_v = !is_q && !is_k && u < units;
      float f[2][8];
      uint32_t o[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[h][e] = x[j][h][e];         // copies keep their bits
          f[h][2 * e] = bf16_lo(x[j][h][e]);
          f[h][2 * e + 1] = bf16_hi(x[j][h][e]);
        }
      if (turned && !is_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& p = PAIRS ? f[e / 4][2 * (e % 4)] : f[0][e];
          float& q = PAIRS ? f[e / 4][2 * (e % 4) + 1] : f[1][e];
          const float p0 = p, q0 = q;
          p = p0 * c[e] - q0 * s[e];
          q = p0 * s[e] + q0 * c[e];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][e] = bf16x2(f[h][2 * e], f[h][2 * e + 1]);
      }
      if (is_q || (is_k && a.k_out)) {
        uint16_t* to = is_q ? a.q_out + t * a.qo_stride + u * a.D : a.k_out + t * a.ko_stride + (u - a.Hq) * a.D;
        store_words(to + d0, o[0]);
        store_words(to + d1, o[1]);
      }
      if constexpr (FMT != kNoCache) {
        const bool in = row0 >= 0 && (is_k || is_v);
        if (__any_sync(0xffffffffu, in)) {
          const long long row = row0 + ((long long)(is_v ? u - a.Hq - a.Hk : u - a.Hq) << a.page_log2);
          store_kv<8, FMT>(a, f[0], o[0], in, is_v, row, d0);
          store_kv<8, FMT>(a, f[1], o[1], in, is_v, row, d1);
        }
      }
    }
    fetch(g0 + U * share);
  }
}

// Heads whose halves, or whose blocks of 32, do not lie so: a lane has one chunk of a head, of 8 values, or 4 where the turned
// part's second half would begin inside 8, and the other half of its pairs comes from another lane. A warp takes a part of a token
// and works out its cosines and sines.
template <int VEC, bool PAIRS, int FMT>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 turn[kRopeWarps][kRopeMaxD / 2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long wid = (long long)blockIdx.x * kRopeWarps + warp;
  const int t = (int)(wid / a.parts), part = (int)(wid - (long long)t * a.parts);
  pdl_trigger();
  pdl_wait();
  if (t >= a.T) return;
  const int heads = 32 / a.lanes, in_warp = lane / a.lanes, ch = lane - in_warp * a.lanes;
  const int d0 = ch * VEC, rot = 2 * a.half, units = in_warp < heads ? a.Hq + a.Hk + a.Hv : 0;
  const int end = min(a.groups, (part + 1) * a.per);

  for (int i = lane; i < a.half; i += 32) turn[warp][i] = turn_of(a, t, i);
  long long row0 = -1;
  if constexpr (FMT != kNoCache) row0 = kv_row(a, t, lane == 0 && part == 0);
  __syncwarp();
  const bool turned = d0 < rot, second = d0 >= a.half;
  float c[VEC], s[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float2 cs = turned ? turn[warp][PAIRS ? d0 / 2 + e / 2 : second ? d0 - a.half + e : d0 + e] : make_float2(1.f, 0.f);
    c[e] = cs.x;
    s[e] = (PAIRS ? (e & 1) == 0 : !second) ? -cs.y : cs.y;
  }
  const int far = turned && !PAIRS ? (second ? lane - a.half / VEC : lane + a.half / VEC) : lane;

  for (int g = part * a.per; g < end; ++g) {
    const int u = g * heads + in_warp;
    const bool is_q = u < min(a.Hq, units), is_k = !is_q && u < min(a.Hq + a.Hk, units), is_v = !is_q && !is_k && u < units;
    uint32_t w[VEC / 2] = {}, o[VEC / 2];
    if (u < units) load_words(w, row_of(a, t, u) + d0);
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const uint32_t other = PAIRS ? (w[e] >> 16) | (w[e] << 16) : __shfl_sync(0xffffffffu, w[e], far & 31);
      f[2 * e] = bf16_lo(w[e]);
      f[2 * e + 1] = bf16_hi(w[e]);
      o[e] = w[e];                      // copies keep their bits
      if (turned && !is_v) {
        f[2 * e] = f[2 * e] * c[2 * e] + bf16_lo(other) * s[2 * e];
        f[2 * e + 1] = f[2 * e + 1] * c[2 * e + 1] + bf16_hi(other) * s[2 * e + 1];
        o[e] = bf16x2(f[2 * e], f[2 * e + 1]);
      }
    }
    if (is_q) store_words(a.q_out + t * a.qo_stride + u * a.D + d0, o);
    if (is_k && a.k_out) store_words(a.k_out + t * a.ko_stride + (u - a.Hq) * a.D + d0, o);
    if constexpr (FMT != kNoCache) {
      const bool in = row0 >= 0 && (is_k || is_v);
      if (__any_sync(0xffffffffu, in))
        store_kv<VEC, FMT>(a, f, o, in, is_v, row0 + ((long long)(is_v ? u - a.Hq - a.Hk : u - a.Hq) << a.page_log2), d0);
    }
  }
}

// The rotary description and the rows, checked and laid out; what has to do with the cache is the caller's.
static int rope_args(RopeArgs& p, const moe_rotary* r, int T, int Hq, int Hk, int Hv, int D, const uint16_t* q,
                     int64_t q_stride, const uint16_t* k, int64_t k_stride, const int32_t* pos, int64_t pos_stride,
                     uint16_t* q_out, int64_t qo_stride, uint16_t* k_out, int64_t ko_stride) {
  if (!r->turns || !pos || (reinterpret_cast<uintptr_t>(r->turns) & 7) || (reinterpret_cast<uintptr_t>(pos) & 3) ||
      pos_stride < T)
    return MOE_ERR_INVALID_ARG;
  auto rows_ok = [&](const uint16_t* x, int64_t stride, int heads) {
    return x && !(reinterpret_cast<uintptr_t>(x) & 15) && stride % 8 == 0 && stride >= (int64_t)heads * D;
  };
  if (Hq && (!rows_ok(q, q_stride, Hq) || !rows_ok(q_out, qo_stride, Hq))) return MOE_ERR_INVALID_ARG;
  if (Hk && (!rows_ok(k, k_stride, Hk) || (k_out && !rows_ok(k_out, ko_stride, Hk)))) return MOE_ERR_INVALID_ARG;
  p.half = r->dim / 2;
  p.axes = r->axes;
  p.back = r->inverse != 0;
  p.factor = r->factor;
  p.turns = r->turns;
  p.axis = r->axis;
  p.T = T, p.D = D, p.Hq = Hq, p.Hk = Hk, p.Hv = Hv;
  p.q = q, p.k = k, p.q_stride = q_stride, p.k_stride = k_stride;
  p.pos = pos, p.pos_stride = pos_stride;
  p.q_out = q_out, p.k_out = k_out, p.qo_stride = qo_stride, p.ko_stride = ko_stride;
  return MOE_OK;
}

static bool rotary_ok(const moe_rotary* r, int D) {
  return r->dim >= 8 && r->dim <= D && r->dim % 8 == 0 && r->axes >= 1 && r->axes <= 4 && std::isfinite(r->factor) &&
         D % 8 == 0 && D <= kRopeMaxD;
}

// The general kernel's lanes take 8 values, or 4 where the second half of a turned head would begin inside 8: half the bytes a load,
// for which the head has to fit 32 lanes.
static int rope_vec(const moe_rotary* r) { return !r->interleaved && r->dim % 16 ? 4 : 8; }

template <int VEC, bool PAIRS>
static void (*rope_kernel_of(int format))(RopeArgs) {
  switch (format) {
    case MOE_KV_BF16: return rope_kernel<VEC, PAIRS, MOE_KV_BF16>;
    case MOE_KV_MXFP8: return rope_kernel<VEC, PAIRS, MOE_KV_MXFP8>;
    case MOE_KV_MXFP4: return rope_kernel<VEC, PAIRS, MOE_KV_MXFP4>;
    default: return rope_kernel<VEC, PAIRS, kNoCache>;
  }
}
template <bool PAIRS>
static void (*rope_paired_of(int format))(RopeArgs) {
  switch (format) {
    case MOE_KV_BF16: return rope_paired_kernel<PAIRS, MOE_KV_BF16>;
    case MOE_KV_MXFP8: return rope_paired_kernel<PAIRS, MOE_KV_MXFP8>;
    case MOE_KV_MXFP4: return rope_paired_kernel<PAIRS, MOE_KV_MXFP4>;
    default: return rope_paired_kernel<PAIRS, kNoCache>;
  }
}

static int launch_rope(RopeArgs& p, bool pairs, int vec, int format, cudaStream_t st) {
  const int rot = 2 * p.half, heads = p.Hq + p.Hk + p.Hv;
  const bool blocks_fit = format == kNoCache || format == MOE_KV_BF16 || (rot % 64 == 0 && p.D % 64 == 0);
  if (rot % 16 == 0 && p.D % 16 == 0 && blocks_fit) {
    p.lanes = p.D / 16;
    p.groups = ceil_div(heads, 32 / p.lanes);
    // Tokens of a block: as many as leave a warp no more than 8 groups of heads and the GPU 4 blocks a multiprocessor.
    p.tokens = kRopeWarps;
    while (p.tokens > 1 && (p.groups > 8 * (kRopeWarps / p.tokens) || p.T < 4ll * num_sms() * p.tokens)) p.tokens /= 2;
    return launch_pdl(pairs ? rope_paired_of<true>(format) : rope_paired_of<false>(format),
                      dim3((unsigned)ceil_div(p.T, p.tokens)), dim3(kRopeWarps * 32), 0, st, p);
  }
  p.lanes = ceil_div(p.D, vec);
  p.groups = ceil_div(heads, 32 / p.lanes);
  // As many groups a warp as leave every multiprocessor 32 warps, at least 2 and at most 16.
  const long long all = (long long)p.T * p.groups, slots = (long long)num_sms() * 32;
  p.per = (int)std::max(2ll, std::min(16ll, all / slots));
  p.parts = ceil_div(p.groups, p.per);
  const long long warps = (long long)p.T * p.parts, blocks = (warps + kRopeWarps - 1) / kRopeWarps;
  if (blocks >= (1ll << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  auto kern = vec == 4 ? rope_kernel_of<4, false>(format)
              : pairs  ? rope_kernel_of<8, true>(format)
                       : rope_kernel_of<8, false>(format);
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(kRopeWarps * 32), 0, st, p);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_rotary_turns(int32_t n, const double* inv_freq, uint64_t* turns) {
  if (n < 0 || (n && (!inv_freq || !turns))) return MOE_ERR_INVALID_ARG;
  // 1 / 2 pi in two doubles: the product's first part is exact with its remainder
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1e6)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double w = std::fabs(inv_freq[i]), t = w * hi, rest = std::fma(w, hi, -t) + w * lo;
    // t - floor(t) is exact and below one; in 64 bits whole but for what lies below 2^-64
    const double f = std::ldexp(t - std::floor(t), 64), whole = std::floor(f);
    const uint64_t n = static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint(f - whole + std::ldexp(rest, 64)));
    turns[i] = inv_freq[i] < 0 ? 0 - n : n;
  }
  return MOE_OK;
}

extern "C" int moe_rope(const moe_rotary* r, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, const uint16_t* q,
                        int64_t q_stride, const uint16_t* k, int64_t k_stride, const int32_t* pos, int64_t pos_stride,
                        uint16_t* q_out, int64_t qo_stride, uint16_t* k_out, int64_t ko_stride, void* stream) {
  if (!r || T < 0 || Hq < 0 || Hkv < 0 || D <= 0) return MOE_ERR_INVALID_ARG;
  const int vec = rope_vec(r);
  if (!rotary_ok(r, D) || D > 32 * vec || Hq > 65535 || Hkv > 65535 || T > kRopeMaxT) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || (Hq == 0 && Hkv == 0)) return MOE_OK;
  if (Hkv && !k_out) return MOE_ERR_INVALID_ARG;
  RopeArgs p{};
  const int rc = rope_args(p, r, T, Hq, Hkv, 0, D, q, q_stride, k, k_stride, pos, pos_stride, q_out, qo_stride, k_out, ko_stride);
  return rc ? rc : launch_rope(p, r->interleaved != 0, vec, kNoCache, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_rope_kv_append(const moe_rotary* r, const moe_kv_cache* cache, int32_t T, int32_t Hq,
                                  const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                  const uint16_t* v, int64_t v_stride, const int32_t* pos, int64_t pos_stride,
                                  const int32_t* slots, uint16_t* q_out, int64_t qo_stride, uint16_t* k_out,
                                  int64_t ko_stride, void* ws, size_t ws_bytes, void* stream) {
  if (!r || !cache || T < 0 || Hq < 0) return MOE_ERR_INVALID_ARG;
  if (!kv_cache_ok(cache) || !rotary_ok(r, cache->D) || Hq > 65535 || cache->Hkv > 65535 || T > kRopeMaxT)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!status_ws_ok(ws, ws_bytes)) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  const int64_t row = (int64_t)cache->Hkv * cache->D;
  if (!v || (reinterpret_cast<uintptr_t>(v) & 15) || v_stride % 8 || v_stride < row || !slots ||
      (reinterpret_cast<uintptr_t>(slots) & 3) || !kv_cache_pointers_ok(cache))
    return MOE_ERR_INVALID_ARG;
  RopeArgs p{};
  const int rc = rope_args(p, r, T, Hq, cache->Hkv, cache->Hkv, cache->D, q, q_stride, k, k_stride, pos, pos_stride,
                           q_out, qo_stride, k_out, ko_stride);
  if (rc) return rc;
  p.v = v, p.v_stride = v_stride;
  p.c = *cache;
  while ((1 << p.page_log2) < cache->page_size) ++p.page_log2;
  p.slots = slots;
  p.status = static_cast<uint32_t*>(ws);
  return launch_rope(p, r->interleaved != 0, rope_vec(r), cache->format, static_cast<cudaStream_t>(stream));
}
