// Attention of a few new rows of every sequence over the paged cache (a decode step, or the verification rows of
// speculative decoding), cut into pieces along the cache and joined.
//
// Bound: HBM. Every visible key and value is read once for all rows and all heads of a group; per key and kv head that
// is 4 D bytes (bf16) or 2.06 D (MXFP8) against 4 D R flops, R = rows * Hq / Hkv: far above what CUDA cores do at full
// bandwidth (R = 8 would need 54 of their ~75 TFLOP/s), so both products run on the tensor cores. This file's kernel takes
// up to 16 rows, with m16n8k16: up to 8 rows as its columns, more as its M (a tcgen05 product has at least 64 rows); above 16
// they go to attention_paged_tc.cu. Pieces of both are joined here.
//
// Resident blocks (two to four a multiprocessor) take item after item, one piece of one (sequence, kv head): a producer warp
// streams pages by TMA through a ring of 64-token stages and runs ahead into the next item, four warps consume it, 16 tokens
// of a stage each. Every warp keeps its own running maximum, sum and output, so that nothing but the ring's barriers is shared
// until an item's end.
//
// One row of 32 heads over 8 kv heads of 128, four sequences of up to 128k bf16 tokens: 201 us, 6.2 TB/s. 160 rows of 64
// heads over 8 of 64, a window of 1024 and 4 first tokens: 63 us, 5.4 TB/s (17 steps a row leave an item little to run
// ahead of). 256 rows over 4096 MXFP8 tokens: 445 us, 5.0 TB/s, the conversion's and the products' latencies. One sequence's
// rows are a matter of latency: 11 us for 1024 to 4096 tokens, the join among them.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "attention.cuh"
#include "attention_paged.cuh"
#include "attention_tc.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kTileTok = 64;          // tokens of a stage
constexpr int kFewRows = 16;          // rows that this kernel takes

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <int D_, bool MX_, bool EIGHT_>
struct PagedCfg {
  static constexpr int D = D_;
  static constexpr bool MX = MX_, EIGHT = EIGHT_;                  // EIGHT: up to 8 rows, as a product's columns
  // Blocks of a multiprocessor. Up to 16 rows take 168 registers, up to 8 rows 128 or less. Measured with 2, 3 and 4 blocks:
  // 256 sequences of 4096 tokens, 32 heads over 8 of 128, MXFP8 651 (16 rows' code), 441, 456 us; 64 over 8 of 64, MXFP8
  // 459 (16 rows' code), 338, 296 us; 160 sequences, a window of 1024, 64 over 8 of 64, bf16 68, 63, 67 us.
  static constexpr int CTAS = !EIGHT ? 2 : MX && D == 64 ? 4 : 3;
  static constexpr int WARPS = 4, ST = kTileTok / WARPS;           // tokens of a stage that a warp takes
  static constexpr int HALVES = MX ? 1 : D / 64;                   // 128-byte (MX: D-byte) column blocks of a row
  static constexpr int ROWB = MX ? D : 128;                        // bytes of a row in a column block
  static constexpr int KV = kTileTok * D * (MX ? 1 : 2);           // bytes of a stage's keys, or values
  static constexpr int SC = MX ? kTileTok * D / 32 : 0;
  static constexpr int STAGE = 2 * KV + (MX ? 1024 : 0);
  static constexpr int STAGES = (CTAS == 4 ? 45056 : CTAS == 3 ? 65536 : 98304) / STAGE;
  static constexpr int PITCH = D + 4;                              // floats of a row in the join buffer
  static constexpr int JOIN = 2 * 8 * PITCH * 4;                   // of two warps 8 rows at a time
  static constexpr int SMEM = STAGES * STAGE + JOIN + 1024;
  static_assert(2 * SC <= 1024, "scales");
};

// A barrier of the consuming warps, and whether any thread says so.
template <int WARPS>
__device__ __forceinline__ bool consumers_any(bool said) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((uint32_t)said), "n"(WARPS * 32) : "memory");
  return r != 0;
}

// Shared address of 16-byte chunk `chunk` (of the row's D values) of token `tok`.
template <class C>
__device__ __forceinline__ uint32_t kv_addr(uint32_t base, int tok, int chunk) {
  if (C::ROWB == 128) return base + (chunk >> 3) * (kTileTok * 128) + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4);
  return base + tok * 64 + ((chunk ^ ((tok >> 1) & 3)) << 4);
}

template <class C>
__device__ __forceinline__ float value_at(const uint8_t* stage_v, const uint8_t* scales, int tok, int d) {
  if (C::MX) {
    const uint32_t at = kv_addr<C>(0, tok, d >> 4) + (d & 15);
    return e4m3(stage_v[at]) * ue8m0(scales[tok * (C::D / 32) + (d >> 5)]);
  }
  const uint32_t at = kv_addr<C>(0, tok, d >> 3) + (d & 7) * 2;
  return bf16_lo(*reinterpret_cast<const uint16_t*>(stage_v + at));
}

// Item `n` of a block, as it lies in shared memory: what the warps need of it, worked out once.
struct FewItem {
  int there, b, hk;
  int pos0, pmin, pmax;                         // positions of the first of all rows, of the first and last that are there
  int first_any, first_all, sink_tiles, win_tile;
  int i0, cnt, piece, pieces;                   // first step, steps; piece of how many
  __device__ __forceinline__ int tok(int i) const {
    const int t = i0 + i;
    return (t < sink_tiles ? t : win_tile + (t - sink_tiles)) * kTileTok;
  }
};

// One 8 x 8 matrix of 16-bit values over the warp's lanes (row lane / 4, columns 2 (lane % 4) and the next), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The consuming warps' work for up to 8 rows: the rows are the columns of both products (scores: 16 tokens x 8 rows, output: 16
// of the D columns x 8 rows), so that half as many products, exponentials and accumulators do as with the rows as M = 16.
// Thread (g, c) = (lane / 4, lane % 4) has the scores of tokens g and g + 8 for rows 2c and 2c + 1.
template <class C>
__device__ __forceinline__ void consume_eight(const PagedArgs& p, uint8_t* smem, float* join, uint64_t* full, uint64_t* empty,
                                              uint64_t* w_full, uint64_t* w_empty, const uint32_t* page_mask,
                                              const FewItem* items, float2 (*sums)[16], volatile uint32_t* abort, int warp,
                                              int lane) {
  constexpr int D = C::D, ST = C::ST, MT = D / 16;
  static_assert(ST == 16, "a warp's tokens of a stage are a product's rows");
  const int g = lane >> 2, c = lane & 3, G = p.G, R = p.R;
  const int in_tile = p.page_size >= kTileTok ? 1 : kTileTok >> p.page_log2;
  const float scale = p.a.scale * 1.4426950408889634f;
  uint32_t qf[D / 16][2];
  auto load_q = [&](int n) {
    if (!__all_sync(0xffffffffu, bar_wait(&w_full[n & 1], (n >> 1) & 1, kPagedWaitNs, abort, DEV_TIMEOUT_FULL)) ||
        !items[n & 1].there)
      return false;
    const bool live = g < R;
    const int r = g / G;
    const uint16_t* row = p.q + ((long long)items[n & 1].b * p.rows + r) * p.q_stride + (long long)(items[n & 1].hk * G + g - r * G) * D;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      // MX: the k of a step are the codes that one thread has at hand (8 in a row, 4 for each of two steps)
      const int d0 = C::MX ? (ks / 2) * 32 + 8 * c + 4 * (ks & 1) : ks * 16 + 2 * c;
      const int d1 = C::MX ? d0 + 2 : d0 + 8;
      qf[ks][0] = live ? *reinterpret_cast<const uint32_t*>(row + d0) : 0;
      qf[ks][1] = live ? *reinterpret_cast<const uint32_t*>(row + d1) : 0;
    }
    return true;
  };
  int tiles = 0;                                // steps so far
  const uint32_t k16 = C::MX ? sixteen() : 0;
  // the warps go on together or not at all, also when one of them has given up
  bool stop = consumers_any<C::WARPS>(!load_q(0));
  for (int n = 0; !stop; ++n) {
    const FewItem& it = items[n & 1];
    const int cnt = it.cnt;
    int pos[2], first[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rho = 2 * c + e;
      pos[e] = rho < R ? it.pos0 + rho / G : -1;
      first[e] = (p.a.window && pos[e] >= p.a.window) ? pos[e] + 1 - p.a.window : 0;
    }
    float o[MT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    // A wait that runs out ends the item for all lanes or none: the vote is cast where each of them is. (In one place, as `if
    // (!__all_sync(mask, bar_wait(...)))`, the code of a step grows by 7 % of its instructions: 256 sequences of 4096 MXFP8
    // tokens 470 us instead of 445.)
    for (int i = 0; i < cnt; ++i, ++tiles) {
      const int s = tiles % C::STAGES;
      if (!bar_wait(&full[s], (tiles / C::STAGES) & 1, kPagedWaitNs, abort, DEV_TIMEOUT_FULL)) {
        __all_sync(0xffffffffu, false);         // told to those that go on below
        break;
      }
      if (!__all_sync(0xffffffffu, true)) break;
      const int loc0 = warp * ST, tok0 = it.tok(i) + loc0;
      const uint8_t* st = smem + s * C::STAGE;
      const uint32_t kb = smem_u32(st), vb = kb + C::KV;
      const uint32_t mask = page_mask[s];
      // every row of the block sees every token of this warp
      const bool whole = tok0 + ST - 1 <= it.pmin && (tok0 >= it.first_all || tok0 + ST <= p.a.sinks) &&
                         mask == (1u << in_tile) - 1u;
      if (tok0 <= it.pmax) {
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};      // of every other product
        if constexpr (!C::MX) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t r[4];
            ldsm4(kv_addr<C>(kb, loc0 + (lane & 15), 2 * ks + (lane >> 4)), r);
            mma_16816(ks & 1 ? sd : sc, r, qf[ks][0], qf[ks][1]);
          }
        } else {
          // Tokens whose scales one factor does not hold have a copy of the code to themselves: a branch inside would keep
          // loads, conversions and products of neighbouring blocks apart.
          const uint8_t* scales = st + 2 * C::KV;
          uint32_t sw[2], most = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = loc0 + g + 8 * h;
            sw[h] = D == 128 ? *reinterpret_cast<const uint32_t*>(scales + t * 4)
                             : *reinterpret_cast<const uint16_t*>(scales + t * 2);
            most |= __vcmpgtu4(sw[h], kScaleFits * 0x01010101u);
          }
          auto scores = [&](auto large) {
#pragma unroll
            for (int bl = 0; bl < D / 32; ++bl) {
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w0, w1;
                const uint32_t at = kv_addr<C>(kb, loc0 + g + 8 * h, 2 * bl + (c >> 1)) + 8 * (c & 1);
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
                const uint32_t by = (sw[h] >> (8 * bl)) & 255u;
                const uint32_t f = (large.value ? scale_bits(by) : (by + 120u) << 7) * 0x10001u;
                x[0][h] = mul_bf16x2(e4m3_pair(w0, w0, kCodes01, k16), f);
                x[0][2 + h] = mul_bf16x2(e4m3_pair(w0, w0, kCodes23, k16), f);
                x[1][h] = mul_bf16x2(e4m3_pair(w1, w1, kCodes01, k16), f);
                x[1][2 + h] = mul_bf16x2(e4m3_pair(w1, w1, kCodes23, k16), f);
                if (large.value) {
                  const uint32_t f2 = scale_rest(by) * 0x10001u;
#pragma unroll
                  for (int e = 0; e < 2; ++e) x[e][h] = mul_bf16x2(x[e][h], f2), x[e][2 + h] = mul_bf16x2(x[e][2 + h], f2);
                }
              }
              mma_16816(sc, x[0], qf[2 * bl][0], qf[2 * bl][1]);
              mma_16816(sd, x[1], qf[2 * bl + 1][0], qf[2 * bl + 1][1]);
            }
          };
          if (__any_sync(0xffffffffu, most != 0)) scores(std::true_type{});
          else scores(std::false_type{});
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] = (sc[e] + sd[e]) * scale;

        // ---- what the rows do not see ----
        uint32_t drop = 0, alone = 0;            // of this warp's tokens: left out of the product; added one by one
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int loc = g + 8 * (e >> 1), t = tok0 + loc;
            const bool there = (mask >> ((loc0 + loc) >> min(p.page_log2, 6))) & 1u;
            const bool see = there && t <= pos[e & 1] && (t >= first[e & 1] || t < p.a.sinks);
            sc[e] = see ? sc[e] : -INFINITY;
          }
          // A weight of zero does not hide a value that is not finite: the product leaves out what no row sees, and
          // what only some rows see where it is not finite.
          const int t = tok0 + lane;
          const bool there = lane < ST && ((mask >> ((loc0 + lane) >> min(p.page_log2, 6))) & 1u);
          const bool any = there && t <= it.pmax && (t >= it.first_any || t < p.a.sinks);
          const bool all = any && t <= it.pmin && (t >= it.first_all || t < p.a.sinks);
          drop = __ballot_sync(0xffffffffu, lane < ST && !any);
          alone = __ballot_sync(0xffffffffu, any && !all);
          for (uint32_t some = alone; some; some &= some - 1) {
            const int loc = __ffs(some) - 1;
            bool fine = true;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
              fine = fine && isfinite(value_at<C>(st + C::KV, st + 2 * C::KV + C::SC, loc0 + loc, lane + 32 * e));
            if (__all_sync(0xffffffffu, fine)) alone &= ~(1u << loc);
          }
          drop |= alone;
        }

        // the values' codes, under way while the weights are worked out: thread (g, c) has the D/8 values from g D/8 on of its
        // four tokens; product j takes the 2j-th of each as its row g, and the next as its row g + 8
        uint32_t w[4][D / 32], by[4];
        if constexpr (C::MX) {
          const uint8_t* scales = st + 2 * C::KV + C::SC;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tk = loc0 + 2 * c + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 128) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                           : "r"(kv_addr<C>(vb, tk, g)) : "memory");
            } else {
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[e][0]), "=r"(w[e][1])
                           : "r"(kv_addr<C>(vb, tk, g >> 1) + 8 * (g & 1)) : "memory");
            }
            by[e] = scales[tk * (D / 32) + g / (256 / D)];
          }
        }
        // ---- softmax ----
        float mx[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(sc[e], sc[2 + e]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
          mx[e] = fmaxf(mx[e], m[e]);
          base[e] = mx[e] == -INFINITY ? 0.f : mx[e];
        }
        if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
          const float k0 = ex2(m[0] - base[0]), k1 = ex2(m[1] - base[1]);
          l[0] *= k0;
          l[1] *= k1;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[j][0] *= k0;
            o[j][1] *= k1;
            o[j][2] *= k0;
            o[j][3] *= k1;
          }
          m[0] = mx[0];
          m[1] = mx[1];
        }
        // the weights are rounded to bf16 for the second product; the sum takes the rounded ones, so that a single large
        // weight divides out exactly
        const uint32_t w0 = bf16x2(ex2(sc[0] - base[0]), ex2(sc[1] - base[1]));
        const uint32_t w1 = bf16x2(ex2(sc[2] - base[0]), ex2(sc[3] - base[1]));
        l[0] += bf16_lo(w0) + bf16_lo(w1);
        l[1] += bf16_hi(w0) + bf16_hi(w1);
        const uint32_t p0 = transposed(w0), p1 = transposed(w1);

        // ---- weighted values ----
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (drop) {
          keep0 = ((drop >> (2 * c)) & 1u ? 0u : 0xffffu) | ((drop >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
          keep1 = ((drop >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((drop >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);
        }
        if constexpr (!C::MX) {
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            uint32_t r[4];
            ldsm4t(kv_addr<C>(vb, loc0 + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)), r);
            if (drop) r[0] &= keep0, r[1] &= keep0, r[2] &= keep1, r[3] &= keep1;
            mma_16816(o[j], r, p0, p1);
          }
        } else {
          const bool large = max(max(by[0], by[1]), max(by[2], by[3])) > kScaleFits;
          auto values = [&](auto rare) {         // rare: some scale is large, or some token left out
            auto fac = [&](uint32_t b) { return rare.value ? scale_bits(b) : (b + 120u) << 7; };
            const uint32_t f0 = fac(by[0]) | fac(by[1]) << 16, f1 = fac(by[2]) | fac(by[3]) << 16;
            uint32_t r0 = 0, r1 = 0;
            if (rare.value) r0 = scale_rest(by[0]) | scale_rest(by[1]) << 16, r1 = scale_rest(by[2]) | scale_rest(by[3]) << 16;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              uint32_t x[4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                constexpr uint32_t kSel[4] = {0xC480, 0xD591, 0xE6A2, 0xF7B3};    // the code of that number of either word
                const int at = 2 * j + h;
                x[h] = mul_bf16x2(e4m3_pair(w[0][at / 4], w[1][at / 4], kSel[at & 3], k16), f0);
                x[2 + h] = mul_bf16x2(e4m3_pair(w[2][at / 4], w[3][at / 4], kSel[at & 3], k16), f1);
                if (rare.value) x[h] = mul_bf16x2(x[h], r0) & keep0, x[2 + h] = mul_bf16x2(x[2 + h], r1) & keep1;
              }
              mma_16816(o[j], x, p0, p1);
            }
          };
          if (__any_sync(0xffffffffu, large || drop != 0)) values(std::true_type{});
          else values(std::false_type{});
        }
        for (; alone; alone &= alone - 1) {
          const int loc = __ffs(alone) - 1, t = tok0 + loc;
          const uint32_t both = __shfl_sync(0xffffffffu, loc & 8 ? w1 : w0, (loc & 7) * 4 + c);
          const bool see0 = t <= pos[0] && (t >= first[0] || t < p.a.sinks);
          const bool see1 = t <= pos[1] && (t >= first[1] || t < p.a.sinks);
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float v = value_at<C>(st + C::KV, st + 2 * C::KV + C::SC, loc0 + loc,
                                          C::MX ? g * (D / 8) + 2 * j + h : j * 16 + g + 8 * h);
              if (see0) o[j][2 * h] = fmaf(bf16_lo(both), v, o[j][2 * h]);
              if (see1) o[j][2 * h + 1] = fmaf(bf16_hi(both), v, o[j][2 * h + 1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ---------------- the warps' parts joined, in the order of their tokens ----------------
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
      if (g == 0) sums[warp][2 * c + e] = make_float2(m[e], l[e]);
    }
    const int piece = it.piece, pieces = it.pieces, hk = it.hk;
    const long long b = it.b;
    const bool more = load_q(n + 1);              // on their way while this item ends
    stop = consumers_any<C::WARPS>(!more || *abort);
    float top[2], tl[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = -INFINITY, tl[e] = 0.f;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) top[e] = fmaxf(top[e], sums[w][2 * c + e].x);
      const float base = top[e] == -INFINITY ? 0.f : top[e];
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) tl[e] += ex2(sums[w][2 * c + e].x - base) * sums[w][2 * c + e].y;
      const float f = ex2(m[e] - base);
#pragma unroll
      for (int j = 0; j < MT; ++j) o[j][e] *= f, o[j][2 + e] *= f;
    }
    // ((0 + 2) + (1 + 3)): the upper two warps hand theirs to the lower two, those one to the other
#pragma unroll
    for (int far = 2; far; far >>= 1) {
      float4* mine = reinterpret_cast<float4*>(join) + (warp & (far - 1)) * MT * 32 + lane;
      if (warp >= far && warp < 2 * far) {
#pragma unroll
        for (int j = 0; j < MT; ++j) mine[j * 32] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      }
      named_bar_sync(1, C::WARPS * 32);
      if (warp < far) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float4 v = mine[j * 32];
          o[j][0] += v.x, o[j][1] += v.y, o[j][2] += v.z, o[j][3] += v.w;
        }
      }
      named_bar_sync(1, C::WARPS * 32);
    }
    if (warp == 0 && !*abort) {
      const long long at = (b * p.a.Hkv + hk) * p.max_pieces + piece;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rho = 2 * c + e;
        if (rho >= R) continue;
        const bool one = pieces == 1;
        const int r = rho / G;
        const float inv = !one ? 1.f : tl[e] == 0.f ? no_weights(p, b, pos[e]) : 1.f / tl[e];
        uint16_t* out = p.out + ((b * p.rows + r) * p.a.Hq + hk * G + rho - r * G) * D;
#pragma unroll
        for (int j = 0; j < MT; j += 2) {
          // of products j and j + 1: MX four columns in a row, else g, g + 8, g + 16 and g + 24 of 32
          const float v[4] = {o[j][e] * inv, o[j][2 + e] * inv, o[j + 1][e] * inv, o[j + 1][2 + e] * inv};
          if (C::MX) {
            const int d = g * (D / 8) + 2 * j;
            if (one) *reinterpret_cast<uint2*>(out + d) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
            else *reinterpret_cast<float4*>(part_of(p, at, D, rho, d / 4)) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int d = j * 16 + g + 8 * k;
              if (one) out[d] = (uint16_t)bf16x2(v[k], 0.f);
              else part_of(p, at, D, rho, d / 4)[d % 4] = v[k];
            }
          }
        }
        if (!one && g == 0) *sums_of(p, at, rho) = make_float2(top[e], tl[e]);
      }
    }
    if (lane == 0) mbar_arrive(&w_empty[n & 1]);
  }
}

// At the end of every warp: who gave up, or saw that another one had, records it.
__device__ __forceinline__ void record_end(const PagedArgs& p, volatile uint32_t* abort) {
  __syncwarp();
  if (threadIdx.x % 32 == 0 && *abort) atomicCAS(p.status, 0u, *abort);
}

template <class C>
__global__ void __launch_bounds__((C::WARPS + 1) * 32, C::CTAS)
paged_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const PagedArgs p) {
  constexpr int D = C::D, ST = C::ST, NT = D / 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], w_full[2], w_empty[2];
  __shared__ uint32_t page_mask[C::STAGES];
  __shared__ FewItem items[2];
  __shared__ float2 sums[C::WARPS][16];         // the warps' maximum (times log2 e) and sum of a row
  __shared__ volatile uint32_t abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* join = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int G = p.G, R = p.R;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::WARPS);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], C::WARPS);
    }
    abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int in_tile = p.page_size >= kTileTok ? 1 : kTileTok >> p.page_log2;     // pages of a step

  if (warp == C::WARPS) {
    // ---------------- items and loads ----------------
    const int rows_of = min(p.page_size, kTileTok);
    int n = 0, issued = 0;
    bool ok = true;
    ItemWalk walk;
    for (long long idx = blockIdx.x; ok; idx += gridDim.x) {
      const int who = walk.lane_of(p, idx);
      if (n >= 2 && !(ok = __all_sync(0xffffffffu, bar_wait(&w_empty[n & 1], ((n >> 1) - 1) & 1, kPagedWaitNs, &abort_flag,
                                                            DEV_TIMEOUT_EMPTY))))
        break;
      if (lane == max(who, 0)) {
        FewItem mine{};                          // no more items: that one is not there
        if (who >= 0) {
          const int u = walk.group + lane, j = (int)(idx - walk.before) - (walk.upto - walk.mine);
          const Pieces& pc = walk.pc;
          mine.there = 1;
          mine.b = u;
          mine.piece = j / p.a.Hkv;
          mine.hk = j - mine.piece * p.a.Hkv;
          mine.pos0 = pc.pos0;
          mine.pmin = pc.pmin, mine.pmax = pc.pmax, mine.first_any = pc.first_any, mine.first_all = pc.first_all;
          mine.sink_tiles = pc.sink_tiles, mine.win_tile = pc.win_tile;
          mine.i0 = pc.begin(mine.piece);
          mine.cnt = pc.steps(mine.piece);
          mine.pieces = pc.count;
        }
        items[n & 1] = mine;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_full[n & 1]);
      if (who < 0) break;
      const FewItem it = items[n & 1];
      ++n;
      const int32_t* table = p.table + (long long)it.b * p.table_width;
      const int last_page = it.pmax >> p.page_log2;
      int base = -1000, ids = 0, next = 0;   // 32 table entries from `base` on, and the 32 behind them
      for (int i = 0; i < it.cnt; ++i, ++issued) {
        const int s = issued % C::STAGES;
        const int tok0 = it.tok(i), page0 = tok0 >> p.page_log2;
        if (page0 < base || page0 + in_tile > base + 32) {
          // in_tile divides 32: a step's pages lie in one group of 32 entries
          const int nb = page0 & ~31;
          ids = nb == base + 32 ? next : (nb + lane <= last_page ? table[nb + lane] : -1);
          base = nb;
          next = nb + 32 + lane <= last_page ? table[nb + 32 + lane] : -1;
        }
        const int id = __shfl_sync(0xffffffffu, ids, (page0 - base + lane) & 31);
        // pages that no row sees are not loaded: past the end, or between the first tokens and the window
        const int t0 = tok0 + lane * rows_of;
        const bool want = lane < in_tile && t0 <= it.pmax &&
                          (t0 + rows_of > it.first_any || t0 < min(p.a.sinks, it.first_all));
        const bool good = want && id >= 0 && id < p.pages;
        if (want && !good) atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
        const uint32_t mask = __ballot_sync(0xffffffffu, good);
        if (issued >= C::STAGES &&
            !(ok = __all_sync(0xffffffffu, bar_wait(&empty[s], (issued / C::STAGES - 1) & 1, kPagedWaitNs, &abort_flag,
                                                    DEV_TIMEOUT_EMPTY))))
          break;
        if (lane == 0) {
          page_mask[s] = mask;
          mbar_arrive_expect_tx(&full[s], __popc(mask) * rows_of * (2 * D * (C::MX ? 1 : 2) + (C::MX ? 2 * D / 32 : 0)) +
                                              (issued == p.hold ? 16 : 0));
        }
        __syncwarp();
        if (good) {
          const int row = (int)(((long long)id * p.a.Hkv + it.hk) << p.page_log2) + (t0 & (p.page_size - 1));
          uint8_t* st = smem + s * C::STAGE;
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h) {
            const uint32_t at = h * kTileTok * C::ROWB + lane * rows_of * C::ROWB;
            tma_load_2d(st + at, &kmap, h * 64, row, &full[s]);
            tma_load_2d(st + C::KV + at, &vmap, h * 64, row, &full[s]);
          }
          if (C::MX) {
            const uint32_t bytes = rows_of * (D / 32);
            uint8_t* sc = st + 2 * C::KV + lane * bytes;
            bulk_load(sc, p.k_s + (long long)row * (D / 32), bytes, &full[s]);
            bulk_load(sc + C::SC, p.v_s + (long long)row * (D / 32), bytes, &full[s]);
          }
        }
      }
    }
    // copies in flight end before the block does, whoever gives up and when
    if (lane == 0)
      for (int j = max(0, issued - C::STAGES); j < issued; ++j)
        mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1, kPagedWaitNs, nullptr, nullptr, DEV_TIMEOUT_DRAIN);
    record_end(p, &abort_flag);
    return;
  }

  // ---------------- consumers ----------------
  if constexpr (C::EIGHT) {
    consume_eight<C>(p, smem, join, full, empty, w_full, w_empty, page_mask, items, sums, &abort_flag, warp, lane);
    record_end(p, &abort_flag);
    return;
  }
  const int g = lane >> 2, c = lane & 3;
  const float scale = p.a.scale * 1.4426950408889634f;
  uint32_t qf[D / 16][4];
  // The queries of item n, once it is known; false: there is none.
  auto load_q = [&](int n) {
    if (!__all_sync(0xffffffffu, bar_wait(&w_full[n & 1], (n >> 1) & 1, kPagedWaitNs, &abort_flag, DEV_TIMEOUT_FULL)) ||
        !items[n & 1].there)
      return false;
    const long long b = items[n & 1].b;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rho = g + 8 * h;
      const bool live = rho < R;
      const int r = rho / G;
      const uint16_t* row = p.q + (b * p.rows + r) * p.q_stride + (long long)(items[n & 1].hk * G + rho - r * G) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // MX: the k of a step are the codes that one thread has at hand (8 in a row, 4 for each of two steps)
        const int d0 = C::MX ? (ks / 2) * 32 + 8 * c + 4 * (ks & 1) : ks * 16 + 2 * c;
        const int d1 = C::MX ? d0 + 2 : d0 + 8;
        qf[ks][h] = live ? *reinterpret_cast<const uint32_t*>(row + d0) : 0;
        qf[ks][2 + h] = live ? *reinterpret_cast<const uint32_t*>(row + d1) : 0;
      }
    }
    return true;
  };
  int tiles = 0;                                // steps so far
  const uint32_t k16 = C::MX ? sixteen() : 0;
  // the warps go on together or not at all, also when one of them has given up
  bool stop = consumers_any<C::WARPS>(!load_q(0));
  for (int n = 0; !stop; ++n) {
    const FewItem& it = items[n & 1];
    const int cnt = it.cnt;
    int pos[2], first[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rho = g + 8 * h;
      pos[h] = rho < R ? it.pos0 + rho / G : -1;
      first[h] = (p.a.window && pos[h] >= p.a.window) ? pos[h] + 1 - p.a.window : 0;
    }
    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int i = 0; i < cnt; ++i, ++tiles) {
      const int s = tiles % C::STAGES;
      if (!bar_wait(&full[s], (tiles / C::STAGES) & 1, kPagedWaitNs, &abort_flag, DEV_TIMEOUT_FULL)) {
        __all_sync(0xffffffffu, false);         // told to those that go on below
        break;
      }
      if (!__all_sync(0xffffffffu, true)) break;
      const int loc0 = warp * ST, tok0 = it.tok(i) + loc0;
      const uint8_t* st = smem + s * C::STAGE;
      const uint32_t kb = smem_u32(st), vb = kb + C::KV;
      const uint32_t mask = page_mask[s];
      // every row of the block sees every token of this warp
      const bool whole = tok0 + ST - 1 <= it.pmin && (tok0 >= it.first_all || tok0 + ST <= p.a.sinks) &&
                         mask == (1u << in_tile) - 1u;
      if (tok0 <= it.pmax) {
        float sc[ST / 8][4];
#pragma unroll
        for (int j = 0; j < ST / 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        if (!C::MX) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int jp = 0; jp < ST / 16; ++jp) {
              uint32_t r[4];
              ldsm4(kv_addr<C>(kb, loc0 + jp * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), r);
              mma_16816(sc[2 * jp], qf[ks], r[0], r[1]);
              mma_16816(sc[2 * jp + 1], qf[ks], r[2], r[3]);
            }
        } else {
          // Tokens whose scales one factor does not hold have a copy of the code to themselves: a branch inside would keep
          // loads, conversions and products of neighbouring blocks apart.
          const uint8_t* scales = st + 2 * C::KV;
          uint32_t sw[ST / 8], most = 0;
#pragma unroll
          for (int j = 0; j < ST / 8; ++j) {
            const int t = loc0 + j * 8 + g;
            sw[j] = D == 128 ? *reinterpret_cast<const uint32_t*>(scales + t * 4)
                             : *reinterpret_cast<const uint16_t*>(scales + t * 2);
            most |= __vcmpgtu4(sw[j], kScaleFits * 0x01010101u);
          }
          auto scores = [&](auto large) {
#pragma unroll
            for (int bl = 0; bl < D / 32; ++bl)
#pragma unroll
              for (int j = 0; j < ST / 8; ++j) {
                uint32_t w0, w1;
                const uint32_t at = kv_addr<C>(kb, loc0 + j * 8 + g, 2 * bl + (c >> 1)) + 8 * (c & 1);
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
                const uint32_t by = (sw[j] >> (8 * bl)) & 255u;
                const uint32_t f = (large.value ? scale_bits(by) : (by + 120u) << 7) * 0x10001u;
                uint32_t x[4] = {mul_bf16x2(e4m3_pair(w0, w0, kCodes01, k16), f), mul_bf16x2(e4m3_pair(w0, w0, kCodes23, k16), f),
                                 mul_bf16x2(e4m3_pair(w1, w1, kCodes01, k16), f), mul_bf16x2(e4m3_pair(w1, w1, kCodes23, k16), f)};
                if (large.value) {
                  const uint32_t f2 = scale_rest(by) * 0x10001u;
#pragma unroll
                  for (int e = 0; e < 4; ++e) x[e] = mul_bf16x2(x[e], f2);
                }
                mma_16816(sc[j], qf[2 * bl], x[0], x[1]);
                mma_16816(sc[j], qf[2 * bl + 1], x[2], x[3]);
              }
          };
          if (__any_sync(0xffffffffu, most != 0)) scores(std::true_type{});
          else scores(std::false_type{});
        }

        // ---- what the rows do not see ----
        unsigned long long drop = 0, alone = 0;      // of this warp's tokens: left out of the product; added one by one
        if (whole) {
#pragma unroll
          for (int j = 0; j < ST / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][e] *= scale;
        } else {
#pragma unroll
          for (int j = 0; j < ST / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int loc = j * 8 + 2 * c + (e & 1), t = tok0 + loc;
              const bool there = (mask >> ((loc0 + loc) >> min(p.page_log2, 6))) & 1u;
              const bool see = there && t <= pos[e >> 1] && (t >= first[e >> 1] || t < p.a.sinks);
              sc[j][e] = see ? sc[j][e] * scale : -INFINITY;
            }
          // A weight of zero does not hide a value that is not finite: the product leaves out what no row sees, and
          // what only some rows see where it is not finite.
#pragma unroll
          for (int w = 0; w < (ST + 31) / 32; ++w) {
            const int loc = w * 32 + lane, t = tok0 + loc;
            const bool there = loc < ST && ((mask >> ((loc0 + loc) >> min(p.page_log2, 6))) & 1u);
            const bool any = there && t <= it.pmax && (t >= it.first_any || t < p.a.sinks);
            const bool all = any && t <= it.pmin && (t >= it.first_all || t < p.a.sinks);
            drop |= (unsigned long long)__ballot_sync(0xffffffffu, loc < ST && !any) << (32 * w);
            alone |= (unsigned long long)__ballot_sync(0xffffffffu, any && !all) << (32 * w);
          }
          for (unsigned long long some = alone; some; some &= some - 1) {
            const int loc = __ffsll(some) - 1;
            bool fine = true;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
              fine = fine && isfinite(value_at<C>(st + C::KV, st + 2 * C::KV + C::SC, loc0 + loc, lane + 32 * e));
            if (__all_sync(0xffffffffu, fine)) alone &= ~(1ull << loc);
          }
          drop |= alone;
        }

        // the values' codes, under way while the weights are worked out
        uint32_t w[4][D / 32], by[4];
        if constexpr (C::MX) {
          const uint8_t* scales = st + 2 * C::KV + C::SC;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tk = loc0 + 2 * c + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 128) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                           : "r"(kv_addr<C>(vb, tk, g)) : "memory");
            } else {
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[e][0]), "=r"(w[e][1])
                           : "r"(kv_addr<C>(vb, tk, g >> 1) + 8 * (g & 1)) : "memory");
            }
            by[e] = scales[tk * (D / 32) + g / (256 / D)];
          }
        }
        // ---- softmax ----
        float mx[2] = {-INFINITY, -INFINITY}, base[2];
#pragma unroll
        for (int j = 0; j < ST / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], sc[j][e]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          mx[h] = fmaxf(mx[h], m[h]);
          base[h] = mx[h] == -INFINITY ? 0.f : mx[h];
        }
        if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
          const float k0 = ex2(m[0] - base[0]), k1 = ex2(m[1] - base[1]);
          l[0] *= k0;
          l[1] *= k1;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            o[j][0] *= k0;
            o[j][1] *= k0;
            o[j][2] *= k1;
            o[j][3] *= k1;
          }
          m[0] = mx[0];
          m[1] = mx[1];
        }
        uint32_t pf[ST / 16][4];
#pragma unroll
        for (int j = 0; j < ST / 8; ++j) {
          // the weights are rounded to bf16 for the second product; the sum takes the rounded ones, so that a single
          // large weight divides out exactly
          const uint32_t w0 = bf16x2(ex2(sc[j][0] - base[0]), ex2(sc[j][1] - base[0]));
          const uint32_t w1 = bf16x2(ex2(sc[j][2] - base[1]), ex2(sc[j][3] - base[1]));
          l[0] += bf16_lo(w0) + bf16_hi(w0);
          l[1] += bf16_lo(w1) + bf16_hi(w1);
          pf[j / 2][(j & 1) * 2] = w0;
          pf[j / 2][(j & 1) * 2 + 1] = w1;
        }

        // ---- weighted values ----
#pragma unroll
        for (int t = 0; t < ST / 16; ++t) {
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (drop) {
            const uint32_t d16 = (uint32_t)(drop >> (16 * t));
            keep0 = ((d16 >> (2 * c)) & 1u ? 0u : 0xffffu) | ((d16 >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
            keep1 = ((d16 >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((d16 >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);
          }
          if (!C::MX) {
#pragma unroll
            for (int np = 0; np < D / 16; ++np) {
              uint32_t r[4];
              ldsm4t(kv_addr<C>(vb, loc0 + t * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * np + (lane >> 4)), r);
              if (drop) r[0] &= keep0, r[1] &= keep1, r[2] &= keep0, r[3] &= keep1;
              mma_16816(o[2 * np], pf[t], r[0], r[1]);
              mma_16816(o[2 * np + 1], pf[t], r[2], r[3]);
            }
          } else {
            // thread (g, c) holds the D/8 values from g D/8 on of its four tokens; product j takes the j-th of each
            const bool large = max(max(by[0], by[1]), max(by[2], by[3])) > kScaleFits;
            auto values = [&](auto rare) {       // rare: some scale is large, or some token left out
              auto fac = [&](uint32_t b) { return rare.value ? scale_bits(b) : (b + 120u) << 7; };
              const uint32_t f0 = fac(by[0]) | fac(by[1]) << 16, f1 = fac(by[2]) | fac(by[3]) << 16;
              uint32_t r0 = 0, r1 = 0;
              if (rare.value) r0 = scale_rest(by[0]) | scale_rest(by[1]) << 16, r1 = scale_rest(by[2]) | scale_rest(by[3]) << 16;
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                constexpr uint32_t kSel[4] = {0xC480, 0xD591, 0xE6A2, 0xF7B3};    // the j-th code of either word
                uint32_t x0 = mul_bf16x2(e4m3_pair(w[0][j / 4], w[1][j / 4], kSel[j & 3], k16), f0);
                uint32_t x1 = mul_bf16x2(e4m3_pair(w[2][j / 4], w[3][j / 4], kSel[j & 3], k16), f1);
                if (rare.value) x0 = mul_bf16x2(x0, r0) & keep0, x1 = mul_bf16x2(x1, r1) & keep1;
                mma_16816(o[j], pf[t], x0, x1);
              }
            };
            if (__any_sync(0xffffffffu, large || drop != 0)) values(std::true_type{});
            else values(std::false_type{});
          }
        }
        for (; alone; alone &= alone - 1) {
          const int loc = __ffsll(alone) - 1, t = tok0 + loc;
          uint32_t w0 = 0, w1 = 0;
#pragma unroll
          for (int j = 0; j < ST / 8; ++j)
            if (j == loc >> 3) w0 = pf[j / 2][(j & 1) * 2], w1 = pf[j / 2][(j & 1) * 2 + 1];
          w0 = __shfl_sync(0xffffffffu, w0, (lane & 28) | ((loc & 7) >> 1));
          w1 = __shfl_sync(0xffffffffu, w1, (lane & 28) | ((loc & 7) >> 1));
          const float p0 = loc & 1 ? bf16_hi(w0) : bf16_lo(w0), p1 = loc & 1 ? bf16_hi(w1) : bf16_lo(w1);
          const bool see0 = t <= pos[0] && (t >= first[0] || t < p.a.sinks);
          const bool see1 = t <= pos[1] && (t >= first[1] || t < p.a.sinks);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float v = value_at<C>(st + C::KV, st + 2 * C::KV + C::SC, loc0 + loc,
                                          C::MX ? (2 * c + e) * (D / 8) + j : j * 8 + 2 * c + e);
              if (see0) o[j][e] = fmaf(p0, v, o[j][e]);
              if (see1) o[j][2 + e] = fmaf(p1, v, o[j][2 + e]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ---------------- the warps' parts joined, in the order of their tokens ----------------
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (c == 0) sums[warp][g + 8 * h] = make_float2(m[h], l[h]);
    }
    const int piece = it.piece, pieces = it.pieces, hk = it.hk;
    const long long b = it.b;
    const bool more = load_q(n + 1);              // on their way while this item ends
    stop = consumers_any<C::WARPS>(!more || abort_flag);
    float top[2], tl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = -INFINITY, tl[h] = 0.f;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) top[h] = fmaxf(top[h], sums[w][g + 8 * h].x);
      const float base = top[h] == -INFINITY ? 0.f : top[h];
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) tl[h] += ex2(sums[w][g + 8 * h].x - base) * sums[w][g + 8 * h].y;
      const float f = ex2(m[h] - base);
#pragma unroll
      for (int j = 0; j < NT; ++j) o[j][2 * h] *= f, o[j][2 * h + 1] *= f;
    }
    // ((0 + 2) + (1 + 3)): the upper two warps hand theirs to the lower two, those one to the other, 8 rows at a time
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int far = 2; far; far >>= 1) {
        float* mine = join + ((warp & (far - 1)) * 8 + g) * C::PITCH;
        if (warp >= far && warp < 2 * far) {
#pragma unroll
          for (int j = 0; j < NT; ++j) *reinterpret_cast<float2*>(mine + j * 8 + 2 * c) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
        }
        named_bar_sync(1, C::WARPS * 32);
        if (warp < far) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float2 v = *reinterpret_cast<const float2*>(mine + j * 8 + 2 * c);
            o[j][2 * h] += v.x, o[j][2 * h + 1] += v.y;
          }
        }
        named_bar_sync(1, C::WARPS * 32);
      }
      const int rho = g + 8 * h;
      if (warp == 0 && rho < R && !abort_flag) {
        const bool one = pieces == 1;
        const int r = rho / G;
        const float inv = !one ? 1.f : tl[h] == 0.f ? no_weights(p, b, pos[h]) : 1.f / tl[h];
        const long long at = (b * p.a.Hkv + hk) * p.max_pieces + piece;
        uint16_t* out = p.out + ((b * p.rows + r) * p.a.Hq + hk * G + rho - r * G) * D;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          // thread (g, c) has of product j the columns 2c and 2c + 1; MX: the j-th of what two threads' values are
          const float v0 = o[j][2 * h] * inv, v1 = o[j][2 * h + 1] * inv;
          if (!C::MX) {
            const int d = j * 8 + 2 * c;
            if (one) *reinterpret_cast<uint32_t*>(out + d) = bf16x2(v0, v1);
            else *reinterpret_cast<float2*>(part_of(p, at, D, rho, d / 4) + d % 4) = make_float2(v0, v1);
          } else {
            const int d = 2 * c * (D / 8) + j;
            if (one) {
              out[d] = (uint16_t)bf16x2(v0, 0.f);
              out[d + D / 8] = (uint16_t)bf16x2(v1, 0.f);
            } else {
              part_of(p, at, D, rho, d / 4)[d % 4] = v0;
              part_of(p, at, D, rho, (d + D / 8) / 4)[d % 4] = v1;
            }
          }
        }
        if (!one && c == 0) *sums_of(p, at, rho) = make_float2(top[h], tl[h]);
      }
    }
    if (lane == 0) mbar_arrive(&w_empty[n & 1]);
  }
  record_end(p, &abort_flag);
}

// The pieces' parts joined in order, a thread per four columns of a row, rows next to each other. Rows of one piece are
// already written.
constexpr int kJoinRows = 8;            // rows of a block ...
constexpr int kJoinCols = 16;           // ... and groups of four columns

template <int D>
__global__ void __launch_bounds__(kJoinRows * kJoinCols) paged_join_kernel(const PagedArgs p) {
  const int G = p.G, R = p.R;
  const int row_blocks = (R + kJoinRows - 1) / kJoinRows;
  const unsigned unit = blockIdx.x / row_blocks;
  const int rho = (int)(blockIdx.x % row_blocks) * kJoinRows + threadIdx.x % kJoinRows;
  const int d4 = blockIdx.y * kJoinCols + threadIdx.x / kJoinRows, hk = (int)(unit % p.a.Hkv);
  const long long b = unit / p.a.Hkv;
  // The lengths are there: the kernel before this one lets it start only after its own wait for what was before.
  const Pieces pc(p, checked_len(p, b, false), min(rho, R - 1) >> p.block_log2);
  pdl_wait();
  if (rho >= R || pc.count == 1) return;
  const long long at = (b * p.a.Hkv + hk) * p.max_pieces;
  // Eight pieces at a time, the next eight under way meanwhile. The last one stands in for those past the end, so that no load
  // waits for a comparison; it is added once.
  const int count = pc.count;
  float2 s[2][8];
  float4 v[2][8];
  auto load = [&](float2 (&sums)[8], float4 (&sum)[8], int i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int piece = min(i + k, count - 1);
      sums[k] = *sums_of(p, at + piece, rho);
      sum[k] = *reinterpret_cast<const float4*>(part_of(p, at + piece, D, rho, d4));
    }
  };
  float m = -INFINITY, tl = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float2 (&sums)[8], const float4 (&sum)[8], int i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i + k >= count) break;
      const float mn = fmaxf(m, sums[k].x), base = mn == -INFINITY ? 0.f : mn;
      const float keep = ex2(m - base), f = ex2(sums[k].x - base);
      m = mn;
      tl = fmaf(f, sums[k].y, tl * keep);
      o.x = fmaf(f, sum[k].x, o.x * keep), o.y = fmaf(f, sum[k].y, o.y * keep);
      o.z = fmaf(f, sum[k].z, o.z * keep), o.w = fmaf(f, sum[k].w, o.w * keep);
    }
  };
  load(s[0], v[0], 0);
  for (int i = 0; i < count; i += 16) {
    if (i + 8 < count) load(s[1], v[1], i + 8);
    add(s[0], v[0], i);
    if (i + 16 < count) load(s[0], v[0], i + 16);
    add(s[1], v[1], i + 8);
  }
  const float inv = tl == 0.f ? no_weights(p, b, pc.pos0 + rho / G) : 1.f / tl;
  *reinterpret_cast<uint2*>(p.out + ((b * p.rows + rho / G) * p.a.Hq + hk * G + rho % G) * D + d4 * 4) =
      make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
}

// Positions are 32 bits wide, and steps are rounded up to 128 tokens behind the last one.
constexpr int kMaxLen = 0x7fffffff - 255;

// Blocks of up to 16 rows take steps of 64 tokens, more rows steps of 128.
static int tile_of(const moe_attention* a, int rows) {
  return rows * (a->Hq / a->Hkv) <= kFewRows ? kTileTok : 2 * kTileTok;
}

// The most pieces a sequence of up to max_len tokens can have.
static int max_pieces_of(const moe_attention* a, int rows, int max_len) {
  const int tile = tile_of(a, rows);
  long long tiles = ((long long)max_len + tile - 1) / tile;
  if (a->window) {
    const long long sinks = ((long long)a->sinks + tile - 1) / tile;
    tiles = std::min(tiles, sinks + ((long long)a->window + rows) / tile + 2);
  }
  // a shorter sequence can have more, where a piece's steps change
  int most = 1;
  for (long long t : {tiles, std::min(tiles, 63ll)}) most = std::max(most, piece_count(tile == kTileTok ? 6 : 7, (int)t));
  return most;
}

static size_t part_rows(const moe_attention* a, int rows, int max_len) {
  const int pieces = max_pieces_of(a, rows, max_len);
  return pieces == 1 ? 0 : (size_t)a->B * a->Hq * rows * pieces;
}

template <class C>
static int launch_cfg(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st) {
  CUtensorMap km, vm;
  const int box = std::min(cache->page_size, kTileTok);
  const CUtensorMapSwizzle swizzle = C::ROWB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  int rc = page_map(&km, cache->k, cache, box, swizzle);
  if (rc || (rc = page_map(&vm, cache->v, cache, box, swizzle))) return rc;
  auto kern = paged_attention_kernel<C>;
  if ((rc = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::SMEM))) return rc;
  const long long items = (long long)p.a.B * p.a.Hkv * p.max_pieces;
  return launch_pdl(kern, dim3((unsigned)std::min(items, (long long)C::CTAS * num_sms())), dim3((C::WARPS + 1) * 32), C::SMEM, st, km, vm, p);
}

template <int D, bool EIGHT>
static int launch_few(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st) {
  return cache->format == MOE_KV_MXFP8 ? launch_cfg<PagedCfg<D, true, EIGHT>>(p, cache, st)
                                       : launch_cfg<PagedCfg<D, false, EIGHT>>(p, cache, st);
}

static int launch_paged(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st) {
  const bool d64 = p.a.D == 64;
  int rc;
  if (p.tile_log2 != 6) rc = launch_paged_tc(p, cache, st);
  else if (p.R <= 8) rc = d64 ? launch_few<64, true>(p, cache, st) : launch_few<128, true>(p, cache, st);
  else rc = d64 ? launch_few<64, false>(p, cache, st) : launch_few<128, false>(p, cache, st);
  if (rc || p.max_pieces == 1) return rc;
  const int R = p.R;
  return launch_pdl(d64 ? paged_join_kernel<64> : paged_join_kernel<128>,
                    dim3((unsigned)(ceil_div(R, kJoinRows) * p.a.B * p.a.Hkv), (unsigned)(p.a.D / 4 / kJoinCols)),
                    dim3(kJoinRows * kJoinCols), 0, st, p);
}

static std::atomic<int> hold_load{-1};

int held_load() { return hold_load; }

}  // namespace moe

using namespace moe;

extern "C" int moe_selftest_attention_hold(int32_t load) {
  hold_load = load;
  return MOE_OK;
}

extern "C" size_t moe_paged_attention_workspace_bytes(const moe_attention* a, int32_t rows, int32_t max_len) {
  if (!attention_ok(a) || rows < 1 || rows > 64 || max_len < 0 || max_len > kMaxLen) return 0;
  const size_t n = part_rows(a, rows, max_len);
  return 256 + align_up(n * a->D * 4, 256) + align_up(n * 8, 256);
}

extern "C" int moe_paged_attention(const moe_attention* a, const moe_kv_cache* cache, int32_t rows, int32_t max_len,
                                   const uint16_t* q, int64_t q_stride, const int32_t* block_table,
                                   int32_t table_width, const int32_t* seq_lens, uint16_t* out, void* ws,
                                   size_t ws_bytes, void* stream) {
  if (!a || !cache) return MOE_ERR_INVALID_ARG;
  if (!attention_ok(a) || !kv_cache_ok(cache) || rows < 1 || rows > 64 || max_len > kMaxLen)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (cache->Hkv != a->Hkv || cache->D != a->D) return MOE_ERR_INVALID_ARG;
  if (max_len < 0 || table_width < 0 || max_len > (int64_t)table_width * cache->page_size) return MOE_ERR_INVALID_ARG;
  if (!status_ws_ok(ws, ws_bytes) || ws_bytes < moe_paged_attention_workspace_bytes(a, rows, max_len))
    return MOE_ERR_WORKSPACE;
  if (a->B == 0) return MOE_OK;
  if (!q || !block_table || !seq_lens || !out || !kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (q_stride < (int64_t)a->Hq * a->D || q_stride % 8) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens)) & 3) return MOE_ERR_INVALID_ARG;
  PagedArgs p{};
  p.a = *a;
  p.pages = cache->pages;
  p.page_size = cache->page_size;
  while ((1 << p.page_log2) < cache->page_size) ++p.page_log2;
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  p.k_s = cache->k_s;
  p.v_s = cache->v_s;
  p.rows = rows;
  p.max_len = max_len;
  p.table_width = table_width;
  p.G = a->Hq / a->Hkv;
  p.R = rows * p.G;
  p.tile_log2 = tile_of(a, rows) == kTileTok ? 6 : 7;
  p.block_log2 = p.tile_log2 == 6 ? 4 : 7;
  p.mblocks = ceil_div(p.R, 1 << p.block_log2);
  p.max_pieces = max_pieces_of(a, rows, max_len);
  // grids and the numbers of pieces stay below 2^31
  if ((int64_t)a->B * a->Hkv * std::max((int64_t)p.mblocks * p.max_pieces, (int64_t)ceil_div(p.R, kJoinRows)) >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  p.q = q;
  p.q_stride = q_stride;
  p.table = block_table;
  p.lens = seq_lens;
  p.out = out;
  p.status = static_cast<uint32_t*>(ws);
  p.hold = held_load();
  const size_t n = part_rows(a, rows, max_len);
  p.part_o = ws_ptr<float>(ws, 256);
  p.part_ml = ws_ptr<float>(ws, 256 + align_up(n * a->D * 4, 256));
  return launch_paged(p, cache, static_cast<cudaStream_t>(stream));
}
