// Attention of whole prompts, packed one behind the other.
//
// Bound: the tensor cores. Per visible (row, key) pair and head 4 D flops; keys come from L2 (a block reads its keys
// once for 256 rows). Both products run on tcgen05 with accumulators in Tensor Memory: S = Q K^T (128 x 128 keys), the
// softmax weights P as bf16 over S's own columns, O += P V with P read from Tensor Memory.
//
// A block has two tiles of 128 rows that share their keys: two heads of a group, or where a group has an odd number of
// heads, 256 rows of one. (Where there are few tiles, a block has one.) While one tile's weights are computed (one warpgroup each, a thread per row), the tensor
// cores work on the other's products:  PV0(i) QK0(i+1) | PV1(i) QK1(i+1).
// Blocks stay (one an SM) and take one item after the other, so that the next item's loads and first products run under
// the last one's end. The output is rescaled only when a row's maximum has grown by more than 2^8 since the last time
// (weights of up to 256 are as exact in bf16 as those up to 1), so that the softmax warps seldom touch it.
//
// A step of 128 keys takes two tiles about 2650 cycles, of which the products run 2048; an item's end 4000 to 5000, in which
// none runs. Three prompts of 12288 tokens together, 32 heads of 128, a window of 4096: 366 us, 1.29 PFLOP/s of visible pairs;
// one of 8192 without a window 338 us, 1.63 PFLOP/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "attention_tc.cuh"
#include "common.cuh"
#include "gemm.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kTileM = 128;             // query rows of a tile
constexpr int kTileN = 128;             // keys of a step
constexpr uint64_t kPrefillWaitNs = 1000000000ull;
constexpr float kRescaleLog2 = 8.f;
constexpr int kShort = 32;              // keys of a step that has few first tokens alone
constexpr int kFewKeys = 512;           // rows that see fewer keep their weights in two parts

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
  int pair;                             // 1: the two tiles are two heads, 0: two blocks of rows
  int hold;                             // see held_load
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

template <int D>
struct PrefillCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = kTileN * D * 2;                      // bytes of a tile of rows, keys or values
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static_assert(STAGES % 2 == 0, "keys in the even stages, values in the odd ones");
  static constexpr int OUT = 8 * 4096;                             // the output's way to global memory, 4 KB a warp
  static constexpr int SMEM = 2 * TILE + STAGES * TILE + OUT + 1024;
  // two softmax warpgroups and one whose first two warps load and issue; of the registers that the block is launched with
  // (168 a thread) the third warpgroup gives up what the others take: 2 x 208 + 88 = 3 x 168
  static constexpr int THREADS = 384;
  // Tensor Memory columns
  static constexpr int S0 = 0, S1 = 128, O0 = 256, O1 = 256 + D;
};

// The columns of one row's result that a listed key decides, by a warp.
template <int D>
__device__ __noinline__ void finish_row(const PrefillArgs& p, const BadKeys& bad, const Span& s, int row, int h) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x % 32, hk = h / (p.a.Hq / p.a.Hkv);
  const long long t = s.q0 + row;
  LaneRow<D> q;
  q.load_bf16(p.q + t * p.q_stride + (long long)h * D, lane);
  uint16_t* out = p.out + (t * p.a.Hq + h) * D + lane * N;
  add_not_finite<D>(bad, q, Visible(s.kn - s.qn + row, p.a.window, p.a.sinks), p.a.scale,
                    [&](int j, LaneRow<D>& k, LaneRow<D>& v) {
                      k.load_bf16(p.k + (long long)(s.k0 + j) * p.k_stride + (long long)hk * D, lane);
                      v.load_bf16(p.v + (long long)(s.k0 + j) * p.v_stride + (long long)hk * D, lane);
                    },
                    [&](int i, float x) { out[i] = (uint16_t)bf16x2(bf16_lo(out[i]) + x, 0.f); });
}

// Which steps of a tile are edges: some row of it does not see some key of the step that begins at j0.
struct Edges {
  int hi, lo, low;
  __device__ __forceinline__ bool at(int j0) const { return j0 > hi || (j0 < lo && j0 > low); }
};

// A block's item: up to 2 x 128 rows of a sequence and the keys that any of them sees, as steps of 128: the first tokens'
// steps, then the window's.
struct Item {
  Span s;
  int r0, h0;                           // first row (of the sequence), first head
  int off, r_end, sink_tiles, win_shift, tiles;
  bool short_sinks;                     // step 0 has the first tokens alone, and no more than 32
  __device__ __forceinline__ Item(const PrefillArgs& p, const int (&slot)[8])
      : s{slot[0], slot[1], slot[2], slot[3]}, r0(slot[4]), h0(slot[5]) {
    off = s.kn - s.qn;                  // position of row 0
    r_end = min(s.qn, r0 + (p.pair ? kTileM : 2 * kTileM));
    const int p_hi = off + r_end - 1;
    const int first_hi = first_of(p, p_hi);
    sink_tiles = (min(p.a.sinks, first_hi) + kTileN - 1) / kTileN;
    const int win_tile = max(first_of(p, off + r0) / kTileN, sink_tiles);
    win_shift = win_tile - sink_tiles;
    short_sinks = sink_tiles == 1 && p.a.sinks <= kShort && first_of(p, off + r0) >= kTileN;
    tiles = p_hi < 0 ? 0 : (p_hi + kTileN) / kTileN - win_shift;
  }
  static __device__ __forceinline__ int first_of(const PrefillArgs& p, int pos) {
    return p.a.window && pos >= p.a.window ? pos + 1 - p.a.window : 0;
  }
  __device__ __forceinline__ int key_of(int i) const { return (i < sink_tiles ? i : i + win_shift) * kTileN; }
  __device__ __forceinline__ int row_of(const PrefillArgs& p, int x) const { return r0 + (p.pair ? 0 : x * kTileM); }
  __device__ __forceinline__ Edges edges(const PrefillArgs& p, int x) const {
    const int t0 = row_of(p, x);
    if (t0 >= r_end) return Edges{0x7fffffff, 0, 0};      // nobody's rows
    return Edges{off + t0 + 1 - kTileN, first_of(p, off + min(t0 + kTileM, r_end) - 1), p.a.sinks - kTileN};
  }
  // Tiles whose first row sees few keys give their weights to the product in two parts in edge steps, rounded and rest;
  // over many keys the roundings even out.
  __device__ __forceinline__ bool split(const PrefillArgs& p, int x) const {
    return off + row_of(p, x) < kFewKeys || (p.a.window && p.a.window < kFewKeys);
  }
};

template <int D, bool ONE>                // ONE: a block has one tile alone (p.pair is 1 too)
__global__ void __launch_bounds__(PrefillCfg<D>::THREADS, 1)
prefill_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const PrefillArgs p) {
  using C = PrefillCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t w_full[2], w_empty[2], q_full, q_empty, s_full[2], p_full[2][2], o_full[2], drain;
  __shared__ uint64_t kv_full[C::STAGES], kv_empty[C::STAGES], v_clean[C::STAGES];
  __shared__ int slots[2][8];                   // items: span, first row, first head, whether there is one
  __shared__ BadKeys bad[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + 2 * C::TILE;
  uint8_t* staging = ring + C::STAGES * C::TILE;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 11);               // the warps of the products, of the cleaning and of the softmax
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 128);
      mbar_init(&p_full[i][1], 128);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
      mbar_init(&v_clean[i], 64);
    }
    abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Only now: a successor that takes Tensor Memory as well must not come before this block has its own, which it would keep
  // until this grid ends.
  pdl_trigger();
  pdl_wait();

  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {       // a whole warp's
    return __all_sync(0xffffffffu, bar_wait(bar, parity, kPrefillWaitNs, &abort_flag, code)) != 0;
  };
  auto item_there = [&](int n) {
    return wait(&w_full[n & 1], (n >> 1) & 1, DEV_TIMEOUT_FULL) && slots[n & 1][6] != 0;
  };
  auto item_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&w_empty[n & 1]);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // ---------------- items and loads ----------------
    if (warp == 8) {
      const int per_item = p.pair ? kTileM : 2 * kTileM;
      const int head_items = p.pair && !ONE ? p.a.Hq / 2 : p.a.Hq;
      int kv = 0, qs = 0;                       // tiles of keys or values, and pairs of tiles of queries, loaded so far
      bool ok = true;
      // The walk along the sequences, 32 at a time from the last ones on; a block's items only go up, so that it goes once.
      int group = (p.a.B + 31) / 32 * 32;       // first sequence of the 32
      int before = 0, total = 0, upto = 0;      // blocks of rows of those that were passed; of the 32; up to this lane's
      Span mine{0, 0, 0, 0};                    // the lane's sequence: lane 0 has the last one
      for (int n = 0; ok; ++n) {
        // Items are numbered from the last rows of the last sequence on, so that long rows are begun first; the heads of
        // the same rows are neighbours and share their keys in L2. Every other round is dealt out backwards: who had the
        // longest item of one round has the shortest of the next.
        const unsigned idx = (unsigned)n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        int want = (int)(idx / (unsigned)head_items), found = 0;
        Span sp{0, 0, 0, 0};
        while (want >= before + total && group > 0) {
          before += total;
          group -= 32;
          const int b = group + 31 - lane;
          mine = b < p.a.B ? span_of(p, b) : Span{0, 0, 0, 0};
          upto = (mine.qn + per_item - 1) / per_item;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
          }
          total = __shfl_sync(0xffffffffu, upto, 31);
        }
        want -= before;
        if (want < total) {
          const int who = __ffs(__ballot_sync(0xffffffffu, want < upto)) - 1;
          found = 1;
          want = __shfl_sync(0xffffffffu, upto, who) - 1 - want;        // of the sequence's items, from its first on
          sp.q0 = __shfl_sync(0xffffffffu, mine.q0, who);
          sp.qn = __shfl_sync(0xffffffffu, mine.qn, who);
          sp.k0 = __shfl_sync(0xffffffffu, mine.k0, who);
          sp.kn = __shfl_sync(0xffffffffu, mine.kn, who);
        }
        if (n >= 2 && !wait(&w_empty[n & 1], ((n >> 1) - 1) & 1, DEV_TIMEOUT_EMPTY)) break;
        const int slot[8] = {sp.q0, sp.qn, sp.k0, sp.kn, want * per_item, (int)(idx % (unsigned)head_items) * (p.pair && !ONE ? 2 : 1), found, 0};
        bad[n & 1].clear(lane);                 // the last item but one, whose list this was, is done
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < 7; ++i) slots[n & 1][i] = slot[i];
          mbar_arrive(&w_full[n & 1]);
        }
        if (!found) break;                      // the later rounds have none either
        const Item it(p, slot);
        if (it.tiles == 0) continue;
        if (qs > 0 && !wait(&q_empty, (qs - 1) & 1, DEV_TIMEOUT_EMPTY)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full, (2 - ONE) * C::TILE);
          for (int x = 0; x < 2 - ONE; ++x)
            for (int d = 0; d < C::HALVES; ++d)
              tma_load_3d(smem + x * C::TILE + d * kTileM * 128, &qmap, d * 64, p.pair ? it.h0 + x : it.h0,
                          it.s.q0 + it.row_of(p, x), &q_full);
        }
        ++qs;
        const int hk = it.h0 / (p.a.Hq / p.a.Hkv);
        for (int i = 0; ok && i < 2 * it.tiles; ++i) {      // K of a step, V of a step, in turn
          const int s = kv % C::STAGES;
          if (kv >= C::STAGES && !(ok = wait(&kv_empty[s], (kv / C::STAGES - 1) & 1, DEV_TIMEOUT_EMPTY))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&kv_full[s], C::TILE + (kv == p.hold ? 16 : 0));
            for (int d = 0; d < C::HALVES; ++d)
              tma_load_3d(ring + s * C::TILE + d * kTileN * 128, i & 1 ? &vmap : &kmap, d * 64, hk,
                          it.s.k0 + it.key_of(i / 2), &kv_full[s]);
          }
          ++kv;
        }
      }
      // copies in flight end before the block does, whoever gives up and when
      if (qs) mbar_wait(&q_full, (qs - 1) & 1, kPrefillWaitNs, nullptr, nullptr, DEV_TIMEOUT_DRAIN);
      for (int j = max(0, kv - C::STAGES); j < kv; ++j)
        mbar_wait(&kv_full[j % C::STAGES], (j / C::STAGES) & 1, kPrefillWaitNs, nullptr, nullptr, DEV_TIMEOUT_DRAIN);
    }
    // ---------------- products ----------------
    // The whole warp goes along and one lane issues: addresses stay uniform, and so in uniform registers. (With one
    // lane alone in the branch each product took 80 to 160 cycles to issue, of the 64 that it runs.)
    if (warp == 9) {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const bool leader = elect_one();
      const uint32_t idesc_qk = idesc_bf16_f32(kTileM, kTileN), idesc_short = idesc_bf16_f32(kTileM, kShort);
      const uint32_t idesc_pv = idesc_bf16_f32(kTileM, D) | (1u << 16);      // V: its D values contiguous, keys apart
      const uint64_t qdesc = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t kdesc = smem_desc(smem_u32(ring), 16, 1024, 2);
      const uint64_t vdesc = smem_desc(smem_u32(ring), kTileN * 128, 1024, 2);
      auto qk = [&](int x, int s, bool brief) {
        if (leader) {
          const uint64_t qx = qdesc + x * (C::TILE >> 4), kx = kdesc + s * (C::TILE >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const int at = ((ks / 4) * kTileN * 128 + (ks % 4) * 32) >> 4;
            mma_bf16(tm + x * (C::S1 - C::S0) + C::S0, qx + at, kx + at, brief ? idesc_short : idesc_qk, ks > 0);
          }
          tc_commit(&s_full[x]);
        }
        __syncwarp();
      };
      // Half h of the keys of a step; its weights are there.
      auto pv = [&](int x, int h, int s, bool more, bool split, bool brief) {
        if (leader) {
          const uint32_t d = tm + x * (C::O1 - C::O0) + C::O0, a = tm + x * (C::S1 - C::S0) + C::S0;
          const uint64_t vx = vdesc + s * (C::TILE >> 4);
          if (!split) {
#pragma unroll
            for (int k4 = 0; k4 < kTileN / 32; ++k4) {
              const int ks = h * kTileN / 32 + k4;
              if (brief && ks >= kShort / 16) break;
              mma_bf16_ts(d, a + ks * 8, vx + ks * (2048 >> 4), idesc_pv, more || k4 > 0);
            }
          } else {
            // of every 32 columns 16 hold the rounded weights of 32 keys, 16 the rests
#pragma unroll
            for (int k4 = 0; k4 < kTileN / 32; ++k4) {
              const int ks = h * kTileN / 32 + k4;
              if (brief && ks >= kShort / 16) break;
              mma_bf16_ts(d, a + ks / 2 * 32 + ks % 2 * 8, vx + ks * (2048 >> 4), idesc_pv, more || k4 > 0);
              mma_bf16_ts(d, a + ks / 2 * 32 + ks % 2 * 8 + 16, vx + ks * (2048 >> 4), idesc_pv, 1);
            }
          }
        }
        __syncwarp();
      };
      auto release = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
      };
      int kv = 0, step = 0, qs = 0;             // tiles of keys or values, steps and pairs of query tiles so far
      auto have = [&](int n) { return wait(&kv_full[n % C::STAGES], (n / C::STAGES) & 1, DEV_TIMEOUT_FULL); };
      bool ok = true;
      for (int n = 0; ok && item_there(n); ++n) {
        const Item it(p, slots[n & 1]);
        item_done(n);
        if (it.tiles == 0) continue;
        ok = wait(&q_full, qs & 1, DEV_TIMEOUT_FULL) && have(kv);
        if (!ok) break;
        ++qs;
        // S lies over the last item's weights: products are executed in the order of their issue
        qk(0, kv % C::STAGES, it.short_sinks);
        if (!ONE) qk(1, kv % C::STAGES, it.short_sinks);
        release(&kv_empty[kv % C::STAGES]);
        if (it.tiles == 1) release(&q_empty);
        const Edges e0 = it.edges(p, 0), e1 = it.edges(p, 1);
        const bool split[2] = {it.split(p, 0), it.split(p, 1)};
        for (int i = 0; ok && i < it.tiles; ++i, ++step) {
          const int vs = (kv + 1) % C::STAGES, ks = (kv + 2) % C::STAGES;
          const bool brief = it.short_sinks && i == 0;
          const bool edge[2] = {e0.at(it.key_of(i)), e1.at(it.key_of(i))};
          ok = wait(&v_clean[vs], ((kv + 1) / C::STAGES) & 1, DEV_TIMEOUT_FULL);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x == 1 && ONE) break;
            if (!ok || !(ok = wait(&p_full[x][0], step & 1, DEV_TIMEOUT_ACCUM))) break;
            tc_fence_after();
            pv(x, 0, vs, i > 0, edge[x] && split[x], brief);
            if (!(ok = wait(&p_full[x][1], step & 1, DEV_TIMEOUT_ACCUM))) break;
            tc_fence_after();
            if (!brief) pv(x, 1, vs, true, edge[x] && split[x], false);
            if (x == 1 || ONE) release(&kv_empty[vs]);
            release(&o_full[x]);
            if (i + 1 < it.tiles) {
              if (x == 0 && !(ok = have(kv + 2))) break;
              qk(x, ks, false);
            }
          }
          if (ok && i + 1 < it.tiles) {         // a stage that was not read is not given back
            release(&kv_empty[ks]);
            if (i + 2 == it.tiles) release(&q_empty);
          }
          kv += 2;
        }
      }
      if (leader) {                             // the products end before the block does, too
        tc_commit(&drain);
        mbar_wait(&drain, 0, kPrefillWaitNs, nullptr, nullptr, DEV_TIMEOUT_DRAIN);
      }
    }
    // ---------------- values that are not finite ----------------
    // A weight of zero does not hide such a value in the product. Where a row of the block does not see every key of a
    // step, they are set to zero and their keys listed, for the rows that do see them.
    if (warp >= 10) {
      const int tid = threadIdx.x - 320;
      int kv = 0;
      bool ok = true;
      for (int n = 0; ok && item_there(n); ++n) {
        const Item it(p, slots[n & 1]);
        const Edges e0 = it.edges(p, 0), e1 = it.edges(p, 1);
        for (int i = 0; i < it.tiles; ++i, kv += 2) {
          // every step's values pass here, edge or not: a barrier's parity tells its next phase from the last one only
          // to a waiter that has seen them all
          const int j0 = it.key_of(i), st = (kv + 1) % C::STAGES;
          if (!(ok = wait(&kv_full[st], ((kv + 1) / C::STAGES) & 1, DEV_TIMEOUT_FULL))) break;
          if (!e0.at(j0) && !e1.at(j0)) {
            mbar_arrive(&v_clean[st]);
            continue;
          }
          uint4* v = reinterpret_cast<uint4*>(ring + st * C::TILE);
          // zero times a value that is not finite is NaN, and stays in the sum
          uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 8
          for (int e = tid; e < C::TILE / 16; e += 64) {
            const uint4 a = v[e];
            sum[0] = fma_bf16x2(a.x, 0, sum[0]);
            sum[1] = fma_bf16x2(a.y, 0, sum[1]);
            sum[2] = fma_bf16x2(a.z, 0, sum[2]);
            sum[3] = fma_bf16x2(a.w, 0, sum[3]);
          }
          if (!__any_sync(0xffffffffu, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0)) {
            mbar_arrive(&v_clean[st]);
            continue;
          }
          bool wrote = false;
#pragma unroll 1
          for (int e = tid; e < C::TILE / 16; e += 64) {
            const uint4 a = v[e];
            // an exponent field of all ones carries into the bit above it when its lowest bit is added
            const uint32_t any = (((a.x & 0x7F807F80u) + 0x00800080u) | ((a.y & 0x7F807F80u) + 0x00800080u) |
                                  ((a.z & 0x7F807F80u) + 0x00800080u) | ((a.w & 0x7F807F80u) + 0x00800080u)) & 0x80008000u;
            // 8 neighbouring lanes hold one key's 64 values: one of them lists it
            const unsigned hits = __ballot_sync(0xffffffffu, any != 0);
            if (any) {
              const uint32_t w[4] = {a.x, a.y, a.z, a.w};
              uint32_t z[4];
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const uint32_t hit = ((w[f] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                z[f] = w[f] & ~((hit >> 15) * 0xFFFFu);
              }
              v[e] = make_uint4(z[0], z[1], z[2], z[3]);
              wrote = true;
              if (__ffs(hits & (0xFFu << (tid & 24))) - 1 == (tid & 31)) bad[n & 1].add(j0 + e / 8 % kTileN);
            }
          }
          if (wrote) fence_async_smem();
          mbar_arrive(&v_clean[st]);
        }
        item_done(n);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------- softmax ----------------
    const int x = warp / 4, tid = threadIdx.x % 128;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + (x ? C::S1 : C::S0) + lanes, to = tmem + (x ? C::O1 : C::O0) + lanes;
    // scores in units of log2 e / scale; a scale below zero turns their sign, zero becomes a scale that tells none apart
    const uint32_t turn = p.a.scale < 0.f ? 0x80000000u : 0u;
    const float c = fmaxf(fabsf(p.a.scale) * 1.4426950408889634f, 1e-37f);
    int step = 0;                               // steps so far
    bool ok = true;
    for (int n = 0; ok && item_there(n); ++n) {
      if (x == 1 && ONE) {
        item_done(n);
        continue;
      }
      int tiles, sink_tiles, win_shift, pos, first;
      bool split;
      Edges edges;
      {
        const Item it(p, slots[n & 1]);
        const int row = it.row_of(p, x) + tid;  // of the sequence
        pos = row < it.r_end ? it.off + row : -1;
        first = Item::first_of(p, pos);
        split = it.split(p, x);
        edges = it.edges(p, x);
        tiles = it.tiles, sink_tiles = it.sink_tiles, win_shift = it.win_shift;
      }
      float m = -INFINITY;                      // the maximum that the weights so far refer to
      uint64_t l2 = pack2(0.f, 0.f);
      for (int i = 0; i < tiles; ++i, ++step) {
        if (!(ok = wait(&s_full[x], step & 1, DEV_TIMEOUT_ACCUM))) break;
        tc_fence_after();
        const int j0 = (i < sink_tiles ? i : i + win_shift) * kTileN;
        float mx = -INFINITY;
        // The maximum that the weights refer to moves only when one has outgrown it; then what has been summed is
        // rescaled.
        auto move_base = [&]() {
          const float mn = fmaxf(m, mx);
          // (-inf) - (-inf): no. Rows that nobody has, or that see nothing, have no say: where the others' maximum moves
          // decides how their weights round.
          if (!__any_sync(0xffffffffu, pos >= 0 && (mn - m) * c > kRescaleLog2)) return true;
          if (i > 0) {
            if (!wait(&o_full[x], (step - 1) & 1, DEV_TIMEOUT_ACCUM)) return false;
            tc_fence_after();
            const float f = m == -INFINITY ? 0.f : ex2((m - mn) * c);
            l2 = mul2(l2, pack2(f, f));
#pragma unroll 1
            for (int e = 0; e < D; e += 16) {
              uint32_t o[16];
              tmem_ld16(to + e, o);
              tmem_ld_wait();
              reg_fence16(o);
#pragma unroll
              for (int d = 0; d < 16; ++d) o[d] = __float_as_uint(__uint_as_float(o[d]) * f);
              tmem_st16(to + e, o);
            }
          }
          m = mn;
          return true;
        };
        uint64_t la = pack2(0.f, 0.f), lb = la, b2 = la, c2 = la;
        auto weights = [&](const uint32_t* s, float (&w)[4]) {
          unpack2(fma2(pack2(__uint_as_float(s[0]), __uint_as_float(s[1])), c2, b2), w[0], w[1]);
          unpack2(fma2(pack2(__uint_as_float(s[2]), __uint_as_float(s[3])), c2, b2), w[2], w[3]);
#pragma unroll
          for (int f = 0; f < 4; ++f) w[f] = ex2(w[f]);
          la = add2(la, pack2(w[0], w[1]));
          lb = add2(lb, pack2(w[2], w[3]));
        };
        // the weights of half h are in Tensor Memory
        auto hand_over = [&](int h) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[x][h]);
        };
        const bool edge = edges.at(j0);
        if (edge || turn) {
          // Hidden in Tensor Memory, 32 scores at a time: little code, and groups that all of the warp's rows see are left.
          // The row sees key j0 + e when e <= hi and (e >= lo or e < low). (Scores that a short step has not computed are
          // hidden with the rest behind the first tokens.)
          const int hi = pos - j0, lo = first - j0, low = p.a.sinks - j0;
          auto below = [](int k) { return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u; };
#pragma unroll 1
          for (int e = 0; e < kTileN; e += 32) {
            const uint32_t see = below(hi + 1 - e) & (~below(lo - e) | below(low - e));
            if (!turn && __all_sync(0xffffffffu, see == 0xffffffffu)) continue;
            uint32_t s[32];
            tmem_ld32(ts + e, s, 0);
            tmem_ld_wait();
            reg_fence32(s, 0);
#pragma unroll
            for (int d = 0; d < 32; ++d) s[d] = (see >> d) & 1u ? s[d] ^ turn : 0xff800000u;
            tmem_st32(ts + e, s, 0);
          }
          tmem_st_wait();
        }
        uint32_t s[128];
#pragma unroll
        for (int e = 0; e < 128; e += 32) tmem_ld32(ts + e, s, e);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 128; e += 32) reg_fence32(s, e);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 8)
#pragma unroll
          for (int f = 0; f < 4; ++f)
            m4[f] = max3(m4[f], __uint_as_float(s[e + 2 * f]), __uint_as_float(s[e + 2 * f + 1]));
        mx = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
        if (!(ok = move_base())) break;
        const float cw = weight_factor(m, c), base = m == -INFINITY ? 0.f : -m * cw;
        b2 = pack2(base, base);
        c2 = pack2(cw, cw);
        if (!edge || !split) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 64 * h; e < 64 * h + 64; e += 4) {
              float w[4];
              weights(s + e, w);
              s[e / 2] = bf16x2(w[0], w[1]);    // s[e / 2] has been read
              s[e / 2 + 1] = bf16x2(w[2], w[3]);
            }
            tmem_st32(ts + 32 * h, s, 32 * h);
            hand_over(h);
          }
        } else {
#pragma unroll 1
          for (int e = 0; e < 128; e += 32) {
            uint32_t s[32], u[32];              // of u, 16 of the rounded weights and 16 of the rests
            tmem_ld32(ts + e, s, 0);
            tmem_ld_wait();
            reg_fence32(s, 0);
#pragma unroll
            for (int d = 0; d < 16; d += 2) {
              float w[4];
              weights(s + 2 * d, w);
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                u[d + f] = bf16x2(w[2 * f], w[2 * f + 1]);
                u[16 + d + f] = bf16x2(w[2 * f] - bf16_lo(u[d + f]), w[2 * f + 1] - bf16_hi(u[d + f]));
              }
            }
            tmem_st32(ts + e, u, 0);
            if (e & 32) hand_over(e / 64);
          }
        }
        l2 = add2(l2, add2(la, lb));
      }
      if (ok && tiles > 0) {
        ok = wait(&o_full[x], (step - 1) & 1, DEV_TIMEOUT_ACCUM);
        tc_fence_after();
      }
      if (!ok) break;

      // what the end of an item needs is worked out here, not kept in registers over the steps
      int ln = lane;
      asm volatile("" : "+r"(ln));
      const Item it(p, slots[n & 1]);
      const int h = p.pair ? it.h0 + x : it.h0, row = it.row_of(p, x) + warp % 4 * 32 + ln;
      const bool live = row < it.r_end;
      float la, lb;
      unpack2(l2, la, lb);
      const float l = la + lb;
      // without weights: zero where a row sees nothing; else all scores were minus infinity, and 0 / 0 is NaN
      const float inv = l != 0.f ? 1.f / l : it.off + row < 0 ? 0.f : __uint_as_float(0x7FC00000u);
      // Rows that see a listed key. (Every value that is not finite was listed before the last product that met it. A score
      // that is NaN makes the sum NaN, and with it the row: that is its result.)
      bool again = false;
      if (it.tiles > 0 && *reinterpret_cast<volatile int*>(&bad[n & 1].some)) {
        const Visible see(live ? it.off + row : -1, p.a.window, p.a.sinks);
        bad[n & 1].each([&](int j) { again = again || see.sees(j); });
        again = again && live && l == l;
      }
      // Through shared memory, so that a warp writes 128-byte pieces of rows: 64 columns of its 32 rows at a time, in
      // chunks of 16 bytes whose order is turned by the row.
      uint4* mine = reinterpret_cast<uint4*>(staging + warp * 4096);
      const unsigned rows_live = __ballot_sync(0xffffffffu, live);
      uint16_t* out = p.out + ((long long)(it.s.q0 + row - ln) * p.a.Hq + h) * D;
      uint32_t o[D];
#pragma unroll
      for (int e = 0; e < D; e += 32) tmem_ld32(to + e, o, e);        // without keys: whatever is there, and not used
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < D; e += 32) reg_fence32(o, e);
      if (it.tiles == 0) {
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = 0;
      }
      const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
#pragma unroll
        for (int d = 0; d < 64; d += 8) {
          uint32_t w[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int e = half * 64 + d + 2 * f;
            float u, v;
            unpack2(mul2(pack2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), inv2), u, v);
            w[f] = bf16x2(u, v);
          }
          mine[ln * 8 + ((d / 8) ^ (ln & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        uint4 t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = e * 4 + ln / 8, ch = ln % 8;
          t[e] = mine[r * 8 + (ch ^ (r & 7))];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = e * 4 + ln / 8, ch = ln % 8;
          if ((rows_live >> r) & 1u)
            *reinterpret_cast<uint4*>(out + (long long)r * p.a.Hq * D + half * 64 + ch * 8) = t[e];
        }
        __syncwarp();
      }
      for (unsigned rows = __ballot_sync(0xffffffffu, again); rows; rows &= rows - 1)
        finish_row<D>(p, bad[n & 1], it.s, row - ln + __ffs(rows) - 1, h);
      item_done(n);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && abort_flag) atomicCAS(p.status, 0u, abort_flag);
}

static int rows_map(CUtensorMap* m, const void* base, int D, int heads, int rows, long long stride) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return MOE_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTileN};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

// The most items that there can be: every sequence may end in a part of a tile.
static long long items_of(const PrefillArgs& p, bool one) {
  const int rows = one || p.pair ? kTileM : 2 * kTileM;
  return ((long long)p.Tq / rows + p.a.B) * (!one && p.pair ? p.a.Hq / 2 : p.a.Hq);
}

template <int D>
static int launch_prefill(const PrefillArgs& p, cudaStream_t st) {
  CUtensorMap qm, km, vm;
  int rc = rows_map(&qm, p.q, D, p.a.Hq, p.Tq, p.q_stride);
  // without keys no tile is loaded; the maps have to describe something all the same
  if (!rc) rc = p.Tk ? rows_map(&km, p.k, D, p.a.Hkv, p.Tk, p.k_stride) : rows_map(&km, p.q, D, p.a.Hq, p.Tq, p.q_stride);
  if (!rc) rc = p.Tk ? rows_map(&vm, p.v, D, p.a.Hkv, p.Tk, p.v_stride) : rows_map(&vm, p.q, D, p.a.Hq, p.Tq, p.q_stride);
  if (rc) return rc;
  // Two tiles a block take 2650 cycles a step, one alone about 1900: one each where there are blocks enough for it (one
  // head, 2048 tokens of 128: 24 us against 29; 32 heads, 128 tokens: 6.4 against 8.7).
  PrefillArgs args = p;
  const bool one = items_of(p, true) <= num_sms();
  if (one) args.pair = 1;
  auto kern = one ? prefill_attention_kernel<D, true> : prefill_attention_kernel<D, false>;
  if ((rc = ensure_smem_limit(reinterpret_cast<const void*>(kern), PrefillCfg<D>::SMEM))) return rc;
  const long long items = items_of(p, one);
  if (items >= (1ll << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return launch_pdl(kern, dim3((unsigned)std::min(items, (long long)num_sms())), dim3(PrefillCfg<D>::THREADS),
                    PrefillCfg<D>::SMEM, st, qm, km, vm, args);
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
                      static_cast<uint32_t*>(ws), (a->Hq / a->Hkv) % 2 == 0, held_load()};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->D == 64 ? launch_prefill<64>(p, st) : launch_prefill<128>(p, st);
}
