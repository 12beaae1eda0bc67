// Attention of many rows over the paged cache: blocks of more than 16 rows (row, head of the group), as the verification
// rows of speculative decoding make them (6 rows and 8 heads to a group are 48).
//
// Bound: HBM, as for few rows, but here the products decide whether it is reached: 4 D R flops a key are more than
// mma.sync does at that rate once R passes 16 or so, and an MXFP8 cache would have to be converted by every warp again.
// So both products run on tcgen05 with the rows as M = 128 (the rows beyond R cost nothing but tensor time, of which
// there is enough: 1024 cycles a step of 128 tokens, against 2800 that its bytes take in bf16 and 1440 in MXFP8). Both
// sides of the limit measured: 24 rows over bf16 take 14 us here and 18 us there (4096 tokens, 8 kv heads), 48 rows over
// MXFP8 76 us here and 248 us there (8 sequences of up to 16k tokens). 16 rows go there: M = 16 wastes nothing of them.
//
// Resident blocks take item after item: one piece of one (sequence, kv head). Its steps go in turn to two chains, each with
// scores, weights and output of its own in Tensor Memory and a warpgroup of its own (a thread per row), so that one
// chain's products run under the other's softmax:  PV0(0) QK0(2) | PV1(1) QK1(3) | PV0(2) QK0(4) ...  The chains' outputs
// are joined at the item's end.
// Pages come by TMA, bf16 straight into the ring that the products read, MXFP8 into a ring of raw codes from where a
// warpgroup converts them once for all rows (four significant bits and a power of two fit bf16: exactly, but for scale bytes 0
// to 2, whose blocks may have codes below bf16's last subnormal, 2^-133, and are rounded to it).
//
// What an MXFP8 step takes, about 2,350 cycles, is shared memory's time for the most part: 270 for the codes to come in, 320
// for them to be read, 512 to be stored converted, 770 for the operands of the products. An item's end takes about 5,000
// more, in which the chains join and write and no product runs; the pieces are long enough for four fifths of the time to
// go to steps. 8 sequences of up to 16k tokens, 48 rows, 8 kv heads of 128: 76 us, 2.6 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "attention_paged.cuh"
#include "attention_tc.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kRowsM = 128;             // rows of a block
constexpr int kStepTok = 128;           // tokens of a step
constexpr int kInfos = 16;              // steps whose tokens are remembered
// Kinds of steps: every row sees every key; does so but for pages out of range; some row does not see some key.
enum : int { kSeen, kHoles, kEdge };
constexpr float kGrow = 8.f;            // the maximum that weights refer to moves when outgrown by 2^8

template <int D_, bool MX_>
struct TcCfg {
  static constexpr int D = D_;
  static constexpr bool MX = MX_;
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = kStepTok * D * 2;                    // a step's keys, or values, in bf16; the queries
  static constexpr int RAW = MX ? (kStepTok * D + kStepTok * (D / 32) + 1023) / 1024 * 1024 : 0;
  static constexpr int RAWS = !MX ? 1 : D == 128 ? 4 : 10;          // stages of raw codes
  static constexpr int ENTRIES = MX ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
  static constexpr int SMEM = TILE + ENTRIES * TILE + RAWS * RAW + 1024;
  static constexpr int THREADS = MX ? 640 : 384;
  // registers: the block is launched with 96 (168) a thread; the two softmax warpgroups take what the others give up
  static constexpr int MORE = MX ? 168 : 208, LESS = MX ? 48 : 88;
  static constexpr int FEEDERS = MX ? 4 : 1;                       // warps that hand a tile to the products
  static constexpr int GROUPS = MX ? 2 : 1;                        // of them, which take tiles in turn
  // Barriers of the entries that the products have read, by tile: a group waits for those of its own tiles alone, and a barrier
  // cannot end its next phase before the group has seen this one.
  static constexpr int ENT_BARS = ENTRIES % GROUPS ? ENTRIES * GROUPS : ENTRIES;
  static constexpr int S0 = 0, S1 = 128, O0 = 256, O1 = 256 + D;   // Tensor Memory columns
  static_assert(RAWS % GROUPS == 0, "a group of feeders sees every phase of its stages");
  static_assert(SMEM + 4096 <= 227 * 1024, "shared memory");
};

// Item `n` of a block, as it lies in shared memory: what the warps need of it, worked out once.
struct PagedItem {
  int there, b, hk, rho0, live;                 // first row of the block, rows there are
  int pos0;                                     // position of row 0 of the sequence's new rows
  int pmax, first_any, sink_tiles, win_tile;
  int first_all, pmin;                          // tokens from first_all to pmin are in all rows' windows
  int i0, cnt, piece, pieces;                   // first step, steps; piece of how many
  __device__ __forceinline__ int tok(int i) const {
    const int t = i0 + i;
    return (t < sink_tiles ? t : win_tile + (t - sink_tiles)) * kStepTok;
  }
};

// The columns of one row's part of an item that a listed key decides, by a warp, which takes one half of them.
template <int D, bool MX>
__device__ __noinline__ void finish_part(const PagedArgs& p, const BadKeys& bad, const PagedItem& it, int rho, int half) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x % 32, G = p.G, r = rho / G;
  const long long row = ((long long)it.b * p.rows + r) * p.a.Hq + it.hk * G + rho % G;
  const long long at = ((long long)it.b * p.a.Hkv + it.hk) * p.max_pieces + it.piece;
  LaneRow<D> q;
  q.load_bf16(p.q + ((long long)it.b * p.rows + r) * p.q_stride + (long long)(it.hk * G + rho % G) * D, lane);
  add_not_finite<D>(bad, q, Visible(it.pos0 + r, p.a.window, p.a.sinks), p.a.scale,
                    [&](int j, LaneRow<D>& k, LaneRow<D>& v) {
                      const int page = p.table[(long long)it.b * p.table_width + (j >> p.page_log2)];
                      const long long t = (((long long)page * p.a.Hkv + it.hk) << p.page_log2) + (j & (p.page_size - 1));
                      if (MX) {
                        k.load_mxfp8(p.k + t * D, p.k_s + t * N, lane);
                        v.load_mxfp8(p.v + t * D, p.v_s + t * N, lane);
                      } else {
                        k.load_bf16(reinterpret_cast<const uint16_t*>(p.k) + t * D, lane);
                        v.load_bf16(reinterpret_cast<const uint16_t*>(p.v) + t * D, lane);
                      }
                    },
                    [&](int i, float x) {
                      if (lane / 16 != half) return;
                      const int d = lane * N + i;
                      if (it.pieces == 1) p.out[row * D + d] = (uint16_t)bf16x2(bf16_lo(p.out[row * D + d]) + x, 0.f);
                      else part_of(p, at, D, rho, d / 4)[d % 4] += x;
                    });
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PagedArgs p) {
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t w_full[2], w_empty[2], q_full, q_empty, s_full[2], p_full[2][2], o_full[2], drain;
  __shared__ uint64_t sums_there, outs_read;
  __shared__ uint64_t landed[C::MX ? C::RAWS : C::ENTRIES], raw_empty[C::RAWS], ready[C::ENTRIES], ent_empty[C::ENT_BARS];
  __shared__ PagedItem items[2];
  __shared__ int4 infos[kInfos];                // of a step: first token, pages there, its kind
  __shared__ BadKeys bad[2];
  __shared__ float2 sums[2][kRowsM];            // the chains' maximum (times log2 e) and sum of a row
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + C::TILE;
  uint8_t* raws = ring + C::ENTRIES * C::TILE;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&drain, 1);
    mbar_init(&sums_there, 256);
    mbar_init(&outs_read, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&w_full[i], 1);
      // the warps of the products, of the queries, of the feeding, of the softmax
      mbar_init(&w_empty[i], 10 + C::FEEDERS * C::GROUPS);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 128);
      mbar_init(&p_full[i][1], 128);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < (C::MX ? C::RAWS : C::ENTRIES); ++i) mbar_init(&landed[i], 1);
    for (int i = 0; i < C::RAWS; ++i) mbar_init(&raw_empty[i], C::FEEDERS);
    for (int i = 0; i < C::ENTRIES; ++i) mbar_init(&ready[i], C::FEEDERS);
    for (int i = 0; i < C::ENT_BARS; ++i) mbar_init(&ent_empty[i], 1);
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
  pdl_wait();
  pdl_trigger();

  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {       // a whole warp's
    return __all_sync(0xffffffffu, bar_wait(bar, parity, kPagedWaitNs, &abort_flag, code)) != 0;
  };
  auto item_there = [&](int n) {
    return wait(&w_full[n & 1], (n >> 1) & 1, DEV_TIMEOUT_FULL) && items[n & 1].there != 0;
  };
  auto item_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&w_empty[n & 1]);
  };
  // the products have read what was in this tile's entry before
  auto ent_free = [&](int tile) {
    const int last = tile - C::ENTRIES;
    return last < 0 || wait(&ent_empty[last % C::ENT_BARS], (last / C::ENT_BARS) & 1, DEV_TIMEOUT_EMPTY);
  };
  // An item's tiles pass in this order: K0 K1 V0 K2 V1 K3 V2 ..., one counter for all.

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::LESS));
    if (warp == 8) {
      // ---------------- items and loads ----------------
      const int in_tile = p.page_size >= kStepTok ? 1 : kStepTok >> p.page_log2;   // pages of a step
      const int rows_of = min(p.page_size, kStepTok);
      int n = 0, tile = 0, steps = 0;
      bool ok = true;
      ItemWalk walk;
      for (long long idx = blockIdx.x; ok; idx += gridDim.x) {
        const int who = walk.lane_of(p, idx);
        if (n >= 2 && !(ok = wait(&w_empty[n & 1], ((n >> 1) - 1) & 1, DEV_TIMEOUT_EMPTY))) break;
        if (lane == max(who, 0)) {
          PagedItem mine{};                     // no more items: that one is not there
          if (who >= 0) {
            const int u = walk.group + lane, b = p.mblocks == 1 ? u : u / p.mblocks;
            const int j = (int)(idx - walk.before) - (walk.upto - walk.mine);
            const Pieces& pc = walk.pc;
            mine.there = 1;
            mine.b = b;
            mine.piece = j / p.a.Hkv;
            mine.hk = j - mine.piece * p.a.Hkv;
            mine.rho0 = (u - b * p.mblocks) * kRowsM;
            mine.live = min(p.R - mine.rho0, kRowsM);
            mine.pos0 = pc.pos0;
            mine.pmin = pc.pmin, mine.pmax = pc.pmax, mine.first_any = pc.first_any, mine.first_all = pc.first_all;
            mine.sink_tiles = pc.sink_tiles, mine.win_tile = pc.win_tile;
            mine.i0 = pc.begin(mine.piece);
            mine.cnt = pc.steps(mine.piece);
            mine.pieces = pc.count;
          }
          items[n & 1] = mine;
        }
        bad[n & 1].clear(lane);                 // the last item but one, whose list this was, is done
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_full[n & 1]);
        if (who < 0) break;
        const PagedItem it = items[n & 1];
        const int all_from = it.first_all, all_to = it.pmin;
        ++n;
        const int cnt = it.cnt;
        const int32_t* table = p.table + (long long)it.b * p.table_width;
        const int last_page = it.pmax >> p.page_log2;
        int base = -1000, ids = 0, next = 0;       // 32 table entries from `base` on, and the 32 behind them
        int held[2] = {-1, -1};                    // page of this lane in the last two steps
        for (int t = 0; t < 2 * cnt + 2; ++t) {    // the turns: K0 K1 V0 K2 V1 ...
          const bool is_v = t >= 2 && !(t & 1);
          const int i = t < 2 ? t : is_v ? (t - 2) / 2 : (t + 1) / 2;
          if (i >= cnt) continue;
          const int tok0 = it.tok(i), t0 = tok0 + lane * rows_of;
          int id = i & 1 ? held[1] : held[0];
          if (!is_v) {
            const int page0 = tok0 >> p.page_log2;
            if (page0 < base || page0 + in_tile > base + 32) {
              const int nb = page0 & ~31;          // in_tile divides 32: a step's pages lie in one group of 32 entries
              ids = nb == base + 32 ? next : (nb + lane <= last_page ? table[nb + lane] : -1);
              base = nb;
              next = nb + 32 + lane <= last_page ? table[nb + 32 + lane] : -1;
            }
            id = __shfl_sync(0xffffffffu, ids, (page0 - base + lane) & 31);
            // pages that no row sees are not loaded: past the end, or between the first tokens and the window
            const bool want = lane < in_tile && t0 <= it.pmax &&
                              (t0 + rows_of > it.first_any || t0 < min(p.a.sinks, all_from));
            const bool good = want && id >= 0 && id < p.pages;
            if (want && !good) atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
            id = good ? id : -1;
            if (i & 1) held[1] = id; else held[0] = id;
          }
          constexpr int N = C::MX ? C::RAWS : C::ENTRIES;
          const int st = tile % N, use = tile / N;
          const unsigned mask = __ballot_sync(0xffffffffu, id >= 0);
          if (!(ok = C::MX ? use == 0 || wait(&raw_empty[st], (use - 1) & 1, DEV_TIMEOUT_EMPTY) : ent_free(tile))) break;
          if (lane == 0) {
            if (!is_v) {
              const bool whole = tok0 + kStepTok - 1 <= all_to && (tok0 >= all_from || tok0 + kStepTok <= p.a.sinks);
              infos[(steps + i) % kInfos] =
                  make_int4(tok0, (int)mask, whole ? (mask == (1u << in_tile) - 1u ? kSeen : kHoles) : kEdge, 0);
            }
            mbar_arrive_expect_tx(&landed[st], __popc(mask) * rows_of * (C::MX ? D + D / 32 : 2 * D) + (tile == p.hold ? 16 : 0));
          }
          __syncwarp();
          if (id >= 0) {
            const int row = (int)(((long long)id * p.a.Hkv + it.hk) << p.page_log2) + (t0 & (p.page_size - 1));
            const CUtensorMap* map = is_v ? &vmap : &kmap;
            if (C::MX) {
              uint8_t* dst = raws + st * C::RAW;
              tma_load_2d(dst + lane * rows_of * D, map, 0, row, &landed[st]);
              bulk_load(dst + kStepTok * D + lane * rows_of * (D / 32), (is_v ? p.v_s : p.k_s) + (long long)row * (D / 32),
                        rows_of * (D / 32), &landed[st]);
            } else {
              uint8_t* dst = ring + st * C::TILE;
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_2d(dst + h * kStepTok * 128 + lane * rows_of * 128, map, h * 64, row, &landed[st]);
            }
          }
          ++tile;
        }
        steps += cnt;
      }
      // copies in flight end before the block does, whoever gives up and when
      for (int j = max(0, tile - (C::MX ? C::RAWS : C::ENTRIES)); j < tile; ++j)
        mbar_wait(&landed[j % (C::MX ? C::RAWS : C::ENTRIES)], (j / (C::MX ? C::RAWS : C::ENTRIES)) & 1, kPagedWaitNs,
                  nullptr, nullptr, DEV_TIMEOUT_DRAIN);
    } else if (warp == 9) {
      // ---------------- products ----------------
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const bool leader = elect_one();
      const uint32_t idesc_qk = idesc_bf16_f32(kRowsM, kStepTok);
      const uint32_t idesc_pv = idesc_bf16_f32(kRowsM, D) | (1u << 16);
      const uint64_t qdesc = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t kdesc = smem_desc(smem_u32(ring), 16, 1024, 2);
      const uint64_t vdesc = smem_desc(smem_u32(ring), kStepTok * 128, 1024, 2);
      int tile = 0, qs = 0, done[2] = {0, 0};   // tiles, queries and steps of the chains so far
      auto have = [&]() { return wait(&ready[tile % C::ENTRIES], (tile / C::ENTRIES) & 1, DEV_TIMEOUT_FULL); };
      auto qk = [&](int x) {
        if (leader) {
          const uint64_t kx = kdesc + (tile % C::ENTRIES) * (C::TILE >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const int at = ((ks / 4) * kStepTok * 128 + (ks % 4) * 32) >> 4;
            mma_bf16(tm + (x ? C::S1 : C::S0), qdesc + at, kx + at, idesc_qk, ks > 0);
          }
          tc_commit(&s_full[x]);
          tc_commit(&ent_empty[tile % C::ENT_BARS]);
        }
        __syncwarp();
        ++tile;
      };
      auto pv = [&](int x, int h, bool more) {
        if (leader) {
          const uint32_t d = tm + (x ? C::O1 : C::O0), a = tm + (x ? C::S1 : C::S0);
          const uint64_t vx = vdesc + (tile % C::ENTRIES) * (C::TILE >> 4);
#pragma unroll
          for (int k4 = 0; k4 < kStepTok / 32; ++k4) {
            const int ks = h * kStepTok / 32 + k4;
            mma_bf16_ts(d, a + ks * 8, vx + ks * (2048 >> 4), idesc_pv, more || k4 > 0);
          }
        }
        __syncwarp();
      };
      bool ok = true;
      for (int n = 0; ok && item_there(n); ++n) {
        const int cnt = items[n & 1].cnt;
        item_done(n);
        if (cnt == 0) continue;
        if (!(ok = wait(&q_full, qs & 1, DEV_TIMEOUT_FULL))) break;
        ++qs;
        tc_fence_after();
        for (int x = 0; ok && x < min(cnt, 2); ++x) {
          if (!(ok = have())) break;
          tc_fence_after();
          qk(x);
        }
        if (cnt <= 2 && leader) tc_commit(&q_empty);
        for (int i = 0; ok && i < cnt; ++i) {
          const int x = i & 1, k = x ? done[1] : done[0];
          if (!(ok = have() && wait(&p_full[x][0], k & 1, DEV_TIMEOUT_ACCUM))) break;
          tc_fence_after();
          pv(x, 0, i > 1);
          if (!(ok = wait(&p_full[x][1], k & 1, DEV_TIMEOUT_ACCUM))) break;
          tc_fence_after();
          pv(x, 1, true);
          if (leader) {
            tc_commit(&ent_empty[tile % C::ENT_BARS]);
            tc_commit(&o_full[x]);
          }
          __syncwarp();
          ++tile;
          if (x) ++done[1]; else ++done[0];
          if (i + 2 < cnt) {
            if (!(ok = have())) break;
            tc_fence_after();
            qk(x);
            if (i + 3 == cnt && leader) tc_commit(&q_empty);
          }
        }
      }
      if (leader) {                             // and so do the products
        tc_commit(&drain);
        mbar_wait(&drain, 0, kPagedWaitNs, nullptr, nullptr, DEV_TIMEOUT_DRAIN);
      }
    } else if (warp == 10) {
      // ---------------- queries ----------------
      // Into the layout of a swizzled TMA tile. Rows beyond R keep what was there: a row of the products depends on its own
      // query alone, and the softmax asks live rows alone.
      int qs = 0;
      bool ok = true;
      for (int n = 0; ok && item_there(n); ++n) {
        const PagedItem& it = items[n & 1];
        if (it.cnt > 0) {
          if (qs > 0 && !(ok = wait(&q_empty, (qs - 1) & 1, DEV_TIMEOUT_EMPTY))) break;
          ++qs;
          const int G = p.G;
          // a scale below zero turns the queries' sign instead
          const uint32_t turn = p.a.scale < 0.f ? 0x80008000u : 0u;
          const uint16_t* q = p.q + (long long)it.b * p.rows * p.q_stride + (long long)it.hk * G * D;
          constexpr int CH = D / 8, RPW = 32 / CH;  // chunks of 16 bytes of a row, rows at a time
          const int ch = lane % CH, live = it.live;
          int r = (it.rho0 + lane / CH) / G, h = it.rho0 + lane / CH - r * G;
          uint8_t* dst = smem + (ch >> 3) * kRowsM * 128;
#pragma unroll 2
          for (int row = lane / CH; row < live; row += RPW) {
            cp_async_16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4), q + r * p.q_stride + h * D + ch * 8, 16);
            h += RPW;
            while (h >= G) h -= G, ++r;
          }
          cp_async_wait_all();
          if (turn) {
            for (int row = lane / CH; row < live; row += RPW) {
              uint4* v = reinterpret_cast<uint4*>(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
              *v = make_uint4(v->x ^ turn, v->y ^ turn, v->z ^ turn, v->w ^ turn);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full);
        }
        item_done(n);
      }
    } else if (C::MX ? warp >= 12 : warp == 11) {
      // ---------------- feeding ----------------
      // Hands every tile to the products, MXFP8 converted. In steps where some row does not see a key, values that are not
      // finite become zero (a weight of zero would not hide them), and the keys that some row sees are listed, for the rows
      // that do see them.
      const int tid = C::MX ? threadIdx.x % 128 : lane, group = C::MX ? warp / 4 - 3 : 0;
      const uint32_t k16 = sixteen();
      int tile = 0, steps = 0;
      bool ok = true;
      for (int n = 0; ok && item_there(n); ++n) {
        const int cnt = items[n & 1].cnt, pmax = items[n & 1].pmax, first_any = items[n & 1].first_any;
        auto list = [&](int tok) {
          if (tok <= pmax && (tok >= first_any || tok < p.a.sinks)) bad[n & 1].add(tok);
        };
        auto feed = [&](int i, bool is_v) {
          const int e = tile % C::ENTRIES, st = C::MX ? tile % C::RAWS : e;
          if (tile % C::GROUPS != group) {      // the other group's
            ++tile;
            return;
          }
          if (!(ok = wait(&landed[st], (tile / (C::MX ? C::RAWS : C::ENTRIES)) & 1, DEV_TIMEOUT_FULL))) return;
          const int4 info = infos[(steps + i) % kInfos];
          const bool edge = is_v && info.z == kEdge;
          uint8_t* dst = ring + e * C::TILE;
          if (C::MX) {
            if (!(ok = ent_free(tile))) return;
            const uint8_t* src = raws + st * C::RAW;
            constexpr int CH = D / 16, RPT = 128 / CH;          // 16 codes at a time; rows of the tile a pass covers
            const int ch = tid % CH, row0 = tid / CH;
            // half of the lanes take their second 8 codes first: the lanes of a load, and of a store, are then in different banks
            const uint32_t flip = ((lane >> 3) ^ (D == 128 ? ch >> 2 : 0)) & 1;
            // a thread's rows are RPT apart, a multiple of 8: their chunks are turned alike
            const uint32_t from = smem_u32(src) + row0 * D + ch * 16 + flip * 8;
            const uint32_t sc = smem_u32(src) + kStepTok * D + row0 * (D / 32) + ch / 2;
            const uint32_t to = smem_u32(dst) + (ch >> 2) * kStepTok * 128 + row0 * 128 +
                                ((((2 * ch + flip) & 7) ^ (row0 & 7)) << 4);
            static_assert(RPT % 8 == 0, "turned alike");
            uint32_t top = 0;
#pragma unroll 1
            for (int r = 0; r < kStepTok; r += 4 * RPT) {
              uint32_t w[4][4], by[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[j][0]), "=r"(w[j][1]) : "r"(from + (r + j * RPT) * D));
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                             : "=r"(w[j][2]), "=r"(w[j][3]) : "r"((from ^ 8) + (r + j * RPT) * D));
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(by[j]) : "r"(sc + (r + j * RPT) * (D / 32)));
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                top = max(top, by[j]);
                const uint32_t f = ((by[j] + 120u) << 7) * 0x10001u;
                uint32_t o[8];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  o[2 * b] = mul_bf16x2(e4m3_pair(w[j][b], w[j][b], kCodes01, k16), f);
                  o[2 * b + 1] = mul_bf16x2(e4m3_pair(w[j][b], w[j][b], kCodes23, k16), f);
                }
                const uint32_t at = to + (r + j * RPT) * 128;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
              }
            }
            // Scales past what one factor holds (values from 57,344 on, and NaN): those chunks once more, in two factors. A
            // value is not finite only there.
            if (__any_sync(0xffffffffu, top > kScaleFits)) {
#pragma unroll 1
              for (int r = 0; r < kStepTok; r += RPT) {
                const int row = row0 + r;
                const uint32_t by = src[kStepTok * D + row * (D / 32) + ch / 2];
                if (by <= kScaleFits) continue;
                if (!((info.y >> (row >> min(p.page_log2, 7))) & 1)) {       // of a page that was not loaded: whatever was here
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + r * 128), "r"(0) : "memory");
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"((to + r * 128) ^ 16), "r"(0) : "memory");
                  continue;
                }
                const uint32_t f = scale_bits(by) * 0x10001u, f2 = scale_rest(by) * 0x10001u;
                bool bad = false;
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                  const uint32_t w = *reinterpret_cast<const uint32_t*>(src + row * D + ch * 16 + (b / 2 ^ flip * 2) * 4);
                  uint32_t o = mul_bf16x2(mul_bf16x2(e4m3_pair(w, w, b & 1 ? kCodes23 : kCodes01, k16), f), f2);
                  const uint32_t hit = ((o & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                  if (edge) {
                    bad = bad || hit;
                    o &= ~((hit >> 15) * 0xFFFFu);
                  }
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(((to + r * 128) ^ (b / 4 * 16)) + b % 4 * 4), "r"(o) : "memory");
                }
                if (bad) list(info.x + row);
              }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[st]);
          } else if (is_v && info.z != kSeen) {
            uint4* v = reinterpret_cast<uint4*>(dst);
            // places of pages that were not loaded hold whatever was here
            const int rows_of = min(p.page_size, kStepTok);
            uint32_t gone = ~(uint32_t)info.y & ((2u << (kStepTok / rows_of - 1)) - 1u);
            if (gone) {
              for (; gone; gone &= gone - 1) {
                const int row = (__ffs(gone) - 1) * rows_of;
                for (int h = 0; h < C::HALVES; ++h)
                  for (int a = lane; a < rows_of * 8; a += 32) v[(h * kStepTok + row) * 8 + a] = make_uint4(0, 0, 0, 0);
              }
              fence_async_smem();
              __syncwarp();
            }
            // zero times a value that is not finite is NaN, and stays in the sum
            uint32_t sum = 0;
#pragma unroll 8
            for (int a = edge ? lane : C::TILE / 16; a < C::TILE / 16; a += 32) {
              const uint4 w = v[a];
              sum = fma_bf16x2(w.x, 0, sum);
              sum = fma_bf16x2(w.y, 0, sum);
              sum = fma_bf16x2(w.z, 0, sum);
              sum = fma_bf16x2(w.w, 0, sum);
            }
            if (__any_sync(0xffffffffu, (sum & 0x7FFF7FFFu) != 0)) {
#pragma unroll 1
              for (int a = lane; a < C::TILE / 16; a += 32) {
                const uint4 w = v[a];
                uint32_t z[4] = {w.x, w.y, w.z, w.w};
                bool bad = false;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const uint32_t hit = ((z[b] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                  bad = bad || hit;
                  z[b] &= ~((hit >> 15) * 0xFFFFu);
                }
                // 8 neighbouring lanes hold one key's 64 values: one of them lists it
                const unsigned hits = __ballot_sync(0xffffffffu, bad) & (0xFFu << (lane & 24));
                if (bad) {
                  v[a] = make_uint4(z[0], z[1], z[2], z[3]);
                  if (__ffs(hits) - 1 == lane) list(info.x + a / 8 % kStepTok);
                }
              }
              fence_async_smem();
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&ready[e]);
          ++tile;
        };
        // one call for all: K0 K1 V0 K2 V1 ... are the turns 0 1 2 3 4 ...; the last but one turn has no K
        for (int t = 0; ok && t < 2 * cnt + 2; ++t) {
          const bool is_v = t >= 2 && !(t & 1);
          const int i = t < 2 ? t : is_v ? (t - 2) / 2 : (t + 1) / 2;
          if (i < cnt) feed(i, is_v);
        }
        steps += cnt;
        item_done(n);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MORE));
    // ---------------- softmax ----------------
    const int x = warp / 4, row = threadIdx.x % 128;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + (x ? C::S1 : C::S0) + lanes, to = tmem + (x ? C::O1 : C::O0) + lanes;
    // scores in units of log2 e / scale; a scale of zero becomes one that tells none apart
    const float c = fmaxf(fabsf(p.a.scale) * 1.4426950408889634f, 1e-37f);
    const uint64_t c2 = pack2(c, c);
    const int G = p.G;
    int done = 0, steps = 0;                    // steps of this chain, and of all, so far
    bool ok = true;
    for (int n = 0; ok && item_there(n); ++n) {
      const int cnt = items[n & 1].cnt;
      const bool live = row < items[n & 1].live, warp_live = __any_sync(0xffffffffu, live);
      const int pos = live ? items[n & 1].pos0 + (items[n & 1].rho0 + row) / G : -1;
      const int first = (p.a.window && pos >= p.a.window) ? pos + 1 - p.a.window : 0;
      float m = -INFINITY;                      // the maximum that the weights so far refer to
      uint64_t l2 = pack2(0.f, 0.f);
      bool any = false;                         // a step of this chain
      for (int i = x; i < cnt; i += 2, ++done) {
        if (!(ok = wait(&s_full[x], done & 1, DEV_TIMEOUT_ACCUM))) break;
        tc_fence_after();
        if (!warp_live) {                       // rows that nobody has: their weights may be anything
          mbar_arrive(&p_full[x][0]);
          mbar_arrive(&p_full[x][1]);
          any = true;
          continue;
        }
        const int4 info = infos[(steps + i) % kInfos];
        if (info.z) {
          // Hidden in Tensor Memory, 32 scores at a time: little code, and groups that all of the warp's rows see are left.
          // The row sees token info.x + e when e <= hi and (e >= lo or e < low), and its page is there.
          const int hi = pos - info.x, lo = first - info.x, low = p.a.sinks - info.x;
          const uint32_t pages = (uint32_t)info.y;
          auto below = [](int k) { return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u; };
#pragma unroll 1
          for (int e = 0; e < kStepTok; e += 32) {
            uint32_t see = below(hi + 1 - e) & (~below(lo - e) | below(low - e));
            for (int d = 0; d < 32; d += 8)     // a page has at least 8 tokens
              if (!((pages >> ((e + d) >> min(p.page_log2, 7))) & 1u)) see &= ~(0xFFu << d);
            if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
            uint32_t s[32];
            tmem_ld32(ts + e, s, 0);
            tmem_ld_wait();
            reg_fence32(s, 0);
#pragma unroll
            for (int d = 0; d < 32; ++d) s[d] = (see >> d) & 1u ? s[d] : 0xff800000u;
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
        const float mn = max3(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]), m);
        // (-inf) - (-inf): no. Rows that nobody has hold an earlier kernel's leftovers and have no say: where the others' maximum
        // moves decides how their weights round.
        if (__any_sync(0xffffffffu, live && (mn - m) * c > kGrow)) {
          if (any) {
            if (!(ok = wait(&o_full[x], (done - 1) & 1, DEV_TIMEOUT_ACCUM))) break;
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
        }
        any = true;
        const float base = m == -INFINITY ? 0.f : -m * c;
        const uint64_t b2 = pack2(base, base);
        uint64_t la = pack2(0.f, 0.f), lb = la;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 64 * h; e < 64 * h + 64; e += 4) {
            float w[4];
            unpack2(fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, b2), w[0], w[1]);
            unpack2(fma2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, b2), w[2], w[3]);
#pragma unroll
            for (int f = 0; f < 4; ++f) w[f] = ex2(w[f]);
            la = add2(la, pack2(w[0], w[1]));
            lb = add2(lb, pack2(w[2], w[3]));
            s[e / 2] = bf16x2(w[0], w[1]);      // s[e / 2] has been read
            s[e / 2 + 1] = bf16x2(w[2], w[3]);
          }
          tmem_st32(ts + 32 * h, s, 32 * h);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[x][h]);
        }
        if (info.z) {
          // A row that sees few keys has them in such steps: there the sum takes the weights as the product does, rounded,
          // so that a single large one divides out exactly. Over many keys the roundings even out.
          la = lb = pack2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            la = add2(la, pack2(bf16_lo(s[e]), bf16_hi(s[e])));
            lb = add2(lb, pack2(bf16_lo(s[e + 1]), bf16_hi(s[e + 1])));
          }
        }
        l2 = add2(l2, add2(la, lb));
      }
      if (ok && any) {
        ok = wait(&o_full[x], (done - 1) & 1, DEV_TIMEOUT_ACCUM);
        tc_fence_after();
      }
      steps += cnt;
      float la, lb;
      unpack2(l2, la, lb);
      const float l = la + lb, top = m == -INFINITY ? -INFINITY : m * c;

      // ---- the chains joined: both have the same rows in the same lanes, and each takes half of the columns ----
      sums[x][row] = make_float2(any ? top : -INFINITY, any ? l : 0.f);
      tc_fence_before();
      mbar_arrive(&sums_there);
      ok = wait(&sums_there, n & 1, DEV_TIMEOUT_ACCUM) && ok;
      tc_fence_after();
      const PagedItem& it = items[n & 1];
      const int rho = it.rho0 + row, r = rho / G;
      const float2 s0 = sums[0][row], s1 = sums[1][row];
      const float both = fmaxf(s0.x, s1.x), base = both == -INFINITY ? 0.f : both;
      const float f0 = ex2(s0.x - base), f1 = ex2(s1.x - base), tl = f0 * s0.y + f1 * s1.y;
      const int e0 = x * (D / 2);
      uint32_t a[D / 2], b[D / 2];
#pragma unroll
      for (int e = 0; e < D / 2; e += 32) {
        tmem_ld32(tmem + C::O0 + lanes + e0 + e, a, e);
        tmem_ld32(tmem + C::O1 + lanes + e0 + e, b, e);
      }
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < D / 2; e += 32) {
        reg_fence32(a, e);
        reg_fence32(b, e);
      }
      tc_fence_before();
      mbar_arrive(&outs_read);                  // the next item's products may write there
      if (ok && live) {
        const bool one = it.pieces == 1;
        const float inv = !one ? 1.f : tl == 0.f ? no_weights(p, it.b, pos) : 1.f / tl;
        const float g0 = f0 * inv, g1 = f1 * inv;
        // a chain without steps has no output: what is there is nobody's
        if (cnt < 2) {
#pragma unroll
          for (int d = 0; d < D / 2; ++d) b[d] = 0;
        }
        if (cnt < 1) {
#pragma unroll
          for (int d = 0; d < D / 2; ++d) a[d] = 0;
        }
#pragma unroll
        for (int d = 0; d < D / 2; d += 2) {
          const uint64_t sum = fma2(pack2(__uint_as_float(b[d]), __uint_as_float(b[d + 1])), pack2(g1, g1),
                                    mul2(pack2(__uint_as_float(a[d]), __uint_as_float(a[d + 1])), pack2(g0, g0)));
          float lo, hi;
          unpack2(sum, lo, hi);
          a[d] = __float_as_uint(lo), a[d + 1] = __float_as_uint(hi);
        }
        if (one) {
          uint16_t* out = p.out + (((long long)it.b * p.rows + r) * p.a.Hq + it.hk * G + rho - r * G) * D + e0;
#pragma unroll
          for (int d = 0; d < D / 2; d += 8) {
            uint32_t w[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) w[f] = bf16x2(__uint_as_float(a[d + 2 * f]), __uint_as_float(a[d + 2 * f + 1]));
            *reinterpret_cast<uint4*>(out + d) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          const long long at = ((long long)it.b * p.a.Hkv + it.hk) * p.max_pieces + it.piece;
          float* part = part_of(p, at, D, rho, e0 / 4);
          const long long next = (long long)p.rows * G * 4;
#pragma unroll
          for (int d = 0; d < D / 2; d += 4)
            *reinterpret_cast<uint4*>(part + d / 4 * next) = make_uint4(a[d], a[d + 1], a[d + 2], a[d + 3]);
          if (x == 0) *sums_of(p, at, rho) = make_float2(both, tl);
        }
      }
      // ---- rows that see a listed key: each chain's warps their half of the columns ----
      if (ok && cnt > 0) {
        if (*reinterpret_cast<volatile int*>(&bad[n & 1].some)) {
          bool again = false;
          const Visible see(live ? pos : -1, p.a.window, p.a.sinks);
          bad[n & 1].each([&](int j) { again = again || see.sees(j); });
          again = again && live && tl == tl;    // a score that is NaN makes the sum NaN, and with it the row
          __syncwarp();                         // what a lane has written another one adds to
          for (unsigned rows = __ballot_sync(0xffffffffu, again); rows; rows &= rows - 1)
            finish_part<D, C::MX>(p, bad[n & 1], it, rho - lane + __ffs(rows) - 1, x);
        }
      }
      ok = wait(&outs_read, n & 1, DEV_TIMEOUT_ACCUM) && ok;
      tc_fence_after();
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

template <int D, bool MX>
static int launch_tc(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st) {
  using C = TcCfg<D, MX>;
  CUtensorMap km, vm;
  const int box = std::min(cache->page_size, kStepTok);
  const CUtensorMapSwizzle swizzle = MX ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  int rc = page_map(&km, cache->k, cache, box, swizzle);
  if (rc || (rc = page_map(&vm, cache->v, cache, box, swizzle))) return rc;
  auto kern = paged_tc_kernel<C>;
  if ((rc = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::SMEM))) return rc;
  const long long items = (long long)p.a.B * p.mblocks * p.a.Hkv * p.max_pieces;
  return launch_pdl(kern, dim3((unsigned)std::min(items, (long long)num_sms())), dim3(C::THREADS), C::SMEM, st, km, vm, p);
}

int launch_paged_tc(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st) {
  const bool mx = cache->format == MOE_KV_MXFP8;
  if (p.a.D == 64) return mx ? launch_tc<64, true>(p, cache, st) : launch_tc<64, false>(p, cache, st);
  return mx ? launch_tc<128, true>(p, cache, st) : launch_tc<128, false>(p, cache, st);
}

}  // namespace moe
