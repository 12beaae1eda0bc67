// What the two kernels of the paged attention share: their arguments, a sequence's pieces, and MXFP8 in bf16.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "gemm.cuh"
#include "ptx.cuh"

namespace moe {

constexpr uint64_t kPagedWaitNs = 1000000000ull;

struct PagedArgs {
  moe_attention a;
  int pages, page_size, page_log2;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_s;
  const uint8_t* v_s;
  int rows, max_len, table_width;
  int G, R;                  // heads of a group; rows (row, head of the group) of a sequence and kv head
  int tile_log2, block_log2; // tokens of a step; rows of a block
  int mblocks, max_pieces;
  const uint16_t* q;
  long long q_stride;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* out;
  uint32_t* status;
  int hold;                             // see held_load
  // Partial results of pieces. Rows are next to each other, because threads of a warp have rows of their own where they are
  // written and where they are joined.
  float* part_o;    // [B, Hkv, max_pieces, D / 4, R, 4]: sums of weighted values
  float* part_ml;   // [B, Hkv, max_pieces, R, 2]: running maximum (times log2 e) and sum
};

// Four columns of row rho's sums, and its maximum and sum, in piece `at` (of all).
__device__ __forceinline__ float* part_of(const PagedArgs& p, long long at, int D, int rho, int d4) {
  return p.part_o + ((at * (D / 4) + d4) * p.R + rho) * 4;
}
__device__ __forceinline__ float2* sums_of(const PagedArgs& p, long long at, int rho) {
  return reinterpret_cast<float2*>(p.part_ml) + at * p.R + rho;
}

// Pieces of equal length, to a step. Steps of 64 tokens (few rows, two blocks a multiprocessor): about 8 a piece, and at most
// 64 pieces. Steps of 128 (one block a multiprocessor): about 4, 8 from 8192 tokens on, and at most 32 pieces. Shorter pieces
// help the smallest batch and cost a large one, whose cache is read apace anyway: 1400 tokens, 64 heads over 8 of 128 bf16
// elements take 11 us for one sequence and 240 us for 256 in pieces of 8 steps, 19 us and 215 us in one piece; four rows of
// 1024 tokens take 13 us and 257 us in pieces of 4 steps of 128, 17 us and 198 us in one of 8. The small call counts here.
__host__ __device__ inline int piece_count(int tile_log2, int tiles) {
  const int log2 = tile_log2 == 6 || tiles >= 64 ? 3 : 2;      // of the steps
  return min(max((tiles + (1 << log2 >> 1)) >> log2, 1), tile_log2 == 6 ? 64 : 32);
}

// What the rows of block mb of a sequence see, as steps, and its pieces. The pieces follow from the sequence's own length
// alone: a row's result is the same in every batch.
struct Pieces {
  int pos0, pmin, pmax;  // positions of the sequence's first new row, of the block's first and last row
  int first_any, first_all;
  int sink_tiles, win_tile, tiles;
  int count, per, longer;    // pieces; steps of each, and how many have one more (the first ones)
  Pieces() = default;
  __device__ __forceinline__ Pieces(const PagedArgs& p, int len, int mb) {
    pos0 = len - p.rows;
    pmin = pos0, pmax = len - 1;
    if (p.mblocks > 1) {
      pmin = pos0 + (mb << p.block_log2) / p.G;
      pmax = pos0 + (min(p.R, (mb + 1) << p.block_log2) - 1) / p.G;
    }
    if (len == 0) pmax = -1;
    first_any = (p.a.window && pmin >= p.a.window) ? pmin + 1 - p.a.window : 0;
    first_all = (p.a.window && pmax >= p.a.window) ? pmax + 1 - p.a.window : 0;
    const int up = (1 << p.tile_log2) - 1;
    sink_tiles = (min(p.a.sinks, first_all) + up) >> p.tile_log2;
    win_tile = max(first_any >> p.tile_log2, sink_tiles);
    tiles = pmax < 0 ? 0 : sink_tiles + ((pmax + up + 1) >> p.tile_log2) - win_tile;
    count = piece_count(p.tile_log2, tiles);
    per = count == 1 ? tiles : (int)((unsigned)tiles / (unsigned)count);
    longer = tiles - per * count;
  }
  __device__ __forceinline__ int begin(int piece) const { return piece * per + min(piece, longer); }
  __device__ __forceinline__ int steps(int piece) const { return per + (piece < longer); }
};

__device__ __forceinline__ int checked_len(const PagedArgs& p, long long b, bool report) {
  const int len = p.lens[b];
  if (len >= 0 && len <= p.max_len) return len;
  if (report) atomicCAS(p.status, 0u, (uint32_t)DEV_BAD_INPUT);
  return 0;
}

// What a row without weights is: zero where it sees nothing. Where it does (its own key, in a page that there is), all scores
// were minus infinity, and 0 / 0 is NaN.
__device__ __forceinline__ float no_weights(const PagedArgs& p, long long b, int pos) {
  if (pos < 0) return 0.f;
  const int page = p.table[b * p.table_width + (pos >> p.page_log2)];
  return page >= 0 && page < p.pages ? __uint_as_float(0x7FC00000u) : 0.f;
}

// The items (sequence, block of rows, piece, head) that there are, numbered without gaps, so that blocks that take every
// grid-th of them differ by one at most. A warp goes along them, 32 blocks of rows at a time; numbers only go up.
struct ItemWalk {
  long long before = 0;  // items of the groups that have been passed
  int group = -32, total = 0;
  Pieces pc;                         // the lane's block of rows,
  int mine = 0, upto = 0;            // its items, these and those before
  // The lane that has item idx, or -1 if there are not as many.
  __device__ __forceinline__ int lane_of(const PagedArgs& p, long long idx) {
    const int lane = threadIdx.x % 32, units = p.a.B * p.mblocks;
    while (idx >= before + total) {
      before += total;
      total = 0;
      group += 32;
      if (group >= units) return -1;
      const int u = group + lane;
      mine = 0;
      if (u < units) {
        const int b = p.mblocks == 1 ? u : u / p.mblocks;
        pc = Pieces(p, checked_len(p, b, true), u - b * p.mblocks);
        mine = pc.count * p.a.Hkv;
      }
      upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int t = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += t;
      }
      total = __shfl_sync(0xffffffffu, upto, 31);
    }
    return __ffs(__ballot_sync(0xffffffffu, idx - before < upto)) - 1;
  }
};

// Two E4M3 codes as bf16 with their values times 2^-120: sign, exponent and fraction in bf16's places (subnormal codes
// become subnormals). `sel` takes, from the lowest byte on, a code, its sign (replicated), another code, its sign; four bits
// further up sign and code lie where bf16 has them. The shift is a product with a 16 that the compiler does not know
// (`sixteen()`): the pipe of the other instructions is the one that conversions are short of.
__device__ __forceinline__ uint32_t sixteen() {
  uint32_t r;
  asm volatile("mov.u32 %0, 16;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t a, uint32_t b, uint32_t sel, uint32_t k16) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return (r * k16) & 0x87F087F0u;
}
constexpr uint32_t kCodes01 = 0x9180, kCodes23 = 0xB3A2;   // codes 0 and 1 (2 and 3) of one word
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A scale byte's factor for e4m3_pair's values, 2^(120 + byte - 127), as bf16 bits: bytes up to 134 fit. What lies
// above (values past 57,344) takes a second factor; byte 255 is NaN.
constexpr uint32_t kScaleFits = 134;
__device__ __forceinline__ uint32_t scale_bits(uint32_t byte) { return (min(byte, kScaleFits) + 120u) << 7; }
__device__ __forceinline__ uint32_t scale_rest(uint32_t byte) {
  return byte == 255u ? 0x7FC0u : byte > kScaleFits ? (byte - kScaleFits + 127u) << 7 : 0x3F80u;
}

// Tensor map of the cache's rows [pages * Hkv * page_size, D], loaded `rows` at a time.
inline int page_map(CUtensorMap* m, const void* base, const moe_kv_cache* c, int rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return MOE_ERR_CUDA;
  const bool mx = c->format == MOE_KV_MXFP8;
  const cuuint64_t dims[2] = {(cuuint64_t)c->D, (cuuint64_t)c->pages * c->Hkv * c->page_size};
  const cuuint64_t stride[1] = {(cuuint64_t)c->D * (mx ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)(mx ? c->D : 64), (cuuint32_t)rows};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r = enc(m, mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void*>(base), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

// The kernel for many rows a block (attention_paged_tc.cu).
int launch_paged_tc(const PagedArgs& p, const moe_kv_cache* cache, cudaStream_t st);

}  // namespace moe
