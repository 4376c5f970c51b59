/*
 * fa_kv4_units.cuh -- how attention over the 4-bit cache is shared out: every
 * sequence's keys, times its heads and row tiles, are one line of 64-key chunks
 * (with some places more for each unit's fixed cost), cut into equal runs for
 * the blocks of the launch whatever the lengths are.  A unit (sequence, head,
 * row tile) that a cut divides leaves fp32 partials, which a second kernel
 * merges.  Everything follows from the lengths on the device.
 */
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>
#include <type_traits>

#include "../../include/fa_api.h"
#include "fa_kv4.cuh"
#include "fa_launch.cuh"

namespace fa {
namespace kv4 {

constexpr int kChunk = 64;          // keys of a unit of work
constexpr int kUnitCost = 6;        // chunks that a unit costs beside its own, for an even split
constexpr int kMinShare = kUnitCost + 1;   // least work of a block, in chunks: any run longer than
                                    // kUnitCost holds keys
constexpr int kMaxSms = 160;
constexpr float kBias = 8.0f;       // P is held as 2^(score - max + kBias): small
                                    // probabilities stay normal numbers of f16
constexpr float kLag = 6.0f;        // the maximum follows once a score passes it by
                                    // this much (log2): P <= 2^14 < 65504


struct AttnParams {
  Cache cache;
  const void* q;
  void* o;
  float* lse;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* block_table;
  float* part_o;          // [blocks, 2, rows, D]
  float* part_lse;        // [blocks, 2, rows]
  struct Meta* meta;      // [blocks]
  int64_t total_q, max_keys;
  float scale;            // |scale|
  int32_t n_seqs, max_pages, page_shift;   // page_shift: log2(page_size), or -1
  int32_t H, G, causal, negate;            // G = H / H_kv
};

// A unit that starts in this block's run and ends in a later block's.
struct Meta {
  int64_t q_row0;    // the sequence's first row of q
  int32_t pieces;    // 0: none
  int32_t head0;     // first query head of the group
  int32_t row0;      // first row (token * G + head) of the tile
  int32_t rows;      // rows of the tile that exist
};

// What turns a score of codes and scales into a power of two.
__device__ __forceinline__ float score_scale(const AttnParams& p) {
  return p.scale * descale_of(p.cache, 0) * 1.4426950408889634f;
}

struct Seq {
  int64_t q_row0;
  int32_t q_len, k_len;    // k_len: keys some row sees
  int32_t keys;            // keys held (the causal offset counts from here)
  int32_t tiles, chunks;   // row tiles; 64-key chunks (at least 1 where there are rows)
};

template <int ROWS>
__device__ __forceinline__ Seq sequence(const AttnParams& p, int s) {
  Seq q;
  const int64_t a = min(max(static_cast<int64_t>(p.cu_q[s]), int64_t(0)), p.total_q);
  const int64_t b = min(max(static_cast<int64_t>(p.cu_q[s + 1]), a), p.total_q);
  q.q_row0 = a;
  q.q_len = static_cast<int32_t>(b - a);
  q.keys = static_cast<int32_t>(min(max(static_cast<int64_t>(p.seqused_k[s]), int64_t(0)), p.max_keys));
  q.k_len = q.keys;
  if (p.causal == FA_CAUSAL_TOP_LEFT) q.k_len = min(q.k_len, q.q_len);
  q.tiles = static_cast<int32_t>((static_cast<int64_t>(q.q_len) * p.G + ROWS - 1) / ROWS);
  q.chunks = q.q_len > 0 ? max(1, (q.k_len + kChunk - 1) / kChunk) : 0;
  return q;
}

// A sequence's work, in chunks: its units' keys and their fixed costs.
__device__ __forceinline__ int64_t work_of(const AttnParams& p, const Seq& q) {
  return q.chunks > 0 ? static_cast<int64_t>(p.cache.H_kv) * q.tiles * (q.chunks + kUnitCost) : 0;
}

// One unit of work: a run of chunks of one (sequence, head, row tile).
struct Unit {
  int64_t q_row0;                   // the sequence's first row of q
  int32_t s, head, row0, rows;      // row0: first row (token * G + head) of the tile
  int32_t key_begin, key_end;
  int32_t keys, q_len, k_len;       // of the sequence, see Seq
  int32_t piece;                    // -1: the whole (sequence, head, tile); else the partial's slot
  int32_t pieces;                   // of a divided one that starts here, else 0
  int32_t more;                     // another unit of this block follows
};

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {   // both >= 0
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// An even split of the work: the first `extra` blocks have share + 1 places.
struct Split {
  int64_t share, extra;
  __device__ __forceinline__ int64_t start(int64_t block) const { return share * block + min(block, extra); }
  __device__ __forceinline__ int64_t block_of(int64_t place) const {
    const int64_t edge = extra * (share + 1);
    return place < edge ? divide(place, share + 1) : extra + divide(place - edge, share);
  }
};

// Where a block is in its run of chunks.
struct Cursor {
  int64_t w, w1, off;       // next place, end; offset in the sequence
  Split split;
  int32_t s;
  Seq sq;
};

// The cursor's next unit (moving on to the sequence that has it).
template <int ROWS>
static __device__ __noinline__ void next_unit(const AttnParams& p, Cursor& c, Unit& u) {
  int64_t all = work_of(p, c.sq);
  while (c.off >= all) {
    c.off -= all;
    c.sq = sequence<ROWS>(p, ++c.s);
    all = work_of(p, c.sq);
  }
  const Seq& sq = c.sq;
  // A unit is kUnitCost places without keys and then its chunks; this block's
  // run covers its places [pos, end).
  const int size = sq.chunks + kUnitCost;
  const int64_t unit = divide(c.off, size);
  const int pos = static_cast<int>(c.off - unit * size);
  const int end = static_cast<int>(min(static_cast<int64_t>(size), pos + (c.w1 - c.w)));
  const int c0 = max(pos - kUnitCost, 0), c1 = end - kUnitCost;
  u.q_row0 = sq.q_row0;
  u.s = c.s;
  u.head = static_cast<int>(divide(unit, sq.tiles));
  u.row0 = static_cast<int>(unit - static_cast<int64_t>(u.head) * sq.tiles) * ROWS;
  u.rows = static_cast<int>(min(static_cast<int64_t>(ROWS), static_cast<int64_t>(sq.q_len) * p.G - u.row0));
  u.key_begin = c0 * kChunk;
  u.key_end = min(c1 * kChunk, sq.k_len);
  u.keys = sq.keys;
  u.q_len = sq.q_len;
  u.k_len = sq.k_len;
  // a block's first unit may continue one, its last may be continued
  u.piece = c0 > 0 ? 0 : c1 < sq.chunks ? 1 : -1;
  u.pieces = 0;
  if (u.piece == 1)   // up to the block that holds the unit's last chunk
    u.pieces = static_cast<int32_t>(c.split.block_of(c.w - pos + size - 1) - blockIdx.x + 1);
  c.w += end - pos;
  c.off += end - pos;
  u.more = c.w1 - c.w > kUnitCost;    // (what is left begins with a unit: has it keys?)
}

// The block's run of the work and the sequence it starts in, and its first two
// units; false where there is no work for it.  For a block of THREADS; scan:
// shared, THREADS / 32 entries; factors: shared, score_scale and V's descale,
// written here so that their loads overlap those of the lengths.
template <int ROWS, int THREADS>
__device__ __forceinline__ bool begin_units(const AttnParams& p, int64_t* scan, Cursor& cursor, Unit* units, float* factors) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n_seqs + THREADS - 1) / THREADS;
  const int s0 = min(p.n_seqs, tid * per), s1 = min(p.n_seqs, s0 + per);
  int64_t mine = 0;
  const float factor[2] = {score_scale(p), descale_of(p.cache, 1)};
  Seq sq = {};
  for (int s = s0; s < s1; ++s) {
    sq = sequence<ROWS>(p, s);
    mine += work_of(p, sq);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += a;
  }
  if (lane == 31) scan[warp] = incl;
  if (tid < 2) factors[tid] = factor[tid];
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int64_t blocks = total == 0 ? 0 : min(static_cast<int64_t>(gridDim.x), max(divide(total, kMinShare), int64_t(1)));
  const int64_t bid = blockIdx.x;
  if (tid == 0) p.meta[bid].pieces = 0;
  if (bid >= blocks) return false;
  const int64_t share = divide(total, blocks);
  const Split split{share, total - share * blocks};
  const int64_t w = split.start(bid);
  if (w >= before && w < before + mine) {   // one thread has the sequence
    int64_t off = w - before;
    int s = s0;
    if (per > 1) {                          // (else sq is the one sequence already)
      for (;; ++s) {
        sq = sequence<ROWS>(p, s);
        const int64_t c = work_of(p, sq);
        if (off < c) break;
        off -= c;
      }
    }
    cursor = Cursor{w, split.start(bid + 1), off, split, s, sq};
    next_unit<ROWS>(p, cursor, units[0]);
    if (units[0].more) next_unit<ROWS>(p, cursor, units[1]);
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Merge of a divided unit's pieces:
//   lse = log sum exp(lse_i),  O = sum exp(lse_i - lse) O_i.
// The first piece is the starting block's second slot, the others the
// following blocks' first slots.  One block a unit; its warps share the rows,
// several on one row where there are few, each over every n-th piece.
constexpr int kMergeWarps = 16;

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_kv4_merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;              // elements a lane
  __shared__ float sum_o[kMergeWarps][D], sum_w[kMergeWarps];
  fa::wait_for_stream();
  fa::let_next_start();
  const Meta mt = p.meta[blockIdx.x];
  const float dv = descale_of(p.cache, 1);
  if (mt.pieces == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int share = 1;                         // warps a row
  while (2 * share * mt.rows <= kMergeWarps && share < 8) share *= 2;
  const int64_t first = blockIdx.x;
  for (int base = 0; base < mt.rows; base += kMergeWarps / share) {
    const int r = base + warp / share, part = warp % share;
    const bool in = r < mt.rows;
    auto at = [&](int i) { return ((first + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + r; };
    float top = -CUDART_INF_F, sum = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    if (in) {
      for (int i = lane; i < mt.pieces; i += 32) top = fmaxf(top, p.part_lse[at(i)]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 8
      for (int i = part; i < mt.pieces; i += share) {
        const int64_t a = at(i);
        const float lse = p.part_lse[a];
        const float wgt = lse == -CUDART_INF_F ? 0.0f : expf(lse - top);
        const float* src = p.part_o + a * D + lane * E;
        sum += wgt;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wgt * src[e];
      }
    }
    if (share > 1) {                     // the row's warps, in order
#pragma unroll
      for (int e = 0; e < E; ++e) sum_o[warp][lane * E + e] = acc[e];
      if (lane == 0) sum_w[warp] = sum;
      __syncthreads();
      if (part == 0 && in) {
        for (int k = 1; k < share; ++k) {
          sum += sum_w[warp + k];
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += sum_o[warp + k][lane * E + e];
        }
      }
    }
    if (in && part == 0) {
      const int row = mt.row0 + r, tok = row / p.G, h = mt.head0 + (row - tok * p.G);
      const float mul = sum == 0.0f ? 0.0f : dv / sum;
      uint16_t* dst = static_cast<uint16_t*>(p.o) + ((mt.q_row0 + tok) * p.H + h) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint32_t w;
        if (std::is_same<T, __half>::value) {
          w = pack_half(acc[e] * mul, acc[e + 1] * mul);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(acc[e] * mul, acc[e + 1] * mul);
          w = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint32_t*>(dst + e) = w;
      }
      if (lane == 0)
        p.lse[static_cast<int64_t>(h) * p.total_q + mt.q_row0 + tok] = sum == 0.0f ? -CUDART_INF_F : top + logf(sum);
    }
    // (share > 1 only where one pass takes all rows: the buffers are not reused)
  }
}

}  // namespace kv4
}  // namespace fa
