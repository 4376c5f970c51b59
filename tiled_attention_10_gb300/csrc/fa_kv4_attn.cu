/*
 * fa_kv4_attn.cu -- fa_fwd_paged_kv4: attention of packed queries over the
 * 4-bit paged cache (include/fa_api.h).  Two ways, by the rows (queries x
 * heads that share a key/value head) a sequence brings to each key:
 *
 * Few rows (decoding, speculative tokens): bound by HBM, 9/16 byte a cached
 * value.  At the measured 6.8 TB/s an SM receives 23 bytes a cycle, 41 values,
 * and each has to become a 16-bit operand: 3.1 lane instructions a value are
 * all the issue slots there are.  So codes go from shared memory to registers
 * and from there straight into the matrix product (mma.sync): tcgen05 takes
 * its operands from shared or tensor memory, and the unpacked values' trip
 * there (4 bytes written and read for each cached 9/16) would take longer than
 * HBM.  The products are oriented so that no value is moved between lanes:
 *     S^T [keys x rows] = K Q^T      K codes in A's place, 16 keys high
 *     O^T [D x rows]   += V^T P^T    V codes in A's place, 16 elements high
 * with 8 rows a tile (N).  The contraction's order is free: each lane takes
 * the 32 (16 at D = 64) consecutive dimensions it can load at once and Q is
 * loaded in the same order.  For V a byte has to hold two keys of one element,
 * not two elements of one key: two bit-selects over words of two keys.  P
 * changes from S^T's accumulator layout to an operand by one 8x8 transposition
 * (movmatrix) for 8 keys.
 *   codes -> f16: cvt e2m1x2 (exact), times the group's scale (exact: 2 x 4
 *   significant bits); bf16 queries become f16 exactly too, each row shifted
 *   by a power of two that its scale takes back.  P in f16 is the only
 *   rounding: 2^-12 of each probability; scores, sums and O are fp32.
 * Work: every sequence's keys, times its heads, are one line of 64-key chunks,
 * cut into equal runs for the resident blocks whatever the lengths are; a
 * (sequence, head) that a cut divides leaves fp32 partials that a second
 * kernel merges.  A block's warps take 32-key steps in turn, each with its own
 * cp.async ring and its own running maximum, and join at the run's end.
 *
 * Many rows (chunked prefill): bound by the matrix products.  The keys and
 * values are unpacked once into a 16-bit workspace (a few per cent of the
 * time) and the tcgen05 forward (fa_fwd_varlen) reads them there.
 */
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/fa_api.h"
#include "fa_kv4.cuh"

namespace {

using fa::kv4::Cache;
using fa::kv4::codes_to_half;
using fa::kv4::mul_half;
using fa::kv4::scales_to_half;

constexpr int kWarps = 4;           // warps of a block
constexpr int kStep = 32;           // keys of a warp's step
constexpr int kChunk = 64;          // keys of a unit of work
constexpr int kMinChunks = 4;       // least chunks worth a block of their own
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
  float sl2;              // |scale| * descale_k * log2(e)
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

__device__ __forceinline__ int64_t chunks_of(const AttnParams& p, const Seq& q) {
  return static_cast<int64_t>(p.cache.H_kv) * q.tiles * q.chunks;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t a0, const uint32_t a1, const uint32_t a2,
                                    const uint32_t a3, const uint32_t b0, const uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D>
struct Stage {
  static constexpr int kCodes = kStep * D / 2;       // bytes of K (or V) codes
  static constexpr int kScales = kStep * D / 16;
  static constexpr int kBytes = 2 * (kCodes + kScales);
  static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
  static constexpr int kChunksRow = D / 32;          // 16-byte pieces of a row of codes
};

// Place of V's row r (of a step) and 16-byte piece c in shared memory: a lane
// reads rows 2 t (t = lane % 4) at 8 g bytes (D = 128; 4 g at 64), g = lane / 4,
// and rows of one parity would share banks in the plain order.
template <int D>
__device__ __forceinline__ int v_place(int r, int c) {
  if (D == 128)
    return ((r & ~3) | ((r & 1) << 1) | ((r >> 1) & 1)) * 64 + ((c ^ (((r >> 2) & 1) << 1)) * 16);
  return ((r & ~7) | ((r & 1) << 2) | ((r >> 1) & 3)) * 32 + c * 16;
}

// The codes and scales of keys [key0, key0 + 32) into a ring stage; keys from
// `end` on, and pages outside the cache, become zeros.
template <int D>
__device__ __forceinline__ void load_step(const AttnParams& p, uint32_t stage, int head, int key0, int end,
                                          const int (&page)[2], int lane) {
  using St = Stage<D>;
  const int ps = p.cache.page_size;
  int64_t row[2];
  bool ok[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int key = key0 + 16 * h;
    const int in_page = p.page_shift >= 0 ? key & (ps - 1) : key % ps;
    ok[h] = page[h] >= 0 && page[h] < p.cache.num_pages;
    row[h] = (static_cast<int64_t>(ok[h] ? page[h] : 0) * p.cache.H_kv + head) * ps + (ok[h] ? in_page : 0);
  }
  constexpr int C = St::kChunksRow, kPer = kStep * C / 32;   // pieces a lane, of K and of V
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = lane + 32 * i, r = piece / C, c = piece % C;
    const int h = i * 2 / kPer;                              // the half that row r is in
    const int64_t at = (row[h] + (r & 15)) * (D / 2) + c * 16;
    const bool in = ok[h] && key0 + r < end;
    const int64_t from = in ? at : 0;
    copy16(stage + r * (D / 2) + c * 16, p.cache.codes[0] + from, in ? 16 : 0);
    copy16(stage + St::kV + v_place<D>(r, c), p.cache.codes[1] + from, in ? 16 : 0);
  }
  // scales: D / 16 bytes a key; 16-byte pieces hold 256 / D keys
  constexpr int KP = 256 / D, N = kStep / KP;                // keys a piece, pieces
  if (lane < 2 * N) {
    const int which = lane / N, piece = lane % N, r = piece * KP, h = r >> 4;
    const int keys = ok[h] ? min(max(end - key0 - r, 0), KP) : 0;
    const int64_t at = keys > 0 ? (row[h] + (r & 15)) * (D / 16) : 0;
    copy16(stage + (which ? St::kVs : St::kKs) + piece * 16, p.cache.scales[which] + at, keys * (D / 16));
  }
}

__device__ __forceinline__ int page_index(const AttnParams& p, int key) {
  return p.page_shift >= 0 ? key >> p.page_shift : key / p.cache.page_size;
}
__device__ __forceinline__ void look_up(const AttnParams& p, const int32_t* table, int key0, int end, int (&page)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int key = key0 + 16 * h;
    page[h] = key < end ? table[page_index(p, key)] : -1;
  }
}

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocks = NT == 1 ? 4 : NT == 2 ? 3 : 2;   // resident blocks an SM
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kRing = kStages * Stage<D>::kBytes;        // a warp's ring
  // at the end of a run a warp's O takes the place of its ring
  static constexpr int kWarpBytes = kRing > kRows * D * 4 ? kRing : kRows * D * 4;
  static constexpr int kSmem = kWarps * kWarpBytes;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, Cfg<D, NT>::kBlocks)
    fa_kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NT>;
  using St = Stage<D>;
  constexpr int kRows = C::kRows;
  constexpr int MT = D / 16;        // 16-element tiles of O^T
  constexpr int QW = D / 8;         // f16 pairs of Q a lane holds for a row
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float w_max[kWarps][kRows], w_sum[kWarps][kRows];
  __shared__ int64_t scan[kWarps], start_off;
  __shared__ int start_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  // ---- this block's run of chunks [w0, w1)
  const int per = (p.n_seqs + kWarps * 32 - 1) / (kWarps * 32);
  const int s0 = min(p.n_seqs, tid * per), s1 = min(p.n_seqs, s0 + per);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += chunks_of(p, sequence<kRows>(p, s));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += a;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), (total + kMinChunks - 1) / kMinChunks);
  const int64_t bid = blockIdx.x;
  if (tid == 0) p.meta[bid].pieces = 0;
  if (bid >= blocks) return;
  int64_t w = total * bid / blocks;
  const int64_t w1 = total * (bid + 1) / blocks;
  if (w >= before && w < before + mine) {
    int64_t off = w - before;
    int s = s0;
    for (;; ++s) {
      const int64_t c = chunks_of(p, sequence<kRows>(p, s));
      if (off < c) break;
      off -= c;
    }
    start_seq = s;
    start_off = off;
  }
  __syncthreads();
  int s = start_seq;
  int64_t off = start_off;

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kWarpBytes;
  uint8_t* const ring_p = smem + warp * C::kWarpBytes;
  float* const warp_o = reinterpret_cast<float*>(ring_p);

  while (w < w1) {
    const Seq sq = sequence<kRows>(p, s);
    const int64_t all = chunks_of(p, sq);
    if (off >= all) {                       // an empty sequence, or this one is done
      off -= all;
      ++s;
      continue;
    }
    const int64_t unit = off / sq.chunks;
    const int c0 = static_cast<int>(off - unit * sq.chunks);
    const int c1 = static_cast<int>(min(static_cast<int64_t>(sq.chunks), c0 + (w1 - w)));
    const int head = static_cast<int>(unit / sq.tiles);
    const int tile_row0 = static_cast<int>(unit - static_cast<int64_t>(head) * sq.tiles) * kRows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), static_cast<int64_t>(sq.q_len) * p.G - tile_row0));
    const int key_begin = c0 * kChunk, key_end = min(c1 * kChunk, sq.k_len);
    const int32_t* table = p.block_table + static_cast<int64_t>(s) * p.max_pages;

    // ---- start the ring
    const int step = kWarps * kStep;
    int next = key_begin + warp * kStep;     // first key of the next step to load
    int page[2];
    look_up(p, table, next, key_end, page);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (next < key_end) load_step<D>(p, ring + i * St::kBytes, head, next, key_end, page, lane);
      copies_commit();
      next += step;
      look_up(p, table, next, key_end, page);
    }

    // ---- Q: this lane's dimensions of row 8 j + g, and the rows' scales
    uint32_t q[NT][QW];
    float sl2[NT][2];
    int limit[NT][2];                       // keys that the lane's two rows see
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = 8 * j + g;
      float rescale = 1.0f;
      const int row = tile_row0 + r;
      const int tok = row / p.G;
      if (r < rows) {
        const int64_t at = ((sq.q_row0 + tok) * p.H + static_cast<int64_t>(head) * p.G + (row - tok * p.G)) * D + t * (D / 4);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at);
#pragma unroll
        for (int i = 0; i < QW / 4; ++i) {
          const uint4 v = src[i];
          q[j][4 * i] = v.x; q[j][4 * i + 1] = v.y; q[j][4 * i + 2] = v.z; q[j][4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < QW; ++i) q[j][i] = 0u;
      }
      if (!std::is_same<T, __half>::value) {
        // bf16: shift the row by a power of two so that its largest value is
        // in [2^8, 2^9) and convert: exact down to 2^-22 of the largest.
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < QW; ++i) top = max(top, max(q[j][i] & 0x7fffu, (q[j][i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max(static_cast<int>(top >> 7), 30), 254);   // biased exponent
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 + 127 - e) << 23);
        rescale = __uint_as_float(static_cast<uint32_t>(e - 8) << 23);
#pragma unroll
        for (int i = 0; i < QW; ++i)
          q[j][i] = pack_half(__uint_as_float(q[j][i] << 16) * up, __uint_as_float(q[j][i] & 0xffff0000u) * up);
      }
      if (p.negate) {
#pragma unroll
        for (int i = 0; i < QW; ++i) q[j][i] ^= 0x80008000u;
      }
      int see = sq.k_len;
      if (p.causal == FA_CAUSAL_TOP_LEFT) see = min(see, tok + 1);
      if (p.causal == FA_CAUSAL_BOTTOM_RIGHT) see = min(see, tok + 1 + sq.keys - sq.q_len);
      // the accumulators of this lane are rows 8 j + 2 t and 8 j + 2 t + 1
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sl2[j][c] = fmaxf(p.sl2 * __shfl_sync(0xffffffffu, rescale, (2 * t + c) * 4), 1e-30f);
        limit[j][c] = __shfl_sync(0xffffffffu, see, (2 * t + c) * 4);
      }
    }
    int full = limit[0][0];                  // keys that all rows of the tile see
#pragma unroll
    for (int j = 0; j < NT; ++j) full = min(full, min(limit[j][0], limit[j][1]));
    full = min(full, __shfl_xor_sync(0xffffffffu, full, 1));
    full = min(full, __shfl_xor_sync(0xffffffffu, full, 2));

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
      m[j][0] = m[j][1] = -CUDART_INF_F;
      l[j][0] = l[j][1] = 0.0f;
    }

    // ---- the steps
    int slot = 0;
    for (int key0 = key_begin + warp * kStep; key0 < key_end; key0 += step) {
      copies_wait<C::kStages - 2>();
      __syncwarp();
      const uint8_t* const st = ring_p + slot * St::kBytes;
      {
        const int into = slot == 0 ? C::kStages - 1 : slot - 1;   // the stage read one step ago
        if (next < key_end) load_step<D>(p, ring + into * St::kBytes, head, next, key_end, page, lane);
        copies_commit();
        next += step;
        look_up(p, table, next, key_end, page);
      }

      // S^T: two tiles of 16 keys
      float sc[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) sc[u][j][0] = sc[u][j][1] = sc[u][j][2] = sc[u][j][3] = 0.0f;
        uint32_t words[2][D / 32], s2[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * u + 8 * h + g;
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + r * 64 + t * 16);
            words[h][0] = v.x; words[h][1] = v.y; words[h][2 % (D / 32)] = v.z; words[h][3 % (D / 32)] = v.w;
            const uint32_t two = scales_to_half(*reinterpret_cast<const uint16_t*>(st + St::kKs + r * 8 + t * 2));
            s2[h][0] = __byte_perm(two, 0u, 0x1010);
            s2[h][1] = __byte_perm(two, 0u, 0x3232);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(st + r * 32 + t * 8);
            words[h][0] = v.x; words[h][1] = v.y;
            const uint32_t b = st[St::kKs + r * 4 + t];
            s2[h][0] = s2[h][1] = scales_to_half(b | (b << 8));
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {          // a word: 8 dimensions, two k16 steps
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_to_half(words[h][i], a[h]);
#pragma unroll
            for (int x = 0; x < 4; ++x) a[h][x] = mul_half(a[h][x], s2[h][i / 2]);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma(sc[u][j], a[0][2 * x], a[1][2 * x], a[0][2 * x + 1], a[1][2 * x + 1], q[j][4 * i + 2 * x], q[j][4 * i + 2 * x + 1]);
        }
      }

      // softmax of the step, P to operands
      const bool edge = key0 + kStep > min(full, key_end);
      uint32_t pb[NT][4];                            // 8 keys each
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (edge) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key0 + 16 * u + 8 * (x >> 1) + g;
              if (key >= limit[j][x & 1] || key >= key_end) sc[u][j][x] = -CUDART_INF_F;
            }
        }
        bool over = false;
        float top[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[c] = fmaxf(fmaxf(sc[0][j][c], sc[0][j][c + 2]), fmaxf(sc[1][j][c], sc[1][j][c + 2])) * sl2[j][c];
          over = over || top[c] > m[j][c] + kLag;
        }
        if (__any_sync(0xffffffffu, over)) {         // move the maximum
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = top[c];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            v = fmaxf(v, m[j][c]);
            const float a = v == -CUDART_INF_F ? 1.0f : exp2_approx(m[j][c] - v);
            m[j][c] = v;
            l[j][c] *= a;
#pragma unroll
            for (int i = 0; i < MT; ++i) { o[j][i][c] *= a; o[j][i][c + 2] *= a; }
          }
        }
        float sub[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) sub[c] = m[j][c] == -CUDART_INF_F ? 0.0f : kBias - m[j][c];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sc[u][j][x] = exp2_approx(fmaf(sc[u][j][x], sl2[j][x & 1], sub[x & 1]));
            l[j][x & 1] += sc[u][j][x];
          }
          pb[j][2 * u] = transpose8(pack_half(sc[u][j][0], sc[u][j][1]));
          pb[j][2 * u + 1] = transpose8(pack_half(sc[u][j][2], sc[u][j][3]));
        }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        constexpr int VW = D / 64;                   // words of a lane's elements of one key
        uint32_t lo[2][VW], hi[2][VW], s2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * u + 8 * h + 2 * t;
          uint32_t x[VW], y[VW], sx, sy;
          if (D == 128) {
            const uint2 a = *reinterpret_cast<const uint2*>(st + St::kV + v_place<D>(r, g >> 1) + (g & 1) * 8);
            const uint2 b = *reinterpret_cast<const uint2*>(st + St::kV + v_place<D>(r + 1, g >> 1) + (g & 1) * 8);
            x[0] = a.x; x[VW - 1] = a.y; y[0] = b.x; y[VW - 1] = b.y;
            sx = st[St::kVs + r * 8 + g];
            sy = st[St::kVs + r * 8 + 8 + g];
          } else {
            x[0] = *reinterpret_cast<const uint32_t*>(st + St::kV + v_place<D>(r, g >> 2) + (g & 3) * 4);
            y[0] = *reinterpret_cast<const uint32_t*>(st + St::kV + v_place<D>(r + 1, g >> 2) + (g & 3) * 4);
            sx = st[St::kVs + r * 4 + (g >> 1)];
            sy = st[St::kVs + r * 4 + 4 + (g >> 1)];
          }
          s2[h] = scales_to_half(sx | (sy << 8));
#pragma unroll
          for (int i = 0; i < VW; ++i) {             // bytes of two keys' codes of one element
            lo[h][i] = (x[i] & 0x0f0f0f0fu) | ((y[i] << 4) & 0xf0f0f0f0u);
            hi[h][i] = ((x[i] >> 4) & 0x0f0f0f0fu) | (y[i] & 0xf0f0f0f0u);
          }
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          uint32_t a[2][2][4];                       // [key half][even / odd element][tile]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_to_half(lo[h][i], a[h][0]);
            codes_to_half(hi[h][i], a[h][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int x = 0; x < 4; ++x) a[h][e][x] = mul_half(a[h][e][x], s2[h]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma(o[j][4 * i + x], a[0][0][x], a[0][1][x], a[1][0][x], a[1][1][x], pb[j][2 * u], pb[j][2 * u + 1]);
        }
      }
      slot = slot == C::kStages - 1 ? 0 : slot + 1;
    }

    // ---- join the warps: rows of O in shared memory, then one sum a row
    copies_wait<0>();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[j][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int r = 8 * j + 2 * t + c;
        if (g == 0) { w_max[warp][r] = m[j][c]; w_sum[warp][r] = v; }
        // elements 16 g + 2 i + {0, 1} (D = 64: 8 g + ...)
        float* dst = warp_o + r * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[j][i][c], o[j][i][c + 2]);
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == sq.chunks;
    const int piece = c0 == 0 ? 1 : 0;               // a block's first unit may continue
                                                     // one, its last may be continued
    for (int i = tid; i < rows * (D / 2); i += kWarps * 32) {
      const int r = i / (D / 2), d = (i % (D / 2)) * 2;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, w_max[k][r]);
      float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float a = w_max[k][r] == -CUDART_INF_F ? 0.0f : exp2f(w_max[k][r] - top);
        const float2 v = *reinterpret_cast<const float2*>(smem + k * C::kWarpBytes + (r * D + d) * 4);
        sum += a * w_sum[k][r];
        x += a * v.x;
        y += a * v.y;
      }
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);   // NaN stays
      const float lse = sum == 0.0f ? -CUDART_INF_F
                                    : (top - kBias + log2f(sum)) * 0.69314718055994530942f;
      if (whole) {
        const int row = tile_row0 + r, tok = row / p.G, h = head * p.G + (row - tok * p.G);
        const int64_t at = (sq.q_row0 + tok) * p.H + h;
        const float dv = p.cache.descale[1] * inv;
        T* dst = static_cast<T*>(p.o) + at * D + d;
        if (std::is_same<T, __half>::value)
          *reinterpret_cast<__half2*>(dst) = __floats2half2_rn(x * dv, y * dv);
        else
          *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(x * dv, y * dv);
        if (d == 0) p.lse[static_cast<int64_t>(h) * p.total_q + sq.q_row0 + tok] = lse;
      } else {
        const int64_t at = (bid * 2 + piece) * kRows + r;
        *reinterpret_cast<float2*>(p.part_o + at * D + d) = make_float2(x * inv, y * inv);
        if (d == 0) p.part_lse[at] = lse;
      }
    }
    if (tid == 0 && c0 == 0 && !whole) {
      // the block that holds the unit's last chunk
      const int64_t last = w + sq.chunks - 1;
      Meta& mt = p.meta[bid];
      mt.q_row0 = sq.q_row0;
      mt.head0 = head * p.G;
      mt.row0 = tile_row0;
      mt.rows = rows;
      mt.pieces = static_cast<int32_t>(((last + 1) * blocks - 1) / total - bid + 1);
    }
    __syncthreads();                                  // the rings may be filled again
    w += c1 - c0;
    off += c1 - c0;
  }
}

// Merge of a divided unit's pieces, one block a row:
//   lse = log sum exp(lse_i),  O = sum exp(lse_i - lse) O_i.
// The first piece is the starting block's second slot, the others the
// following blocks' first slots.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(4 * D) fa_kv4_merge_kernel(const __grid_constant__ AttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Meta mt = p.meta[blockIdx.x];
  const int r = blockIdx.y;
  if (mt.pieces == 0 || r >= mt.rows) return;
  __shared__ float sum_o[4][D], sum_w[4];
  const int d = threadIdx.x % D, part = threadIdx.x / D;
  const int64_t first = blockIdx.x;
  auto at = [&](int i) { return ((first + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + r; };
  __shared__ float tops[4 * D / 32];
  float top = -CUDART_INF_F;
  for (int i = threadIdx.x; i < mt.pieces; i += 4 * D) top = fmaxf(top, p.part_lse[at(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4 * D / 32; ++i) top = fmaxf(top, tops[i]);
  float acc = 0.0f, sum = 0.0f;
#pragma unroll 4
  for (int i = part; i < mt.pieces; i += 4) {
    const int64_t a = at(i);
    const float lse = p.part_lse[a];
    const float wgt = lse == -CUDART_INF_F ? 0.0f : expf(lse - top);
    sum += wgt;
    acc += wgt * p.part_o[a * D + d];
  }
  sum_o[part][d] = acc;
  if (d == 0) sum_w[part] = sum;
  __syncthreads();
  if (part != 0) return;
  acc = (sum_o[0][d] + sum_o[1][d]) + (sum_o[2][d] + sum_o[3][d]);
  sum = (sum_w[0] + sum_w[1]) + (sum_w[2] + sum_w[3]);
  const int row = mt.row0 + r, tok = row / p.G, h = mt.head0 + (row - tok * p.G);
  const float v = sum == 0.0f ? 0.0f : acc / sum * p.cache.descale[1];
  T* dst = static_cast<T*>(p.o) + ((mt.q_row0 + tok) * p.H + h) * D + d;
  if (std::is_same<T, __half>::value)
    *reinterpret_cast<__half*>(dst) = __float2half_rn(v);
  else
    *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(v);
  if (d == 0)
    p.lse[static_cast<int64_t>(h) * p.total_q + mt.q_row0 + tok] = sum == 0.0f ? -CUDART_INF_F : top + logf(sum);
}

// ---------------------------------------------------------------- unpacking
constexpr int kUnpackThreads = 256;
constexpr int kUnpackRows = 32;           // packed rows of a block

struct UnpackParams {
  Cache cache;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* block_table;
  int32_t* cu_k;            // [n_seqs + 1], written
  void* out[2];             // [total_k, H_kv, D]
  int64_t total_q, total_k, max_keys;
  int32_t n_seqs, max_pages;
};

template <typename T, int D>
__global__ void __launch_bounds__(kUnpackThreads) fa_kv4_unpack_kernel(const __grid_constant__ UnpackParams p) {
  extern __shared__ int32_t cu[];         // [n_seqs + 1] key rows before each sequence
  __shared__ int64_t warp_sum[kUnpackThreads / 32];
  __shared__ int64_t where[kUnpackRows];  // row (page, 0, row of the page) in the cache, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_seqs;
  // keys of a sequence: none where it brings no queries
  auto keys = [&](int s) -> int64_t {
    return p.cu_q[s + 1] > p.cu_q[s] ? min(max(static_cast<int64_t>(p.seqused_k[s]), int64_t(0)), p.max_keys) : 0;
  };
  const int per = (n + kUnpackThreads - 1) / kUnpackThreads;
  const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += keys(s);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += a;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t at = incl - mine;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int s = s0; s < s1; ++s) {
    cu[s] = static_cast<int32_t>(min(at, p.total_k));
    at += keys(s);
  }
  if (s0 < n && s1 == n) cu[n] = static_cast<int32_t>(min(at, p.total_k));
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = tid; s <= n; s += kUnpackThreads) p.cu_k[s] = cu[s];

  // and zeros behind the last sequence, where its last tile of 128 keys ends
  const int64_t used = cu[n], rows = min(used + 128, p.total_k);
  const int groups = p.cache.H_kv * (D / 16);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kUnpackRows; base < rows;
       base += static_cast<int64_t>(gridDim.x) * kUnpackRows) {
    __syncthreads();
    if (tid < kUnpackRows) {
      int64_t row = -1;
      const int64_t i = base + tid;
      if (i < used) {
        int lo = 0, hi = n;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cu[mid] <= i) lo = mid; else hi = mid;
        }
        const int key = static_cast<int>(i - cu[lo]), ps = p.cache.page_size;
        const int col = key / ps;
        const int page = p.block_table[static_cast<int64_t>(lo) * p.max_pages + col];
        if (page >= 0 && page < p.cache.num_pages)
          row = static_cast<int64_t>(page) * p.cache.H_kv * ps + (key - col * ps);
      }
      where[tid] = row;
    }
    __syncthreads();
    const int todo = static_cast<int>(min(static_cast<int64_t>(kUnpackRows), rows - base));
    const int which = blockIdx.y;
    for (int i = tid; i < todo * groups; i += kUnpackThreads) {
      const int r = i / groups, rest = i - r * groups, head = rest / (D / 16), gr = rest % (D / 16);
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0u;
      if (where[r] >= 0) {
        const int64_t row = where[r] + static_cast<int64_t>(head) * p.cache.page_size;
        const uint2 codes = *reinterpret_cast<const uint2*>(p.cache.codes[which] + row * (D / 2) + gr * 8);
        const uint32_t s = p.cache.scales[which][row * (D / 16) + gr];
        const uint32_t s2 = scales_to_half(s | (s << 8));
        const float dv = p.cache.descale[which];
        uint32_t h[2][4];
        codes_to_half(codes.x, h[0]);
        codes_to_half(codes.y, h[1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t v = mul_half(h[j / 4][j % 4], s2);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
          if (std::is_same<T, __half>::value) {
            w[j] = pack_half(f.x * dv, f.y * dv);
          } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * dv, f.y * dv);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[which]) + ((base + r) * groups + rest) * 16);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// ---------------------------------------------------------------- host
// Rows of a sequence (queries x G) up to which the cache is read as it is:
// measured below.
constexpr int64_t kStreamRows = 64;
constexpr int64_t kMaxUnpackSeqs = 16384;

bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Streaming multiprocessors of the current device (at most kMaxSms are used).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return std::min(n, kMaxSms);
}

int tiles_for(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

struct Layout {
  size_t part_o, part_lse, meta, bytes;
};
Layout stream_layout(int64_t D, int nt) {
  const size_t blocks = static_cast<size_t>(kMaxSms) * (nt == 1 ? 4 : nt == 2 ? 3 : 2);
  Layout l;
  l.part_o = 0;
  l.part_lse = round256(blocks * 2 * 8 * nt * D * 4);
  l.meta = l.part_lse + round256(blocks * 2 * 8 * nt * 4);
  l.bytes = l.meta + round256(blocks * sizeof(Meta));
  return l;
}
struct UnpackLayout {
  size_t k, v, bytes;
};
UnpackLayout unpack_layout(int64_t n_seqs, int64_t total_k, int64_t H_kv, int64_t D) {
  const size_t rows = round256(static_cast<size_t>(std::max<int64_t>(total_k, 1)) * H_kv * D * 2);
  UnpackLayout l;
  l.k = round256(static_cast<size_t>(n_seqs + 1) * 4);
  l.v = l.k + rows;
  l.bytes = l.v + rows;
  return l;
}

template <typename T, int D, int NT>
cudaError_t launch_stream(const AttnParams& p, int sms, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(fa_kv4_attn_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms * C::kBlocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, fa_kv4_attn_kernel<T, D, NT>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3(static_cast<unsigned>(sms * C::kBlocks), C::kRows);
  mc.blockDim = dim3(4 * D);
  mc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  mc.attrs = attr;
  mc.numAttrs = 1;
  return cudaLaunchKernelEx(&mc, fa_kv4_merge_kernel<T, D, C::kRows>, p);
}

template <typename T, int D>
cudaError_t launch_stream_rows(const AttnParams& p, int nt, int sms, cudaStream_t stream) {
  return nt == 1   ? launch_stream<T, D, 1>(p, sms, stream)
         : nt == 2 ? launch_stream<T, D, 2>(p, sms, stream)
                   : launch_stream<T, D, 4>(p, sms, stream);
}

template <typename T, int D>
cudaError_t launch_unpack(const UnpackParams& p, int sms, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.n_seqs + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(fa_kv4_unpack_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kMaxUnpackSeqs + 1) * 4));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  const int64_t want = std::max<int64_t>(1, (p.total_k + kUnpackRows - 1) / kUnpackRows);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(want, sms * 4)), 2);
  cfg.blockDim = dim3(kUnpackThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, fa_kv4_unpack_kernel<T, D>, p);
}

}  // namespace

extern "C" {

fa_status_t fa_fwd_paged_kv4_workspace_size(int64_t n_seqs, int64_t max_seqlen_q, int64_t total_k,
                                            int64_t H, int64_t H_kv, int64_t D,
                                            size_t* workspace_bytes) {
  if (!workspace_bytes || n_seqs < 1 || max_seqlen_q < 1 || total_k < 0 || H < 1 || D < 1 ||
      H_kv < 1 || H % H_kv != 0)
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  const int64_t kMaxRows = (int64_t(1) << 31) - 256;
  if (max_seqlen_q > kMaxRows || total_k > kMaxRows || H > 65536 || n_seqs > INT32_MAX - 1)
    return FA_ERR_UNSUPPORTED;
  const int64_t rows = max_seqlen_q * (H / H_kv);
  *workspace_bytes = rows <= kStreamRows ? stream_layout(D, tiles_for(rows)).bytes
                                         : unpack_layout(n_seqs, total_k, H_kv, D).bytes;
  return FA_OK;
}

fa_status_t fa_fwd_paged_kv4(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                             const uint8_t* v_codes, const uint8_t* v_scales, void* o, float* lse,
                             const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                             const int32_t* block_table, int64_t n_seqs, int64_t max_pages_per_seq,
                             int64_t page_size, int64_t num_pages, int64_t total_q,
                             int64_t max_seqlen_q, int64_t total_k, int64_t H, int64_t H_kv,
                             int64_t D, float scale, int causal, fa_dtype_t dtype, float descale_k,
                             float descale_v, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  if (!k_codes || !k_scales || !v_codes || !v_scales || !cu_seqlens_q || !seqused_k ||
      !block_table || !workspace || (total_q != 0 && (!q || !o || !lse)))
    return FA_ERR_INVALID_ARG;
  if (n_seqs < 1 || total_q < 0 || max_seqlen_q < 1 || total_k < 0 || H < 1 || D < 1 || H_kv < 1 ||
      H % H_kv != 0 || max_pages_per_seq < 1 || num_pages < 1 || page_size < 16)
    return FA_ERR_INVALID_ARG;
  if (causal < 0 || causal > 2) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP8E4M3)
    return FA_ERR_INVALID_ARG;
  const float lo = std::ldexp(1.0f, -100), hi = std::ldexp(1.0f, 100);
  if (!(descale_k >= lo && descale_k <= hi && descale_v >= lo && descale_v <= hi)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(scale * descale_k)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_DTYPE_FP8E4M3 || !fa::kv4::page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
  if (off(q, 16) || off(o, 16) || off(k_codes, 16) || off(v_codes, 16) || off(k_scales, 16) ||
      off(v_scales, 16) || off(lse, 4) || off(cu_seqlens_q, 4) || off(seqused_k, 4) || off(block_table, 4))
    return FA_ERR_MISALIGNED;
  const int64_t kMaxRows = (int64_t(1) << 31) - 256;
  if (total_q > kMaxRows || total_k > kMaxRows || max_seqlen_q > kMaxRows || H > 65536 ||
      n_seqs > INT32_MAX - 1 || max_pages_per_seq > INT32_MAX || num_pages > INT32_MAX ||
      page_size > 65536 || max_pages_per_seq * page_size > kMaxRows)
    return FA_ERR_UNSUPPORTED;
  size_t need = 0;
  const fa_status_t st = fa_fwd_paged_kv4_workspace_size(n_seqs, max_seqlen_q, total_k, H, H_kv, D, &need);
  if (st != FA_OK) return st;
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (off(workspace, 256)) return FA_ERR_MISALIGNED;
  const int64_t G = H / H_kv, rows = max_seqlen_q * G;
  if (rows > kStreamRows && n_seqs > kMaxUnpackSeqs) return FA_ERR_UNSUPPORTED;
  if (total_q == 0) return FA_OK;

  const int sms = sm_count();
  if (sms < 1) return FA_ERR_CUDA;
  Cache c = {};
  c.codes[0] = const_cast<uint8_t*>(k_codes); c.codes[1] = const_cast<uint8_t*>(v_codes);
  c.scales[0] = const_cast<uint8_t*>(k_scales); c.scales[1] = const_cast<uint8_t*>(v_scales);
  c.num_pages = num_pages;
  c.page_size = static_cast<int32_t>(page_size);
  c.H_kv = static_cast<int32_t>(H_kv);
  char* ws = static_cast<char*>(workspace);

  if (rows > kStreamRows) {
    const UnpackLayout l = unpack_layout(n_seqs, total_k, H_kv, D);
    UnpackParams u = {};
    u.cache = c;
    // K keeps its exact values (its descale goes into the softmax scale); V
    // takes its descale here, a second rounding to 16 bits (half a step) that
    // O's own rounding outweighs.
    u.cache.descale[0] = 1.0f;
    u.cache.descale[1] = descale_v;
    u.cu_q = cu_seqlens_q; u.seqused_k = seqused_k; u.block_table = block_table;
    u.cu_k = reinterpret_cast<int32_t*>(ws);
    u.out[0] = ws + l.k; u.out[1] = ws + l.v;
    u.total_q = total_q; u.total_k = total_k;
    u.max_keys = max_pages_per_seq * page_size;
    u.n_seqs = static_cast<int32_t>(n_seqs);
    u.max_pages = static_cast<int32_t>(max_pages_per_seq);
    cudaError_t e;
    if (dtype == FA_DTYPE_F16)
      e = D == 64 ? launch_unpack<__half, 64>(u, sms, stream) : launch_unpack<__half, 128>(u, sms, stream);
    else
      e = D == 64 ? launch_unpack<__nv_bfloat16, 64>(u, sms, stream) : launch_unpack<__nv_bfloat16, 128>(u, sms, stream);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    return fa_fwd_varlen(q, u.out[0], u.out[1], o, lse, cu_seqlens_q, u.cu_k, n_seqs, total_q, total_k,
                         max_seqlen_q, H, H_kv, D, scale * descale_k, causal, dtype, nullptr, nullptr,
                         nullptr, stream);
  }

  const int nt = tiles_for(rows);
  const Layout l = stream_layout(D, nt);
  AttnParams p = {};
  p.cache = c;
  p.cache.descale[0] = descale_k;
  p.cache.descale[1] = descale_v;
  p.q = q; p.o = o; p.lse = lse;
  p.cu_q = cu_seqlens_q; p.seqused_k = seqused_k; p.block_table = block_table;
  p.part_o = reinterpret_cast<float*>(ws + l.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + l.part_lse);
  p.meta = reinterpret_cast<Meta*>(ws + l.meta);
  p.total_q = total_q;
  p.max_keys = max_pages_per_seq * page_size;
  p.sl2 = std::fabs(scale) * descale_k * 1.4426950408889634f;
  p.negate = scale < 0.0f ? 1 : 0;
  p.n_seqs = static_cast<int32_t>(n_seqs);
  p.max_pages = static_cast<int32_t>(max_pages_per_seq);
  p.page_shift = -1;
  if ((page_size & (page_size - 1)) == 0)
    for (p.page_shift = 0; (int64_t(1) << p.page_shift) < page_size;) ++p.page_shift;
  p.H = static_cast<int32_t>(H);
  p.G = static_cast<int32_t>(G);
  p.causal = causal;
  cudaError_t e;
  if (dtype == FA_DTYPE_F16)
    e = D == 64 ? launch_stream_rows<__half, 64>(p, nt, sms, stream) : launch_stream_rows<__half, 128>(p, nt, sms, stream);
  else
    e = D == 64 ? launch_stream_rows<__nv_bfloat16, 64>(p, nt, sms, stream)
                : launch_stream_rows<__nv_bfloat16, 128>(p, nt, sms, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
