/*
 * fa_kv4_attn.cu -- fa_fwd_paged_kv4: attention of packed queries over the
 * 4-bit paged cache (include/fa_api.h).  Three ways, by the rows (queries x
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
 *   significant bits); bf16 queries become f16 too, each row shifted by a power
 *   of two that its scale takes back: exactly, but for elements below 2^-22 of
 *   the row's largest, which keep fewer bits.  Beside that P in f16 is the only
 *   rounding: 2^-11 of each probability; scores, sums and O are fp32.
 * Work: every sequence's keys, times its heads, are one line of 64-key chunks,
 * cut into equal runs for the resident blocks whatever the lengths are; a
 * (sequence, head) that a cut divides leaves fp32 partials that a second
 * kernel merges.  A block's warps take 32-key steps in turn, each with its own
 * cp.async ring and its own running maximum, and join at the run's end.
 *
 * More rows (17 to 128, to 512 over long sequences): fa_kv4_wide.cu.
 *
 * Many rows (chunked prefill): bound by the matrix products.  The keys and
 * values are unpacked once into a 16-bit workspace (a tenth of the time),
 * exactly, and the tcgen05 forward of packed sequences reads them there.  That
 * one holds P in the queries' type, as everywhere in this library: a rounding of
 * 2^-8 of each probability for bf16, of 2^-11 for f16 (2^-25 of the row's largest
 * for those below 2^-14 of it).
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
#include "fa_kv4_units.cuh"
#include "fa_kv4_wide.cuh"

namespace fa {
// The packed forward with a factor on O, and one each on the scores and on O
// that are read on the device where the pointers are not null (fa_api.cu).
fa_status_t fwd_varlen_scaled(const void* q, const void* k, const void* v, void* o, float* lse,
                              const int32_t* cu_q, const int32_t* cu_k, int64_t n_seqs,
                              int64_t total_q, int64_t total_k, int64_t max_seqlen_q, int64_t H,
                              int64_t H_kv, int64_t D, float scale, int causal, fa_dtype_t dtype,
                              float o_scale, const float* scale_at, const float* o_scale_at,
                              cudaStream_t stream);
// The current device's error word for bounded waits, and their limit (fa_api.cu).
fa_status_t wait_control(uint32_t** err, uint64_t* limit_ns);
}  // namespace fa

namespace {

using namespace fa::kv4;

constexpr int kStep = 32;           // keys of a warp's step
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes of which the first `bytes` come from src, zeros behind them.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, int bytes) {
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

// Where the next step's keys are: pages of its two halves (one lookup when
// pages hold 32 keys or more) and the first key's row in its page.  A step ahead
// of a sequence's last key may be past 2^31 (unsigned here).
struct Place {
  int page[2], in_page;
};
__device__ __forceinline__ Place look_up(const AttnParams& p, uint32_t table, uint32_t key0, uint32_t end) {
  Place at = {{-1, -1}, 0};
  if (key0 < end) {
    const uint32_t ps = p.cache.page_size;
    const uint32_t col = p.page_shift >= 0 ? key0 >> p.page_shift : key0 / ps;
    at.in_page = key0 - col * ps;
    at.page[0] = p.block_table[table + col];
    at.page[1] = ps >= kStep ? at.page[0] : key0 + 16 < end ? p.block_table[table + col + 1] : -1;
  }
  return at;
}

// A lane's sources and destinations in a step's copies.
struct Lane {
  uint32_t v_dst, s_dst;     // offsets in a stage of its first piece of V and its piece of scales
};

// The codes and scales of keys [key0, key0 + 32) into a ring stage; keys from
// `end` on, and pages outside the cache, become zeros.  Rows of a page are
// one run of memory, so a lane's pieces lie 512 bytes apart.
template <int D>
__device__ __forceinline__ void load_step(const AttnParams& p, const Lane& me, uint32_t stage, int head, int key0,
                                          int end, const Place& at, int lane) {
  using St = Stage<D>;
  constexpr int C = St::kChunksRow, kHalf = 16 * C / 32;     // pieces of K (or V) a lane takes of 16 keys
  constexpr int KP = 256 / D, N = kStep / KP;                // keys a piece of scales holds, pieces
  const uint32_t pages = static_cast<uint32_t>(p.cache.num_pages), ps = p.cache.page_size;
  uint32_t row[2];
  row[0] = (static_cast<uint32_t>(at.page[0]) * p.cache.H_kv + head) * ps + at.in_page;
  row[1] = row[0] + 16;
  if (ps < kStep) row[1] = (static_cast<uint32_t>(at.page[1]) * p.cache.H_kv + head) * ps;
  const bool ok0 = static_cast<uint32_t>(at.page[0]) < pages, ok1 = static_cast<uint32_t>(at.page[1]) < pages;
  if (ok0 && ok1 && key0 + kStep <= end) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t off = static_cast<uint64_t>(row[h]) * (D / 2) + lane * 16;
      const uint8_t *k = p.cache.codes[0] + off, *v = p.cache.codes[1] + off;
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        copy16(stage + lane * 16 + (h * kHalf + i) * 512, k + i * 512);
        copy16(stage + me.v_dst + (h * kHalf + i) * 512, v + i * 512);
      }
    }
    if (2 * N == 32 || lane < 2 * N) {
      const int h = (lane % N) * KP / 16;
      copy16(stage + me.s_dst, p.cache.scales[lane / N % 2] + static_cast<uint64_t>(row[h] + (lane % N) * KP - 16 * h) * (D / 16));
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool ok = h ? ok1 : ok0;
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const int r = (lane + 32 * i) / C;                     // row of the half
      const bool in = ok && key0 + 16 * h + r < end;
      const uint64_t off = in ? static_cast<uint64_t>(row[h]) * (D / 2) + i * 512 + lane * 16 : 0;
      copy16_or_zero(stage + lane * 16 + (h * kHalf + i) * 512, p.cache.codes[0] + off, in ? 16 : 0);
      copy16_or_zero(stage + me.v_dst + (h * kHalf + i) * 512, p.cache.codes[1] + off, in ? 16 : 0);
    }
  }
  if (lane < 2 * N) {
    const int r = (lane % N) * KP, h = r >> 4;
    const int keys = (h ? ok1 : ok0) ? min(max(end - key0 - r, 0), KP) : 0;
    const uint64_t off = keys > 0 ? static_cast<uint64_t>(row[h] + r - 16 * h) * (D / 16) : 0;
    copy16_or_zero(stage + me.s_dst, p.cache.scales[lane / N % 2] + off, keys * (D / 16));
  }
}

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  // Warps of a block and resident blocks an SM: 12 warps of up to 168 registers
  // (8 rows use 144, 130 at D = 64; 16 rows 160 at 64, and at 128 all 168 with 12
  // bytes spilled).  With 8 rows, 128 sequences of 8192 keys (floor 178 us):
  // 4 blocks of 3 warps 210 us, 2 x 8 (128 registers) 214, 6 x 2 211, 2 x 4 224;
  // 4000 of 256 keys, where units end often: 383, 557, 354, 525; one of 65536:
  // 28, 26, 32, 27.
  static constexpr int kWarps = NT == 1 ? 3 : 4;
  static constexpr int kBlocks = NT == 1 ? 4 : 3;
  // A warp's ring: three stages; at the end of a unit its O lies in the third
  // one's place (and behind it), while the next unit's first two steps are
  // already on their way to the other two.
  static constexpr int kStages = 3;
  static constexpr int kOut = 2 * Stage<D>::kBytes;
  static constexpr int kWarpBytes = kOut + (Stage<D>::kBytes > kRows * D * 4 ? Stage<D>::kBytes : kRows * D * 4);
  static constexpr int kQ = kWarps * kWarpBytes;                  // the unit's Q, f16, in operand order
  static constexpr int kSmem = kQ + kRows * D * 2;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kWarps * 32, Cfg<D, NT>::kBlocks)
    fa_kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NT>;
  using St = Stage<D>;
  constexpr int kRows = C::kRows, kWarps = C::kWarps;
  constexpr int MT = D / 16;        // 16-element tiles of O^T
  constexpr int QW = D / 8;         // f16 pairs of a row of Q in one lane's dimensions
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float w_max[kWarps][kRows], w_sum[kWarps][kRows], row_scale[kRows];
  __shared__ int row_limit[kRows];
  __shared__ float factors[2];            // of the scores, of V
  __shared__ int64_t scan[kWarps];
  __shared__ Cursor cursor;
  __shared__ Unit units[4];               // of a ring: this one, the next two
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  fa::wait_for_stream();
  fa::let_next_start();

  if (!begin_units<kRows, kWarps * 32>(p, scan, cursor, units, factors)) return;

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kWarpBytes;
  uint8_t* const ring_p = smem + warp * C::kWarpBytes;
  Lane me;
  {
    constexpr int CR = St::kChunksRow, KP = 256 / D, N = kStep / KP;
    me.v_dst = St::kV + v_place<D>(lane / CR, lane % CR);
    const int which = lane / N % 2, piece = lane % N;
    me.s_dst = (which ? St::kVs : St::kKs) + piece * 16;
  }
  // this lane's reads of a stage, relative to it
  const int k_at = D == 128 ? g * 64 + t * 16 : g * 32 + t * 8;
  const int ks_at = St::kKs + (D == 128 ? g * 8 + t * 2 : g * 4 + t);
  const int v0_at = St::kV + (D == 128 ? v_place<D>(2 * t, g >> 1) + (g & 1) * 8 : v_place<D>(2 * t, g >> 2) + (g & 3) * 4);
  const int v1_at = v0_at + 128;            // v_place of row 2 t + 1 at both D
  const int vs_at = St::kVs + (D == 128 ? t * 16 + g : t * 8 + (g >> 1));
  uint8_t* const q_smem = smem + C::kQ;
  const int step = kWarps * kStep;

  Place at;                                 // of the next step to load
  uint32_t table;                           // the sequence's row of the block table
  auto start_ring = [&](const Unit& u) {
    const uint32_t end = u.key_end;
    table = static_cast<uint32_t>(u.s) * static_cast<uint32_t>(p.max_pages);
    uint32_t next = u.key_begin + warp * kStep;
    at = look_up(p, table, next, end);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (next < end) load_step<D>(p, me, ring + i * St::kBytes, u.head, next, end, at, lane);
      copies_commit();
      next += step;
      at = look_up(p, table, next, end);
    }
  };

  // Q: warp j takes rows 8 j .. 8 j + 7 of a unit; lane (g, t) its dimensions of
  // row 8 j + g.  Loaded before the last unit's rows are joined, turned into
  // operands after that.
  constexpr int kQTiles = (NT + kWarps - 1) / kWarps;
  uint4 q_raw[kQTiles][QW / 4];
  auto load_q = [&](const Unit& u) {
#pragma unroll
    for (int i = 0; i < kQTiles; ++i) {
      const int r = 8 * (warp + i * kWarps) + g, row = u.row0 + r, tok = row / p.G;
#pragma unroll
      for (int x = 0; x < QW / 4; ++x) q_raw[i][x] = make_uint4(0u, 0u, 0u, 0u);
      if (r < u.rows) {
        const int64_t from = ((u.q_row0 + tok) * p.H + static_cast<int64_t>(u.head) * p.G + (row - tok * p.G)) * D + t * (D / 4);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + from);
#pragma unroll
        for (int x = 0; x < QW / 4; ++x) q_raw[i][x] = src[x];
      }
    }
  };
  auto turn_q = [&](const Unit& u) {
#pragma unroll
    for (int i = 0; i < kQTiles; ++i) {
      const int j = warp + i * kWarps;
      if (j >= NT) break;                   // the same for the whole warp
      uint32_t q[QW];
#pragma unroll
      for (int x = 0; x < QW / 4; ++x) {
        q[4 * x] = q_raw[i][x].x; q[4 * x + 1] = q_raw[i][x].y; q[4 * x + 2] = q_raw[i][x].z; q[4 * x + 3] = q_raw[i][x].w;
      }
      float rescale = 1.0f;
      if (!std::is_same<T, __half>::value) {
        // bf16: shift the row by a power of two so that its largest value is
        // in [2^8, 2^9) and convert: exact down to 2^-22 of the largest.
        uint32_t top = 0u;
#pragma unroll
        for (int x = 0; x < QW; ++x) top = max(top, max(q[x] & 0x7fffu, (q[x] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max(static_cast<int>(top >> 7), 30), 254);   // biased exponent
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 + 127 - e) << 23);
        rescale = __uint_as_float(static_cast<uint32_t>(e - 8) << 23);
#pragma unroll
        for (int x = 0; x < QW; ++x)
          q[x] = pack_half(__uint_as_float(q[x] << 16) * up, __uint_as_float(q[x] & 0xffff0000u) * up);
      }
      if (p.negate) {
#pragma unroll
        for (int x = 0; x < QW; ++x) q[x] ^= 0x80008000u;
      }
      // [8 dimensions of a lane][lane]: 16 bytes, the two k16 steps of a word of codes
#pragma unroll
      for (int x = 0; x < QW / 4; ++x)
        *reinterpret_cast<uint4*>(q_smem + ((j * (QW / 4) + x) * 32 + lane) * 16) =
            make_uint4(q[4 * x], q[4 * x + 1], q[4 * x + 2], q[4 * x + 3]);
      const int r = 8 * j + g, tok = (u.row0 + r) / p.G;
      int see = u.k_len;
      if (p.causal == FA_CAUSAL_TOP_LEFT) see = min(see, tok + 1);
      if (p.causal == FA_CAUSAL_BOTTOM_RIGHT) see = min(see, tok + 1 + u.keys - u.q_len);
      if (t == 0) {
        row_scale[r] = fmaxf(factors[0] * rescale, 1e-30f);
        row_limit[r] = see;
      }
    }
  };

  start_ring(units[0]);
  load_q(units[0]);
  turn_q(units[0]);
  __syncthreads();
  for (int turn = 0;; turn = (turn + 1) & 3) {
    const Unit& un = units[turn];
    int key_begin = un.key_begin, key_end = un.key_end, head = un.head;
    // kept in registers: not to be read from shared memory again at every step
    asm volatile("" : "+r"(key_begin), "+r"(key_end), "+r"(head));
    // one warp looks for the unit after the next (known to all at the next one)
    if (lane == 0 && warp == (turn % kWarps) && un.more && units[(turn + 1) & 3].more)
      next_unit<kRows>(p, cursor, units[(turn + 2) & 3]);
    __syncwarp();
    // this lane's accumulators are rows 8 j + 2 t and 8 j + 2 t + 1
    float sl2[NT][2];
    int full = key_end;                      // keys that all rows see
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sl2[j][c] = row_scale[8 * j + 2 * t + c];
        full = min(full, row_limit[8 * j + 2 * t + c]);
      }
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
      // Shared memory is read well ahead of use, in the order written here (the
      // votes and copies below keep the compiler from moving reads over them).
      uint32_t words[2][2][D / 32], k_scale[2][2];   // [16 keys][8 keys]
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * u + 8 * h;
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + k_at + r * 64);
            words[u][h][0] = v.x; words[u][h][1] = v.y; words[u][h][2 % (D / 32)] = v.z; words[u][h][3 % (D / 32)] = v.w;
            k_scale[u][h] = *reinterpret_cast<const uint16_t*>(st + ks_at + r * 8);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(st + k_at + r * 32);
            words[u][h][0] = v.x; words[u][h][1] = v.y;
            k_scale[u][h] = st[ks_at + r * 4] * 0x101u;
          }
        }
      {
        const int into = slot == 0 ? C::kStages - 1 : slot - 1;   // the stage read one step ago
        const int next = key0 + (C::kStages - 1) * step;
        if (next < key_end) load_step<D>(p, me, ring + into * St::kBytes, head, next, key_end, at, lane);
        copies_commit();
        at = look_up(p, table, static_cast<uint32_t>(next) + step, key_end);
      }

      // S^T: two tiles of 16 keys
      float sc[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) sc[u][j][0] = sc[u][j][1] = sc[u][j][2] = sc[u][j][3] = 0.0f;
        uint32_t s2[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t two = scales_to_half(k_scale[u][h]);
          s2[h][0] = __byte_perm(two, 0u, 0x1010);
          s2[h][1] = __byte_perm(two, 0u, 0x3232);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {          // a word: 8 dimensions, two k16 steps
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_to_half(words[u][h][i], a[h]);
#pragma unroll
            for (int x = 0; x < 4; ++x) a[h][x] = mul_half(a[h][x], s2[h][i / 2]);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 b = *reinterpret_cast<const uint4*>(q_smem + ((j * (QW / 4) + i) * 32 + lane) * 16);
            mma(sc[u][j], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
            mma(sc[u][j], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
          }
        }
      }
      // V of 16 keys: this lane's elements of keys 2 t, 2 t + 1 of each 8
      constexpr int VW = D / 64;                     // words of a lane's elements of one key
      uint32_t vx[2][2][VW], vy[2][2][VW], v_scale[2][2];
      auto load_v = [&](int u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * u + 8 * h;
          if (D == 128) {
            const uint2 a = *reinterpret_cast<const uint2*>(st + v0_at + r * 64);
            const uint2 b = *reinterpret_cast<const uint2*>(st + v1_at + r * 64);
            vx[u][h][0] = a.x; vx[u][h][VW - 1] = a.y; vy[u][h][0] = b.x; vy[u][h][VW - 1] = b.y;
            v_scale[u][h] = st[vs_at + r * 8] | (st[vs_at + r * 8 + 8] << 8);
          } else {
            vx[u][h][0] = *reinterpret_cast<const uint32_t*>(st + v0_at + r * 32);
            vy[u][h][0] = *reinterpret_cast<const uint32_t*>(st + v1_at + r * 32);
            v_scale[u][h] = st[vs_at + r * 4] | (st[vs_at + r * 4 + 4] << 8);
          }
        }
      };
      load_v(0);

      // softmax of the step, P to operands
      const bool edge = key0 + kStep > full;
      uint32_t pb[NT][4];                            // 8 keys each
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (edge) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int limit = min(row_limit[8 * j + 2 * t + c], key_end) - key0 - g;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (8 * x >= limit) sc[x >> 1][j][c + 2 * (x & 1)] = -CUDART_INF_F;
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
      load_v(1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t s2[2] = {scales_to_half(v_scale[u][0]), scales_to_half(v_scale[u][1])};
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          uint32_t a[2][2][4];                       // [key half][even / odd element][tile]
#pragma unroll
          for (int h = 0; h < 2; ++h) {              // bytes of two keys' codes of one element
            const uint32_t x = vx[u][h][i], y = vy[u][h][i];
            codes_to_half((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[h][0]);
            codes_to_half(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[h][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int x4 = 0; x4 < 4; ++x4) a[h][e][x4] = mul_half(a[h][e][x4], s2[h]);
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

    // ---- the next unit's first keys start their way while this one ends
    const bool more = un.more;
    __syncwarp();                           // all lanes have read the ring's stages
    if (more) start_ring(units[(turn + 1) & 3]);

    // ---- join the warps: rows of O in shared memory, then one sum a row
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
        float* dst = reinterpret_cast<float*>(ring_p + C::kOut) + r * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[j][i][c], o[j][i][c + 2]);
      }
    __syncthreads();
    if (more) load_q(units[(turn + 1) & 3]);
    for (int i = tid; i < un.rows * (D / 2); i += kWarps * 32) {
      const int r = i / (D / 2), d = (i % (D / 2)) * 2;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, w_max[k][r]);
      float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float a = w_max[k][r] == -CUDART_INF_F ? 0.0f : exp2f(w_max[k][r] - top);
        const float2 v = *reinterpret_cast<const float2*>(smem + k * C::kWarpBytes + C::kOut + (r * D + d) * 4);
        sum += a * w_sum[k][r];
        x += a * v.x;
        y += a * v.y;
      }
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);   // NaN stays
      const float lse = sum == 0.0f ? -CUDART_INF_F
                                    : (top - kBias + log2f(sum)) * 0.69314718055994530942f;
      if (un.piece < 0) {
        const int row = un.row0 + r, tok = row / p.G, h = head * p.G + (row - tok * p.G);
        const int64_t to = (un.q_row0 + tok) * p.H + h;
        const float dv = factors[1] * inv;
        T* dst = static_cast<T*>(p.o) + to * D + d;
        if (std::is_same<T, __half>::value)
          *reinterpret_cast<__half2*>(dst) = __floats2half2_rn(x * dv, y * dv);
        else
          *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(x * dv, y * dv);
        if (d == 0) p.lse[static_cast<int64_t>(h) * p.total_q + un.q_row0 + tok] = lse;
      } else {
        const int64_t to = (blockIdx.x * int64_t(2) + un.piece) * kRows + r;
        *reinterpret_cast<float2*>(p.part_o + to * D + d) = make_float2(x * inv, y * inv);
        if (d == 0) p.part_lse[to] = lse;
      }
    }
    if (tid == 0 && un.pieces > 0)
      p.meta[blockIdx.x] = Meta{un.q_row0, un.pieces, head * p.G, un.row0, un.rows};
    if (!more) break;
    turn_q(units[(turn + 1) & 3]);
    __syncthreads();                        // O has been read, Q is written
  }
}

// ---------------------------------------------------------------- unpacking
// The keys and values of the sequences that bring queries, packed, in 16 bits:
// 4 bytes of codes give 16 out, so writing is most of what it does (283 MB
// moved in 64 us, 65 % of HBM; the forward behind it takes 598).
constexpr int kUnpackThreads = 256;
constexpr int kUnpackRows = 32;           // packed rows of a block

struct UnpackParams {
  Cache cache;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* block_table;
  int32_t* cu_k;            // [n_seqs + 1], written
  void* out[2];             // [total_k, H_kv, D]
  int64_t total_k, max_keys;
  int32_t n_seqs, max_pages;
};

template <typename T, int D>
__global__ void __launch_bounds__(kUnpackThreads) fa_kv4_unpack_kernel(const __grid_constant__ UnpackParams p) {
  extern __shared__ int32_t cu[];         // [n_seqs + 1] key rows before each sequence
  __shared__ int64_t warp_sum[kUnpackThreads / 32];
  __shared__ int64_t where[2][kUnpackRows];   // row (page, 0, row of the page) in the cache, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_seqs;
  fa::wait_for_stream();
  fa::let_next_start();
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
  // Where a tile's rows are is looked up while the tile before it is unpacked.
  auto look = [&](int64_t base, int64_t* to) {
    if (tid >= kUnpackRows) return;
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
    to[tid] = row;
  };
  const int which = blockIdx.y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kUnpackRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kUnpackRows;
  look(base, where[0]);
  __syncthreads();
  for (int b = 0; base < rows; base += step, b ^= 1) {
    look(base + step, where[b ^ 1]);
    fa::kv4::unpack_rows<T, D, kUnpackThreads, false>(p.cache, which, where[b],
                                               static_cast<int>(min(static_cast<int64_t>(kUnpackRows), rows - base)),
                                               static_cast<uint16_t*>(p.out[which]) + base * p.cache.H_kv * D);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host
// Rows of a sequence (queries x G) up to which the cache is read straight into
// mma.sync operands, up to which it is unpacked on the way to tcgen05, and up to
// which it is so where the sequences are long (total_k a sequence): a workspace
// of 16-bit rows costs what it writes and reads, a 128-row tile its unpacking.
// us, tiles / workspace, D 128, H 32 / 8:
//   128 sequences of 8192 keys: 16 rows 294, 32 rows 458 (506 in mma.sync operands),
//     64 rows 456, 128 rows 477 / 1575, 256 rows 919 / 1628, 512 rows 1816 / 2305
//   32 of 2048: 256 rows 104 / 142, 512 rows 175 / 197
//   8 of 2048: 256 rows 48 / 50, 512 rows 66 / 51 (few units: the rule takes the
//     slower way here)
//   one of 65536: 256 rows 101 / 687, 512 rows 142 / 691
//   256 of 256: 128 rows 133 / 152, 256 rows 242 / 165
// The rule goes by total_k, the caller's bound on all keys, and so by the mean.
constexpr int64_t kNarrowRows = 16, kStreamRows = 128, kLongStreamRows = 512, kLongKeys = 2048;
bool streams(int64_t rows, int64_t n_seqs, int64_t total_k) {
  return rows <= (total_k / kLongKeys >= n_seqs ? kLongStreamRows : kStreamRows);
}
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

// 8-row tiles of a unit; 0: the many-rows kernel.
int tiles_for(int64_t rows) { return rows <= 8 ? 1 : rows <= kNarrowRows ? 2 : 0; }

struct Layout {
  size_t part_o, part_lse, meta, bytes;
};
Layout stream_layout(int64_t D, int nt) {
  const size_t blocks = static_cast<size_t>(kMaxSms) * (nt == 1 ? 4 : nt == 2 ? 3 : 1);     // Cfg::kBlocks
  const size_t rows = blocks * 2 * (nt ? 8 * nt : kWideRows);
  Layout l;
  l.part_o = 0;
  l.part_lse = round256(rows * D * 4);
  l.meta = l.part_lse + round256(rows * 4);
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
  cudaError_t e = fa::allow_smem<fa_kv4_attn_kernel<T, D, NT>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(sms * C::kBlocks));
  const fa::Launch c(grid, C::kWarps * 32, C::kSmem, stream);
  e = cudaLaunchKernelEx(&c.cfg, fa_kv4_attn_kernel<T, D, NT>, p);
  if (e != cudaSuccess) return e;
  const fa::Launch mc(grid, kMergeWarps * 32, 0, stream);
  return cudaLaunchKernelEx(&mc.cfg, fa_kv4_merge_kernel<T, D, C::kRows>, p);
}

template <typename T, int D>
cudaError_t launch_stream_rows(const AttnParams& p, int nt, int sms, cudaStream_t stream) {
  return nt == 1 ? launch_stream<T, D, 1>(p, sms, stream) : launch_stream<T, D, 2>(p, sms, stream);
}

template <typename T, int D>
cudaError_t launch_unpack(const UnpackParams& p, int sms, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.n_seqs + 1) * 4;
  if (smem > fa::kFreeSmem) {
    const cudaError_t e = cudaFuncSetAttribute(fa_kv4_unpack_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kMaxUnpackSeqs + 1) * 4));
    if (e != cudaSuccess) return e;
  }
  const int64_t want = std::max<int64_t>(1, (p.total_k + kUnpackRows - 1) / kUnpackRows);
  const fa::Launch c(dim3(static_cast<unsigned>(std::min<int64_t>(want, sms * 4)), 2), kUnpackThreads, smem, stream);
  return cudaLaunchKernelEx(&c.cfg, fa_kv4_unpack_kernel<T, D>, p);
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
  // What a step with fewer sequences, queries or keys needs too: the layouts of
  // fewer rows, and unpacked keys where only their number keeps this one from it.
  *workspace_bytes = stream_layout(D, tiles_for(rows)).bytes;
  if (rows > kStreamRows) {
    const int64_t keys = rows > kLongStreamRows ? total_k : std::min(total_k, kLongKeys * n_seqs);
    *workspace_bytes = std::max(*workspace_bytes, unpack_layout(n_seqs, keys, H_kv, D).bytes);
  }
  return FA_OK;
}

}  // extern "C"

namespace {

fa_status_t attend(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                   const uint8_t* v_codes, const uint8_t* v_scales, void* o, float* lse,
                   const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                   const int32_t* block_table, int64_t n_seqs, int64_t max_pages_per_seq,
                   int64_t page_size, int64_t num_pages, int64_t total_q, int64_t max_seqlen_q,
                   int64_t total_k, int64_t H, int64_t H_kv, int64_t D, float scale, int causal,
                   fa_dtype_t dtype, const Descales& d, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
  const float descale_k = d.value[0], descale_v = d.value[1];
  if (!k_codes || !k_scales || !v_codes || !v_scales || !cu_seqlens_q || !seqused_k ||
      !block_table || !workspace || (total_q != 0 && (!q || !o || !lse)))
    return FA_ERR_INVALID_ARG;
  if (n_seqs < 1 || total_q < 0 || max_seqlen_q < 1 || total_k < 0 || H < 1 || D < 1 || H_kv < 1 ||
      H % H_kv != 0 || max_pages_per_seq < 1 || num_pages < 1 || page_size < 16)
    return FA_ERR_INVALID_ARG;
  if (causal < 0 || causal > 2) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP8E4M3)
    return FA_ERR_INVALID_ARG;
  const fa_status_t ds = check_descales(d);
  if (ds != FA_OK) return ds;
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
  // Queries are read by blocks that may run after another has written its rows.
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
  const uintptr_t span = static_cast<uintptr_t>(total_q) * H * D * 2;
  if (q0 < o0 + span && o0 < q0 + span) return FA_ERR_INVALID_ARG;
  size_t need = 0;
  const fa_status_t st = fa_fwd_paged_kv4_workspace_size(n_seqs, max_seqlen_q, total_k, H, H_kv, D, &need);
  if (st != FA_OK) return st;
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (off(workspace, 256)) return FA_ERR_MISALIGNED;
  const int64_t G = H / H_kv, rows = max_seqlen_q * G;
  if (!streams(rows, n_seqs, total_k) && n_seqs > kMaxUnpackSeqs) return FA_ERR_UNSUPPORTED;
  // a row's index in the cache is a 32-bit number (2^32 rows of D = 64, K and V, take 309 GB)
  if (num_pages > static_cast<int64_t>(0xffffffffu) / (page_size * H_kv)) return FA_ERR_UNSUPPORTED;
  if (n_seqs > static_cast<int64_t>(0xffffffffu) / max_pages_per_seq) return FA_ERR_UNSUPPORTED;
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

  if (!streams(rows, n_seqs, total_k)) {
    const UnpackLayout l = unpack_layout(n_seqs, total_k, H_kv, D);
    UnpackParams u = {};
    u.cache = c;
    // Keys and values keep their exact values: K's descale goes into the softmax
    // scale, V's into the factor of O before its rounding.
    u.cu_q = cu_seqlens_q; u.seqused_k = seqused_k; u.block_table = block_table;
    u.cu_k = reinterpret_cast<int32_t*>(ws);
    u.out[0] = ws + l.k; u.out[1] = ws + l.v;
    u.total_k = total_k;
    u.max_keys = max_pages_per_seq * page_size;
    u.n_seqs = static_cast<int32_t>(n_seqs);
    u.max_pages = static_cast<int32_t>(max_pages_per_seq);
    cudaError_t e;
    if (dtype == FA_DTYPE_F16)
      e = D == 64 ? launch_unpack<__half, 64>(u, sms, stream) : launch_unpack<__half, 128>(u, sms, stream);
    else
      e = D == 64 ? launch_unpack<__nv_bfloat16, 64>(u, sms, stream) : launch_unpack<__nv_bfloat16, 128>(u, sms, stream);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    return fa::fwd_varlen_scaled(q, u.out[0], u.out[1], o, lse, cu_seqlens_q, u.cu_k, n_seqs, total_q, total_k,
                                 max_seqlen_q, H, H_kv, D, scale * descale_k, causal, dtype, descale_v, d.at[0],
                                 d.at[1], stream);
  }

  const int nt = tiles_for(rows);
  const Layout l = stream_layout(D, nt);
  AttnParams p = {};
  p.cache = c;
  for (int i = 0; i < 2; ++i) { p.cache.descale[i] = d.value[i]; p.cache.descale_at[i] = d.at[i]; }
  p.q = q; p.o = o; p.lse = lse;
  p.cu_q = cu_seqlens_q; p.seqused_k = seqused_k; p.block_table = block_table;
  p.part_o = reinterpret_cast<float*>(ws + l.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + l.part_lse);
  p.meta = reinterpret_cast<Meta*>(ws + l.meta);
  p.total_q = total_q;
  p.max_keys = max_pages_per_seq * page_size;
  p.scale = std::fabs(scale);
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
  if (nt == 0) {
    uint32_t* err = nullptr;
    uint64_t limit_ns = 0;
    if (fa::wait_control(&err, &limit_ns) != FA_OK) return FA_ERR_CUDA;
    e = launch_wide(p, static_cast<int>(D), dtype == FA_DTYPE_F16, sms, err, limit_ns, stream);
  } else if (dtype == FA_DTYPE_F16)
    e = D == 64 ? launch_stream_rows<__half, 64>(p, nt, sms, stream) : launch_stream_rows<__half, 128>(p, nt, sms, stream);
  else
    e = D == 64 ? launch_stream_rows<__nv_bfloat16, 64>(p, nt, sms, stream)
                : launch_stream_rows<__nv_bfloat16, 128>(p, nt, sms, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status_t fa_fwd_paged_kv4(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                             const uint8_t* v_codes, const uint8_t* v_scales, void* o, float* lse,
                             const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                             const int32_t* block_table, int64_t n_seqs, int64_t max_pages_per_seq,
                             int64_t page_size, int64_t num_pages, int64_t total_q,
                             int64_t max_seqlen_q, int64_t total_k, int64_t H, int64_t H_kv,
                             int64_t D, float scale, int causal, fa_dtype_t dtype, float descale_k,
                             float descale_v, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  return attend(q, k_codes, k_scales, v_codes, v_scales, o, lse, cu_seqlens_q, seqused_k, block_table,
                n_seqs, max_pages_per_seq, page_size, num_pages, total_q, max_seqlen_q, total_k, H, H_kv,
                D, scale, causal, dtype, Descales{{descale_k, descale_v}, {}}, workspace, workspace_bytes,
                stream);
}

fa_status_t fa_fwd_paged_kv4_devscale(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                                      const uint8_t* v_codes, const uint8_t* v_scales, void* o,
                                      float* lse, const int32_t* cu_seqlens_q,
                                      const int32_t* seqused_k, const int32_t* block_table,
                                      int64_t n_seqs, int64_t max_pages_per_seq, int64_t page_size,
                                      int64_t num_pages, int64_t total_q, int64_t max_seqlen_q,
                                      int64_t total_k, int64_t H, int64_t H_kv, int64_t D,
                                      float scale, int causal, fa_dtype_t dtype,
                                      const float* descale_k, const float* descale_v,
                                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attend(q, k_codes, k_scales, v_codes, v_scales, o, lse, cu_seqlens_q, seqused_k, block_table,
                n_seqs, max_pages_per_seq, page_size, num_pages, total_q, max_seqlen_q, total_k, H, H_kv,
                D, scale, causal, dtype, Descales{{1.0f, 1.0f}, {descale_k, descale_v}}, workspace,
                workspace_bytes, stream);
}

}  // extern "C"
