/*
 * fa_kv4_wide.cu -- attention over the 4-bit cache for units of many rows
 * (queries x heads that share a key/value head, up to 128 a tile): the products
 * on tcgen05, the cached values unpacked on their way to them.
 *
 * With few rows HBM's time for a 128-key block (784 cycles an SM) is far above
 * the products', and mma.sync straight from registers serves (fa_kv4_attn.cu).
 * From 17 rows on its products and registers cost more than that, while here a
 * block costs nearly the same for any number of rows up to 128.  Measured with
 * 128 sequences of 8192 keys (H_kv 8, D 128): 458 us with 32 rows, 477 with 128
 * (1.15 PFLOP/s); HBM alone would take 178.  D = 64, 256 such sequences: 787 us.
 * A block takes 2000 cycles: the softmax warps are busy all of them (a row of 128
 * scores a thread, so that 32 rows are one warp's, on one of four sub-partitions),
 * the issue of the 16 products and its waits about 1600, an unpacking warp about
 * 1100.  What each step gave when it was made: the softmax in pairs of fp32
 * (f32x2) 512 us to 460; a page looked up without a branch around it, 450; the
 * next unit's first rows loaded while a unit ends, 336 us for 1000 sequences of 256
 * keys instead of 346 (12,000 cycles a unit of two blocks, most of them one
 * latency after another: Q, S, softmax twice, output).  The schedule hangs on
 * small things: where the scale comes from moves it by 1 to 2 % (451 us as a
 * launch parameter, 457 from shared memory).  Tried and
 * slower: P against the maximum so far with a check behind it (550), two softmax
 * warpgroups, on alternate blocks (487) or on half of each block's keys (457, 501
 * with 128 rows; faster at D = 64, 702 for 256 sequences against 788),
 * S^T = K Q^T with tiles of 64 rows and K's tiles in tensor memory (510, and
 * twice that for 128 rows).
 *
 * One block a SM, sixteen warps:
 *   warps 0-3   one query row a thread: Q to shared memory (f16), softmax of the
 *               S tiles from tensor memory, P back into tensor memory, output
 *   warps 4-7   unpack K, warps 8-11 V: a key row a lane, its codes loaded two
 *               128-key blocks ahead, written as f16 in the 128-byte swizzle
 *   warp  12    issues S(j) = Q K_j^T and then O += P(j-1) V_(j-1)
 *   warp  13    finds the unit after the next
 * (warps 4-15 give up registers to the softmax's, whose threads hold a row of S).
 * Tensor memory: S in two buffers of 128 columns (P overwrites the first half
 * of its own), O in 128.  Rounding as in fa_kv4_attn.cu: P in f16 only.
 * The units come from the same even split of the work, with the same merge.
 */
#include <atomic>
#include <cstdint>

#include "fa_kv4_units.cuh"
#include "fa_kv4_wide.cuh"
#include "fa_ptx.cuh"
#include "fa_tmem_io.cuh"

namespace {

using namespace fa::kv4;

constexpr int kRows = kWideRows;            // rows of a tile
constexpr int kBlockKeys = 128;
constexpr int kSoftmaxWarps = 4, kUnpackWarps = 4, kMmaWarp = kSoftmaxWarps + 2 * kUnpackWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;
// Registers a thread, of 512 for the four warpgroups.
constexpr int kSoftmaxRegs = 216, kUnpackRegs = 104, kOtherRegs = 88;
static_assert(kSoftmaxRegs + 2 * kUnpackRegs + kOtherRegs <= 4 * 128, "more than the launch has");
static_assert(kSoftmaxRegs >= 128 && kUnpackRegs <= 128 && kOtherRegs <= 128, "an increase has to be one, a decrease too");
constexpr uint32_t kTmemS = 0, kTmemO = 256;

template <int D>
struct WideCfg {
  static constexpr int kSlab = 128 * 128;                  // 128 rows x 64 f16 elements
  static constexpr int kTile = kSlab * (D / 64);           // 128 rows x D
  static constexpr int kQ = 0, kK = kTile, kV = 3 * kTile; // Q; two of K, two of V
  static constexpr int kSmem = 5 * kTile + 1024;           // (aligned to 1024 by hand)
  static constexpr uint32_t kIdescQK = fa::umma_idesc(0, false, 128, kBlockKeys);
  static constexpr uint32_t kIdescPV = fa::umma_idesc(0, true, 128, D);
};

// Barriers, each a phase an event: K / V buffer written, K / V buffer read, S
// ready, P ready, O updated with P and V of a buffer (all per buffer: a phase
// two blocks old is over when a block's S is there, one block old it need not be).
enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kODone = 12, kDrain = 14, kBarriers = 15 };

// Byte of element piece `piece` (8 elements of 16 bits) of row r in a tile of
// 128-byte rows, 128-byte swizzle, 64 elements a slab.
__device__ __forceinline__ uint32_t tile_at(int r, int piece) {
  return static_cast<uint32_t>((piece >> 3) * (128 * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// mbar_wait of a whole warp, with one answer: a warp that gives up does so as
// one, before its next tcgen05 instruction.  mbar_wait's try_wait may itself
// sleep for longer than this kernel's longest wait, so limits below kPollBelow,
// which a test of giving up sets, take an instantiation that polls (5 % slower).
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, const fa::WaitCtl& c) {
  const uint64_t t0 = fa::global_timer_ns();
  while (!fa::mbar_test_wait(bar, parity)) {
    if (*c.abort) return false;
    if (fa::global_timer_ns() - t0 > c.limit_ns) {
      atomicOr(c.err, fa::kErrTimeout);
      *c.abort = 1;
      return false;
    }
  }
  return true;
}
template <bool POLL>
__device__ __forceinline__ bool warp_wait_by(uint32_t bar, uint32_t parity, const fa::WaitCtl& c) {
  return __all_sync(0xffffffffu, POLL ? poll(bar, parity, c) : fa::mbar_wait(bar, parity, c));
}
constexpr uint64_t kPollBelow = 100000;

// One key row's codes and scales.
template <int D>
struct KeyRow {
  uint4 codes[D / 32];
  uint2 scales;
};

template <typename T, int D, bool POLL>
__global__ void __launch_bounds__(kThreads, 1) fa_kv4_wide_kernel(const __grid_constant__ AttnParams p, uint32_t* err, uint64_t limit_ns) {
  using C = WideCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t barriers[kBarriers];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, drain_flag;
  __shared__ float factors[2];            // of the scores, of V
  __shared__ int64_t scan[kThreads / 32];
  __shared__ Cursor cursor;
  __shared__ Unit units[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = (fa::smem_addr(smem_raw) + 1023u) & ~1023u;
  auto bar = [&](int i) { return fa::smem_addr(&barriers[i]); };
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      fa::mbar_init(bar(kKFull + s), kUnpackWarps);
      fa::mbar_init(bar(kVFull + s), kUnpackWarps);
      fa::mbar_init(bar(kKEmpty + s), 1);
      fa::mbar_init(bar(kVEmpty + s), 1);
      fa::mbar_init(bar(kSFull + s), 1);
      fa::mbar_init(bar(kPFull + s), kSoftmaxWarps);
      fa::mbar_init(bar(kODone + s), 1);
    }
    fa::mbar_init(bar(kDrain), 1);
    abort_flag = drain_flag = 0;
    fa::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    fa::tmem_alloc(fa::smem_addr(&tmem_slot), 512);
    fa::tmem_relinquish();
  }
  fa::tc_fence_before();
  __syncthreads();
  fa::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const fa::WaitCtl wc{limit_ns, err, &abort_flag};
  auto warp_wait = [](uint32_t b, uint32_t parity, const fa::WaitCtl& c) { return warp_wait_by<POLL>(b, parity, c); };
  fa::wait_for_stream();
  fa::let_next_start();

  if (!begin_units<kRows, kThreads>(p, scan, cursor, units, factors)) {
    if (warp == kMmaWarp) fa::tmem_dealloc(tmem, 512);
    return;
  }
  // The end of a unit, of all roles: does another follow?
  auto next = [&](bool ok, bool more) {
    __syncwarp();
    fa::tc_fence_before();
    const bool stop = __syncthreads_or(!ok || !more);
    fa::tc_fence_after();
    return !stop;
  };
  uint32_t done = 0;                        // 128-key blocks before this unit
  if (warp < kSoftmaxWarps) {
    fa::reg_alloc_inc<kSoftmaxRegs>();
    for (int turn = 0;; turn = (turn + 1) & 3) {
      const Unit& un = units[turn];
      const int key_begin = un.key_begin, key_end = un.key_end, head = un.head, rows = un.rows;
      const uint32_t n = static_cast<uint32_t>((key_end - key_begin + kBlockKeys - 1) / kBlockKeys);
      // ---- Q: a row a thread, f16 (bf16 rows shifted by a power of two)
      const int r = tid, row = un.row0 + r, tok = row / p.G;
      uint32_t q[D / 2];
#pragma unroll
      for (int i = 0; i < D / 2; ++i) q[i] = 0u;
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            ((un.q_row0 + tok) * p.H + static_cast<int64_t>(head) * p.G + (row - tok * p.G)) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = src[i];
          q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
        }
      }
      float rescale = factors[0];
      if (!std::is_same<T, __half>::value) {
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) top = max(top, max(q[i] & 0x7fffu, (q[i] >> 16) & 0x7fffu));
        const int e = min(max(static_cast<int>(top >> 7), 30), 254);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 + 127 - e) << 23);
        rescale *= __uint_as_float(static_cast<uint32_t>(e - 8) << 23);
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
          q[i] = pack_half(__uint_as_float(q[i] << 16) * up, __uint_as_float(q[i] & 0xffff0000u) * up);
      }
      const uint32_t flip = p.negate ? 0x80008000u : 0u;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        st_shared_v4(smem + C::kQ + tile_at(r, i), q[4 * i] ^ flip, q[4 * i + 1] ^ flip, q[4 * i + 2] ^ flip, q[4 * i + 3] ^ flip);
      asm volatile("bar.sync 1, 160;" ::: "memory");        // Q is there: the issuing warp joins

      // ---- softmax
      const float sl2 = fmaxf(rescale, 1e-30f);
      int see = un.k_len;
      if (p.causal == FA_CAUSAL_TOP_LEFT) see = min(see, tok + 1);
      if (p.causal == FA_CAUSAL_BOTTOM_RIGHT) see = min(see, tok + 1 + un.keys - un.q_len);
      const int limit = min(see, key_end);
      const bool active = warp * 32 < rows;
      const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
      const uint32_t tO = tmem + lanes + kTmemO;
      float m = -CUDART_INF_F, l = 0.0f;
      bool ok = true;
      for (uint32_t j = 0; j < n; ++j) {
        const uint32_t at = done + j, slot = at & 1;
        if (!warp_wait(bar(kSFull + slot), (at >> 1) & 1, wc)) { ok = false; break; }
        if (active) {
          fa::tc_fence_after();
          const uint32_t tS = tmem + lanes + kTmemS + slot * 128;
          const int key0 = key_begin + static_cast<int>(j) * kBlockKeys;
          const int lim = limit - key0;                      // columns this row sees
          const bool edge = __any_sync(0xffffffffu, lim < kBlockKeys);
          float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_x32(tS + c * 32, v[c]);
          fa::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_dep_x32(v[c]);
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= lim) v[c][i] = __float_as_uint(-CUDART_INF_F);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              tops[c] = fa::max3(tops[c], __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * sl2;
          if (__any_sync(0xffffffffu, top > m + kLag)) {     // move the maximum: rescale O
            const float to = fmaxf(m, top);
            const float a = to == -CUDART_INF_F ? 1.0f : fa::ex2(m - to);
            m = to;
            l *= a;
            if (j > 0) {
              if (!warp_wait(bar(kODone + (slot ^ 1u)), ((at - 1) >> 1) & 1, wc)) ok = false;
              fa::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_x32(tO + c * 32, o);
                fa::tmem_wait_ld();
                reg_dep_x32(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                tmem_st_x32(tO + c * 32, o);
              }
            }
          }
          const float sub = m == -CUDART_INF_F ? 0.0f : kBias - m;
          const uint64_t sl2s = fa::f2_pack(sl2, sl2), subs = fa::f2_pack(sub, sub);
          uint64_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = c * 64 + 2 * i;
              float x, y;
              fa::f2_unpack(fa::f2_fma(fa::f2_pack(__uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1])), sl2s, subs), x, y);
              x = fa::ex2(x);
              y = fa::ex2(y);
              sum[i & 3] = fa::f2_add(sum[i & 3], fa::f2_pack(x, y));
              pk[i] = pack_half(x, y);
            }
            tmem_st_x32(tS + c * 32, pk);
          }
          float x, y;
          fa::f2_unpack(fa::f2_add(fa::f2_add(sum[0], sum[1]), fa::f2_add(sum[2], sum[3])), x, y);
          l += x + y;
          fa::tmem_wait_st();
          fa::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) fa::mbar_arrive(bar(kPFull + slot));
      }

      // ---- output
      if (ok && active) {
        // the last block of each buffer
        for (uint32_t b = n > 2 ? n - 2 : 0; b < n; ++b) ok = warp_wait(bar(kODone + ((done + b) & 1)), ((done + b) >> 1) & 1, wc) && ok;
        fa::tc_fence_after();
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        const float lse = l == 0.0f ? -CUDART_INF_F : (m - kBias + log2f(l)) * 0.69314718055994530942f;
        const bool whole = un.piece < 0;
        const float mul = whole ? factors[1] * inv : inv;
        const int h = head * p.G + (row - tok * p.G);
        const int64_t to = whole ? (un.q_row0 + tok) * p.H + h : (blockIdx.x * int64_t(2) + un.piece) * kRows + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld_x32(tO + c * 32, o);
            fa::tmem_wait_ld();
            reg_dep_x32(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          // (a row without keys multiplies by 0 what other rows' blocks may have left)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = l == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[i]) * mul);
          if (ok && r < rows) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + to * D + c * 32);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  w[x] = pack16<T>(__uint_as_float(o[8 * i + 2 * x]), __uint_as_float(o[8 * i + 2 * x + 1]));
                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + to * D + c * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
        if (ok && r < rows) {
          if (whole) p.lse[static_cast<int64_t>(h) * p.total_q + un.q_row0 + tok] = lse;
          else p.part_lse[to] = lse;
        }
        fa::tc_fence_before();
      }
      if (tid == 0 && un.pieces > 0)
        p.meta[blockIdx.x] = Meta{un.q_row0, un.pieces, head * p.G, un.row0, rows};
      done += n;                            // all phases follow the blocks before this unit
      if (!next(ok, un.more)) break;
    }
  } else if (warp < kMmaWarp) {
    // ---- unpack: this lane's key row of each block, of K or of V
    fa::reg_alloc_dec<kUnpackRegs>();
    const int which = warp >= kSoftmaxWarps + kUnpackWarps;
    const int r = (warp - kSoftmaxWarps - which * kUnpackWarps) * 32 + lane;
    const int full = which ? kVFull : kKFull, empty = which ? kVEmpty : kKEmpty;
    const uint32_t tiles = smem + (which ? C::kV : C::kK);
    const int ps = p.cache.page_size;
    int key_begin, key_end, head;           // of the unit being loaded
    uint32_t n, table, last;
    // A step's page is looked up before it is known whether the step is there
    // (of the unit's last key then): no branch, so nothing waits for the page.
    // (Blocks ahead of the last key may be past 2^31: compared as unsigned numbers.)
    auto key_of = [&](uint32_t j) { return static_cast<int>(static_cast<uint32_t>(key_begin) + j * kBlockKeys + r); };
    auto page_of = [&](uint32_t j) {
      const int key = static_cast<int>(min(static_cast<uint32_t>(key_of(j)), last));
      return __ldg(p.block_table + (table + (p.page_shift >= 0 ? key >> p.page_shift : key / ps)));
    };
    auto fetch = [&](uint32_t j, int page, KeyRow<D>& k) {
      const int key = key_of(j);
      const int in_page = p.page_shift >= 0 ? key & (ps - 1) : key % ps;
      const uint32_t at = (static_cast<uint32_t>(page) * p.cache.H_kv + head) * ps + in_page;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) k.codes[i] = make_uint4(0u, 0u, 0u, 0u);
      k.scales = make_uint2(0u, 0u);
      if (static_cast<uint32_t>(key) < static_cast<uint32_t>(key_end) && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.cache.num_pages)) {
        const uint4* c = reinterpret_cast<const uint4*>(p.cache.codes[which] + static_cast<uint64_t>(at) * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) k.codes[i] = __ldg(c + i);
        const uint8_t* s = p.cache.scales[which] + static_cast<uint64_t>(at) * (D / 16);
        if (D == 128) k.scales = __ldg(reinterpret_cast<const uint2*>(s));
        else k.scales.x = __ldg(reinterpret_cast<const uint32_t*>(s));
      }
    };
    auto put = [&](const KeyRow<D>& k, uint32_t tile) {
      const uint32_t scale[2] = {k.scales.x, k.scales.y};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {k.codes[i].x, k.codes[i].y, k.codes[i].z, k.codes[i].w};
        const uint32_t two = scales_to_half((scale[i / 2] >> (16 * (i % 2))) & 0xffffu);   // of 32 elements
        const uint32_t s2[2] = {__byte_perm(two, 0u, 0x1010), __byte_perm(two, 0u, 0x3232)};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t h[4];
          codes_to_half(w[x], h);
#pragma unroll
          for (int y = 0; y < 4; ++y) h[y] = mul_half(h[y], s2[x / 2]);
          st_shared_v4(tile + tile_at(r, 4 * i + x), h[0], h[1], h[2], h[3]);
        }
      }
    };
    KeyRow<D> ring[2];
    int page;
    // A unit's first two blocks on their way: while the unit before it ends.
    auto begin = [&](const Unit& un) {
      key_begin = un.key_begin;
      key_end = un.key_end;
      last = max(key_end, 1) - 1;
      head = un.head;
      n = static_cast<uint32_t>((key_end - key_begin + kBlockKeys - 1) / kBlockKeys);
      table = static_cast<uint32_t>(un.s) * static_cast<uint32_t>(p.max_pages);
      fetch(0, page_of(0), ring[0]);
      fetch(1, page_of(1), ring[1]);
      page = page_of(2);
    };
    begin(units[0]);
    for (int turn = 0;; turn = (turn + 1) & 3) {
      bool ok = true;
      auto step = [&](uint32_t j, KeyRow<D>& k) {
        const uint32_t at = done + j, slot = at & 1;
        if (!warp_wait(bar(empty + slot), ((at >> 1) & 1) ^ 1u, wc)) { ok = false; return; }
        put(k, tiles + slot * C::kTile);
        fetch(j + 2, page, k);
        page = page_of(j + 3);
        __syncwarp();
        if (lane == 0) fa::mbar_arrive(bar(full + slot));
      };
      for (uint32_t j = 0; j < n && ok; j += 2) {
        step(j, ring[0]);
        if (j + 1 < n && ok) step(j + 1, ring[1]);
      }
      done += n;                            // all phases follow the blocks before this unit
      const bool more = units[turn].more;
      if (more) begin(units[(turn + 1) & 3]);
      if (!next(ok, more)) break;
    }
  } else {
    fa::reg_alloc_dec<kOtherRegs>();
    const bool leader = fa::elect_one();
    constexpr uint32_t hi = fa::umma_desc_hi_sw128(1024);
    const uint32_t q_lo = fa::umma_desc_lo(smem + C::kQ, 16);
    for (int turn = 0;; turn = (turn + 1) & 3) {
      const Unit& un = units[turn];
      const int key_begin = un.key_begin, key_end = un.key_end;
      const uint32_t n = static_cast<uint32_t>((key_end - key_begin + kBlockKeys - 1) / kBlockKeys);
      bool ok = true;
      if (warp == kMmaWarp) {
        // ---- products
        asm volatile("bar.sync 1, 160;" ::: "memory");        // Q
        fence_async_smem();
        for (uint32_t j = 0; j <= n && ok; ++j) {
          if (j < n) {
            const uint32_t at = done + j, slot = at & 1;
            ok = warp_wait(bar(kKFull + slot), (at >> 1) & 1, wc);
            if (!ok) break;
            fence_async_smem();
            fa::tc_fence_after();
            const uint32_t k_lo = fa::umma_desc_lo(smem + C::kK + slot * C::kTile, 16);
  #pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = static_cast<uint32_t>(((kk * 32 / 128) * C::kSlab + (kk * 32) % 128) >> 4);
              if (leader) fa::umma_ss_w<false>(tmem + kTmemS + slot * 128, q_lo + off, hi, k_lo + off, hi, C::kIdescQK, kk > 0);
            }
            fa::umma_commit_if(leader, bar(kSFull + slot));
            fa::umma_commit_if(leader, bar(kKEmpty + slot));
          }
          if (j > 0) {
            const uint32_t at = done + j - 1, slot = at & 1;
            ok = warp_wait(bar(kVFull + slot), (at >> 1) & 1, wc) && warp_wait(bar(kPFull + slot), (at >> 1) & 1, wc);
            if (!ok) break;
            fence_async_smem();
            fa::tc_fence_after();
            const uint32_t v_lo = fa::umma_desc_lo(smem + C::kV + slot * C::kTile, C::kSlab);
  #pragma unroll
            for (int kk = 0; kk < kBlockKeys / 16; ++kk)
              if (leader)
                fa::umma_ts_w<false>(tmem + kTmemO, tmem + kTmemS + slot * 128 + kk * 8, v_lo + static_cast<uint32_t>((kk * 16 * 128) >> 4), hi,
                                     C::kIdescPV, j > 1 || kk > 0);
            fa::umma_commit_if(leader, bar(kVEmpty + slot));
            fa::umma_commit_if(leader, bar(kODone + slot));
          }
        }
      } else if (warp == kMmaWarp + 1 && lane == 0 && un.more && units[(turn + 1) & 3].more) {
        next_unit<kRows>(p, cursor, units[(turn + 2) & 3]);
      }
      done += n;                            // all phases follow the blocks before this unit
      if (!next(ok, un.more)) break;
    }
    if (warp == kMmaWarp) {
      // Whichever role ended the block, products on their way, and their arrivals at
      // its barriers, end before its memory is freed.
      fa::umma_commit_if(leader, bar(kDrain));
      warp_wait(bar(kDrain), 0, fa::WaitCtl{2000000000ull, err, &drain_flag});
      fa::tmem_dealloc(tmem, 512);
    }
  }
}

template <typename T, int D, bool POLL>
cudaError_t launch_by(const AttnParams& p, int sms, uint32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  constexpr int smem = WideCfg<D>::kSmem;
  cudaError_t e = fa::allow_smem<fa_kv4_wide_kernel<T, D, POLL>>(smem);
  if (e != cudaSuccess) return e;
  const fa::Launch c(dim3(sms), kThreads, smem, stream);
  e = cudaLaunchKernelEx(&c.cfg, fa_kv4_wide_kernel<T, D, POLL>, p, err, limit_ns);
  if (e != cudaSuccess) return e;
  const fa::Launch mc(dim3(sms), kMergeWarps * 32, 0, stream);
  return cudaLaunchKernelEx(&mc.cfg, fa_kv4_merge_kernel<T, D, kRows>, p);
}
template <typename T, int D>
cudaError_t launch(const AttnParams& p, int sms, uint32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  return limit_ns < kPollBelow ? launch_by<T, D, true>(p, sms, err, limit_ns, stream)
                               : launch_by<T, D, false>(p, sms, err, limit_ns, stream);
}

}  // namespace

namespace fa {
namespace kv4 {
cudaError_t launch_wide(const AttnParams& p, int D, bool f16, int sms, uint32_t* err, uint64_t limit_ns, cudaStream_t stream) {
  if (f16) return D == 64 ? launch<__half, 64>(p, sms, err, limit_ns, stream) : launch<__half, 128>(p, sms, err, limit_ns, stream);
  return D == 64 ? launch<__nv_bfloat16, 64>(p, sms, err, limit_ns, stream) : launch<__nv_bfloat16, 128>(p, sms, err, limit_ns, stream);
}
}  // namespace kv4
}  // namespace fa
