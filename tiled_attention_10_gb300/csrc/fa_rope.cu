/*
 * fa_rope.cu -- fa_qk_norm_rope and its backward (formulas in include/fa_api.h):
 * RMS norm of each query and key head and the rotation by position, one pass
 * over the data.
 *
 * Bound by HBM: 8 or so operations a value against 4 bytes moved (forward; 6
 * backward).  So one read and one write of each value:
 *   - forward, a block takes a few tokens, works out their cosines and sines a
 *     pair a thread, and its warps walk the tokens' query and then key heads, 512
 *     bytes a step, the next step's loads under way in registers.  16384 tokens
 *     of 32 + 8 heads of 128 in bf16: 60 us (5.6 TB/s, 82 % of a plain copy);
 *   - backward, a warp takes tokens one after another (with few tokens, a part of
 *     one's heads); its rows of x and dy come by cp.async through a ring of steps
 *     in shared memory that runs on over heads and tokens: 91 us for the same
 *     tokens (5.5 TB/s, 81 %), 99 with loads ahead in registers, which hid no more
 *     than one step's time;
 *   - a head vector lies in D / 8 lanes (16 at D = 128, 8 at 64), so sums over
 *     a head are 4 or 3 shuffles; a lane holds both values of its rotation
 *     pairs (four elements of the first half and their partners of the second,
 *     two 8-byte accesses), so the rotation needs none.
 * The angle: a position times the frequency, in turns modulo 1, as a 64-bit
 * fixed-point product (wrapping is the reduction), so no position is too far
 * for 32-bit sine and cosine; in integers, as this GPU has few fp64 units.
 */
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa_api.h"
#include "fa_launch.cuh"

namespace {

constexpr int kFwdWarps = 8;          // warps of a block, forward
constexpr int kBwdWarps = 4;          // and backward
constexpr int kMaxPairs = 64;
constexpr int kBwdResident = 4;       // blocks of the backward an SM holds
constexpr int kBwdBlocks = 152 * kBwdResident;   // backward grid: rows of the weight gradients' partial sums

struct RopeParams {
  const void* x[2];        // q, k: the forward's inputs
  const void* dy[2];       // backward: gradients of the outputs
  void* out[2];            // outputs, or gradients of the inputs
  const void* weight[2];   // [D] or null
  fa_strides_t st_x[2], st_dy[2], st_out[2];
  const int32_t* positions;
  const double* inv_freq;
  float* partial;          // backward: [blocks, 2, D] weight gradient partials, or null
  int64_t B, S;
  int32_t heads[2];
  int32_t share;           // warps that share a token
  int32_t rot;             // rotated elements
  float eps;
  uint8_t axis[kMaxPairs]; // axis of each pair
};

// A lane's 8 values of a row: two runs of 4 elements.
struct Raw {
  uint2 lo, hi;
};
template <typename T> struct Pack;
template <> struct Pack<__half> {
  static __device__ __forceinline__ void load2(uint32_t w, float& a, float& b) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = t.x; b = t.y;
  }
  static __device__ __forceinline__ uint32_t store2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ __half one(float x) { return __float2half_rn(x); }
};
template <> struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ void load2(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t store2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float x) { return __float2bfloat16_rn(x); }
};
// Two fp32 values in a register pair: one instruction for both (the issue slots
// are what comes closest to HBM's time here).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float both(F2 x) {
  const float2 v = split(x);
  return v.x + v.y;
}

// A lane's 8 values as pairs: lo 0 1, lo 2 3, hi 0 1, hi 2 3.
template <typename T>
__device__ __forceinline__ void unpack(const Raw& r, F2 (&f)[4]) {
  const uint32_t w[4] = {r.lo.x, r.lo.y, r.hi.x, r.hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    Pack<T>::load2(w[i], a, b);
    f[i] = f2(a, b);
  }
}

// Which elements a lane holds: 4 from lo and 4 from hi.  Interleaved pairs are
// neighbours, so a run of 8; else the pairs (i, i + rot / 2) of 4 values of i,
// and runs of 8 of what is not rotated.
struct Elements {
  int lo, hi, pair;     // pair: the first of the lane's pairs, or -1
};
template <bool INTERLEAVED>
__device__ __forceinline__ Elements elements(int rot, int sub) {
  if (INTERLEAVED || sub * 8 >= rot) return Elements{sub * 8, sub * 8 + 4, sub * 8 < rot ? sub * 4 : -1};
  return Elements{sub * 4, rot / 2 + sub * 4, sub * 4};
}
__device__ __forceinline__ Raw load_row(const uint16_t* row, const Elements& e) {
  return Raw{*reinterpret_cast<const uint2*>(row + e.lo), *reinterpret_cast<const uint2*>(row + e.hi)};
}
template <typename T>
__device__ __forceinline__ void store_row(uint16_t* row, const Elements& e, const F2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = split(f[i]);
    w[i] = Pack<T>::store2(v.x, v.y);
  }
  *reinterpret_cast<uint2*>(row + e.lo) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + e.hi) = make_uint2(w[2], w[3]);
}

// Sum over the LANES lanes that hold one head vector.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A frequency in radians as a fraction of a turn in units of 2^-64, modulo a
// turn.  With f = m 2^(e - 63), m in [2^63, 2^64), and K = 2^66 / (2 pi):
// f / (2 pi) 2^64 = (m K 2^-64) 2^(e - 1).
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7ff) - 1023;
  const uint64_t m = (bits << 11) | (1ull << 63), K = 0xA2F9836E4E44152Aull;
  const uint64_t hi = __umul64hi(m, K);
  uint64_t fixed = 0ull;               // zero and tiny; 2^64 and more, infinite and NaN
  if (e <= 1 && e > -63) fixed = hi >> (1 - e);
  if (e > 1 && e < 64) fixed = (hi << (e - 1)) | ((m * K) >> (65 - e));
  return (bits >> 63) ? 0ull - fixed : fixed;
}

// cos and sin of pair i of a token.
__device__ __forceinline__ float2 angle(const RopeParams& p, int64_t token, int i) {
  const int64_t pos = p.positions[p.axis[i] * (p.B * p.S) + token];
  // The product modulo 2^64 is the angle modulo a turn; its top half as a
  // signed number counts half turns of 2^-31.
  const int32_t half_turns = static_cast<int32_t>((static_cast<uint64_t>(pos) * turns_of(p.inv_freq[i])) >> 32);
  float s, c;
  sincospif(static_cast<float>(half_turns) * 4.656612873077392578125e-10f, &s, &c);
  return make_float2(c, s);
}

// The cosines and sines of a block's tokens, a pair a thread.
__device__ __forceinline__ void block_angles(const RopeParams& p, int64_t token0, float2 (*table)[kMaxPairs]) {
  const int i = threadIdx.x % kMaxPairs;
  if (i >= p.rot / 2) return;
  for (int k = threadIdx.x / kMaxPairs; k < kFwdWarps / p.share; k += kFwdWarps * 32 / kMaxPairs)
    if (token0 + k < p.B * p.S) table[k][i] = angle(p, token0 + k, i);
}

// The cosines and sines of a token, two pairs a lane of the warp.
__device__ __forceinline__ void warp_angles(const RopeParams& p, int64_t token, float2* table, int lane) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 32 * j < p.rot / 2) table[lane + 32 * j] = angle(p, token, lane + 32 * j);
}

// A lane's four pairs: cosines and sines (turned back with direction -1).  A lane
// without pairs turns nothing: by a cosine of 1 and a sine of 0, an infinity would
// make its neighbour NaN.  (PART: there may be such lanes.  Asked in every kernel,
// that cost the full rotations 2 to 4 %.)
struct Turn {
  F2 cs[2], sn[2], minus_sn[2];     // of pairs 0 1 and 2 3
};
__device__ __forceinline__ Turn load_turn(const float2* table, const Elements& e, float direction) {
  Turn t;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 a = e.pair >= 0 ? table[e.pair + 2 * j] : make_float2(1.0f, 0.0f);
    const float2 b = e.pair >= 0 ? table[e.pair + 2 * j + 1] : make_float2(1.0f, 0.0f);
    t.cs[j] = f2(a.x, b.x);
    t.sn[j] = f2(direction * a.y, direction * b.y);
    t.minus_sn[j] = f2(-direction * a.y, -direction * b.y);
  }
  return t;
}
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(F2 (&y)[4], const Turn& t) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (INTERLEAVED) {                // y[2 j] and y[2 j + 1] are pairs 2 j and 2 j + 1
      const float2 c = split(t.cs[j]), s = split(t.sn[j]), u = split(y[2 * j]), v = split(y[2 * j + 1]);
      y[2 * j] = f2(u.x * c.x - u.y * s.x, u.y * c.x + u.x * s.x);
      y[2 * j + 1] = f2(v.x * c.y - v.y * s.y, v.y * c.y + v.x * s.y);
    } else {
      const F2 a = y[j], b = y[j + 2];
      y[j] = fma2(b, t.minus_sn[j], a * t.cs[j]);
      y[j + 2] = fma2(a, t.sn[j], b * t.cs[j]);
    }
  }
}

// Both weight vectors as fp32 in shared memory (ones where there is none), by the block.
template <int WARPS, typename T, int D>
__device__ __forceinline__ void block_weights(const RopeParams& p, float (*table)[D]) {
  for (int i = threadIdx.x; i < 2 * D; i += WARPS * 32) {
    const T* src = static_cast<const T*>(p.weight[i / D]);
    table[i / D][i % D] = src ? static_cast<float>(src[i % D]) : 1.0f;
  }
}
__device__ __forceinline__ void load_weight(const float* table, const Elements& e, F2 (&w)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(table + e.lo), b = *reinterpret_cast<const float4*>(table + e.hi);
  w[0] = f2(a.x, a.y); w[1] = f2(a.z, a.w);
  w[2] = f2(b.x, b.y); w[3] = f2(b.z, b.w);
}

__device__ __forceinline__ int64_t row_base(const fa_strides_t& st, int64_t b, int64_t s) {
  return b * st.batch + s * st.seq;
}

// A warp's heads of one kind, [first, last): its part of the token's list of
// query heads and then key heads, PER at a time.
template <int PER>
__device__ __forceinline__ void heads_of(const RopeParams& p, int part, int which, int& first, int& last) {
  const int nq = (p.heads[0] + PER - 1) / PER, nk = (p.heads[1] + PER - 1) / PER;
  const int a = (nq + nk) * part / p.share, b = (nq + nk) * (part + 1) / p.share;
  first = PER * (which ? max(a - nq, 0) : min(a, nq));
  last = min(PER * (which ? max(b - nq, 0) : min(b, nq)), p.heads[which]);
}

constexpr int kFwdRows = 2;   // rows a lane loads ahead

template <typename T, int D, bool INTERLEAVED, bool NORM, bool PART>
__global__ void __launch_bounds__(kFwdWarps * 32, 4) fa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;   // lanes a head, heads a warp at once
  __shared__ float2 table[kFwdWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  fa::wait_for_stream();
  fa::let_next_start();
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * (kFwdWarps / p.share);
  const int mine = warp / p.share, part = warp % p.share;
  const bool real = token0 + mine < p.B * p.S;
  const uint32_t token = real ? static_cast<uint32_t>(token0 + mine) : 0u;
  const uint32_t b = token / static_cast<uint32_t>(p.S), s = token - b * static_cast<uint32_t>(p.S);
  const Elements e = elements<INTERLEAVED>(p.rot, sub);

  Turn t;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    int first, last;
    heads_of<PER>(p, part, which, first, last);
    if (!real) last = 0;
    const int64_t x_step = p.st_x[which].head, out_step = p.st_out[which].head;
    const uint16_t* src = static_cast<const uint16_t*>(p.x[which]) + row_base(p.st_x[which], b, s);
    uint16_t* dst = static_cast<uint16_t*>(p.out[which]) + row_base(p.st_out[which], b, s);
    Raw raw[kFwdRows];
    auto load = [&](int h0) {
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        const int h = h0 + i * PER + slot;
        raw[i] = Raw{};
        if (h < last) raw[i] = load_row(src + h * x_step, e);
      }
    };
    load(first);
    if (which == 0) {
      if (NORM) block_weights<kFwdWarps, T, D>(p, weights);
      block_angles(p, token0, table);
      __syncthreads();
      t = load_turn(table[mine], e, 1.0f);
    }
    F2 w[4];
    if (NORM) load_weight(weights[which], e, w);
    for (int h0 = first; h0 < last; h0 += PER * kFwdRows) {
      Raw now[kFwdRows];
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) now[i] = raw[i];
      load(h0 + PER * kFwdRows);
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        const int h = h0 + i * PER + slot;
        F2 y[4];
        unpack<T>(now[i], y);
        if (NORM) {
          const F2 ss = fma2(y[3], y[3], fma2(y[2], y[2], fma2(y[1], y[1], y[0] * y[0])));
          const float r = rsqrtf(head_sum<LANES>(both(ss)) * (1.0f / D) + p.eps);
          const F2 rr = f2(r, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = y[j] * rr * w[j];
        }
        if (!PART || e.pair >= 0) turn<INTERLEAVED>(y, t);
        if (h < last) store_row<T>(dst + h * out_step, e, y);
      }
    }
  }
}

// A warp's work: tasks id, id + step, ... below tasks; task = (token, part of
// its steps).  A token's steps: PER query heads each, then PER key heads each.
template <int PER>
struct Walk {
  int64_t task, step, tasks;
  int32_t at, end, nq;          // step in the token, the task's end, steps of query heads
  uint32_t b, s, token;

  __device__ __forceinline__ Walk(const RopeParams& p) {
    step = static_cast<int64_t>(gridDim.x) * kBwdWarps;
    tasks = p.B * p.S * p.share;
    nq = (p.heads[0] + PER - 1) / PER;
    task = static_cast<int64_t>(blockIdx.x) * kBwdWarps + threadIdx.x / 32 - step;
    at = end = 0;
    advance_task(p);
  }
  __device__ __forceinline__ bool more() const { return task < tasks; }
  // The next task that has steps (a part may have none).
  __device__ __forceinline__ void advance_task(const RopeParams& p) {
    const int n = nq + (p.heads[1] + PER - 1) / PER;
    do {
      task += step;
      if (task >= tasks) return;
      token = static_cast<uint32_t>(task) / static_cast<uint32_t>(p.share);
      const int part = static_cast<int>(static_cast<uint32_t>(task) - token * p.share);
      at = n * part / p.share;
      end = n * (part + 1) / p.share;
    } while (at >= end);
    b = token / static_cast<uint32_t>(p.S);
    s = token - b * static_cast<uint32_t>(p.S);
  }
  __device__ __forceinline__ int kind() const { return at >= nq; }
  __device__ __forceinline__ int head() const { return (at >= nq ? at - nq : at) * PER; }
};

constexpr int kStepBytes = 512;         // PER heads of one tensor

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {   // zeros behind `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The copies' side of a walk: steps of dy and, where X, x into ring stages.
// Addresses move on by a head stride; they are worked out where a run of one kind
// of heads begins.
template <int D, bool X>
struct Feed {
  static constexpr int LANES = D / 8, PER = 32 / LANES;
  Walk<PER> w;
  const uint16_t *x, *dy;
  int h, h_end, left;             // this lane's head, heads, steps left of the run (0: none)

  __device__ __forceinline__ Feed(const RopeParams& p, int lane) : w(p), x(nullptr), dy(nullptr), h(0), h_end(0), left(0) {
    begin_run(p, lane);
  }
  __device__ __forceinline__ void begin_run(const RopeParams& p, int lane) {
    if (!w.more()) return;
    const int k = w.kind();
    h = w.head() + lane / LANES;
    h_end = p.heads[k];
    left = k ? w.end - w.at : min(w.end, w.nq) - w.at;
    w.at += left;
    const int64_t e = (lane % LANES) * 8;
    if (X) x = static_cast<const uint16_t*>(p.x[k]) + row_base(p.st_x[k], w.b, w.s) + h * p.st_x[k].head + e;
    dy = static_cast<const uint16_t*>(p.dy[k]) + row_base(p.st_dy[k], w.b, w.s) + h * p.st_dy[k].head + e;
  }
  // One step (nothing once the work is all under way), as a group of its own.
  __device__ __forceinline__ void step(const RopeParams& p, uint32_t stage, int lane) {
    if (left > 0) {
      const int k = w.at > w.nq;
      const int bytes = h < h_end ? 16 : 0;
      copy16(stage + lane * 16, bytes ? dy : static_cast<const uint16_t*>(p.dy[0]), bytes);
      dy += p.st_dy[k].head * PER;
      if (X) {
        copy16(stage + kStepBytes + lane * 16, bytes ? x : static_cast<const uint16_t*>(p.x[0]), bytes);
        x += p.st_x[k].head * PER;
      }
      h += PER;
      if (--left == 0) {
        if (w.at >= w.end) w.advance_task(p);
        begin_run(p, lane);
      }
    }
    copies_commit();
  }
};

constexpr int kStages = 7;

template <typename T, int D, bool INTERLEAVED, bool NORM, bool PART>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdResident) fa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  constexpr int kBytes = 2 * kStepBytes;
  __shared__ __align__(128) uint8_t ring[kBwdWarps][kStages * kBytes];
  __shared__ float2 tables[kBwdWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  fa::wait_for_stream();
  fa::let_next_start();
  const Elements e = elements<INTERLEAVED>(p.rot, sub);
  const uint32_t stages = static_cast<uint32_t>(__cvta_generic_to_shared(ring[warp]));
  Feed<D, NORM> ahead(p, lane);
  Walk<PER> now(p);
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) ahead.step(p, stages + i * kBytes, lane);
  if (NORM) {
    block_weights<kBwdWarps, T, D>(p, weights);
    __syncthreads();
  }
  F2 dw[2][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j / 4][j % 4] = f2(0.0f, 0.0f);
  int stage = 0;
  while (now.more()) {
    warp_angles(p, now.token, tables[warp], lane);
    __syncwarp();
    const Turn t = load_turn(tables[warp], e, -1.0f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {                 // query heads, key heads
      const int run = k ? now.end - now.at : min(now.end, now.nq) - now.at;
      if (run <= 0) continue;
      const int h_end = p.heads[k];
      F2 w[4];
      if (NORM) load_weight(weights[k], e, w);
      const int64_t out_step = p.st_out[k].head;
      uint16_t* const dst = static_cast<uint16_t*>(p.out[k]) + row_base(p.st_out[k], now.b, now.s);
      int h = now.head() + slot;
      for (int i = 0; i < run; ++i, h += PER) {
        copies_wait<kStages - 2>();
        __syncwarp();
        const uint8_t* const st = ring[warp] + stage * kBytes;
        F2 g[4], xv[4];
        unpack<T>(load_row(reinterpret_cast<const uint16_t*>(st) + slot * D, e), g);
        if (NORM) unpack<T>(load_row(reinterpret_cast<const uint16_t*>(st + kStepBytes) + slot * D, e), xv);
        ahead.step(p, stages + (stage == 0 ? kStages - 1 : stage - 1) * kBytes, lane);
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if (!PART || e.pair >= 0) turn<INTERLEAVED>(g, t);
        if (NORM) {
          F2 u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = g[j] * w[j];
          const F2 ss = fma2(xv[3], xv[3], fma2(xv[2], xv[2], fma2(xv[1], xv[1], xv[0] * xv[0])));
          const F2 dot = fma2(u[3], xv[3], fma2(u[2], xv[2], fma2(u[1], xv[1], u[0] * xv[0])));
          const float r = rsqrtf(head_sum<LANES>(both(ss)) * (1.0f / D) + p.eps);
          const float c = head_sum<LANES>(both(dot)) * (1.0f / D) * r * r;
          // h < h_end only: a lane without a row holds zeros, which add
          // nothing to dw unless r is infinite (0 * inf)
          if (h < h_end) {
            const F2 rr = f2(r, r), cc = f2(-c, -c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dw[k][j] = fma2(g[j] * rr, xv[j], dw[k][j]);
              g[j] = rr * fma2(xv[j], cc, u[j]);
            }
          }
        }
        if (h < h_end) store_row<T>(dst + h * out_step, e, g);
      }
      now.at += run;
    }
    now.advance_task(p);
    __syncwarp();                                 // the table has been read
  }

  if (NORM && p.partial) {
    // The block's sums in a fixed order: lanes of the same elements, then warps
    // (in the rings' place: all copies have landed).
    copies_wait<0>();
    __syncthreads();
    float (*sums)[2][D] = reinterpret_cast<float (*)[2][D]>(&ring[0][0]);
    static_assert(sizeof(ring) >= kBwdWarps * 2 * D * 4, "the sums fit in the rings");
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 two = split(dw[which][j / 2]);
        float v = j % 2 ? two.y : two.x;
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (slot == 0) sums[warp][which][j < 4 ? e.lo + j : e.hi + j - 4] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kBwdWarps * 32) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kBwdWarps; ++k) v += (&sums[k][0][0])[i];
      p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
    }
  }
}

// Weight gradients: element i of both vectors over the blocks' partial sums,
// 32 threads an element; 2 D / 32 blocks of 1024 threads.  Bound by latency: 6.5
// us for 608 blocks' sums at D = 128, the next call's first blocks beside it.
template <typename T>
__global__ void __launch_bounds__(1024) fa_rope_dw_kernel(const float* partial, int blocks, int D,
                                                          T* dwq, T* dwk) {
  __shared__ float sums[32][33];
  fa::wait_for_stream();
  fa::let_next_start();
  const int e = threadIdx.x & 31, k = threadIdx.x >> 5;
  const float* src = partial + blockIdx.x * 32 + e;     // element of 2 D
  float v = 0.0f;
#pragma unroll 4
  for (int r = k; r < blocks; r += 32) v += src[static_cast<int64_t>(r) * 2 * D];
  sums[k][e] = v;
  __syncthreads();
  v = sums[e][k];                                       // warp k: element k
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int i = blockIdx.x * 32 + k;
  T* out = i < D ? dwq : dwk;
  if (e == 0 && out) out[i < D ? i : i - D] = Pack<T>::one(v);
}

bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Last byte + 1 of a tensor of 16-bit elements.
uintptr_t end_of(const void* p, const fa_strides_t& st, int64_t B, int64_t H, int64_t S, int64_t D) {
  return reinterpret_cast<uintptr_t>(p) +
         2 * static_cast<uintptr_t>((B - 1) * st.batch + (H - 1) * st.head + (S - 1) * st.seq + D);
}
bool same(const fa_strides_t& a, const fa_strides_t& b) {
  return a.batch == b.batch && a.head == b.head && a.seq == b.seq;
}

struct Tensor {
  const void* p;
  fa_strides_t st;
  int64_t heads;
};
// Do A's rows (at sum of i_k stride_k) and B's (at d + sum of j_k stride_k)
// share elements, each row D wide?  Dimensions from the largest stride down;
// at each only the few index differences that bring the inner spans together
// are followed.
struct Dim {
  int64_t stride, na, nb;
};
bool rows_meet(int64_t d, const Dim* dim, int n, int64_t D) {
  if (n == 0) return d > -D && d < D;
  int64_t ea = D, eb = D;
  for (int k = 1; k < n; ++k) {
    ea += (dim[k].na - 1) * dim[k].stride;
    eb += (dim[k].nb - 1) * dim[k].stride;
  }
  // d + delta * stride in (-eb, ea), delta = j - i
  const double s = static_cast<double>(dim[0].stride);
  int64_t lo = static_cast<int64_t>(std::floor((-eb - d) / s)), hi = static_cast<int64_t>(std::ceil((ea - d) / s));
  lo = std::max(lo, -(dim[0].na - 1));
  hi = std::min(hi, dim[0].nb - 1);
  if (hi - lo > 64) return true;
  for (int64_t t = lo; t <= hi; ++t) {
    const int64_t e = d + t * dim[0].stride;
    if (e > -eb && e < ea && rows_meet(e, dim + 1, n - 1, D)) return true;
  }
  return false;
}
// Two tensors share memory.  Views of one buffer with the same strides (a
// fused projection's q and k) are told apart row by row; for others the spans
// decide.
bool meet(const Tensor& a, const Tensor& b, int64_t B, int64_t S, int64_t D) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  if (a0 >= end_of(b.p, b.st, B, b.heads, S, D) || b0 >= end_of(a.p, a.st, B, a.heads, S, D))
    return false;
  const int64_t sa[3] = {a.st.batch, a.st.head, a.st.seq}, sb[3] = {b.st.batch, b.st.head, b.st.seq};
  const int64_t na[3] = {B, a.heads, S}, nb[3] = {B, b.heads, S};
  Dim dim[3];
  int n = 0;
  for (int k = 0; k < 3; ++k) {
    if (na[k] == 1 && nb[k] == 1) continue;
    if (na[k] > 1 && nb[k] > 1 && sa[k] != sb[k]) return true;
    dim[n++] = Dim{na[k] > 1 ? sa[k] : sb[k], na[k], nb[k]};
  }
  std::sort(dim, dim + n, [](const Dim& x, const Dim& y) { return x.stride > y.stride; });
  return rows_meet(static_cast<int64_t>(b0 - a0) / 2, dim, n, D);
}

fa_status_t check_common(int64_t B, int64_t S, int64_t H, int64_t H_kv, int64_t D, int64_t rot,
                         int64_t n_axes, const uint8_t* pair_axis, const int32_t* positions,
                         const double* inv_freq, const void* qw, const void* kw, int norm,
                         float eps, fa_dtype_t dtype) {
  if (B < 0 || S < 0 || H < 1 || H_kv < 1 || D < 1 || rot < 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP8E4M3)
    return FA_ERR_INVALID_ARG;
  if (!norm && rot == 0) return FA_ERR_INVALID_ARG;
  if (!norm && (qw || kw)) return FA_ERR_INVALID_ARG;
  if (norm && !(std::isfinite(eps) && eps >= 0.0f)) return FA_ERR_INVALID_ARG;
  if (rot > 0 && (!inv_freq || (!positions && B > 0 && S > 0))) return FA_ERR_INVALID_ARG;
  if (rot > D) return FA_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > 4) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (rot % 16 != 0 || dtype == FA_DTYPE_FP8E4M3) return FA_ERR_UNSUPPORTED;
  if (pair_axis)
    for (int64_t i = 0; i < rot / 2; ++i)
      if (pair_axis[i] >= n_axes) return FA_ERR_INVALID_ARG;
  if (H > (1 << 20) || H_kv > (1 << 20)) return FA_ERR_UNSUPPORTED;
  if (B > 0 && S > 0 && S > ((int64_t(1) << 31) - 1) / B) return FA_ERR_UNSUPPORTED;
  if (off(positions, 4) || off(inv_freq, 8) || off(qw, 2) || off(kw, 2)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa_status_t check_tensors(const Tensor* t, int n) {
  for (int i = 0; i < n; ++i) {
    const int64_t v[3] = {t[i].st.batch, t[i].st.head, t[i].st.seq};
    for (int64_t x : v) {
      if (x < 1) return FA_ERR_INVALID_ARG;
      if (x % 8 != 0) return FA_ERR_MISALIGNED;
      if (x > (int64_t(1) << 38)) return FA_ERR_UNSUPPORTED;
    }
    if (off(t[i].p, 16)) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

void fill(RopeParams& p, const int32_t* positions, const double* inv_freq, int64_t B, int64_t S,
          int64_t H, int64_t H_kv, int64_t rot, const uint8_t* pair_axis, float eps,
          const void* qw, const void* kw) {
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.B = B; p.S = S;
  p.heads[0] = static_cast<int32_t>(H);
  p.heads[1] = static_cast<int32_t>(H_kv);
  p.rot = static_cast<int32_t>(rot);
  p.eps = eps;
  p.weight[0] = qw; p.weight[1] = kw;
  if (pair_axis) std::memcpy(p.axis, pair_axis, static_cast<size_t>(rot / 2));
}

// Warps that share a token: more while the tokens alone would not give each of
// 152 SMs its 32 warps.  At 16384 tokens, 32 + 8 heads of 128:
// forward 60.0 us with one, 60.7 with two, 74.7 with four.
int fwd_share(int64_t tokens) {
  return tokens >= 152 * 64 ? 1 : tokens >= 152 * 16 ? 2 : tokens >= 152 * 8 ? 4 : 8;
}

// Backward: parts a token's steps are cut into, so that there are tasks for all
// warps of the grid: as few as that takes, two steps each at least (and steps *
// parts a 32-bit number: a million heads a token are allowed).
int bwd_share(int64_t tokens, int64_t steps) {
  const int64_t want = (int64_t(kBwdBlocks) * kBwdWarps + tokens - 1) / tokens;
  return static_cast<int>(std::max<int64_t>(1, std::min({want, (steps + 1) / 2, INT32_MAX / steps})));
}
int64_t steps_of(int64_t H, int64_t H_kv, int64_t D) {
  const int64_t per = 256 / D;
  return (H + per - 1) / per + (H_kv + per - 1) / per;
}

template <typename T, int D, bool PART>
cudaError_t launch_fwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, cudaStream_t stream) {
  const fa::Launch c(dim3(static_cast<unsigned>(grid)), kFwdWarps * 32, 0, stream);
  if (interleaved)
    return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, true, true, PART>, p)
                : cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, true, false, PART>, p);
  return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, false, true, PART>, p)
              : cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, false, false, PART>, p);
}
template <typename T, int D>
cudaError_t launch_fwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, cudaStream_t stream) {
  return p.rot < D ? launch_fwd<T, D, true>(p, interleaved, norm, grid, stream)
                   : launch_fwd<T, D, false>(p, interleaved, norm, grid, stream);
}

template <typename T, int D, bool PART>
cudaError_t launch_bwd_rows(const RopeParams& p, bool interleaved, bool norm, int64_t grid, cudaStream_t stream) {
  const fa::Launch c(dim3(static_cast<unsigned>(grid)), kBwdWarps * 32, 0, stream);
  if (interleaved)
    return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, true, true, PART>, p)
                : cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, true, false, PART>, p);
  return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, false, true, PART>, p)
              : cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, false, false, PART>, p);
}
template <typename T, int D>
cudaError_t launch_bwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, void* dwq,
                       void* dwk, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (grid > 0)
    e = p.rot < D ? launch_bwd_rows<T, D, true>(p, interleaved, norm, grid, stream)
                  : launch_bwd_rows<T, D, false>(p, interleaved, norm, grid, stream);
  if (e != cudaSuccess || !(dwq || dwk)) return e;
  const fa::Launch c(dim3(2 * D / 32), 1024, 0, stream);
  return cudaLaunchKernelEx(&c.cfg, fa_rope_dw_kernel<T>, static_cast<const float*>(p.partial),
                            static_cast<int>(grid), D, static_cast<T*>(dwq), static_cast<T*>(dwk));
}

size_t bwd_workspace(int64_t D) { return static_cast<size_t>(kBwdBlocks) * 2 * D * 4; }

}  // namespace

extern "C" {

fa_status_t fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                            const void* q_weight, const void* k_weight, const int32_t* positions,
                            const double* inv_freq, int64_t B, int64_t S, int64_t H, int64_t H_kv,
                            int64_t D, int64_t rot_dim, int64_t n_axes, const uint8_t* pair_axis,
                            int interleaved, int norm, float eps, const fa_strides_t* strides,
                            fa_dtype_t dtype, cudaStream_t stream) {
  if (!strides) return FA_ERR_INVALID_ARG;
  fa_status_t st = check_common(B, S, H, H_kv, D, rot_dim, n_axes, pair_axis, positions, inv_freq,
                                q_weight, k_weight, norm, eps, dtype);
  if (st != FA_OK) return st;
  if (B == 0 || S == 0) return FA_OK;
  if (!q || !k || !q_out || !k_out) return FA_ERR_INVALID_ARG;
  const Tensor t[4] = {{q, strides[0], H}, {k, strides[1], H_kv}, {q_out, strides[2], H}, {k_out, strides[3], H_kv}};
  st = check_tensors(t, 4);
  if (st != FA_OK) return st;
  for (int o = 2; o < 4; ++o)
    for (int i = 0; i < o; ++i) {
      if (i == o - 2 && t[i].p == t[o].p && same(t[i].st, t[o].st)) continue;   // in place
      if (meet(t[i], t[o], B, S, D)) return FA_ERR_INVALID_ARG;
    }

  RopeParams p = {};
  p.x[0] = q; p.x[1] = k;
  p.out[0] = q_out; p.out[1] = k_out;
  for (int i = 0; i < 2; ++i) { p.st_x[i] = strides[i]; p.st_out[i] = strides[2 + i]; }
  fill(p, positions, inv_freq, B, S, H, H_kv, rot_dim, pair_axis, eps, q_weight, k_weight);
  p.share = fwd_share(B * S);
  const int per_block = kFwdWarps / p.share;
  const int64_t grid = (B * S + per_block - 1) / per_block;
  cudaError_t e;
  if (dtype == FA_DTYPE_F16)
    e = D == 64 ? launch_fwd<__half, 64>(p, interleaved, norm, grid, stream)
                : launch_fwd<__half, 128>(p, interleaved, norm, grid, stream);
  else
    e = D == 64 ? launch_fwd<__nv_bfloat16, 64>(p, interleaved, norm, grid, stream)
                : launch_fwd<__nv_bfloat16, 128>(p, interleaved, norm, grid, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_qk_norm_rope_bwd_workspace_size(int64_t D, size_t* workspace_bytes) {
  if (!workspace_bytes || D < 1) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  *workspace_bytes = bwd_workspace(D);
  return FA_OK;
}

fa_status_t fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                                const void* k, void* dq, void* dk, const void* q_weight,
                                const void* k_weight, void* dq_weight, void* dk_weight,
                                const int32_t* positions, const double* inv_freq, int64_t B,
                                int64_t S, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                                int64_t n_axes, const uint8_t* pair_axis, int interleaved, int norm,
                                float eps, const fa_strides_t* strides, fa_dtype_t dtype,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!strides) return FA_ERR_INVALID_ARG;
  fa_status_t st = check_common(B, S, H, H_kv, D, rot_dim, n_axes, pair_axis, positions, inv_freq,
                                q_weight, k_weight, norm, eps, dtype);
  if (st != FA_OK) return st;
  const bool want_dw = dq_weight || dk_weight;
  if (!norm && want_dw) return FA_ERR_INVALID_ARG;
  if (off(dq_weight, 2) || off(dk_weight, 2)) return FA_ERR_MISALIGNED;
  if (want_dw) {
    if (!workspace || workspace_bytes < bwd_workspace(D)) return FA_ERR_INVALID_ARG;
    if (off(workspace, 256)) return FA_ERR_MISALIGNED;
  }
  const bool empty = B == 0 || S == 0;
  if (!empty) {
    if (!dq_out || !dk_out || !dq || !dk || (norm && (!q || !k))) return FA_ERR_INVALID_ARG;
    const Tensor t[6] = {{dq_out, strides[0], H}, {dk_out, strides[1], H_kv}, {dq, strides[4], H},
                         {dk, strides[5], H_kv}, {q, strides[2], H}, {k, strides[3], H_kv}};
    st = check_tensors(t, norm ? 6 : 4);
    if (st != FA_OK) return st;
    for (int o = 2; o < 4; ++o)
      for (int i = 0; i < (norm ? 6 : 4); ++i) {
        if (i == o || (i == 3 && o == 2)) continue;
        if (i == o - 2 && t[i].p == t[o].p && same(t[i].st, t[o].st)) continue;  // in place
        if (meet(t[i], t[o], B, S, D)) return FA_ERR_INVALID_ARG;
      }
  }

  RopeParams p = {};
  p.x[0] = q; p.x[1] = k;
  p.dy[0] = dq_out; p.dy[1] = dk_out;
  p.out[0] = dq; p.out[1] = dk;
  for (int i = 0; i < 2; ++i) {
    p.st_dy[i] = strides[i];
    p.st_x[i] = strides[2 + i];
    p.st_out[i] = strides[4 + i];
  }
  fill(p, positions, inv_freq, B, S, H, H_kv, rot_dim, pair_axis, eps, q_weight, k_weight);
  p.partial = want_dw ? static_cast<float*>(workspace) : nullptr;
  int64_t grid = 0;
  if (!empty) {
    p.share = bwd_share(B * S, steps_of(H, H_kv, D));
    grid = std::min<int64_t>((B * S * p.share + kBwdWarps - 1) / kBwdWarps, kBwdBlocks);
  }
  cudaError_t e;
  if (dtype == FA_DTYPE_F16)
    e = D == 64 ? launch_bwd<__half, 64>(p, interleaved, norm, grid, dq_weight, dk_weight, stream)
                : launch_bwd<__half, 128>(p, interleaved, norm, grid, dq_weight, dk_weight, stream);
  else
    e = D == 64 ? launch_bwd<__nv_bfloat16, 64>(p, interleaved, norm, grid, dq_weight, dk_weight, stream)
                : launch_bwd<__nv_bfloat16, 128>(p, interleaved, norm, grid, dq_weight, dk_weight, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
