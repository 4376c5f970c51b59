/*
 * fa_rope.cu -- fa_qk_norm_rope and its backward (formulas in include/fa_api.h):
 * RMS norm of each query and key head and the rotation by position, one pass
 * over the data.
 *
 * Bound by HBM: 8 or so operations a value against 4 bytes moved (forward; 6
 * backward).  So one read and one write of each value, with the next rows'
 * loads always in flight:
 *   - a head vector lies in D / 8 lanes (16 at D = 128, 8 at 64), so sums over
 *     a head are 4 or 3 shuffles; a lane holds both values of its rotation
 *     pairs (four elements of the first half and their partners of the second,
 *     two 8-byte accesses), so the rotation needs none;
 *   - one block works out the cosines and sines of its one to four tokens, a
 *     pair a thread, in shared memory; then each warp walks heads of one token
 *     with that token's values and the weights in registers;
 *   - with few tokens more warps share one.
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

constexpr int kWarps = 8;
constexpr int kMaxPairs = 64;
constexpr int kBwdResident = 2;       // blocks of the backward an SM holds
constexpr int kBwdBlocks = 152 * kBwdResident;   // its grid: rows of the weight gradients' partial sums

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
  int32_t share;           // warps that share a token: 1, 2, 4 or 8
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
template <typename T>
__device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) {
  Pack<T>::load2(r.lo.x, f[0], f[1]);
  Pack<T>::load2(r.lo.y, f[2], f[3]);
  Pack<T>::load2(r.hi.x, f[4], f[5]);
  Pack<T>::load2(r.hi.y, f[6], f[7]);
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
__device__ __forceinline__ void store_row(uint16_t* row, const Elements& e, const float (&f)[8]) {
  *reinterpret_cast<uint2*>(row + e.lo) = make_uint2(Pack<T>::store2(f[0], f[1]), Pack<T>::store2(f[2], f[3]));
  *reinterpret_cast<uint2*>(row + e.hi) = make_uint2(Pack<T>::store2(f[4], f[5]), Pack<T>::store2(f[6], f[7]));
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
  if (e > 1 && e <= 64) fixed = (hi << (e - 1)) | ((m * K) >> (65 - e));
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
  for (int k = threadIdx.x / kMaxPairs; k < kWarps / p.share; k += kWarps * 32 / kMaxPairs)
    if (token0 + k < p.B * p.S) table[k][i] = angle(p, token0 + k, i);
}

// A lane's four pairs: cosines and sines (turned back with direction -1).
struct Turn {
  float cs[4], sn[4];
};
__device__ __forceinline__ Turn load_turn(const float2* table, const Elements& e, float direction) {
  Turn t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = e.pair >= 0 ? table[e.pair + j] : make_float2(1.0f, 0.0f);
    t.cs[j] = v.x;
    t.sn[j] = direction * v.y;
  }
  return t;
}
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&y)[8], const Turn& t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float& a = y[INTERLEAVED ? 2 * j : j];
    float& b = y[INTERLEAVED ? 2 * j + 1 : j + 4];
    const float x = a * t.cs[j] - b * t.sn[j];
    b = b * t.cs[j] + a * t.sn[j];
    a = x;
  }
}

// Both weight vectors as fp32 in shared memory (ones where there is none), by the block.
template <typename T, int D>
__device__ __forceinline__ void block_weights(const RopeParams& p, float (*table)[D]) {
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    const T* src = static_cast<const T*>(p.weight[i / D]);
    table[i / D][i % D] = src ? static_cast<float>(src[i % D]) : 1.0f;
  }
}
__device__ __forceinline__ void load_weight(const float* table, const Elements& e, float (&w)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(table + e.lo), b = *reinterpret_cast<const float4*>(table + e.hi);
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
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

template <typename T, int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kWarps * 32, 4) fa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;   // lanes a head, heads a warp at once
  __shared__ float2 table[kWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  fa::wait_for_stream();
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * (kWarps / p.share);
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
      if (NORM) block_weights<T, D>(p, weights);
      block_angles(p, token0, table);
      __syncthreads();
      t = load_turn(table[mine], e, 1.0f);
    }
    float w[8];
    if (NORM) load_weight(weights[which], e, w);
    for (int h0 = first; h0 < last; h0 += PER * kFwdRows) {
      Raw now[kFwdRows];
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) now[i] = raw[i];
      load(h0 + PER * kFwdRows);
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        const int h = h0 + i * PER + slot;
        float y[8];
        unpack<T>(now[i], y);
        if (NORM) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += y[j] * y[j];
          const float r = rsqrtf(head_sum<LANES>(ss) * (1.0f / D) + p.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = y[j] * r * w[j];
        }
        turn<INTERLEAVED>(y, t);
        if (h < last) store_row<T>(dst + h * out_step, e, y);
      }
    }
  }
}

constexpr int kBwdRows = 2;

template <typename T, int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kWarps * 32, kBwdResident) fa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  __shared__ float2 table[2][kWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  fa::wait_for_stream();
  const Elements e = elements<INTERLEAVED>(p.rot, sub);
  const int per_block = kWarps / p.share, mine = warp / p.share, part = warp % p.share;
  const int64_t tokens = p.B * p.S;
  float dw[2][8];
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[j / 8][j % 8] = 0.0f;

  if (NORM) block_weights<T, D>(p, weights);      // (read behind the first barrier)
  int buffer = 0;
  for (int64_t token0 = static_cast<int64_t>(blockIdx.x) * per_block; token0 < tokens;
       token0 += static_cast<int64_t>(gridDim.x) * per_block, buffer ^= 1) {
    const bool real = token0 + mine < tokens;
    const uint32_t token = real ? static_cast<uint32_t>(token0 + mine) : 0u;
    const uint32_t b = token / static_cast<uint32_t>(p.S), s = token - b * static_cast<uint32_t>(p.S);
    Turn t;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      int first, last;
      heads_of<PER>(p, part, which, first, last);
      if (!real) last = 0;
      const int64_t x_step = p.st_x[which].head, dy_step = p.st_dy[which].head, out_step = p.st_out[which].head;
      const uint16_t* x = static_cast<const uint16_t*>(p.x[which]) + row_base(p.st_x[which], b, s);
      const uint16_t* dy = static_cast<const uint16_t*>(p.dy[which]) + row_base(p.st_dy[which], b, s);
      uint16_t* dst = static_cast<uint16_t*>(p.out[which]) + row_base(p.st_out[which], b, s);
      Raw rx[kBwdRows], rg[kBwdRows];
      auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          const int h = h0 + i * PER + slot;
          rx[i] = rg[i] = Raw{};
          if (h < last) {
            rg[i] = load_row(dy + h * dy_step, e);
            if (NORM) rx[i] = load_row(x + h * x_step, e);
          }
        }
      };
      load(first);
      if (which == 0) {       // (the other buffer's readers have passed this barrier since)
        block_angles(p, token0, table[buffer]);
        __syncthreads();
        t = load_turn(table[buffer][mine], e, -1.0f);
      }
      float w[8];
      if (NORM) load_weight(weights[which], e, w);
      for (int h0 = first; h0 < last; h0 += PER * kBwdRows) {
        Raw nx[kBwdRows], ng[kBwdRows];
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) { nx[i] = rx[i]; ng[i] = rg[i]; }
        load(h0 + PER * kBwdRows);
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          const int h = h0 + i * PER + slot;
          float g[8];
          unpack<T>(ng[i], g);
          turn<INTERLEAVED>(g, t);
          if (NORM) {
            float xv[8];
            unpack<T>(nx[i], xv);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              ss += xv[j] * xv[j];
              dot += g[j] * w[j] * xv[j];
            }
            const float r = rsqrtf(head_sum<LANES>(ss) * (1.0f / D) + p.eps);
            const float c = head_sum<LANES>(dot) * (1.0f / D) * r * r;
            // h < last only: a lane without a row holds zeros, which add
            // nothing to dw unless r is infinite (0 * inf)
            if (h < last) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                dw[which][j] += g[j] * xv[j] * r;
                g[j] = r * (g[j] * w[j] - xv[j] * c);
              }
            }
          }
          if (h < last) store_row<T>(dst + h * out_step, e, g);
        }
      }
    }
  }

  if (NORM && p.partial) {
    // The block's sums in a fixed order: lanes of the same elements, then warps.
    __shared__ float sums[kWarps][2][D];
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = dw[which][j];
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (slot == 0) sums[warp][which][j < 4 ? e.lo + j : e.hi + j - 4] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += (&sums[k][0][0])[i];
      p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
    }
  }
}

// Weight gradients: element i of both vectors over the blocks' partial sums,
// 32 threads an element; 2 D / 32 blocks of 1024 threads.
template <typename T>
__global__ void __launch_bounds__(1024) fa_rope_dw_kernel(const float* partial, int blocks, int D,
                                                          T* dwq, T* dwk) {
  __shared__ float sums[32][33];
  fa::wait_for_stream();
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
// 152 SMs its 32 warps (backward: 16).  At 16384 tokens, 32 + 8 heads of 128:
// forward 60.0 us with one, 60.7 with two, 74.7 with four.
int share_for(int64_t tokens) {
  return tokens >= 152 * 64 ? 1 : tokens >= 152 * 16 ? 2 : tokens >= 152 * 8 ? 4 : 8;
}

template <typename T, int D>
cudaError_t launch_fwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, cudaStream_t stream) {
  const fa::Launch c(dim3(static_cast<unsigned>(grid)), kWarps * 32, 0, stream);
  if (interleaved)
    return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, true, true>, p)
                : cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, true, false>, p);
  return norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, false, true>, p)
              : cudaLaunchKernelEx(&c.cfg, fa_rope_fwd_kernel<T, D, false, false>, p);
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, void* dwq,
                       void* dwk, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    const fa::Launch c(dim3(static_cast<unsigned>(grid)), kWarps * 32, 0, stream);
    if (interleaved)
      e = norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, true, true>, p)
               : cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, true, false>, p);
    else
      e = norm ? cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, false, true>, p)
               : cudaLaunchKernelEx(&c.cfg, fa_rope_bwd_kernel<T, D, false, false>, p);
  }
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
  p.share = share_for(B * S);
  const int per_block = kWarps / p.share;
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
    p.share = share_for(B * S);
    const int per_block = kWarps / p.share;
    grid = std::min<int64_t>((B * S + per_block - 1) / per_block, kBwdBlocks);
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
