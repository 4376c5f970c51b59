/*
 * fa_rope.cu -- fa_qk_norm_rope and its backward (formulas in include/fa_api.h):
 * RMS norm of each query and key head and the rotation by position, one pass
 * over the data.
 *
 * Bound by HBM: 8 or so operations a value against 4 bytes moved (forward; 6
 * backward).  So one read and one write of each value, 16 bytes a lane, and
 * several rows in flight a lane:
 *   - a head vector lies in D / 8 lanes (16 at D = 128, 8 at 64), 8 values a
 *     lane, so sums over a head are 3 or 4 shuffles;
 *   - a warp takes one token and walks its heads, so the token's cosines and
 *     sines are worked out once (two pairs a lane, exchanged through shared
 *     memory) and stay in registers over all heads;
 *   - with few tokens the heads of one are cut into parts for several warps.
 * A value's partner in its rotation pair is in the same lane (interleaved) or
 * rot_dim / 16 lanes away (one shuffle).
 * The angle: a position times the frequency, in turns modulo 1, as a 64-bit
 * fixed-point product (wrapping is the reduction), so no position is too far
 * for 32-bit sine and cosine.
 */
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa_api.h"

namespace {

constexpr int kWarps = 8;
constexpr int kMaxPairs = 64;
constexpr int kBwdBlocks = 152 * 2;   // rows of the weight gradients' partial sums

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
  int32_t parts;           // warps that share a token's heads
  int32_t rot;             // rotated elements
  float eps;
  uint8_t axis[kMaxPairs]; // axis of each pair
};

template <typename T> struct Pack;
template <> struct Pack<__half> {
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(h[i]);
      f[2 * i] = t.x; f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ __half one(float x) { return __float2half_rn(x); }
};
template <> struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float x) { return __float2bfloat16_rn(x); }
};

// Sum over the LANES lanes that hold one head vector.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This lane's cosines and (signed) sines of one token: value e turns as
// e * cs[.] + partner * sn[.].
template <bool INTERLEAVED>
struct Turn {
  static constexpr int N = INTERLEAVED ? 4 : 8;   // pairs that a lane's 8 values touch
  float cs[N], sn[N];
};

// cos and sin of the token's pairs into table[0 .. rot / 2), by the warp.
__device__ __forceinline__ void angles(const RopeParams& p, int64_t token, float2* table, int lane) {
  const int64_t tokens = p.B * p.S;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    if (i < p.rot / 2) {
      double turns = p.inv_freq[i] * 0.15915494309189534561;   // 1 / (2 pi)
      turns -= floor(turns);
      const uint64_t fixed = (turns >= 0.0 && turns < 1.0) ? __double2ull_rn(turns * 18446744073709551616.0) : 0ull;
      const int64_t pos = p.positions[p.axis[i] * tokens + token];
      // The product modulo 2^64 is the angle modulo a turn; its top half as a
      // signed number counts half turns of 2^-31.
      const int32_t half_turns = static_cast<int32_t>((static_cast<uint64_t>(pos) * fixed) >> 32);
      float s, c;
      sincospif(static_cast<float>(half_turns) * 4.656612873077392578125e-10f, &s, &c);
      table[i] = make_float2(c, s);
    }
  }
}

// The lane's turn from the table; sub: lane within the head's lanes.  Values
// that are not rotated turn by nothing (cos 1, sin 0, own value as partner).
template <bool INTERLEAVED>
__device__ __forceinline__ void load_turn(const RopeParams& p, const float2* table, int sub,
                                          float direction, Turn<INTERLEAVED>& t) {
  const int e0 = sub * 8;
#pragma unroll
  for (int j = 0; j < Turn<INTERLEAVED>::N; ++j) {
    float2 v = make_float2(1.0f, 0.0f);
    float sign = direction;
    if (e0 < p.rot) {
      if (INTERLEAVED) {
        v = table[e0 / 2 + j];
      } else {
        const bool upper = e0 >= p.rot / 2;
        v = table[(upper ? e0 - p.rot / 2 : e0) + j];
        sign = upper ? direction : -direction;
      }
    }
    t.cs[j] = v.x;
    t.sn[j] = sign * v.y;
  }
}

template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&y)[8], const Turn<INTERLEAVED>& t, int partner) {
  if (INTERLEAVED) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = y[2 * j], b = y[2 * j + 1];
      y[2 * j] = a * t.cs[j] - b * t.sn[j];
      y[2 * j + 1] = b * t.cs[j] + a * t.sn[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float o = __shfl_sync(0xffffffffu, y[j], partner);
      y[j] = y[j] * t.cs[j] + o * t.sn[j];
    }
  }
}

// The lane whose values are this lane's partners.
__device__ __forceinline__ int partner_lane(const RopeParams& p, int lane, int sub) {
  const int e0 = sub * 8;
  if (e0 >= p.rot) return lane;
  const int d = p.rot / 16;
  return e0 < p.rot / 2 ? lane + d : lane - d;
}

template <typename T>
__device__ __forceinline__ void load_weight(const RopeParams& p, int which, int sub, float (&w)[8]) {
  if (p.weight[which]) {
    uint4 v;
    const uint16_t* src = static_cast<const uint16_t*>(p.weight[which]) + sub * 8;
    uint16_t* dst = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
    for (int j = 0; j < 8; ++j) dst[j] = src[j];   // a weight vector may start anywhere
    Pack<T>::load(v, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
  }
}

__device__ __forceinline__ int64_t row_base(const fa_strides_t& st, int64_t b, int64_t s) {
  return b * st.batch + s * st.seq;
}

constexpr int kFwdRows = 4;   // rows in flight a lane

template <typename T, int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kWarps * 32) fa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;   // lanes a head, heads a warp at once
  __shared__ float2 tables[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t token = task / p.parts;
  const int part = static_cast<int>(task - token * p.parts);
  if (token >= p.B * p.S) return;
  const int64_t b = token / p.S, s = token - b * p.S;

  if (p.rot > 0) angles(p, token, tables[warp], lane);
  __syncwarp();
  Turn<INTERLEAVED> t;
  load_turn<INTERLEAVED>(p, tables[warp], sub, 1.0f, t);
  const int partner = partner_lane(p, lane, sub);

#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float w[8];
    if (NORM) load_weight<T>(p, which, sub, w);
    const uint16_t* src = static_cast<const uint16_t*>(p.x[which]) + row_base(p.st_x[which], b, s) + sub * 8;
    uint16_t* dst = static_cast<uint16_t*>(p.out[which]) + row_base(p.st_out[which], b, s) + sub * 8;
    const int stride = PER * p.parts;
    for (int h0 = part * PER; h0 < p.heads[which]; h0 += stride * kFwdRows) {
      uint4 raw[kFwdRows];
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        const int h = h0 + i * stride + slot;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.heads[which]) raw[i] = *reinterpret_cast<const uint4*>(src + h * p.st_x[which].head);
      }
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        if (h0 + i * stride >= p.heads[which]) break;   // the same for the whole warp
        const int h = h0 + i * stride + slot;
        float y[8];
        Pack<T>::load(raw[i], y);
        if (NORM) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += y[j] * y[j];
          const float r = rsqrtf(head_sum<LANES>(ss) * (1.0f / D) + p.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = y[j] * r * w[j];
        }
        turn<INTERLEAVED>(y, t, partner);
        if (h < p.heads[which])
          *reinterpret_cast<uint4*>(dst + h * p.st_out[which].head) = Pack<T>::store(y);
      }
    }
  }
}

constexpr int kBwdRows = 2;

template <typename T, int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kWarps * 32) fa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = D / 8, PER = 32 / LANES;
  __shared__ float2 tables[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LANES, slot = lane / LANES;
  const int partner = partner_lane(p, lane, sub);
  const int64_t tasks = p.B * p.S * p.parts;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i / 8][i % 8] = 0.0f;

  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t token = task / p.parts;
    const int part = static_cast<int>(task - token * p.parts);
    const int64_t b = token / p.S, s = token - b * p.S;
    __syncwarp();                                 // the last task's table has been read
    if (p.rot > 0) angles(p, token, tables[warp], lane);
    __syncwarp();
    Turn<INTERLEAVED> t;
    load_turn<INTERLEAVED>(p, tables[warp], sub, -1.0f, t);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float w[8];
      if (NORM) load_weight<T>(p, which, sub, w);
      const uint16_t* x = static_cast<const uint16_t*>(p.x[which]) + row_base(p.st_x[which], b, s) + sub * 8;
      const uint16_t* dy = static_cast<const uint16_t*>(p.dy[which]) + row_base(p.st_dy[which], b, s) + sub * 8;
      uint16_t* dst = static_cast<uint16_t*>(p.out[which]) + row_base(p.st_out[which], b, s) + sub * 8;
      const int stride = PER * p.parts;
      for (int h0 = part * PER; h0 < p.heads[which]; h0 += stride * kBwdRows) {
        uint4 rx[kBwdRows], rg[kBwdRows];
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          const int h = h0 + i * stride + slot;
          rx[i] = rg[i] = make_uint4(0u, 0u, 0u, 0u);
          if (h < p.heads[which]) {
            rg[i] = *reinterpret_cast<const uint4*>(dy + h * p.st_dy[which].head);
            if (NORM) rx[i] = *reinterpret_cast<const uint4*>(x + h * p.st_x[which].head);
          }
        }
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          if (h0 + i * stride >= p.heads[which]) break;
          const int h = h0 + i * stride + slot;
          float g[8];
          Pack<T>::load(rg[i], g);
          turn<INTERLEAVED>(g, t, partner);
          if (NORM) {
            float xv[8];
            Pack<T>::load(rx[i], xv);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              ss += xv[j] * xv[j];
              dot += g[j] * w[j] * xv[j];
            }
            const float r = rsqrtf(head_sum<LANES>(ss) * (1.0f / D) + p.eps);
            const float c = head_sum<LANES>(dot) * (1.0f / D) * r * r;
            // h < heads only: a lane without a row holds zeros, which add
            // nothing to dw unless r is infinite (0 * inf)
            if (h < p.heads[which]) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                dw[which][j] += g[j] * xv[j] * r;
                g[j] = r * (g[j] * w[j] - xv[j] * c);
              }
            }
          }
          if (h < p.heads[which])
            *reinterpret_cast<uint4*>(dst + h * p.st_out[which].head) = Pack<T>::store(g);
        }
      }
    }
  }

  if (NORM && p.partial) {
    // The block's sums in a fixed order: lanes of the same elements, warps.
    __shared__ float sums[kWarps][2][D];
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = dw[which][j];
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (slot == 0) sums[warp][which][sub * 8 + j] = v;
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
// eight threads an element; grid 2 D / 32 blocks of 256 threads.
template <typename T>
__global__ void __launch_bounds__(256) fa_rope_dw_kernel(const float* partial, int blocks, int D,
                                                         T* dwq, T* dwk) {
  __shared__ float sums[8][32];
  const int e = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + e;     // of 2 D
  float v = 0.0f;
  for (int r = k; r < blocks; r += 8) v += partial[static_cast<int64_t>(r) * 2 * D + i];
  sums[k][e] = v;
  __syncthreads();
  if (k == 0) {
    v = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v += sums[j][e];
    T* out = i < D ? dwq : dwk;
    if (out) out[i < D ? i : i - D] = Pack<T>::one(v);
  }
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
  if (B > 0 && S > 0 && S > (int64_t(1) << 40) / B) return FA_ERR_UNSUPPORTED;
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

// Warps a token: enough tasks for 16 warps on each of 152 SMs, each with one
// pass over the query heads at least.
int parts_for(int64_t tokens, int64_t H, int per) {
  const int64_t passes = std::max<int64_t>(1, (H + per - 1) / per);
  const int64_t want = (152 * 16 + tokens - 1) / tokens;
  return static_cast<int>(std::max<int64_t>(1, std::min(want, passes)));
}

cudaLaunchConfig_t config(int64_t grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  return cfg;
}

template <typename T, int D>
cudaError_t launch_fwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = config(grid, kWarps * 32, stream);
  if (interleaved)
    return norm ? cudaLaunchKernelEx(&cfg, fa_rope_fwd_kernel<T, D, true, true>, p)
                : cudaLaunchKernelEx(&cfg, fa_rope_fwd_kernel<T, D, true, false>, p);
  return norm ? cudaLaunchKernelEx(&cfg, fa_rope_fwd_kernel<T, D, false, true>, p)
              : cudaLaunchKernelEx(&cfg, fa_rope_fwd_kernel<T, D, false, false>, p);
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeParams& p, bool interleaved, bool norm, int64_t grid, void* dwq,
                       void* dwk, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    cudaLaunchConfig_t cfg = config(grid, kWarps * 32, stream);
    if (interleaved)
      e = norm ? cudaLaunchKernelEx(&cfg, fa_rope_bwd_kernel<T, D, true, true>, p)
               : cudaLaunchKernelEx(&cfg, fa_rope_bwd_kernel<T, D, true, false>, p);
    else
      e = norm ? cudaLaunchKernelEx(&cfg, fa_rope_bwd_kernel<T, D, false, true>, p)
               : cudaLaunchKernelEx(&cfg, fa_rope_bwd_kernel<T, D, false, false>, p);
  }
  if (e != cudaSuccess || !(dwq || dwk)) return e;
  cudaLaunchConfig_t cfg = config(2 * D / 32, 256, stream);
  return cudaLaunchKernelEx(&cfg, fa_rope_dw_kernel<T>, static_cast<const float*>(p.partial),
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
  p.parts = parts_for(B * S, H, static_cast<int>(256 / D));
  const int64_t grid = (B * S * p.parts + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return FA_ERR_UNSUPPORTED;
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
    p.parts = parts_for(B * S, H, static_cast<int>(256 / D));
    grid = std::min<int64_t>((B * S * p.parts + kWarps - 1) / kWarps, kBwdBlocks);
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
