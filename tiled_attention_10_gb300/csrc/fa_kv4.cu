/*
 * fa_kv4.cu -- fa_kv4_write and fa_kv4_read: rows of keys and values into and
 * out of the 4-bit cache (formulas in include/fa_api.h).
 *
 * HBM's time is the floor (2 bytes a value one way, 9/16 the other).  Writing, a
 * thread takes groups of 16 values: two 16-byte loads (the next group's ahead),
 * one store of 8 bytes of codes and one byte of scale, so that the codes fall into
 * whole rows.  Reading, it takes 8 values a time, so that each store of a warp
 * fills whole lines.  8192 tokens of 8 heads of 128 take 13.8 us to write and 11.6
 * to read, from HBM 6.3 each; issue slots are used for 52 and 44 %, DRAM for 28 and
 * 9 % (what is written stays in L2 at first).  No unit is full: the blocks live for
 * two groups or pieces a thread, in 2.7 and 1.7 waves, and each begins with a slot's
 * load, a division and a barrier.
 *
 * The nearest code is decided exactly.  16-bit inputs lie on a border between
 * two codes (or two scales) often, and one rounding of x / (scale * descale)
 * in fp32 would settle those by its own error.  So the fp32 quotient is only
 * a first guess, cut to a few bits: every border has fewer, so the guess is
 * either on the right side of it or the border itself, and then the sign of
 * the remainder x - guess * scale * descale, which one fma gives exactly,
 * moves it a little off the border.
 */
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fa_api.h"
#include "fa_kv4.cuh"
#include "fa_launch.cuh"

namespace {

using fa::kv4::Descales;
constexpr int kThreads = 256;

struct RowParams {
  fa::kv4::Cache cache;
  const void* in[2];       // write: K, V rows
  void* out[2];            // read: K, V rows
  int64_t token_stride[2], head_stride[2];   // elements (write)
  const int64_t* slot_map;
  int64_t n_tokens;
  int32_t tile;            // tokens of a block
  int64_t n_slots;
};

// Two fp32 values in a register pair: one instruction for both.
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
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {      // to 1 or 2 ulp: a guess's factor
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// amax / (6 g) for the scale: q is that up to 2^-21; the result's place among
// numbers of at most 10 bits is that of the exact quotient.
__device__ __forceinline__ float place_scale(float q, float g, float amax) {
  const uint32_t h = (__float_as_uint(q) + 0x1000u) & 0xffffe000u;
  const float rest = fmaf(-(__uint_as_float(h) * 6.0f), g, amax);
  return __uint_as_float(h + (rest > 0.0f ? 1u : 0u) - (rest < 0.0f ? 1u : 0u));
}
// a / (scale g) in [0, 8] for two codes, likewise: the borders are multiples of
// 1/4, so the guess is cut to multiples of 2^-6 (by adding and taking away 2^17
// and a half) and moved off by 2^-8.
__device__ __forceinline__ float2 place_codes(float2 q, F2 scale, F2 minus_g, F2 a) {
  const F2 c = f2(196608.0f, 196608.0f), minus_c = f2(-196608.0f, -196608.0f);
  const F2 h = add2(add2(f2(q.x, q.y), c), minus_c);
  const float2 rest = split(fma2(mul2(h, scale), minus_g, a));
  float2 side;                                    // 0, 1/2 or 1: below, on, above
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(side.x) : "f"(rest.x), "f"(8.507059173023462e37f), "f"(0.5f));
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(side.y) : "f"(rest.y), "f"(8.507059173023462e37f), "f"(0.5f));
  return split(fma2(f2(side.x, side.y), f2(0.0078125f, 0.0078125f), add2(h, f2(-0.00390625f, -0.00390625f))));
}

// Row index (page, head 0, row of the page) of a slot.
__device__ __forceinline__ int64_t cache_row(const fa::kv4::Cache& c, int64_t slot) {
  const int64_t page = slot <= 0xffffffffll ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(c.page_size)
                                            : slot / c.page_size;
  return page * c.H_kv * c.page_size + (slot - page * c.page_size);
}

template <typename T> __device__ __forceinline__ float2 unpack(uint32_t w);
template <> __device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// The largest magnitude of 16 values, NaN passed over.
template <typename T> __device__ __forceinline__ float largest(const uint32_t (&w)[8]);
template <> __device__ __forceinline__ float largest<__half>(const uint32_t (&w)[8]) {
  __half2 m = __float2half2_rn(0.0f);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&w[j])));
  return fmaxf(__low2float(m), __high2float(m));
}
template <> __device__ __forceinline__ float largest<__nv_bfloat16>(const uint32_t (&w)[8]) {
  __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
  return fmaxf(__low2float(m), __high2float(m));
}

// One group of 16 values: its codes and its scale.
template <typename T>
__device__ __forceinline__ void encode(const uint32_t (&raw)[8], float g, uint2& codes, uint32_t& code) {
  const float amax = largest<T>(raw);
  const float want = place_scale(fminf(amax * reciprocal(6.0f * g), 1024.0f), g, amax);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(want));
  code = two;
  const uint32_t h2 = fa::kv4::scales_to_half(two);
  const float scale = __low2float(*reinterpret_cast<const __half2*>(&h2));
  codes = make_uint2(0u, 0u);
  if (scale == 0.0f) return;
  const float inv = reciprocal(scale * g);
  const F2 scale2 = f2(scale, scale), minus_g = f2(-g, -g);
  float y[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = unpack<T>(raw[j]);
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y));
    const float2 q = make_float2(fminf(a.x * inv, 8.0f), fminf(a.y * inv, 8.0f));   // (NaN becomes 8)
    const float2 r = place_codes(q, scale2, minus_g, f2(a.x, a.y));
    y[2 * j] = copysignf(r.x, x.x);
    y[2 * j + 1] = copysignf(r.y, x.y);
  }
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w[j])
        : "f"(y[8 * j]), "f"(y[8 * j + 1]), "f"(y[8 * j + 2]), "f"(y[8 * j + 3]), "f"(y[8 * j + 4]),
          "f"(y[8 * j + 5]), "f"(y[8 * j + 6]), "f"(y[8 * j + 7]));
  codes = make_uint2(w[0], w[1]);
}

// A block writes `tile` tokens (at most 32) of K or of V; a thread walks groups.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_write_kernel(const __grid_constant__ RowParams p) {
  constexpr int G = D / 16, R = kThreads / G;       // groups of a head; (token, head) rows at once
  __shared__ int64_t row[32];
  fa::wait_for_stream();
  fa::let_next_start();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.tile), p.n_tokens - first));
  if (threadIdx.x < n) {
    const int64_t slot = p.slot_map[first + threadIdx.x];
    row[threadIdx.x] = slot >= 0 && slot < p.n_slots ? cache_row(p.cache, slot) : -1;
  }
  const int which = blockIdx.y, group = threadIdx.x % G;
  const int h_step = R % p.cache.H_kv, t_step = R / p.cache.H_kv;
  int t = threadIdx.x / G / p.cache.H_kv, h = threadIdx.x / G % p.cache.H_kv;
  const float g = fa::kv4::descale_of(p.cache, which);
  const uint16_t* const src = static_cast<const uint16_t*>(p.in[which]) + first * p.token_stride[which] + group * 16;
  uint4 next[2];
  auto load = [&]() {
    if (t < n) {
      const uint4* from = reinterpret_cast<const uint4*>(src + t * p.token_stride[which] + h * p.head_stride[which]);
      next[0] = from[0];
      next[1] = from[1];
    }
  };
  load();
  __syncthreads();
  while (t < n) {
    const uint32_t raw[8] = {next[0].x, next[0].y, next[0].z, next[0].w, next[1].x, next[1].y, next[1].z, next[1].w};
    const int64_t at = row[t];
    const int head = h;
    t += t_step;
    h += h_step;
    if (h >= p.cache.H_kv) { h -= p.cache.H_kv; ++t; }
    load();
    if (at < 0) continue;
    uint2 codes;
    uint32_t scale;
    encode<T>(raw, g, codes, scale);
    const uint64_t r = static_cast<uint64_t>(at) + static_cast<uint32_t>(head) * static_cast<uint32_t>(p.cache.page_size);
    *reinterpret_cast<uint2*>(p.cache.codes[which] + r * (D / 2) + group * 8) = codes;
    p.cache.scales[which][r * G + group] = static_cast<uint8_t>(scale);
  }
}

// A block reads `tile` tokens (at most 32) of K or of V.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_read_kernel(const __grid_constant__ RowParams p) {
  __shared__ int64_t row[32];
  fa::wait_for_stream();
  fa::let_next_start();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.tile), p.n_tokens - first));
  if (threadIdx.x < n) {
    const int64_t slot = p.slot_map[first + threadIdx.x];
    row[threadIdx.x] = slot >= 0 && slot < p.n_slots ? cache_row(p.cache, slot) : -1;
  }
  __syncthreads();
  const int which = blockIdx.y;
  fa::kv4::unpack_rows<T, D, kThreads, true>(p.cache, which, row, n,
                                       static_cast<uint16_t*>(p.out[which]) + first * p.cache.H_kv * D);
}

bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

fa_status_t check_rows(const void* k, const void* v, const int64_t* slot_map, const uint8_t* kc,
                       const uint8_t* ks, const uint8_t* vc, const uint8_t* vs, const Descales& d,
                       int64_t n_tokens, int64_t H_kv, int64_t D, int64_t page_size,
                       int64_t num_pages, fa_dtype_t dtype) {
  if (!kc || !ks || !vc || !vs) return FA_ERR_INVALID_ARG;
  if (n_tokens < 0 || H_kv < 1 || D < 1 || num_pages < 1 || page_size < 16) return FA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!k || !v || !slot_map)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP8E4M3)
    return FA_ERR_INVALID_ARG;
  const fa_status_t st = check_descales(d);
  if (st != FA_OK) return st;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_DTYPE_FP8E4M3 || !fa::kv4::page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
  if (off(k, 16) || off(v, 16) || off(slot_map, 8) || off(kc, 16) || off(vc, 16) || off(ks, 16) || off(vs, 16))
    return FA_ERR_MISALIGNED;
  if (page_size > 65536 || num_pages > INT32_MAX || H_kv > 65536 || n_tokens > INT32_MAX)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

RowParams params(const uint8_t* kc, const uint8_t* ks, const uint8_t* vc, const uint8_t* vs,
                 const Descales& d, const int64_t* slot_map, int64_t n_tokens, int64_t H_kv,
                 int64_t D, int64_t page_size, int64_t num_pages) {
  RowParams p = {};
  p.cache.codes[0] = const_cast<uint8_t*>(kc); p.cache.codes[1] = const_cast<uint8_t*>(vc);
  p.cache.scales[0] = const_cast<uint8_t*>(ks); p.cache.scales[1] = const_cast<uint8_t*>(vs);
  for (int i = 0; i < 2; ++i) { p.cache.descale[i] = d.value[i]; p.cache.descale_at[i] = d.at[i]; }
  p.cache.num_pages = num_pages;
  p.cache.page_size = static_cast<int32_t>(page_size);
  p.cache.H_kv = static_cast<int32_t>(H_kv);
  p.slot_map = slot_map;
  p.n_tokens = n_tokens;
  // 32 tokens a block, or fewer while that leaves SMs idle
  p.tile = 32;
  while (p.tile > 1 && n_tokens < int64_t(p.tile) * 152 * 4) p.tile /= 2;
  p.n_slots = num_pages * page_size;
  return p;
}

template <typename K>
fa_status_t launch(K kernel, const RowParams& p, int64_t blocks, cudaStream_t stream) {
  const fa::Launch c(dim3(static_cast<unsigned>(blocks), 2), kThreads, 0, stream);
  return cudaLaunchKernelEx(&c.cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t write_rows(const void* k, const void* v, const int64_t* slot_map, uint8_t* k_codes,
                  uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, const Descales& d,
                  int64_t n_tokens, int64_t H_kv, int64_t D, int64_t page_size, int64_t num_pages,
                  const fa_strides_t* strides, fa_dtype_t dtype, cudaStream_t stream) {
  if (!strides) return FA_ERR_INVALID_ARG;
  const fa_status_t st = check_rows(k, v, slot_map, k_codes, k_scales, v_codes, v_scales, d, n_tokens,
                                    H_kv, D, page_size, num_pages, dtype);
  if (st != FA_OK) return st;
  for (int i = 0; i < 2; ++i) {
    if (strides[i].seq < 1 || strides[i].head < 1) return FA_ERR_INVALID_ARG;
    if (strides[i].seq % 8 != 0 || strides[i].head % 8 != 0) return FA_ERR_MISALIGNED;
    if (strides[i].seq > (int64_t(1) << 38) || strides[i].head > (int64_t(1) << 38))
      return FA_ERR_UNSUPPORTED;
  }
  if (n_tokens == 0) return FA_OK;
  RowParams p = params(k_codes, k_scales, v_codes, v_scales, d, slot_map, n_tokens, H_kv, D, page_size,
                       num_pages);
  p.in[0] = k; p.in[1] = v;
  for (int i = 0; i < 2; ++i) { p.token_stride[i] = strides[i].seq; p.head_stride[i] = strides[i].head; }
  const int64_t blocks = (n_tokens + p.tile - 1) / p.tile;
  if (dtype == FA_DTYPE_F16)
    return D == 64 ? launch(fa_kv4_write_kernel<__half, 64>, p, blocks, stream)
                   : launch(fa_kv4_write_kernel<__half, 128>, p, blocks, stream);
  return D == 64 ? launch(fa_kv4_write_kernel<__nv_bfloat16, 64>, p, blocks, stream)
                 : launch(fa_kv4_write_kernel<__nv_bfloat16, 128>, p, blocks, stream);
}

fa_status_t read_rows(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                 const uint8_t* v_scales, const int64_t* slot_map, void* k_out, void* v_out,
                 const Descales& d, int64_t n_tokens, int64_t H_kv, int64_t D, int64_t page_size,
                 int64_t num_pages, fa_dtype_t dtype, cudaStream_t stream) {
  const fa_status_t st = check_rows(k_out, v_out, slot_map, k_codes, k_scales, v_codes, v_scales, d,
                                    n_tokens, H_kv, D, page_size, num_pages, dtype);
  if (st != FA_OK) return st;
  if (n_tokens == 0) return FA_OK;
  RowParams p = params(k_codes, k_scales, v_codes, v_scales, d, slot_map, n_tokens, H_kv, D, page_size,
                       num_pages);
  p.out[0] = k_out; p.out[1] = v_out;
  const int64_t blocks = (n_tokens + p.tile - 1) / p.tile;
  if (dtype == FA_DTYPE_F16)
    return D == 64 ? launch(fa_kv4_read_kernel<__half, 64>, p, blocks, stream)
                   : launch(fa_kv4_read_kernel<__half, 128>, p, blocks, stream);
  return D == 64 ? launch(fa_kv4_read_kernel<__nv_bfloat16, 64>, p, blocks, stream)
                 : launch(fa_kv4_read_kernel<__nv_bfloat16, 128>, p, blocks, stream);
}

}  // namespace

extern "C" {

fa_status_t fa_kv4_write(const void* k, const void* v, const int64_t* slot_map, uint8_t* k_codes,
                         uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, float descale_k,
                         float descale_v, int64_t n_tokens, int64_t H_kv, int64_t D,
                         int64_t page_size, int64_t num_pages, const fa_strides_t* strides,
                         fa_dtype_t dtype, cudaStream_t stream) {
  return write_rows(k, v, slot_map, k_codes, k_scales, v_codes, v_scales, Descales{{descale_k, descale_v}, {}},
               n_tokens, H_kv, D, page_size, num_pages, strides, dtype, stream);
}

fa_status_t fa_kv4_write_devscale(const void* k, const void* v, const int64_t* slot_map,
                                  uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                                  uint8_t* v_scales, const float* descale_k, const float* descale_v,
                                  int64_t n_tokens, int64_t H_kv, int64_t D, int64_t page_size,
                                  int64_t num_pages, const fa_strides_t* strides, fa_dtype_t dtype,
                                  cudaStream_t stream) {
  return write_rows(k, v, slot_map, k_codes, k_scales, v_codes, v_scales,
               Descales{{1.0f, 1.0f}, {descale_k, descale_v}}, n_tokens, H_kv, D, page_size, num_pages,
               strides, dtype, stream);
}

fa_status_t fa_kv4_read(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, const int64_t* slot_map, void* k_out, void* v_out,
                        float descale_k, float descale_v, int64_t n_tokens, int64_t H_kv, int64_t D,
                        int64_t page_size, int64_t num_pages, fa_dtype_t dtype,
                        cudaStream_t stream) {
  return read_rows(k_codes, k_scales, v_codes, v_scales, slot_map, k_out, v_out,
              Descales{{descale_k, descale_v}, {}}, n_tokens, H_kv, D, page_size, num_pages, dtype, stream);
}

fa_status_t fa_kv4_read_devscale(const uint8_t* k_codes, const uint8_t* k_scales,
                                 const uint8_t* v_codes, const uint8_t* v_scales,
                                 const int64_t* slot_map, void* k_out, void* v_out,
                                 const float* descale_k, const float* descale_v, int64_t n_tokens,
                                 int64_t H_kv, int64_t D, int64_t page_size, int64_t num_pages,
                                 fa_dtype_t dtype, cudaStream_t stream) {
  return read_rows(k_codes, k_scales, v_codes, v_scales, slot_map, k_out, v_out,
              Descales{{1.0f, 1.0f}, {descale_k, descale_v}}, n_tokens, H_kv, D, page_size, num_pages, dtype,
              stream);
}

}  // extern "C"
