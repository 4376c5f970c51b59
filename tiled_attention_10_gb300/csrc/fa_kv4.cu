/*
 * fa_kv4.cu -- fa_kv4_write and fa_kv4_read: rows of keys and values into and
 * out of the 4-bit cache (formulas in include/fa_api.h).
 *
 * Bound by HBM (2 bytes a value one way, 9/16 the other).  Writing, a thread
 * takes one group of 16 values: two 16-byte loads, one store of 8 bytes of codes
 * and one byte of scale, so that the codes fall into whole rows.  Reading, it
 * takes 8 values a time, so that each store of a warp fills whole lines.
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

constexpr int kThreads = 256;

struct RowParams {
  fa::kv4::Cache cache;
  const void* in[2];       // write: K, V rows
  void* out[2];            // read: K, V rows
  int64_t token_stride[2], head_stride[2];   // elements (write)
  const int64_t* slot_map;
  int64_t n_tokens, n_groups;   // groups: n_tokens * H_kv * D / 16
  int32_t tile;            // read: tokens of a block
  int64_t n_slots;
};

// amax / (6 g) for the scale: q is that up to 2^-22; the result's place among
// numbers of at most 10 bits is that of the exact quotient.
__device__ __forceinline__ float place_scale(float q, float g, float amax) {
  const uint32_t h = (__float_as_uint(q) + 0x1000u) & 0xffffe000u;
  const float rest = fmaf(-(__uint_as_float(h) * 6.0f), g, amax);
  return __uint_as_float(h + (rest > 0.0f ? 1u : 0u) - (rest < 0.0f ? 1u : 0u));
}
// a / (scale g) in [0, 8] for a code, likewise: the borders are multiples of
// 1/4, so the guess is cut to multiples of 2^-6 (by adding and taking away 2^17
// and a half) and moved off by 2^-8.
__device__ __forceinline__ float place_code(float q, float scale, float g, float a) {
  const float h = (q + 196608.0f) - 196608.0f;
  const float rest = fmaf(-(h * scale), g, a);
  float side;                                     // 0, 1/2 or 1: below, on, above
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(side) : "f"(rest), "f"(8.507059173023462e37f), "f"(0.5f));
  return fmaf(side, 0.0078125f, h - 0.00390625f);
}

// Where a group lives: its token, head and group within the row.
template <int D>
struct Group {
  int64_t token;
  int32_t head, g;
  __device__ __forceinline__ Group(int64_t i, int H_kv) {
    constexpr int G = D / 16;
    g = static_cast<int>(i % G);
    const int64_t r = i / G;
    token = r <= 0xffffffffll ? static_cast<uint32_t>(r) / static_cast<uint32_t>(H_kv) : r / H_kv;
    head = static_cast<int>(r - token * H_kv);
  }
};
// Row index (page, head, row of the page) of a slot's head.
__device__ __forceinline__ int64_t cache_row(const fa::kv4::Cache& c, int64_t slot, int head) {
  const int64_t page = slot <= 0xffffffffll ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(c.page_size)
                                            : slot / c.page_size;
  return (page * c.H_kv + head) * c.page_size + (slot - page * c.page_size);
}

template <typename T> __device__ __forceinline__ float2 unpack(uint32_t w);
template <> __device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_write_kernel(const __grid_constant__ RowParams p) {
  fa::wait_for_stream();
  fa::let_next_start();
  const int which = blockIdx.y;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.n_groups) return;
  const Group<D> at(i, p.cache.H_kv);
  const int64_t slot = p.slot_map[at.token];
  if (slot < 0 || slot >= p.n_slots) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.in[which]) +
                                                    at.token * p.token_stride[which] +
                                                    at.head * p.head_stride[which] + at.g * 16);
  const uint4 r0 = src[0], r1 = src[1];
  const uint32_t raw[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
  float x[16], amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = unpack<T>(raw[j]);
    x[2 * j] = v.x; x[2 * j + 1] = v.y;
    amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));   // fmaxf passes NaN over
  }
  const float g = p.cache.descale[which];
  const float want = place_scale(fminf(amax * __frcp_rn(6.0f * g), 1024.0f), g, amax);
  uint16_t code;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(0.0f), "f"(want));
  const uint32_t h2 = fa::kv4::scales_to_half(code);
  const float scale = __low2float(*reinterpret_cast<const __half2*>(&h2));
  uint32_t lo = 0u, hi = 0u;
  if (scale > 0.0f) {
    const float inv = __frcp_rn(scale * g);
    float y[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float a = fabsf(x[j]);
      y[j] = copysignf(place_code(fminf(a * inv, 8.0f), scale, g, a), x[j]);   // fminf: NaN becomes 8
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
    lo = w[0]; hi = w[1];
  }
  const int64_t row = cache_row(p.cache, slot, at.head);
  *reinterpret_cast<uint2*>(p.cache.codes[which] + row * (D / 2) + at.g * 8) = make_uint2(lo, hi);
  p.cache.scales[which][row * (D / 16) + at.g] = static_cast<uint8_t>(code);
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
    row[threadIdx.x] = slot >= 0 && slot < p.n_slots ? cache_row(p.cache, slot, 0) : -1;
  }
  __syncthreads();
  const int which = blockIdx.y;
  fa::kv4::unpack_rows<T, D, kThreads>(p.cache, which, row, n,
                                       static_cast<uint16_t*>(p.out[which]) + first * p.cache.H_kv * D);
}

bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

fa_status_t check_rows(const void* k, const void* v, const int64_t* slot_map, const uint8_t* kc,
                       const uint8_t* ks, const uint8_t* vc, const uint8_t* vs, float dk, float dv,
                       int64_t n_tokens, int64_t H_kv, int64_t D, int64_t page_size,
                       int64_t num_pages, fa_dtype_t dtype) {
  if (!kc || !ks || !vc || !vs) return FA_ERR_INVALID_ARG;
  if (n_tokens < 0 || H_kv < 1 || D < 1 || num_pages < 1 || page_size < 16) return FA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!k || !v || !slot_map)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP8E4M3)
    return FA_ERR_INVALID_ARG;
  const float lo = std::ldexp(1.0f, -100), hi = std::ldexp(1.0f, 100);
  if (!(dk >= lo && dk <= hi && dv >= lo && dv <= hi)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_DTYPE_FP8E4M3 || !fa::kv4::page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
  if (off(k, 16) || off(v, 16) || off(slot_map, 8) || off(kc, 16) || off(vc, 16) || off(ks, 16) || off(vs, 16))
    return FA_ERR_MISALIGNED;
  if (page_size > 65536 || num_pages > INT32_MAX || H_kv > 65536 || n_tokens > INT32_MAX ||
      n_tokens * H_kv * (D / 16) > static_cast<int64_t>(INT32_MAX) * kThreads)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

RowParams params(const uint8_t* kc, const uint8_t* ks, const uint8_t* vc, const uint8_t* vs,
                 float dk, float dv, const int64_t* slot_map, int64_t n_tokens, int64_t H_kv,
                 int64_t D, int64_t page_size, int64_t num_pages) {
  RowParams p = {};
  p.cache.codes[0] = const_cast<uint8_t*>(kc); p.cache.codes[1] = const_cast<uint8_t*>(vc);
  p.cache.scales[0] = const_cast<uint8_t*>(ks); p.cache.scales[1] = const_cast<uint8_t*>(vs);
  p.cache.descale[0] = dk; p.cache.descale[1] = dv;
  p.cache.num_pages = num_pages;
  p.cache.page_size = static_cast<int32_t>(page_size);
  p.cache.H_kv = static_cast<int32_t>(H_kv);
  p.slot_map = slot_map;
  p.n_tokens = n_tokens;
  p.n_groups = n_tokens * H_kv * (D / 16);
  p.n_slots = num_pages * page_size;
  return p;
}

template <typename K>
fa_status_t launch(K kernel, const RowParams& p, int64_t blocks, cudaStream_t stream) {
  const fa::Launch c(dim3(static_cast<unsigned>(blocks), 2), kThreads, 0, stream);
  return cudaLaunchKernelEx(&c.cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status_t fa_kv4_write(const void* k, const void* v, const int64_t* slot_map, uint8_t* k_codes,
                         uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, float descale_k,
                         float descale_v, int64_t n_tokens, int64_t H_kv, int64_t D,
                         int64_t page_size, int64_t num_pages, const fa_strides_t* strides,
                         fa_dtype_t dtype, cudaStream_t stream) {
  if (!strides) return FA_ERR_INVALID_ARG;
  const fa_status_t st = check_rows(k, v, slot_map, k_codes, k_scales, v_codes, v_scales, descale_k,
                                    descale_v, n_tokens, H_kv, D, page_size, num_pages, dtype);
  if (st != FA_OK) return st;
  for (int i = 0; i < 2; ++i) {
    if (strides[i].seq < 1 || strides[i].head < 1) return FA_ERR_INVALID_ARG;
    if (strides[i].seq % 8 != 0 || strides[i].head % 8 != 0) return FA_ERR_MISALIGNED;
    if (strides[i].seq > (int64_t(1) << 38) || strides[i].head > (int64_t(1) << 38))
      return FA_ERR_UNSUPPORTED;
  }
  if (n_tokens == 0) return FA_OK;
  RowParams p = params(k_codes, k_scales, v_codes, v_scales, descale_k, descale_v, slot_map,
                       n_tokens, H_kv, D, page_size, num_pages);
  p.in[0] = k; p.in[1] = v;
  for (int i = 0; i < 2; ++i) { p.token_stride[i] = strides[i].seq; p.head_stride[i] = strides[i].head; }
  const int64_t blocks = (p.n_groups + kThreads - 1) / kThreads;
  if (dtype == FA_DTYPE_F16)
    return D == 64 ? launch(fa_kv4_write_kernel<__half, 64>, p, blocks, stream)
                   : launch(fa_kv4_write_kernel<__half, 128>, p, blocks, stream);
  return D == 64 ? launch(fa_kv4_write_kernel<__nv_bfloat16, 64>, p, blocks, stream)
                 : launch(fa_kv4_write_kernel<__nv_bfloat16, 128>, p, blocks, stream);
}

fa_status_t fa_kv4_read(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, const int64_t* slot_map, void* k_out, void* v_out,
                        float descale_k, float descale_v, int64_t n_tokens, int64_t H_kv, int64_t D,
                        int64_t page_size, int64_t num_pages, fa_dtype_t dtype,
                        cudaStream_t stream) {
  const fa_status_t st = check_rows(k_out, v_out, slot_map, k_codes, k_scales, v_codes, v_scales,
                                    descale_k, descale_v, n_tokens, H_kv, D, page_size, num_pages, dtype);
  if (st != FA_OK) return st;
  if (n_tokens == 0) return FA_OK;
  RowParams p = params(k_codes, k_scales, v_codes, v_scales, descale_k, descale_v, slot_map,
                       n_tokens, H_kv, D, page_size, num_pages);
  p.out[0] = k_out; p.out[1] = v_out;
  // 32 tokens a block, or fewer while that leaves SMs idle
  p.tile = 32;
  while (p.tile > 1 && n_tokens < int64_t(p.tile) * 152 * 2) p.tile /= 2;
  const int64_t blocks = (n_tokens + p.tile - 1) / p.tile;
  if (dtype == FA_DTYPE_F16)
    return D == 64 ? launch(fa_kv4_read_kernel<__half, 64>, p, blocks, stream)
                   : launch(fa_kv4_read_kernel<__half, 128>, p, blocks, stream);
  return D == 64 ? launch(fa_kv4_read_kernel<__nv_bfloat16, 64>, p, blocks, stream)
                 : launch(fa_kv4_read_kernel<__nv_bfloat16, 128>, p, blocks, stream);
}

}  // extern "C"
