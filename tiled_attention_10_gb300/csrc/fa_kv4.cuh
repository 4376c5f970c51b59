/*
 * fa_kv4.cuh -- the paged cache of 4-bit values: its layout and the conversions
 * of its codes (include/fa_api.h states the format).
 */
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/fa_api.h"

namespace fa {
namespace kv4 {

struct Cache {
  uint8_t* codes[2];    // K, V: [num_pages, H_kv, page_size, D / 2]
  uint8_t* scales[2];   // K, V: [num_pages, H_kv, page_size, D / 16]
  float descale[2];
  const float* descale_at[2];   // where the descales are on the device, or null: the numbers above
  int64_t num_pages;
  int32_t page_size, H_kv;
};

// Descales are in [2^-100, 2^100]: a host's are refused outside, a device's moved
// to the nearer end (NaN to the lower), so that no value becomes NaN by them.
constexpr float kMinDescale = 0x1p-100f, kMaxDescale = 0x1p100f;
__device__ __forceinline__ float descale_from(const float* at) {
  return fminf(fmaxf(*at, kMinDescale), kMaxDescale);
}
__device__ __forceinline__ float descale_of(const Cache& c, int which) {   // (after wait_for_stream)
  return c.descale_at[which] ? descale_from(c.descale_at[which]) : c.descale[which];
}

// Four bytes of codes (eight values) as four f16 pairs, low nibble first; and
// two e4m3 scales as one f16 pair.  Both conversions are exact, and so is the
// f16 product of the two: 2 and 4 significant bits, at most 6 * 448.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t scales_to_half(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t mul_half(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T> __device__ __forceinline__ uint32_t pack16(float a, float b);
template <> __device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// a * b rounded to odd: the exact product where it is one, else the neighbour
// whose last bit is set (the product cut short, with a bit for the rest), so that
// rounding it to 16 bits gives the exact product's nearest: a second rounding to
// nearest would take a product next to a tie for the tie.
__device__ __forceinline__ float mul_to_odd(float a, float b) {
  const float p = __fmul_rz(a, b);
  return __uint_as_float(__float_as_uint(p) | (fmaf(a, b, -p) != 0.0f ? 1u : 0u));
}

// Whether any code * scale times g, in fp32, is a tie of the type T that the exact
// product is not; only such a g needs mul_to_odd (of random ones 1 in 500 for f16;
// 8192 tokens of 8 heads of 128 written and read: 21.9 us, 23.6 with it).  For a
// whole warp, a significand of code * scale a lane: 8..15, and three times those.
// An inexact product whose last set bit is bit `low` is a tie of bf16 at 15, of f16
// at 12, or at more where f16 is subnormal: there the bit is 2^-25, the product
// below 2^(-1 - low), and reached if that is not below g times the least
// code * scale, 2^-10.
template <typename T>
__device__ __forceinline__ bool rounds_twice(float g) {
  const int lane = threadIdx.x & 31;
  const float n = static_cast<float>((8 + (lane & 7)) * ((lane & 8) ? 3 : 1)), p = n * g;
  const int low = __ffs(static_cast<int>(__float_as_uint(p) | 0x800000u)) - 1;
  bool tie = low == 15;
  if (std::is_same<T, __half>::value)
    tie = low == 12 || (low > 12 && __uint_as_float(static_cast<uint32_t>(126 - low) << 23) >= g * 0x1p-10f);
  return __any_sync(0xffffffffu, tie && fmaf(n, g, -p) != 0.0f);
}

// Rows of the cache as dense 16-bit rows out[r][head][D], r < n <= 32, by a block
// of THREADS: row[r] is the index (page, head 0, row of the page) of token r in
// the cache, negative for a row of zeros.  A thread unpacks 8 values at a time
// (4 bytes of codes, one store of 16); consecutive threads take consecutive
// pieces of the output, so the stores fill whole lines.  SCALED: times the descale
// (else code * scale, which needs no rounding).
template <typename T, int D, int THREADS, bool SCALED>
__device__ __forceinline__ void unpack_rows(const Cache& c, int which, const int64_t* row, int n, void* out) {
  constexpr int P = D / 8, kAhead = 4;              // pieces of a head; pieces in flight
  constexpr int R = THREADS / P;                    // (token, head) rows the block takes at once
  const int piece = threadIdx.x % P;
  const int h_step = R % c.H_kv, t_step = R / c.H_kv;
  int t = threadIdx.x / P / c.H_kv, h = threadIdx.x / P % c.H_kv;
  const float g = SCALED ? descale_of(c, which) : 1.0f;
  const bool careful = SCALED && rounds_twice<T>(g);
  uint4* dst = reinterpret_cast<uint4*>(out) + threadIdx.x;
  while (t < n) {
    uint32_t codes[kAhead], scale[kAhead];
    int last = 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      codes[k] = scale[k] = 0u;
      if (t < n) {
        last = k + 1;
        const int64_t at = row[t];
        if (at >= 0) {
          const uint64_t r = static_cast<uint64_t>(at) + static_cast<uint32_t>(h) * static_cast<uint32_t>(c.page_size);
          codes[k] = *reinterpret_cast<const uint32_t*>(c.codes[which] + r * (D / 2) + piece * 4);
          scale[k] = c.scales[which][r * (D / 16) + piece / 2];
        }
      }
      t += t_step;
      h += h_step;
      if (h >= c.H_kv) { h -= c.H_kv; ++t; }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k < last) {
        uint32_t v[4], w[4];
        float2 f[4];
        codes_to_half(codes[k], v);
        const uint32_t s2 = scales_to_half(scale[k] * 0x101u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = mul_half(v[j], s2);
          f[j] = __half22float2(*reinterpret_cast<const __half2*>(&x));
        }
        if (careful) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack16<T>(mul_to_odd(f[j].x, g), mul_to_odd(f[j].y, g));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack16<T>(f[j].x * g, f[j].y * g);
        }
        dst[static_cast<int64_t>(k) * THREADS] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    dst += static_cast<int64_t>(kAhead) * THREADS;
  }
}

// An entry point's descales: numbers, or where they are on the device (null: the numbers).
struct Descales {
  float value[2];
  const float* at[2];
};
inline fa_status_t check_descales(const Descales& d) {
  for (int i = 0; i < 2; ++i) {
    if (!(d.value[i] >= kMinDescale && d.value[i] <= kMaxDescale)) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d.at[i]) % 4 != 0) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

// The paged attention's page sizes: tiles of 16 keys lie in one page.
inline bool page_size_ok(int64_t ps) {
  return ps >= 16 && ((ps <= 128 && 128 % ps == 0) || ps % 128 == 0);
}

}  // namespace kv4
}  // namespace fa
