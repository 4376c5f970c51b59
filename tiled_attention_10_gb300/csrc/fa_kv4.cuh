/*
 * fa_kv4.cuh -- the paged cache of 4-bit values: its layout and the conversions
 * of its codes (include/fa_api.h states the format).
 */
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {
namespace kv4 {

struct Cache {
  uint8_t* codes[2];    // K, V: [num_pages, H_kv, page_size, D / 2]
  uint8_t* scales[2];   // K, V: [num_pages, H_kv, page_size, D / 16]
  float descale[2];
  int64_t num_pages;
  int32_t page_size, H_kv;
};

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

// The paged attention's page sizes: tiles of 16 keys lie in one page.
inline bool page_size_ok(int64_t ps) {
  return ps >= 16 && ((ps <= 128 && 128 % ps == 0) || ps % 128 == 0);
}

}  // namespace kv4
}  // namespace fa
