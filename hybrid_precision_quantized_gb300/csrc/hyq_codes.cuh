// Codes of the pages as fp16 values, two at a time, for the kernels that form c s + z.
#pragma once

#include "hyq_common.cuh"

namespace {

__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes as an fp16 pair, exactly: their bits under 1024, less 1024.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {  // nibbles 0 and 4
  return hadd2_u((w & 0x000F000Fu) | 0x64006400u, 0xE400E400u);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {  // nibbles 1 and 5, which count 16 each
  return hfma2_u((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}
__device__ __forceinline__ uint32_t even_codes(uint32_t w) {  // bytes 0 and 2
  return hadd2_u((w & 0x00FF00FFu) | 0x64006400u, 0xE400E400u);
}
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) {  // bytes 1 and 3
  return hadd2_u(__byte_perm(w, 0x64646464u, 0x4341), 0xE400E400u);
}
__device__ __forceinline__ uint32_t u4at(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// Halves 0 or 1 of a word, twice.
__device__ __forceinline__ uint32_t both(uint32_t w, int half) { return __byte_perm(w, 0, half ? 0x3232 : 0x1010); }

}  // namespace
