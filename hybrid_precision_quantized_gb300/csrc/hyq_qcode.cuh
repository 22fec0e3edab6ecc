// Step, zero and code decisions of the group quantiser (Quant_B of Algorithm 4,
// see hyq_quant.cu), shared by the kernels that quantise rows.
#pragma once

#include "hyq_common.cuh"
#include "hyq_f2.cuh"

namespace {

// Rounding by addition: for |t| < 2^22, fl32(t + 1.5 * 2^23) is
// 1.5 * 2^23 + rint(t) (the sum's ulp is 1, ties to even), so its bit
// pattern is kMagicBits + rint(t).
constexpr float kMagic = 12582912.f;
constexpr uint32_t kMagicBits = 0x4B400000u;
__host__ __device__ constexpr uint32_t magic_sum8() {
  uint32_t s = 0;
  for (int p = 0; p < 8; ++p) s += kMagicBits << (4 * p);
  return s;
}
constexpr uint32_t kMagicSum = magic_sum8();

__device__ __forceinline__ uint32_t lo32(uint64_t v) { return (uint32_t)v; }
__device__ __forceinline__ uint32_t hi32(uint64_t v) { return (uint32_t)(v >> 32); }

// The code is the grid point z + c s nearest to x, ties to the even c.  It is
// found from t = fl32(fl32(x - z) * r), r = RN(1/s), whose relative error is
// at most about 3 * 2^-24 (|t| < 2^8 where it matters: under 5e-5), so
// rint(t) is the exact answer unless t lies within kNearTie of a half
// integer; those elements are decided exactly (exact_code).
constexpr float kNearTie = 0.5f - 0.000244140625f;  // 1/2 - 2^-12

// Step of a group: the smallest FP16 value s with qmax s >= mx - mn (the
// subtraction, the division and the FP16 conversion all round up, which gives
// exactly that value: qmax h is exact in FP32 for every FP16 h).
__device__ __forceinline__ __half group_step(float mn, float mx, float qmax) {
  return __float2half_ru(__fdiv_ru(__fsub_ru(mx, mn), qmax));
}

// Exact decision near the midpoint k + 1/2, k = floor(t): in float64 the
// midpoint z + (k + 1/2) s is exact (s and z are FP16 values: a multiple of
// 2^-25 below 2^25 in magnitude) and the sign of x minus it is exact.
__device__ __forceinline__ float exact_code(float x, float z, float s, float t) {
  const float k = floorf(t);
  const double d = (double)x - ((double)z + ((double)k + 0.5) * (double)s);
  if (d > 0.0) return k + 1.f;
  if (d < 0.0) return k;
  return (__float2int_rz(k) & 1) ? k + 1.f : k;  // a tie: the even one
}

// Bit patterns kMagicBits + code of the two BF16 elements of w (x: low half),
// for a group whose (x - z) * r all lie in (-0.5, 15.5): there the clamp of
// the code decision is the identity and the added magic rounds exactly as
// rint does.  nz2 = (-z, -z), r2 = (r, r).  The magic add is a scalar
// __fadd_rn, which is never contracted with the product into a fused
// multiply-add (that would round the unrounded product).  `near` is set when
// either element lies within kNearTie of a midpoint (the caller then takes
// the exact path for the whole word).
__device__ __forceinline__ uint2 code_bits2(uint32_t w, uint64_t nz2, uint64_t r2, bool& near) {
  const uint64_t x2 = (uint64_t)(w << 16) | ((uint64_t)(w & 0xffff0000u) << 32);
  const uint64_t t2 = f2_mul(f2_add(x2, nz2), r2);
  const float t0 = __uint_as_float(lo32(t2)), t1 = __uint_as_float(hi32(t2));
  const float b0 = __fadd_rn(t0, kMagic), b1 = __fadd_rn(t1, kMagic);
  near |= fabsf(__fsub_rn(t0, __fsub_rn(b0, kMagic))) > kNearTie ||
          fabsf(__fsub_rn(t1, __fsub_rn(b1, kMagic))) > kNearTie;
  return make_uint2(__float_as_uint(b0), __float_as_uint(b1));
}

// Code word from b[p] = kMagicBits + code of nibble p: the shift-add chain
// sums b[p] << 4p modulo 2^32, which is the word plus sum_p kMagicBits << 4p.
__device__ __forceinline__ uint32_t pack_nibbles(const uint32_t (&b)[8]) {
  uint32_t w = b[7];
#pragma unroll
  for (int p = 6; p >= 0; --p) w = (w << 4) + b[p];
  return w - kMagicSum;
}

// r = 1 / s rounded, and 0 exactly when the step s is 0; qmax = 2^B - 1.
__device__ __forceinline__ uint32_t code_of(float x, float z, float r, float s, float qmax = 15.f) {
  if (r == 0.f) return 0u;
  const float t = __fmul_rn(__fsub_rn(x, z), r);
  float c = rintf(t);
  if (fabsf(__fsub_rn(t, c)) > kNearTie) c = exact_code(x, z, s, t);
  c = fminf(fmaxf(c, 0.f), qmax);
  return (uint32_t)c;
}

}  // namespace
