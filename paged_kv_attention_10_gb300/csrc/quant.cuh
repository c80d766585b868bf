// e4m3 with a power-of-two scale per row and head, and small host/device helpers the 8-bit cache's
// kernels share.
//
// A cache row (one slot, one head) x holds x8 = e4m3(x * 2^-k) and the scale 2^k, with the smallest
// k >= -126 for which max |x| <= 448 * 2^k.  The scale is a power of two so that scaling is exact
// both ways: a row is rounded once, when it is written, and bf16(x8 * 2^k) reads it back without a
// second rounding.  A free (not power-of-two) scale would not make e4m3 more accurate: its relative
// step is the same in every binade.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pkv {

// The scale exponent of a row from the bits of its largest finite |x| (fp32): with |x| = f * 2^e,
// f in [1, 2), max |x| <= 448 * 2^k = 1.75 * 2^(k+8) holds for k = e - 8 when f <= 1.75 and for
// k = e - 7 otherwise; adding 0x1fffff to the bits carries into the exponent exactly when
// f > 1.75.  At least -126, so that 2^k and 2^-k are normal (a row of zeros gets 2^-126).
PKV_DEV int e4m3_scale_exp(uint32_t amax_bits) {
  return max((int)((amax_bits + 0x1fffffu) >> 23) - 135, -126);
}
constexpr int kE4m3MaxExp = 120;  // of the largest fp32 numbers: values above 240 * 2^120 are held as that
PKV_DEV float exp2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }  // k in [-126, 127]

// |x| as bits, 0 where x is not finite (the scale of a row ignores infinities and NaNs).
PKV_DEV uint32_t finite_abs_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// Four values to e4m3, round to nearest even, byte i = x[i].  Non-finite values become NaN (the
// format has no infinity; the saturating conversion would store 448 for one).
PKV_DEV uint32_t pack_e4m3x4(float x0, float x1, float x2, float x3) {
  auto nan_if_inf = [](float x) { return fabsf(x) == INFINITY ? __uint_as_float(0x7fffffffu) : x; };
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(nan_if_inf(x0)), "f"(nan_if_inf(x1)), "f"(nan_if_inf(x2)), "f"(nan_if_inf(x3)));
  return r;
}

// Bytes 0,1 (lo) and 2,3 (hi) of v as f16 pairs; exact.
PKV_DEV void unpack_e4m3x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Division of a 31-bit number by a number fixed at launch: multiply by the rounded-up reciprocal
// and shift (Granlund and Montgomery, "Division by invariant integers using multiplication").
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < div) ++shift;
    mul = (uint32_t)((((1ull << shift) - div) << 32) / div + 1);
  }
  PKV_DEV uint32_t quot(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
  PKV_DEV void divmod(uint32_t n, uint32_t& q, uint32_t& r) const {
    q = quot(n);
    r = n - q * d;
  }
};

}  // namespace pkv

namespace pkv_host {
bool valid_pool8(const pkv_pool_fp8* p);  // non-null, positive sizes, head_dim % 8 == 0, 16-byte aligned
}  // namespace pkv_host
