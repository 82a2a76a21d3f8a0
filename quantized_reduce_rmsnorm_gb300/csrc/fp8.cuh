// fp8.cuh -- 8-bit floating point (e4m3) with a scale for each block, device helpers.
//
// A block is 128 neighbouring elements of a row (an activation) or of each of 128
// neighbouring rows (a weight); the last of a row or of the rows may be smaller.  With m
// its largest |x| the scale is s = max(m / 448, 2^-60), a binary32 number, and a code
// is the e4m3 value nearest to x / s (the binary32 quotient; ties to even; 448 is the
// largest).  With the lower limit a block of zeros needs no case of its own and the
// product of two scales is a normal number.  A block with an infinity or a NaN has
// the scale NaN, so all of it reads back as NaN.
//
// x / s is taken as q = x r and one correction q + (x - q s) r, r = 1 / s rounded to
// nearest: the remainder is exact, so the result is the quotient's rounding (Markstein,
// IBM J. Res. Dev. 34, 1990), three operations a value and not a division.  They are
// taken with -r, so that what comes is the quotient's negative and a zero's sign survives
// the sums; the codes' signs are turned afterwards, four at once.
#pragma once

#include "mx4.cuh"

namespace fc {

// The scale of a block whose largest |x| has these bits.
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  return amax_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                  : fmaxf(__fdiv_rn(__uint_as_float(amax_bits), 448.0f), 0x1p-60f);
}
// Sixteen values by their scale, to codes.
template <bool F32>
__device__ __forceinline__ uint4 fp8_encode16(const Raw<F32, 16>& x, float scale) {
  const float2 r = dup2(-__frcp_rn(scale)), s = dup2(scale);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 v = pair<F32, 16>(x, 2 * i + k);
      float2 q = pmul(v, r);
      q = pfma(pfma(q, s, v), r, q);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[k]) : "f"(q.y), "f"(q.x));
    }
    w[i] = (h[0] | static_cast<uint32_t>(h[1]) << 16) ^ 0x80808080u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Sixteen codes to values times the scale.
__device__ __forceinline__ void fp8_decode16(const uint4& c, float scale, float2 (&v)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[i] >> 16 * k)));
      float lo, hi;
      asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
          : "=f"(lo), "=f"(hi)
          : "r"(h));
      v[2 * i + k] = pmul(make_float2(lo, hi), dup2(scale));
    }
}

}  // namespace fc
