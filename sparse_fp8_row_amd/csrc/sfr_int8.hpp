// Device functions of the row quantizer to 8-bit integers, shared by its kernels
// and by the linear layer that quantizes its activation itself, so both write
// the same codes.
#pragma once

#include "sfr_quant.hpp"

namespace sfr {

// Codes of a row are those of the exact quotient 127 x / amax.  With x = a 2^p
// and amax = b 2^q (a, b whole, under 2^8) the quotient is a half-integer
// exactly or at least 2^-16 of itself away from one, so a quotient within 2^-20
// that is exact on half-integers decides every code.  Here it is one binary32
// product by the reciprocal, corrected once: t = t0 + r y with r = 127 x - t0 amax
// exact.  Where the true quotient t* is a half-integer the correction leaves
// |r| 2^-23, below half a step of t*, so t* is returned.  Rows are taken by the
// exponent of amax (x 2^-e, amax 2^-e in [1, 2)), so nothing over- or underflows
// that could reach code 1.
struct RowScale {
  float an, y;  // amax 2^-e and its reciprocal
  int e;
  bool live;  // false: a row of zeros, or one that is not finite
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale s;
  const float amax = bf16_to_f32(amax_bits);
  s.live = amax_bits != 0 && amax_bits < 0x7F80u;
  s.e = s.live ? __builtin_amdgcn_frexp_expf(amax) - 1 : 0;
  s.an = s.live ? ldexpf(amax, -s.e) : 1.0f;
  s.y = 1.0f / s.an;
  return s;
}

// The row's scale: 0 for zeros, NaN for a row that holds a NaN or an infinity.
__device__ __forceinline__ float scale_value(uint32_t amax_bits) {
  return amax_bits < 0x7F80u ? bf16_to_f32(amax_bits) / 127.0f : __builtin_nanf("");
}

// Low byte of the result: the code.  Adding 1.5 * 2^23 rounds to a whole number,
// ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t code(uint32_t bf16, const RowScale& s) {
  const float a = 127.0f * ldexpf(bf16_to_f32(bf16), -s.e);
  const float t0 = a * s.y;
  const float t = __builtin_fmaf(__builtin_fmaf(-t0, s.an, a), s.y, t0);
  return __float_as_uint(t + 12582912.0f);
}

__device__ __forceinline__ uint2 cast8_int8(const uint4& c, const RowScale& s) {
  if (!s.live) return make_uint2(0, 0);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    pair[i] = __builtin_amdgcn_perm(code(w[i] >> 16, s), code(w[i] & 0xFFFFu, s), 0x0C0C0400u);
  return make_uint2(pair[0] | pair[1] << 16, pair[2] | pair[3] << 16);
}

}  // namespace sfr
