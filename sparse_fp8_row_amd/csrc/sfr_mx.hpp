// Device functions of the MX block formats (blocks of 32 values along a row
// share one power-of-two scale, stored as the biased exponent byte E8M0) and
// of the gated block's activation functions.  Shared by the stand-alone
// quantizer, the gated linear layer's epilogue and the 4-bit kernels, so all
// produce and read the same codes by the same arithmetic.
#pragma once

#include "sfr_device.hpp"

namespace sfr {

enum { MX_E4M3 = 0, MX_E5M2 = 1, MX_E2M1 = 2 };
enum { ACT_SILU = 0, ACT_GELU_TANH = 1, ACT_RELU = 2 };
constexpr int MX_BLOCK = 32;
// Smallest scale byte written (2^-110): every decoded value is then zero or a
// normal bf16 number, so decoding to bf16 is exact in all three formats.
constexpr int MX_MIN_CODE = 17;
// Scale byte of a block that holds a NaN or an infinity; it decodes to NaN.
constexpr int MX_NAN_CODE = 255;

// Scale byte of a block whose largest magnitude has the binary32 pattern
// `abits` (sign bit clear): the smallest 2^e with amax <= fmax * 2^e.  fmax is
// 1.75 * 2^8 (e4m3), 1.75 * 2^15 (e5m2) or 1.5 * 2^2 (e2m1), so e is the
// exponent of amax less fmax's, plus one when amax's fraction is above
// fmax's.
template <int FMT>
__device__ __forceinline__ int mx_scale_code(uint32_t abits) {
  constexpr int top = FMT == MX_E4M3 ? 8 : FMT == MX_E5M2 ? 15 : 2;
  constexpr uint32_t frac = FMT == MX_E2M1 ? 0x400000u : 0x600000u;
  const int e = (int)(abits >> 23);
  const int code = e - top + ((abits & 0x7FFFFFu) > frac ? 1 : 0);
  return e == 255 ? MX_NAN_CODE : max(code, MX_MIN_CODE);
}

// 2^-(code - 127), the factor that takes values to the element format's range
// (exact: a power of two).  0 for the NaN code, whose elements are written as
// zeros.
__device__ __forceinline__ float mx_inverse(int code) {
  return code == MX_NAN_CODE ? 0.0f : __uint_as_float((uint32_t)(254 - code) << 23);
}

// Largest element of a block: one that would decode to 2^128, past binary32
// and bf16, is stored as the element below.  Only blocks of the highest scale
// (amax above 1.75 or 1.5 * 2^127) reach it.  0 for the NaN code.
template <int FMT>
__device__ __forceinline__ float mx_limit(int code) {
  constexpr int top = FMT == MX_E4M3 ? 246 : FMT == MX_E5M2 ? 239 : 252;
  constexpr float all = FMT == MX_E4M3 ? 448.0f : FMT == MX_E5M2 ? 57344.0f : 6.0f;
  constexpr float high = FMT == MX_E4M3 ? 240.0f : FMT == MX_E5M2 ? 28672.0f : 3.0f;
  return code <= top ? all : code == MX_NAN_CODE ? 0.0f : high;
}

// v / scale within the limit (the median of the three); a block without a
// finite scale has limit 0, which also turns NaN (from infinity times 0) to
// a zero.
__device__ __forceinline__ float mx_scaled(float v, float inv, float limit) {
  return limit == 0.0f ? 0.0f : __builtin_amdgcn_fmed3f(v * inv, -limit, limit);
}

// The scale as a binary32 operand of the hardware converters, which take its
// exponent field: byte 0 is 2^-127, and with byte 255, the exponent of
// infinities, they return NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t code) { return __uint_as_float(code << 23); }

// Four scaled values (|v| <= fmax) -> four FP8 bytes, nearest even.
template <int FMT>
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d) {
  constexpr int F = FMT == MX_E4M3 ? FMT_E4M3 : FMT_E5M2;
  return (uint32_t)cvt_pk_fp8<F, true>(c, d, cvt_pk_fp8<F, false>(a, b, 0));
}

// Eight scaled values (|v| <= 6) -> eight e2m1 codes, element i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t mx_pack8_e2m1(const float (&v)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
  return w;
}

// Two stored FP8 elements (bytes 0,1 or 2,3 of w) times the block's scale, as two bf16 values.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t mx_widen2(uint32_t w, float scale) {
  if constexpr (FMT == MX_E4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)w, scale, HI));
}

// Eight stored e2m1 elements times the block's scale, as eight bf16 values.
__device__ __forceinline__ uint4 mx_widen8_e2m1(uint32_t w, float scale) {
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3)));
}

// Eight FP8 elements and their block's scale byte, as eight bf16 values.
template <int FMT>
__device__ __forceinline__ uint4 mx_widen8_fp8(uint2 c, uint32_t code) {
  const float f = mx_scale_value(code);
  return make_uint4(mx_widen2<FMT, false>(c.x, f), mx_widen2<FMT, true>(c.x, f), mx_widen2<FMT, false>(c.y, f),
                    mx_widen2<FMT, true>(c.y, f));
}

// ---------------------------------------------------------------------------
// Activation functions.  silu(g) = g s(g); gelu_tanh(g) = g s(2 c (g + 0.044715
// g^3)) with c = sqrt(2 / pi) (0.5 (1 + tanh z) is s(2 z)); s the logistic
// function.  GELU's polynomial takes g clamped to +-20, past which s is 0 or 1
// in binary32, so that it cannot overflow; the factor g itself stays
// unclamped and carries NaN.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == ACT_RELU) {
    return g < 0.0f ? 0.0f : g;  // keeps NaN
  } else if constexpr (ACT == ACT_SILU) {
    return g * logistic(g);
  } else {
    const float t = fminf(fmaxf(g, -20.0f), 20.0f);
    return g * logistic(1.5957691216057308f * (t + 0.044715f * t * t * t));
  }
}

// act(g) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float& a, float& d) {
  if constexpr (ACT == ACT_RELU) {
    a = g < 0.0f ? 0.0f : g;
    d = g > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_SILU) {
    const float s = logistic(g);
    a = g * s;
    d = s * (1.0f + g * (1.0f - s));
  } else {
    const float t = fminf(fmaxf(g, -20.0f), 20.0f);
    const float s = logistic(1.5957691216057308f * (t + 0.044715f * t * t * t));
    a = g * s;
    d = s + g * (s * (1.0f - s)) * (1.5957691216057308f * (1.0f + 0.134145f * t * t));
  }
}

}  // namespace sfr
