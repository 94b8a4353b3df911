// Codes of the 8-bit cache: value = code * scale, the scale a power of two.
//
// E4M3: sign, 4 bits of exponent (bias 7), 3 of mantissa, largest 448.  INT8: -127 .. 127.
// Either code is exact in fp16, and a code times its scale is exact in bf16.
#pragma once

#include <cuda_fp16.h>

#include "rkv_device.cuh"

namespace rkv {

constexpr float kLowestScale = 1.1754943508222875e-38f;  // 2^-126: a block of zeros

// Two bytes of w (its lower or upper half) as a pair of fp16 numbers, the codes' values.
template <int kFormat>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kFormat == RKV_Q8_E4M3) {
    asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 1024 + (code + 128) is an fp16 number with the biased code for its lowest bits
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __float2half2_rn(1152.f);
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  }
}

// The same times a power of two f (which an INT8 code costs nothing for).
template <int kFormat>
__device__ __forceinline__ void decode4_times(uint32_t w, __half2 f, __half2 bias_f, uint32_t& lo, uint32_t& hi) {
  __half2 x, y;
  if (kFormat == RKV_Q8_E4M3) {
    uint32_t a, b;
    decode4<kFormat>(w, a, b);
    x = __hmul2(*reinterpret_cast<__half2*>(&a), f);
    y = __hmul2(*reinterpret_cast<__half2*>(&b), f);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    x = __hfma2(*reinterpret_cast<__half2*>(&a), f, bias_f);  // bias_f = -1152 f
    y = __hfma2(*reinterpret_cast<__half2*>(&b), f, bias_f);
  }
  lo = *reinterpret_cast<uint32_t*>(&x);
  hi = *reinterpret_cast<uint32_t*>(&y);
}

// Four values, divided by the scale already and in the codes' range, as codes: nearest, ties
// to even.
template <int kFormat>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (kFormat == RKV_Q8_E4M3) {
    uint32_t w;
    asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
        " mov.b32 %0, {x, y};\n}\n"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
  }
  const uint32_t x = (uint32_t)__float2int_rn(a) & 0xffu, y = (uint32_t)__float2int_rn(b) & 0xffu;
  const uint32_t z = (uint32_t)__float2int_rn(c) & 0xffu, v = (uint32_t)__float2int_rn(d) & 0xffu;
  return x | (y << 8) | (z << 16) | (v << 24);
}

// The scale of a block of largest magnitude `top` (fp32 bits, finite): 2^e with e =
// ceil(log2(top / largest code)), at least 2^-126.  448 = 1.75 2^8 and 127 = 1.984375 2^6: e
// is top's exponent - 8 or - 6, one more where its mantissa lies above 1.75 or 1.984375,
// which an addition carries into the exponent.
template <int kFormat>
__device__ __forceinline__ float scale_of(uint32_t top) {
  const int e = kFormat == RKV_Q8_E4M3 ? (int)((top + 0x1fffffu) >> 23) - 8 : (int)((top + 0x1ffffu) >> 23) - 6;
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}
// 1 / scale, exact (0 < scale <= 2^122, a power of two).
__device__ __forceinline__ float inverse_scale(float scale) {
  return __uint_as_float((254u << 23) - __float_as_uint(scale));
}

}  // namespace rkv
