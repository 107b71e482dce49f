// fp4.cuh - E2M1 codes and the values they stand for, eight elements at a time: what the
// row quantizer and the attention cache share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "kernels.h"

namespace mx {

// n / d for the d that (mul, shift) was made for (host: fast_div).
__device__ __forceinline__ uint32_t div_u32(uint32_t n, FastDiv f) {
  const uint32_t t = __umulhi(f.mul, n);
  return f.shift < 0 ? n : (t + ((n - t) >> 1)) >> f.shift;
}

// Eight floats times f -> eight E2M1 codes, the first in the low bits.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8], float f) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f),
        "f"(v[6] * f), "f"(v[7] * f));
  return r;
}

// Eight elements as loaded, their values, and the bits of the largest magnitude as a
// float: at or above Inf's bits when any element is Inf or NaN.
template <typename T>
struct Unit {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
  // magnitudes of either 16-bit type order as unsigned numbers, NaN last: two at a time
  __device__ __forceinline__ uint32_t amax() const {
    constexpr uint32_t kMag = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(raw.x & kMag, raw.y & kMag), __vmaxu2(raw.z & kMag, raw.w & kMag));
    return max(m & 0xFFFFu, m >> 16);
  }
  static __device__ __forceinline__ uint32_t amax_bits(uint32_t m) {
    if constexpr (std::is_same<T, __half>::value)
      return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    else
      return m << 16;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};
template <>
struct Unit<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t amax() const {
    float v[8];
    values(v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ uint32_t amax_bits(uint32_t m) { return m; }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// 2^(s - 127) of scale byte s: 0 is the subnormal 2^-127, 0xFF NaN.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 0     ? __uint_as_float(0x00400000u)
         : s < 255u ? __uint_as_float(s << 23)
                    : __uint_as_float(0x7FC00000u);
}
// The four bytes of w, two codes each, as fp16 pairs (low code in the low half).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes times f in bf16, exact where f is a scale (one mantissa bit). Exponent and upper
// mantissa bits of an fp16 code are those of a bf16 number 2^112 times smaller.
__device__ __forceinline__ uint4 e2m1_values_bf16(uint32_t codes, float f) {
  const uint32_t f2 = (__float_as_uint(f) >> 16) * 0x10001u;
  uint32_t w[4];
  codes_f16(codes, w);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = mul_bf16x2(mul_bf16x2((w[e] >> 3 & 0x0FFF0FFFu) | (w[e] & 0x80008000u), 0x77807780u), f2);  // 2^112
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace mx
