// quantize_fp4.cu - rows of bf16 / fp16 / fp32 -> MXFP4 (E2M1, two codes to a
// byte, + one UE8M0 scale per 32 along K), optionally with the values that the
// codes stand for in bf16.
//
// Per 32-block: e = floor(log2 amax) - 2 (the largest E2M1 binade is 2^2),
// clamped below at -127; codes = E2M1 round-to-nearest-even of x 2^-e,
// saturating at +-6; scale byte e + 127. x 2^-e is exact (a power of two), so
// the only rounding is the one to E2M1. A block with an Inf or NaN gets scale
// byte 0xFF (the scale format's NaN) and zero codes: E2M1 has no NaN of its own.
// The value c 2^e has one mantissa bit, so bf16 holds it exactly (its smallest,
// 2^-128, is a bf16 subnormal).
//
// Bound by memory: 2 (4) bytes in, 0.53 out, and 2 more for the values. Four threads
// share a block, eight elements each: one 16-byte load (32 bytes
// for fp32), two xor-shuffles for the block's amax, one 4-byte store of codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;
// From this many units on (8 Mi elements) a thread takes four, whose loads are in
// flight together: 16381 x 8192 bf16 70.7 -> 57.5 us, with y 103 -> 90 us (6.7 TB/s, a
// plain copy's rate), 1024 x 8192 4.9 -> 4.2 us; 512 x 8192 takes 3.7 us either way and
// smaller calls need the blocks. Streaming loads and stores (.cs) were slower: 62 and
// 95 us.
constexpr uint32_t kManyUnits = 1u << 20;

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

// The value of E2M1 code c (sign in bit 3): the magnitude's exponent and mantissa
// bits are those of a float 2^126 times smaller, shifted into place; one exact
// multiplication restores the exponent (and makes code 1 the subnormal 0.5).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const float m = __uint_as_float((c & 7u) << 22) * __uint_as_float(253u << 23);
  return __uint_as_float(__float_as_uint(m) | ((c & 8u) << 28));
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

// kUnits 8-element units per thread, kThreads apart: their loads are in flight together.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_fp4_kernel(const T* x, long ldx, int M, int K, uint32_t* __restrict__ q,
                             uint8_t* __restrict__ scales, int swizzled, uint4* __restrict__ y, uint32_t units,
                             FastDiv per_row, uint32_t unit_blocks) {
  pdl_launch_dependents();
  if (blockIdx.x >= unit_blocks) {
    // rows [M, ceil128(M)) of the swizzled scales: zero, four to a thread
    const uint32_t words = ((static_cast<uint32_t>(K) >> 5) + 3) >> 2;  // of a row
    const uint32_t i = (blockIdx.x - unit_blocks) * kThreads + threadIdx.x;
    pdl_wait();
    if (i < (-M & 127) * words)
      *reinterpret_cast<uint32_t*>(scales + swz_offset(M + i / words, i % words * 4, words * 4)) = 0u;
    return;
  }
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;  // 8-element unit, row-major
  const uint32_t upr = static_cast<uint32_t>(K) >> 3;
  const uint32_t nblk = static_cast<uint32_t>(K) >> 5;
  const uint32_t cpad4 = (nblk + 3) & ~3u;
  uint32_t row[kUnits], col[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    row[i] = div_u32(u0 + i * kThreads, per_row);
    col[i] = u0 + i * kThreads - row[i] * upr;
  }
  pdl_wait();
  Unit<T> in[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (u0 + i * kThreads < units)
      in[i].load(x + static_cast<size_t>(row[i]) * ldx + col[i] * 8);
    else
      in[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = u0 + i * kThreads;
    // units % 4 == 0 and a block's four threads are neighbours: they are in range together
    const bool valid = u < units;
    uint32_t amax = in[i].amax();
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    amax = Unit<T>::amax_bits(amax);
    const bool finite = amax < 0x7F800000u;
    const uint32_t s = finite ? static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - 2, 0)) : 0xFFu;
    float v[8];
    in[i].values(v);
    const uint32_t codes = finite ? cvt_e2m1x8(v, mx_inv_scale(s)) : 0u;
    if (!valid) continue;
    q[u] = codes;
    if (y != nullptr) {
      // 2^(s - 127): s = 0 is the subnormal 2^-127, 0xFF is NaN
      const float f = s == 0   ? __uint_as_float(0x00400000u)
                      : finite ? __uint_as_float(s << 23)
                               : __uint_as_float(0x7FC00000u);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = e2m1_value(codes >> (8 * e)) * f, b = e2m1_value(codes >> (8 * e + 4)) * f;
        w[e] = __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xFFFF0000u);  // exact: the low halves are zero
      }
      y[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if ((col[i] & 3) != 0) continue;
    const uint32_t blk = col[i] >> 2;
    scales[swizzled ? swz_offset(row[i], blk, cpad4) : row[i] * static_cast<size_t>(nblk) + blk] =
        static_cast<uint8_t>(s);
    if (swizzled && blk == nblk - 1)
      for (uint32_t c = nblk; c < cpad4; ++c) scales[swz_offset(row[i], c, cpad4)] = 0;  // padding columns
  }
}

}  // namespace

// Division by d as a multiplication, for every 32-bit n: with l = ceil(log2 d)
// and m = floor(2^32 (2^l - d) / d) + 1, n / d = (t + (n - t) / 2) >> (l - 1)
// where t is the high word of m n (Granlund and Montgomery, 1994).
FastDiv fast_div(uint32_t d) {
  int l = 0;
  while ((uint64_t{1} << l) < d) ++l;
  return FastDiv{static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - d)) / d + 1), l - 1};
}

cudaError_t launch_quantize_rows_fp4(const void* x, long ldx, int x_type, int M, int K, void* q, void* scales,
                                     int swizzled, void* y, cudaStream_t stream) {
  const uint32_t units = static_cast<uint32_t>(static_cast<long>(M) * K / 8);
  const bool many = units >= kManyUnits;
  const uint32_t per_block = kThreads * (many ? 4 : 1);
  cudaLaunchConfig_t cfg = {};
  const uint32_t unit_blocks = (units + per_block - 1) / per_block;
  const uint32_t pad_words = swizzled ? (-M & 127) * ((K / 32 + 3) / 4) : 0;
  cfg.gridDim = dim3(unit_blocks + (pad_words + kThreads - 1) / kThreads);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const FastDiv per_row = fast_div(static_cast<uint32_t>(K / 8));
  auto go = [&](auto kernel, auto* p) {
    return cudaLaunchKernelEx(&cfg, kernel, p, ldx, M, K, static_cast<uint32_t*>(q), static_cast<uint8_t*>(scales),
                              swizzled, static_cast<uint4*>(y), units, per_row, unit_blocks);
  };
  auto pick = [&](auto* p) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    return many ? go(quantize_rows_fp4_kernel<T, 4>, p) : go(quantize_rows_fp4_kernel<T, 1>, p);
  };
  if (x_type == kTypeF32) return pick(static_cast<const float*>(x));
  if (x_type == kTypeF16) return pick(static_cast<const __half*>(x));
  return pick(static_cast<const __nv_bfloat16*>(x));
}

}  // namespace mx
