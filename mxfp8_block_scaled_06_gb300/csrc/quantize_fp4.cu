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
#include <type_traits>

#include "fp4.cuh"
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
    if (y != nullptr) y[u] = e2m1_values_bf16(codes, scale_value(s));
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
