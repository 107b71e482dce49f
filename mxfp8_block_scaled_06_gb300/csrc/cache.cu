// cache.cu - the attention cache in MXFP4: rows of keys and values quantized into its
// pages as they are written, and read back.
//
// A pool holds [pages][heads][page_size] rows of d / 2 bytes of E2M1 codes, and another
// the d / 32 scale bytes of each row: a page's rows of one head lie together, so the
// attention reads a head's tokens in runs of whole pages. A slot is page * page_size +
// place. The rule of a 32-block is the row quantizer's (quantize_fp4.cu).
//
// Both are bound by memory: 2 bytes an element in (or out), 0.53 out (in), and 2 more where
// the values are wanted too. Four threads share a block, eight elements each, as in the
// row quantizer.
#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

// Where unit u (eight elements) of [rows][heads][d] lies.
struct Place {
  uint32_t row, head, col;
};
__device__ __forceinline__ Place place_of(uint32_t u, const CacheRows& a) {
  const uint32_t rh = div_u32(u, a.per_head);
  Place p;
  p.col = u - rh * a.head_units;
  p.row = div_u32(rh, a.per_row);
  p.head = rh - p.row * a.heads;
  return p;
}

// The row of a slot within a pool of rows of `bytes` bytes.
__device__ __forceinline__ size_t row_at(uint32_t slot, uint32_t head, const CacheRows& a, long page_stride,
                                         uint32_t bytes) {
  const uint32_t page = div_u32(slot, a.per_page);
  return static_cast<size_t>(page) * page_stride +
         (static_cast<size_t>(head) * a.page_size + (slot - page * a.page_size)) * bytes;
}

// blockIdx.y: 0 keys, 1 values.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheRows a) {
  pdl_launch_dependents();
  const CacheSide& side = a.side[blockIdx.y];
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  Place at[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) at[i] = place_of(u0 + i * kThreads, a);
  pdl_wait();
  Unit<T> in[kUnits];
  int64_t slot[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (u0 + i * kThreads < a.units) {
      in[i].load(static_cast<const T*>(side.x) + static_cast<size_t>(at[i].row) * side.ldx +
                 static_cast<size_t>(at[i].head) * side.ldx_head + at[i].col * 8);
      slot[i] = a.slots[at[i].row];
    } else {
      in[i].zero();
      slot[i] = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = u0 + i * kThreads;
    // a block's four threads are neighbours, and units % 4 == 0: they are in range together
    uint32_t amax = in[i].amax();
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    amax = Unit<T>::amax_bits(amax);
    const bool finite = amax < 0x7F800000u;
    const uint32_t s = finite ? static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - 2, 0)) : 0xFFu;
    float v[8];
    in[i].values(v);
    const uint32_t codes = finite ? cvt_e2m1x8(v, mx_inv_scale(s)) : 0u;
    if (u >= a.units) continue;
    if (side.y != nullptr) static_cast<uint4*>(side.y)[u] = e2m1_values_bf16(codes, scale_value(s));
    if (slot[i] < 0) continue;
    if (slot[i] >= a.slot_count) {
      if (at[i].head == 0 && at[i].col == 0) atomicOr(a.status, kStatusBadInput);
      continue;
    }
    const uint32_t sl = static_cast<uint32_t>(slot[i]);
    *reinterpret_cast<uint32_t*>(side.codes + row_at(sl, at[i].head, a, side.page_stride, a.head_units * 4) +
                                 at[i].col * 4) = codes;
    if ((at[i].col & 3u) == 0)
      side.scales[row_at(sl, at[i].head, a, side.scale_page_stride, a.head_units >> 2) + (at[i].col >> 2)] =
          static_cast<uint8_t>(s);
  }
}

template <typename T>
__device__ __forceinline__ void store_values(T* out, uint32_t codes, float f);
template <>
__device__ __forceinline__ void store_values(__nv_bfloat16* out, uint32_t codes, float f) {
  *reinterpret_cast<uint4*>(out) = e2m1_values_bf16(codes, f);
}
template <>
__device__ __forceinline__ void store_values(__half* out, uint32_t codes, float f) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 p = __floats2half2_rn(e2m1_value(codes >> (8 * e)) * f, e2m1_value(codes >> (8 * e + 4)) * f);
    w[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store_values(float* out, uint32_t codes, float f) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e2m1_value(codes >> (4 * e)) * f;
  reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T, int kUnits>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheRows a) {
  pdl_launch_dependents();
  const CacheSide& side = a.side[blockIdx.y];
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  Place at[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) at[i] = place_of(u0 + i * kThreads, a);
  pdl_wait();
  uint32_t codes[kUnits], scale[kUnits];
  bool here[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t slot = u0 + i * kThreads < a.units ? a.slots[at[i].row] : -1;
    here[i] = slot >= 0 && slot < a.slot_count;
    if (slot >= a.slot_count && at[i].head == 0 && at[i].col == 0) atomicOr(a.status, kStatusBadInput);
    if (!here[i]) continue;
    const uint32_t sl = static_cast<uint32_t>(slot);
    codes[i] = *reinterpret_cast<const uint32_t*>(
        side.codes + row_at(sl, at[i].head, a, side.page_stride, a.head_units * 4) + at[i].col * 4);
    scale[i] = side.scales[row_at(sl, at[i].head, a, side.scale_page_stride, a.head_units >> 2) + (at[i].col >> 2)];
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (here[i])
      store_values(static_cast<T*>(side.y) + static_cast<size_t>(u0 + i * kThreads) * 8, codes[i],
                   scale_value(scale[i]));
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, const CacheRows& a, int units_a_thread, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const uint32_t per_block = kThreads * units_a_thread;
  cfg.gridDim = dim3((a.units + per_block - 1) / per_block, a.sides);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

CacheRows with_divisions(CacheRows a) {
  a.units = static_cast<uint32_t>(static_cast<int64_t>(a.rows) * a.heads * a.head_units);
  a.per_head = fast_div(a.head_units);
  a.per_row = fast_div(a.heads);
  a.per_page = fast_div(a.page_size);
  return a;
}

}  // namespace

cudaError_t launch_cache_write(const CacheRows& args, int x_type, cudaStream_t stream) {
  const CacheRows a = with_divisions(args);
  const bool many = a.units >= kCacheManyUnits;
  auto pick = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return many ? launch(cache_write_kernel<T, 4>, a, 4, stream) : launch(cache_write_kernel<T, 1>, a, 1, stream);
  };
  if (x_type == kTypeF32) return pick(static_cast<float*>(nullptr));
  if (x_type == kTypeF16) return pick(static_cast<__half*>(nullptr));
  return pick(static_cast<__nv_bfloat16*>(nullptr));
}

cudaError_t launch_cache_read(const CacheRows& args, int out_type, cudaStream_t stream) {
  const CacheRows a = with_divisions(args);
  const bool many = a.units >= kCacheManyUnits;
  auto pick = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return many ? launch(cache_read_kernel<T, 4>, a, 4, stream) : launch(cache_read_kernel<T, 1>, a, 1, stream);
  };
  if (out_type == kTypeF32) return pick(static_cast<float*>(nullptr));
  if (out_type == kTypeF16) return pick(static_cast<__half*>(nullptr));
  return pick(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace mx
