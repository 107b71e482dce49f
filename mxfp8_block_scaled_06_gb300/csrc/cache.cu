// cache.cu - the attention cache in MXFP4: rows of keys and values quantized into its
// pages as they are written, and read back.
//
// A pool holds [pages][heads][page_size] rows of d / 2 bytes of E2M1 codes, and another
// the d / 32 scale bytes of each row: a page's rows of one head lie together, so the
// attention reads a head's tokens in runs of whole pages. A slot is page * page_size +
// place. The rule of a 32-block is the row quantizer's (quantize_fp4.cu).
//
// Both are bound by memory: 2 bytes an element in (or out), 0.53 out (in), and 2 more where
// the values are wanted too. A thread has sixteen elements, half a block, which it loads or stores as 32
// bytes: with eight (16 bytes) the places' divisions and addresses came twice as often, and took 40 us instead of
// 30 for 32749 rows of 8 heads of 128 written, 43 instead of 30 for as many read (5.6 TB/s, of 6.8 that a copy
// has; where rows fit the L2 cache, 16381 of them, 6.4). Codes become fp16, and bf16 from there by shifts and
// exact products, in 27 instructions for eight; one by one they took 56.
#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256, kReadUnits = 2, kWriteUnits = 2;

// Where unit u (sixteen elements) of [rows][heads][d] lies.
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

// 32 bytes, at once where they are aligned.
__device__ __forceinline__ void store32(void* to, uint4 a, uint4 b, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(to)[0] = a;
    static_cast<uint4*>(to)[1] = b;
  }
}
// Sixteen codes times f.
__device__ __forceinline__ void store_values(__nv_bfloat16* out, uint2 codes, float f, bool whole) {
  store32(out, e2m1_values_bf16(codes.x, f), e2m1_values_bf16(codes.y, f), whole);
}
__device__ __forceinline__ float2 code_values(uint32_t pair, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&pair));
  return make_float2(v.x * f, v.y * f);
}
__device__ __forceinline__ uint4 values_f16(uint32_t codes, float f) {
  uint32_t w[4];
  codes_f16(codes, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 p = __float22half2_rn(code_values(w[e], f));
    w[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_values(__half* out, uint2 codes, float f, bool whole) {
  store32(out, values_f16(codes.x, f), values_f16(codes.y, f), whole);
}
__device__ __forceinline__ void store_values(float* out, uint2 codes, float f, bool whole) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
    codes_f16(i == 0 ? codes.x : codes.y, w);
    uint4 v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 a = code_values(w[2 * e], f), b = code_values(w[2 * e + 1], f);
      v[e] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
    store32(out + 8 * i, v[0], v[1], whole);
  }
}

// Sixteen elements.
__device__ __forceinline__ void load32(const void* from, uint4& a, uint4& b, bool whole) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(from));
  } else {
    a = static_cast<const uint4*>(from)[0];
    b = static_cast<const uint4*>(from)[1];
  }
}
template <typename T>
__device__ __forceinline__ void load_units(const T* from, Unit<T> (&to)[2], bool whole) {
  load32(from, to[0].raw, to[1].raw, whole);
}
__device__ __forceinline__ void load_units(const float* from, Unit<float> (&to)[2], bool whole) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint4 a, b;
    load32(from + 8 * j, a, b, whole);
    to[j].a = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
    to[j].b = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
  }
}

// blockIdx.y: 0 keys, 1 values. Two threads share a block.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheRows a) {
  pdl_launch_dependents();
  const CacheSide& side = a.side[blockIdx.y];
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  const bool whole_x = ((reinterpret_cast<uintptr_t>(side.x) | side.ldx * sizeof(T) | side.ldx_head * sizeof(T)) & 31) == 0;
  const bool whole_y = (reinterpret_cast<uintptr_t>(side.y) & 31) == 0;
  Place at[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) at[i] = place_of(u0 + i * kThreads, a);
  pdl_wait();
  Unit<T> in[kUnits][2];
  int64_t slot[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (u0 + i * kThreads < a.units) {
      load_units(static_cast<const T*>(side.x) + static_cast<size_t>(at[i].row) * side.ldx +
                     static_cast<size_t>(at[i].head) * side.ldx_head + at[i].col * 16,
                 in[i], whole_x);
      slot[i] = a.slots[at[i].row];
    } else {
      in[i][0].zero();
      in[i][1].zero();
      slot[i] = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = u0 + i * kThreads;
    // a block's two threads are neighbours, and units % 2 == 0: they are in range together
    uint32_t amax = max(in[i][0].amax(), in[i][1].amax());
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = Unit<T>::amax_bits(amax);
    const bool finite = amax < 0x7F800000u;
    const uint32_t s = finite ? static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - 2, 0)) : 0xFFu;
    uint32_t codes[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v[8];
      in[i][j].values(v);
      codes[j] = finite ? cvt_e2m1x8(v, mx_inv_scale(s)) : 0u;
    }
    if (u >= a.units) continue;
    if (side.y != nullptr)
      store_values(static_cast<__nv_bfloat16*>(side.y) + static_cast<size_t>(u) * 16, make_uint2(codes[0], codes[1]),
                   scale_value(s), whole_y);
    if (slot[i] < 0) continue;
    if (slot[i] >= a.slot_count) {
      if (at[i].head == 0 && at[i].col == 0) atomicOr(a.status, kStatusBadInput);
      continue;
    }
    const uint32_t sl = static_cast<uint32_t>(slot[i]);
    *reinterpret_cast<uint2*>(side.codes + row_at(sl, at[i].head, a, side.page_stride, a.head_units * 8) +
                              at[i].col * 8) = make_uint2(codes[0], codes[1]);
    if ((at[i].col & 1u) == 0)
      side.scales[row_at(sl, at[i].head, a, side.scale_page_stride, a.head_units >> 1) + (at[i].col >> 1)] =
          static_cast<uint8_t>(s);
  }
}

template <typename T, int kUnits>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheRows a) {
  pdl_launch_dependents();
  const CacheSide& side = a.side[blockIdx.y];
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  const bool whole = (reinterpret_cast<uintptr_t>(side.y) & 31) == 0;
  Place at[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) at[i] = place_of(u0 + i * kThreads, a);
  pdl_wait();
  int64_t slot[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) slot[i] = u0 + i * kThreads < a.units ? a.slots[at[i].row] : -1;
  uint2 codes[kUnits];
  uint32_t scale[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (slot[i] >= a.slot_count) {
      if (at[i].head == 0 && at[i].col == 0) atomicOr(a.status, kStatusBadInput);
      slot[i] = -1;
    }
    if (slot[i] < 0) continue;
    const uint32_t sl = static_cast<uint32_t>(slot[i]);
    codes[i] = *reinterpret_cast<const uint2*>(
        side.codes + row_at(sl, at[i].head, a, side.page_stride, a.head_units * 8) + at[i].col * 8);
    scale[i] = side.scales[row_at(sl, at[i].head, a, side.scale_page_stride, a.head_units >> 1) + (at[i].col >> 1)];
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (slot[i] >= 0)
      store_values(static_cast<T*>(side.y) + static_cast<size_t>(u0 + i * kThreads) * 16, codes[i], scale_value(scale[i]),
                   whole);
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
    return many ? launch(cache_write_kernel<T, kWriteUnits>, a, kWriteUnits, stream) : launch(cache_write_kernel<T, 1>, a, 1, stream);
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
    return many ? launch(cache_read_kernel<T, kReadUnits>, a, kReadUnits, stream) : launch(cache_read_kernel<T, 1>, a, 1, stream);
  };
  if (out_type == kTypeF32) return pick(static_cast<float*>(nullptr));
  if (out_type == kTypeF16) return pick(static_cast<__half*>(nullptr));
  return pick(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace mx
