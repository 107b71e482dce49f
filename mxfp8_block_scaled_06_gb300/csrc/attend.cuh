// attend.cuh - what the two kernels of the attention over the MXFP4 cache share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kAttendTile = 128;  // tokens of a tile

struct Seq {
  int q0, n;        // query tokens
  int len;          // cached tokens
  int start;        // first token that any row may see, rounded down to 16
  int tiles;        // of [start, len), one at least
  int row_tiles;
  bool bad;
};
// rows: of a unit.
__device__ __forceinline__ Seq seq_of(const AttendArgs& a, int b, int rows) {
  Seq s;
  int q1;
  if (a.q_offsets != nullptr) {
    s.q0 = a.q_offsets[b];
    q1 = a.q_offsets[b + 1];
  } else {
    s.n = a.T / a.B;
    s.q0 = b * s.n;
    q1 = s.q0 + s.n;
  }
  const int64_t most = static_cast<int64_t>(a.table_cols) * a.page_size;
  const int len = a.lengths[b];
  s.bad = s.q0 < 0 || q1 > a.T || q1 < s.q0 || len < 0 || len > most;
  s.n = s.q0 < 0 || q1 > a.T || q1 < s.q0 ? 0 : q1 - s.q0;
  s.len = len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
  const int64_t first = static_cast<int64_t>(s.len) - s.n - a.window + 1;
  s.start = a.window > 0 && first > 0 ? min(static_cast<int>(first), s.len) & ~15 : 0;
  s.tiles = max((s.len - s.start + kAttendTile - 1) / kAttendTile, 1);
  s.row_tiles = (s.n * a.group + rows - 1) / rows;
  return s;
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
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t p, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(static_cast<uint16_t>(v)) : "memory");
}

// The power of two that brings a row's largest magnitude (its bits as they are, sign off)
// into [2^14, 2^15); at most 2^100, as 2^-that has to be a normal number.
__device__ __forceinline__ int query_shift(uint32_t bits, int f16) {
  const int e = f16 ? static_cast<int>(bits >> 10) - 15 : static_cast<int>(bits >> 7) - 127;
  return min(14 - e, 100);
}
__device__ __forceinline__ uint32_t max_bits(uint4 v) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag));
  return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ uint32_t query_f16(uint32_t w, int f16, float f) {
  float lo, hi;
  if (f16) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = v.x, hi = v.y;
  } else {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
  }
  return pack_f16(lo * f, hi * f);
}
__device__ __forceinline__ uint4 query_f16(uint4 v, int f16, float f) {
  return make_uint4(query_f16(v.x, f16, f), query_f16(v.y, f16, f), query_f16(v.z, f16, f), query_f16(v.w, f16, f));
}
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int f16) {
  if (f16) return pack_f16(lo, hi);
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack_out8(const float* v, float f, int f16) {
  return make_uint4(pack_out(v[0] * f, v[1] * f, f16), pack_out(v[2] * f, v[3] * f, f16),
                    pack_out(v[4] * f, v[5] * f, f16), pack_out(v[6] * f, v[7] * f, f16));
}

}  // namespace mx
