// rope.cu - rotary positions: the table of cosines and sines, and the rotation of
// part of each head.
//
// Pair i of d_rope / 2 turns by p f_i radians at position p. The rotation of a pair is
//   a' = a cos - b sin,  b' = b cos + a sin
// in float32, each product and each sum rounded on its own (as the projection behind the
// attention undoes it, wo_a.cu), rounded once to the element type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

// ------------------------------------------------------------------ table
// An angle is kept as a 64-bit fraction of a turn: turn = 2^64 f / (2 pi), so that
// p * turn mod 2^64 is the angle without its whole turns, exactly but for turn's own
// rounding (2^-53 of it: 1e-10 radians at position 2^20). The top two bits, rounded, are the
// quadrant; the signed rest, at most an eighth of a turn, becomes a float, whose sine
// and cosine are the Taylor polynomials of degree 9 and 10: on pi / 4 their errors are
// below 2e-9 and 2e-10, a thirtieth of half a step of float32.
//
// Bound by its stores: 4 d_rope bytes a position (163840 positions of 64 dimensions 9.2 us, 4.6 TB/s).
// Double precision, a 64th of the float32 rate here, stays on the host.
constexpr int kTableThreads = 256;

struct Turns {
  uint64_t turn[kRopeMaxDim / 2];
};

__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(Turns turns, int max_pos, int half, int rows, float magnitude, float* __restrict__ cos_sin) {
  // `rows` positions of a block at once, `half` threads to each; a thread keeps its pair
  pdl_launch_dependents();
  __shared__ uint64_t turn[kRopeMaxDim / 2];
  for (int i = threadIdx.x; i < half; i += kTableThreads) turn[i] = turns.turn[i];
  __syncthreads();
  const int i = threadIdx.x % half, r = threadIdx.x / half;
  pdl_wait();
  if (r >= rows) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  const uint64_t g = turn[i], g_step = g * static_cast<uint64_t>(step);
  int64_t p = static_cast<int64_t>(blockIdx.x) * rows + r;
  uint64_t phase = g * static_cast<uint64_t>(p);
  float* out = cos_sin + p * (2 * half) + i;
  for (; p < max_pos; p += step, phase += g_step, out += step * (2 * half)) {
    const uint32_t quadrant = static_cast<uint32_t>((phase + (uint64_t{1} << 61)) >> 62);
    const uint64_t rest = phase - (static_cast<uint64_t>(quadrant) << 62);
    const float hi = static_cast<float>(static_cast<int32_t>(rest >> 32));
    const float x = fmaf(static_cast<float>(static_cast<uint32_t>(rest)), 0x1p-32f, hi) *
                    static_cast<float>(6.283185307179586 / 4294967296.0);
    const float z = x * x;
    float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(s, z, 1.f / 120.f);
    s = fmaf(s, z, -1.f / 6.f);
    s = fmaf(s * z, x, x);
    float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(c, z, -1.f / 720.f);
    c = fmaf(c, z, 1.f / 24.f);
    c = fmaf(c, z, -0.5f);
    c = fmaf(c, z, 1.f);
    const bool swap = quadrant & 1u;
    float cs = swap ? s : c, sn = swap ? c : s;
    // quadrants 1 and 2 have a negative cosine, 2 and 3 a negative sine
    cs = __uint_as_float(__float_as_uint(cs) ^ (((quadrant + 1) & 2u) << 30));
    sn = __uint_as_float(__float_as_uint(sn) ^ ((quadrant & 2u) << 30));
    out[0] = cs * magnitude;
    out[half] = sn * magnitude;
  }
}

// --------------------------------------------------------------- rotation
// Bound by memory, an element in and out: 8191 tokens of 32 heads of 128 out of wider rows 23.6 us, 5.9 TB/s (86 % of
// a copy's rate).
constexpr int kRopeThreads = 256;

// V elements of T, loaded and stored as one word of V * sizeof(T) bytes.
template <int kBytes>
struct Word;
template <>
struct Word<2> {
  using type = unsigned short;
};
template <>
struct Word<4> {
  using type = uint32_t;
};
template <>
struct Word<8> {
  using type = uint2;
};
template <>
struct Word<16> {
  using type = uint4;
};

template <typename T, int V>
union Vec {
  typename Word<V * sizeof(T)>::type word;
  T e[V];
  __device__ Vec() {}
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float& o) { o = v; }
__device__ __forceinline__ void from_float(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// N floats from p, four or two at once where V elements of the heads are (then p is
// aligned too: d_rope is a multiple of 2 V or V, and the table is 16-byte aligned).
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else if constexpr (N == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x, v[1] = f.y;
  } else {
    v[0] = p[0];
  }
}

// A thread has one chunk of V elements (of V pairs where the halves are apart) of kHeads
// heads of a token, kHeads apart from the next thread's: the token's cosines and sines
// are loaded once for all of them. Chunks [0, turned) are rotated, the others copied.
template <typename T, int V, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeRows a) {
  pdl_launch_dependents();
  const uint32_t u = blockIdx.x * kRopeThreads + threadIdx.x;
  const uint32_t row = div_u32(u, a.per_row);  // (token, group of heads)
  const uint32_t chunk = u - row * a.chunks;
  const uint32_t t = div_u32(row, a.per_token);
  const uint32_t h0 = (row - t * a.head_groups) * kHeads;
  if (u >= a.units) return;
  const int nh = min(kHeads, a.heads - static_cast<int>(h0));
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(t) * a.ldx + static_cast<size_t>(h0) * a.ldx_head;
  T* out = static_cast<T*>(a.out) + static_cast<size_t>(t) * a.ldo + static_cast<size_t>(h0) * a.ldo_head;
  using Word_t = typename Word<V * sizeof(T)>::type;
  if (chunk >= a.turned) {
    uint32_t e = (chunk - a.turned) * V;
    if (e >= a.first) e += a.d_rope;
    Word_t w[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < nh) w[h] = *reinterpret_cast<const Word_t*>(x + static_cast<size_t>(h) * a.ldx_head + e);
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < nh) *reinterpret_cast<Word_t*>(out + static_cast<size_t>(h) * a.ldo_head + e) = w[h];
    return;
  }
  const uint32_t half = a.d_rope >> 1;
  int64_t pos = a.positions[t];
  if (pos < 0 || pos >= a.max_pos) {
    if (chunk == 0 && h0 == 0) atomicOr(a.status, kStatusBadInput);
    pos = 0;
  }
  const float* cs = a.cos_sin + pos * a.d_rope;
  const uint32_t e = a.first + chunk * V;
  if constexpr (kInterleaved) {
    constexpr int P = V / 2;
    float c[P], s[P];
    load_floats(cs + chunk * P, c);
    load_floats(cs + half + chunk * P, s);
    Vec<T, V> v[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < nh) v[h].word = *reinterpret_cast<const Word_t*>(x + static_cast<size_t>(h) * a.ldx_head + e);
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h >= nh) break;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float p = to_float(v[h].e[2 * i]), q = to_float(v[h].e[2 * i + 1]), w = a.inverse ? -s[i] : s[i];
        from_float(__fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, w)), v[h].e[2 * i]);
        from_float(__fadd_rn(__fmul_rn(q, c[i]), __fmul_rn(p, w)), v[h].e[2 * i + 1]);
      }
      *reinterpret_cast<Word_t*>(out + static_cast<size_t>(h) * a.ldo_head + e) = v[h].word;
    }
  } else {
    float c[V], s[V];
    load_floats(cs + chunk * V, c);
    load_floats(cs + half + chunk * V, s);
    Vec<T, V> p[kHeads], q[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < nh) {
        p[h].word = *reinterpret_cast<const Word_t*>(x + static_cast<size_t>(h) * a.ldx_head + e);
        q[h].word = *reinterpret_cast<const Word_t*>(x + static_cast<size_t>(h) * a.ldx_head + e + half);
      }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h >= nh) break;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = to_float(p[h].e[i]), g = to_float(q[h].e[i]), w = a.inverse ? -s[i] : s[i];
        from_float(__fsub_rn(__fmul_rn(f, c[i]), __fmul_rn(g, w)), p[h].e[i]);
        from_float(__fadd_rn(__fmul_rn(g, c[i]), __fmul_rn(f, w)), q[h].e[i]);
      }
      *reinterpret_cast<Word_t*>(out + static_cast<size_t>(h) * a.ldo_head + e) = p[h].word;
      *reinterpret_cast<Word_t*>(out + static_cast<size_t>(h) * a.ldo_head + e + half) = q[h].word;
    }
  }
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel kernel, dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTable& t, int sm_count, float* cos_sin, cudaStream_t stream) {
  Turns turns = {};
  const int half = t.d_rope / 2;
  const double pi = 3.14159265358979323846;
  // pairs that turn more often than beta_fast times in the original context keep their
  // frequency, those that turn less often than beta_slow are interpolated, and between the
  // two the share goes linearly with the pair's number (Peng et al., 2023)
  double lo = 0, hi = 0;
  if (t.scaling == kRopeYarn) {
    auto at = [&](double beta) { return t.d_rope * std::log(t.original / (2 * pi * beta)) / (2 * std::log(t.base)); };
    lo = std::max(std::floor(at(t.beta_fast)), 0.0);
    hi = std::min(std::ceil(at(t.beta_slow)), t.d_rope - 1.0);
  }
  for (int i = 0; i < half; ++i) {
    double f = std::pow(t.base, -2.0 * i / t.d_rope);
    if (t.scaling == kRopeLinear) f /= t.factor;
    if (t.scaling == kRopeYarn) {
      const double r = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1 - r) + f / t.factor * r;
    }
    const double turn = f / (2 * pi);
    // whole turns of a position change nothing; 2^64 itself does not fit
    turns.turn[i] = static_cast<uint64_t>((turn - std::floor(turn)) * 18446744073709551616.0);
  }
  const int rows = std::max(kTableThreads / half, 1);
  const int64_t blocks = (static_cast<int64_t>(t.max_pos) + rows - 1) / rows;
  const int grid = static_cast<int>(std::min<int64_t>(blocks, 8 * sm_count));
  return launch_pdl(rope_table_kernel, dim3(grid), dim3(kTableThreads), stream, turns, t.max_pos, half, rows,
                    t.magnitude, cos_sin);
}

namespace {

template <typename T, int V, bool kInterleaved>
cudaError_t rope_run(RopeRows a, cudaStream_t stream) {
  a.turned = static_cast<uint32_t>(kInterleaved ? a.d_rope / V : a.d_rope / 2 / V);
  // in place the other elements are already there
  const bool copies = a.x != a.out;
  a.chunks = a.turned + (copies ? static_cast<uint32_t>(a.d - a.d_rope) / V : 0u);
  auto go = [&](auto kernel, int heads) {
    a.head_groups = (a.heads + heads - 1) / heads;
    const int64_t units = static_cast<int64_t>(a.tokens) * a.head_groups * a.chunks;
    if (units >= int64_t{1} << 32) return cudaErrorInvalidValue;  // refused before (api.cu)
    a.units = static_cast<uint32_t>(units);
    a.per_row = fast_div(a.chunks);
    a.per_token = fast_div(a.head_groups);
    return launch_pdl(kernel, dim3(static_cast<uint32_t>((units + kRopeThreads - 1) / kRopeThreads)),
                      dim3(kRopeThreads), stream, a);
  };
  // several heads to a thread only where that leaves enough threads for all SMs
  const int64_t one = static_cast<int64_t>(a.tokens) * a.heads * a.chunks;
  return a.heads >= 4 && one >= kRopeManyUnits ? go(rope_kernel<T, V, kInterleaved, 4>, 4) : go(rope_kernel<T, V, kInterleaved, 1>, 1);
}

template <typename T>
cudaError_t rope_pick(const RopeRows& a, int vec, cudaStream_t stream) {
  constexpr int kMost = 16 / sizeof(T);
  if (a.interleaved) {
    if (vec >= kMost) return rope_run<T, kMost, true>(a, stream);
    if (vec == 4) return rope_run<T, 4, true>(a, stream);
    return rope_run<T, 2, true>(a, stream);
  }
  if (vec >= kMost) return rope_run<T, kMost, false>(a, stream);
  if (vec == 4) return rope_run<T, 4, false>(a, stream);
  if (vec == 2) return rope_run<T, 2, false>(a, stream);
  return rope_run<T, 1, false>(a, stream);
}

}  // namespace

// Elements that every chunk can be moved by at once: a power of two that divides all
// offsets and strides.
int rope_vec(const RopeRows& a, int size) {
  uint64_t all = static_cast<uint64_t>(a.d) | static_cast<uint64_t>(a.first) | static_cast<uint64_t>(a.ldx) |
                 static_cast<uint64_t>(a.ldx_head) | static_cast<uint64_t>(a.ldo) | static_cast<uint64_t>(a.ldo_head) |
                 static_cast<uint64_t>(a.interleaved ? a.d_rope : a.d_rope / 2) |
                 reinterpret_cast<uintptr_t>(a.x) / size | reinterpret_cast<uintptr_t>(a.out) / size;
  int v = 1;
  while (v < 16 / size && (all & v) == 0) v *= 2;
  return v;
}

cudaError_t launch_rope(const RopeRows& a, int x_type, cudaStream_t stream) {
  const int vec = rope_vec(a, x_type == kTypeF32 ? 4 : 2);
  if (x_type == kTypeF32) return rope_pick<float>(a, vec, stream);
  if (x_type == kTypeF16) return rope_pick<__half>(a, vec, stream);
  return rope_pick<__nv_bfloat16>(a, vec, stream);
}

}  // namespace mx
