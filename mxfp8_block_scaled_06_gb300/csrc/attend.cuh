// attend.cuh - what the three kernels of the attention over the MXFP4 cache share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

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
// Waits for loaded values before later loads are issued: a wait that came after those would be for
// them as well (of six counters, loads of one kind share one), a whole memory latency.
__device__ __forceinline__ void arrived(uint32_t v) { asm volatile("" ::"r"(v) : "memory"); }
__device__ __forceinline__ uint32_t folded(uint4 v) { return (v.x ^ v.y) ^ (v.z ^ v.w); }
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

// ------------------------------------------------------------- runs of work
// Places in front of a unit's tiles, for its queries and results: runs are to be equal in time, not in tiles. (61
// sequences of up to 4096 tokens, grouped heads: 58 us without, 52 with one or two; with four queries each 146,
// 131, 122; 48 sequences of up to 32768 latents 127, 123, 128.)
template <int D>
constexpr int kUnitExtra = D <= 128 ? 2 : 1;
template <int D>
__device__ __forceinline__ int64_t seq_work(const AttendArgs& a, const Seq& s) {
  return static_cast<int64_t>(s.tiles + kUnitExtra<D>) * s.row_tiles * a.heads;
}

struct Found {
  int b;          // the sequence that holds the tile
  int64_t first;  // number of its first tile
};
struct ScanShared {
  int64_t warp[16];
  Found found;
};
// The work of as many sequences as threads from c on, added up: this thread's sequence's, what is before it,
// and all.
template <int kRows, int kWarps, typename Work>
__device__ __forceinline__ int64_t scan_work(const AttendArgs& a, ScanShared& sh, int c, Work work, bool& bad,
                                             int64_t& before, int64_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = c + threadIdx.x;
  int64_t w = 0;
  if (b < a.B) {
    const Seq s = seq_of(a, b, kRows);
    w = work(a, s);
    bad |= s.bad;
  }
  int64_t sum = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) sh.warp[warp] = sum;
  __syncthreads();
  before = sum - w;
  all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sh.warp[i];
    all += sh.warp[i];
  }
  __syncthreads();
  return w;
}
// Tiles of each CTA's run: an equal share.
__device__ __forceinline__ int64_t run_of(int64_t total, int ctas) { return (total + ctas - 1) / ctas; }
// All work, and the sequence in which the run of this CTA begins (where it has one).
template <int kRows, int kWarps, typename Work>
__device__ __forceinline__ Found find_run(const AttendArgs& a, ScanShared& sh, Work work, int64_t& total) {
  constexpr int kThreads = 32 * kWarps;
  bool bad = false;
  int64_t before, all;
  const int64_t w = scan_work<kRows, kWarps>(a, sh, 0, work, bad, before, all);
  total = all;
  for (int c = kThreads; c < a.B; c += kThreads) {
    int64_t x;
    scan_work<kRows, kWarps>(a, sh, c, work, bad, x, all);
    total += all;
  }
  if (blockIdx.x == 0 && bad) atomicOr(a.status, kStatusBadInput);
  const int64_t at = run_of(total, gridDim.x) * blockIdx.x;
  if (before <= at && at < before + w) sh.found = Found{static_cast<int>(threadIdx.x), before};
  if (a.B > kThreads) {
    scan_work<kRows, kWarps>(a, sh, 0, work, bad, before, all);
    int64_t base = all;
    for (int c = kThreads; c < a.B; c += kThreads, base += all) {
      const int64_t v = scan_work<kRows, kWarps>(a, sh, c, work, bad, before, all);
      if (base + before <= at && at < base + before + v) sh.found = Found{c + static_cast<int>(threadIdx.x), base + before};
    }
  }
  __syncthreads();
  return sh.found;
}

// A unit: so many query rows of a kv head, row i the query token (row0 + i) / group.
struct AttendUnit {
  int head, row0, rows;  // rows: all of this sequence and head
  __device__ __forceinline__ bool row(const AttendArgs& a, const Seq& s, int i, int& token, int& q_head) const {
    const int r = row0 + i;
    token = r / a.group;
    q_head = head * a.group + r - token * a.group;
    token += s.q0;
    return r < rows;
  }
};

// A cut of a unit: written by the CTA whose run begins there.
struct Cut {
  int first, last;  // the CTAs that have parts of it; last < 0: the run does not begin within a unit
  int later;        // whether the first CTA's part is its second
  int head, row0, rows, q0;
  int pad;
};

// Floats of one CTA's part of a unit: the rows' maxima, sums, and weighted sums.
template <int D, int kRows>
constexpr int kPartFloats = kRows * (D + 2);
__host__ __device__ constexpr size_t cut_bytes(int ctas) { return static_cast<size_t>(ctas) * sizeof(Cut); }

// ------------------------------------------------------------- joining
// Block c is that of the cut where the run of CTA c + 1 begins. A unit of n parts has n - 1 cuts, whose
// blocks (one each, or one for 32 pieces) share its rows' pieces of 128 dimensions (64 at d = 64). A warp adds up a piece of
// some parts in the order of the runs; where there are many, 2 to 8 warps share a piece.
constexpr int kJoinThreads = 256, kAtOnce = 4;
template <int D, int kRows>
constexpr int kJoinBlocks = kRows * D / (D < 128 ? D : 128) > 32 ? kRows * D / (D < 128 ? D : 128) / 32 : 1;  // of a cut
template <int D, int kRows>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, int ctas) {
  constexpr int kPiece = D < 128 ? D : 128, kVec = kPiece / 32;  // floats of a thread
  constexpr int kPieces = kRows * D / kPiece, kWarpsHere = kJoinThreads / 32;
  __shared__ float sums[kWarpsHere][kPiece];
  __shared__ float2 tops[kWarpsHere];
  pdl_launch_dependents();
  pdl_wait();
  const Cut cut = reinterpret_cast<const Cut*>(a.partial)[blockIdx.x + 1];
  if (cut.last < 0) return;
  const float* parts0 = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(a.partial) + cut_bytes(ctas));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = cut.last - cut.first + 1, blocks = (n - 1) * gridDim.y;
  const int block = (static_cast<int>(blockIdx.x) - cut.first) * gridDim.y + blockIdx.y;
  const int team = n > 64 ? 8 : n > 32 ? 4 : n > 16 ? 2 : 1;  // warps to a piece
  const int at_once = kWarpsHere / team, share = warp % team;
  const int each = (n + team - 1) / team, p0 = min(share * each, n), p1 = min(p0 + each, n);
  auto part = [&](int p) {
    return parts0 + (static_cast<size_t>(cut.first + p) * 2 + (p == 0 ? cut.later : 0)) * kPartFloats<D, kRows>;
  };
  for (int x0 = block * at_once; x0 < kPieces; x0 += blocks * at_once) {
    const int piece = x0 + warp / team, r = piece / (D / kPiece), d = piece % (D / kPiece) * kPiece + lane * kVec;
    const bool here = piece < kPieces && cut.row0 + r < cut.rows;
    float top = -INFINITY, sum = 0.f, v[kVec] = {};
    if (here) {
#pragma unroll 1
      for (int p = p0; p < p1; p += kAtOnce) {
        // all loads first; behind the last part, that one again, which is not used
        float m[kAtOnce], l[kAtOnce], y[kAtOnce][kVec];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const float* from = part(min(p + i, p1 - 1));
          m[i] = from[r], l[i] = from[kRows + r];
          if constexpr (kVec == 4) {
            const float4 z = *reinterpret_cast<const float4*>(from + 2 * kRows + r * D + d);
            y[i][0] = z.x, y[i][1] = z.y, y[i][2] = z.z, y[i][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(from + 2 * kRows + r * D + d);
            y[i][0] = z.x, y[i][1] = z.y;
          }
        }
        float most = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) most = fmaxf(most, m[i]);
        // a row that saw nothing yet, or here, adds nothing, or the NaN that it saw
        const float keep = top == -INFINITY ? (sum != sum ? sum : 0.f) : exp2f(top - most);
        sum *= keep;
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] *= keep;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (p + i >= p1) break;
          const float f = m[i] == -INFINITY ? (l[i] != l[i] ? l[i] : 0.f) : exp2f(m[i] - most);
          sum += l[i] * f;
#pragma unroll
          for (int e = 0; e < kVec; ++e) v[e] += y[i][e] * f;
        }
        top = most;
      }
    }
    if (team > 1) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sums[warp][lane * kVec + e] = v[e];
      if (lane == 0) tops[warp] = make_float2(top, sum);
      __syncthreads();
      if (share == 0) {
        for (int i = 1; i < team; ++i) {
          const float2 t = tops[warp + i];
          const float most = fmaxf(top, t.x);
          const float keep = top == -INFINITY ? (sum != sum ? sum : 0.f) : exp2f(top - most);
          const float f = t.x == -INFINITY ? (t.y != t.y ? t.y : 0.f) : exp2f(t.x - most);
          sum = sum * keep + t.y * f;
#pragma unroll
          for (int e = 0; e < kVec; ++e) v[e] = v[e] * keep + sums[warp + i][lane * kVec + e] * f;
          top = most;
        }
      }
      __syncthreads();
    }
    if (!here || share != 0) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int q_row = cut.row0 + r, q_token = q_row / a.group, token = cut.q0 + q_token;
    const int q_head = cut.head * a.group + q_row - q_token * a.group;
    uint16_t* out = a.out + static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head + d;
    if constexpr (kVec == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_out(v[0] * inv, v[1] * inv, a.q_f16), pack_out(v[2] * inv, v[3] * inv, a.q_f16));
    else
      *reinterpret_cast<uint32_t*>(out) = pack_out(v[0] * inv, v[1] * inv, a.q_f16);
    if (a.lse != nullptr && d == 0)
      a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (top + log2f(sum)) * 0.6931471805599453f;
  }
}

// No more CTAs than places: every sequence has at most a block of rows more than its share.
inline int attend_ctas(const AttendArgs& a, int rows, int extra, int ctas) {
  const int64_t tiles = (static_cast<int64_t>(a.table_cols) * a.page_size + 15 + kAttendTile - 1) / kAttendTile;
  const int64_t units = (static_cast<int64_t>(a.T) * a.group / rows + std::min(a.B, a.T)) * a.heads;
  return static_cast<int>(std::min<int64_t>(ctas, (std::max<int64_t>(1, tiles) + extra) * units));
}

// A launch behind the previous kernel of the stream, which it may overlap.
template <typename Kernel, typename... Args>
cudaError_t launch_overlapping(Kernel kernel, dim3 grid, int threads, int bytes, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int kRows>
cudaError_t launch_join(const AttendArgs& a, int ctas, cudaStream_t stream) {
  return launch_overlapping(attend_join_kernel<D, kRows>, dim3(ctas - 1, kJoinBlocks<D, kRows>), kJoinThreads, 0, stream, a,
                            ctas);
}

}  // namespace mx
