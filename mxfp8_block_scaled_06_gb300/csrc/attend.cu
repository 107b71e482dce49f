// attend.cu - attention of few query rows over the MXFP4 cache.
//
//   out[r] = sum over visible t of softmax_t(scale q[r].k[t]) v[t]
//
// The rows of a kv head (its group of query heads, of each query token) fill the 16 rows
// of mma.sync.m16n8k16, which reads its second operand from registers: the codes go from
// shared memory through cvt.f16x2.e2m1x2 and one multiplication by their scale straight
// into the products, without a stop in shared memory at 16 bits (for the 5th-generation
// tensor cores the dequantized tile would have to be written and read there: at d = 512
// 28 bytes of shared memory traffic for each byte of cache).
//
// In 16 bits. fp16 holds what is multiplied, under powers of two that keep all rounding
// out but where it says so:
//   keys    code * 2^(s - S + 7), s the block's scale and S the row's largest: exact down
//           to S - 30, nothing below S - 31 (2^-31 of the row's largest block); the score
//           takes 2^(S - 7) back in float32. Values the same.
//   queries times the power of two that brings the row's largest into [2^14, 2^15):
//           exact down to 2^-31 of it.
//   weights p = exp2(x + S_v - u + 8) rounded to fp16 (11 bits, where a bf16 weight would
//           have 8): x the score, S_v the value row's scale, u the running maximum of
//           x + S_v. So what is rounded, and below 2^-22 of the largest loses bits, is a
//           token's contribution, not its weight. The weights' sum is of float32 exponentials.
//
// Tokens go by in tiles of 128, 32 to each of four warps, through a ring filled by
// 16-byte asynchronous copies. Up to d = 128 a warp is on its own: it keeps the queries
// and its sums in registers, and four warps' results are joined at the end. Above, a
// warp computes the scores of its 32 tokens, hands the weights on through shared memory,
// and sums a quarter of the dimensions over all 128.
//
// The work of all sequences is cut into equal runs of tiles, one for each resident CTA,
// whatever the lengths; a run may end within a sequence. What a CTA has of a unit
// (sequence, kv head, 16 rows) that is not all its own goes to a workspace, from which a
// second kernel adds it up in the order of the tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attend.cuh"

namespace mx {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kSub = 32;                 // tokens of a warp's part of a tile
constexpr int kTile = kWarps * kSub;
static_assert(kTile == kAttendTile, "tiles of the sequences' work");
constexpr float kWeightBits = 8.f;       // weights are up to 2^8, scales up to 2^7
constexpr float kSumBits = 15.f;

// ------------------------------------------------------------- the work
__device__ __forceinline__ int64_t seq_work(const AttendArgs& a, const Seq& s) {
  return static_cast<int64_t>(s.tiles) * s.row_tiles * a.heads;
}

struct Found {
  int b;          // the sequence that holds the tile (B: none)
  int64_t first;  // number of its first tile
};
struct ScanShared {
  int64_t warp[kWarps];
  int64_t total;
  Found found;
};
// Work of all sequences; every thread of the block gets it.
__device__ int64_t total_work(const AttendArgs& a, ScanShared& sh, bool report) {
  int64_t sum = 0;
  bool bad = false;
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const Seq s = seq_of(a, b);
    sum += seq_work(a, s);
    bad |= s.bad;
  }
  if (report && bad) atomicOr(a.status, kStatusBadInput);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += sh.warp[w];
  __syncthreads();
  return sum;
}
// The sequence that holds tile `index` of the work.
__device__ Found find_work(const AttendArgs& a, ScanShared& sh, int64_t index) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh.found = Found{a.B, 0};
  int64_t base = 0;
  for (int c = 0; c < a.B && base <= index; c += kThreads) {
    const int b = c + threadIdx.x;
    const int64_t w = b < a.B ? seq_work(a, seq_of(a, b)) : 0;
    int64_t sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) sh.warp[warp] = sum;
    __syncthreads();
    int64_t before = base, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += sh.warp[i];
      all += sh.warp[i];
    }
    if (before + sum - w <= index && index < before + sum) sh.found = Found{b, before + sum - w};
    base += all;
    __syncthreads();
  }
  __syncthreads();
  return sh.found;
}
// Tiles of each CTA's run.
__device__ __forceinline__ int64_t run_of(int64_t total, int ctas) { return (total + ctas - 1) / ctas; }

// A unit: 16 query rows of a kv head. Row i is query token (16 r + i) / group.
struct Unit16 {
  int head, row0, rows;  // rows: all of this sequence and head
  __device__ __forceinline__ bool row(const AttendArgs& a, const Seq& s, int i, int& token, int& q_head) const {
    const int r = row0 + i;
    token = r / a.group;
    q_head = head * a.group + r - token * a.group;
    token += s.q0;
    return r < rows;
  }
};

// ------------------------------------------------------------- pieces
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Row t of a 16-token group lies at t * (d / 2), its 16-byte chunk c at c ^ flip(t): the
// eight tokens {0..3, 8..11} of one chunk (scores) and the four tokens {0..3} of two
// neighbouring chunks (sums), like those of the other halves, lie in 32 different banks.
template <int D>
__device__ __forceinline__ uint32_t flip(uint32_t t) {
  const uint32_t b3 = (t >> 3) & 1u;
  if constexpr (D == 64) return b3;
  if constexpr (D == 128) return (t & 2u) | b3;
  return ((t & 3u) << 1) | b3;
}

// fp16 bits of 2^(s - top + 7) for scale byte s: 0 below 2^-24, NaN for byte 255.
__device__ __forceinline__ uint32_t scale_f16(uint32_t s, int top) {
  const int e = static_cast<int>(s) - top + 22;  // biased exponent
  const uint32_t v = e >= 1 ? static_cast<uint32_t>(e) << 10 : e > -10 ? 1u << (9 + e) : 0u;
  return s == 255u ? 0x7E00u : v;
}

template <int D, bool kShared>
struct Layout {
  static constexpr bool kCoop = D > 128;
  static constexpr int kSides = kShared ? 1 : 2;
  static constexpr int kBlocks = D / 32;
  static constexpr int kCodes = kSub * D / 2;       // bytes of a warp's part of a stage
  static constexpr int kRaw = kSub * kBlocks;       // scale bytes
  static constexpr int kPart = kSides * (kCodes + kRaw);
  static constexpr int kStages = kCoop ? 2 : 4;
  static constexpr int kRing = kStages * kWarps * kPart;
  // fp16 scales of a warp's 32 tokens, block after block: two groups of eight words
  // {token i, token i + 8}, i in the order 0 4 1 5 2 6 3 7; 96 bytes apart, so that two
  // neighbouring blocks' words lie in different banks
  static constexpr int kScaleStride = 96;
  static constexpr int kScales = kBlocks * kScaleStride;
  static constexpr int kTokens = kSub * 8;  // {2^(S_k - 127), S_v - 127} of each token
  static constexpr int kSide = kSides * kScales + kTokens;  // of a warp
  static constexpr int kDump = kWarps * kAttendRows * (D + 4) * 4;
  static constexpr int kQ = kCoop ? kAttendRows * D * 2 : 0;
  static constexpr int kP = kCoop ? kTile / 16 * 512 : 0;
  static constexpr int kRingArea = !kCoop && kDump > kRing ? kDump : kRing;
  static constexpr int kOffSide = kRingArea;
  static constexpr int kOffQ = kOffSide + kWarps * kSide;
  static constexpr int kOffP = kOffQ + kQ;
  static constexpr int kOffRows = kOffP + kP;                  // [warp][16] {max x, max x + S_v}, or {m, l}
  static constexpr int kOffScale = kOffRows + kWarps * kAttendRows * 8;  // [16] row factors
  static constexpr int kBytes = kOffScale + kAttendRows * 4;
};

// Floats of one CTA's part of a unit: the rows' maxima, sums, and weighted sums.
template <int D>
constexpr int kPartFloats = kAttendRows * (D + 2);

// ------------------------------------------------------------- the kernel
template <int D, bool kShared>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs a) {
  using L = Layout<D, kShared>;
  constexpr bool kCoop = L::kCoop;
  constexpr int kBlocks = L::kBlocks;
  constexpr int kStages = L::kStages;
  constexpr int kChunks = kCoop ? D / 64 / kWarps : D / 64;  // 64 dimensions each, of a warp's sums
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanShared scan;
  const uint32_t base = smem_u32(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t side0 = base + L::kOffSide + warp * L::kSide;  // this warp's fp16 scales
  const uint32_t tokens0 = side0 + L::kSides * L::kScales;
  float2* rows_sh = reinterpret_cast<float2*>(smem + L::kOffRows);
  float* factor_sh = reinterpret_cast<float*>(smem + L::kOffScale);

  pdl_wait();
  const int64_t total = total_work(a, scan, blockIdx.x == 0);
  const int64_t run = run_of(total, gridDim.x);
  int64_t at = run * blockIdx.x;
  const int64_t stop = min(at + run, total);
  if (at >= stop) {
    pdl_launch_dependents();
    return;
  }
  const Found found = find_work(a, scan, at);
  int b = found.b;
  int64_t seq_first = found.first;
  Seq s = seq_of(a, b);

  while (at < stop) {
    while (at >= seq_first + seq_work(a, s)) {  // sequences without queries have no work
      seq_first += seq_work(a, s);
      s = seq_of(a, ++b);
    }
    const int64_t in = at - seq_first;
    const int unit = static_cast<int>(in / s.tiles);
    const int tile0 = static_cast<int>(in - static_cast<int64_t>(unit) * s.tiles);
    const int tile1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), tile0 + (stop - at)));
    // a CTA has two parts of units at most: the one its run begins within, and a later one
    const int part = at == run * blockIdx.x ? 0 : 1;
    at += tile1 - tile0;
    Unit16 un;
    un.head = unit / s.row_tiles;
    un.row0 = (unit - un.head * s.row_tiles) * kAttendRows;
    un.rows = s.n * a.group;
    const int t_begin = s.start + tile0 * kTile;
    const int t_end = min(s.start + tile1 * kTile, s.len);

    // ---- queries and what each row sees
    int lo[2], hi[2];
    bool valid[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      int token, q_head;
      valid[r] = un.row(a, s, g + 8 * r, token, q_head);
      const int pos = s.len - s.n + token - s.q0;
      hi[r] = !valid[r] ? 0 : a.causal ? min(pos + 1, s.len) : s.len;
      lo[r] = a.window > 0 ? pos - a.window + 1 : 0;
    }
    // whether a tile may hold tokens that not every row sees
    const bool masked = a.window > 0 || (a.causal && s.n > 1);
    uint32_t qf[kCoop ? 1 : kBlocks][2][4];
    float factor[2];
    if constexpr (kCoop) {
      __syncthreads();  // the previous unit's queries are read
#pragma unroll
      for (int i = 0; i < kAttendRows / kWarps; ++i) {
        const int r = warp * (kAttendRows / kWarps) + i;
        int token, q_head;
        const bool ok = un.row(a, s, r, token, q_head);
        const uint16_t* q = a.q + static_cast<size_t>(token) * a.ldq + static_cast<size_t>(q_head) * a.ldq_head;
        uint4 v[D / 256];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < D / 256; ++j) {
          v[j] = ok ? *reinterpret_cast<const uint4*>(q + (lane + 32 * j) * 8) : make_uint4(0, 0, 0, 0);
          most = max(most, max_bits(v[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
        const int shift = query_shift(most, a.q_f16);
        const float f = pow2(shift);
#pragma unroll
        for (int j = 0; j < D / 256; ++j) {
          const int ch = lane + 32 * j;  // eight dimensions: block ch / 4, thread ch % 4 of a row's four
          sts128(base + L::kOffQ + ((((ch >> 2) * 2 + (r >> 3)) * 32) + (r & 7) * 4 + (ch & 3)) * 16,
                 query_f16(v[j], a.q_f16, f));
        }
        if (lane == 0) factor_sh[r] = pow2(-shift - 7) * a.scale_log2;
      }
      __syncthreads();
      factor[0] = factor_sh[g];
      factor[1] = factor_sh[g + 8];
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        int token, q_head;
        const bool ok = un.row(a, s, g + 8 * r, token, q_head);
        const uint16_t* q = a.q + static_cast<size_t>(token) * a.ldq + static_cast<size_t>(q_head) * a.ldq_head;
        uint4 v[kBlocks];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
          v[j] = ok ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * c) : make_uint4(0, 0, 0, 0);
          most = max(most, max_bits(v[j]));
        }
        most = max(most, __shfl_xor_sync(kFull, most, 1));
        most = max(most, __shfl_xor_sync(kFull, most, 2));
        const int shift = query_shift(most, a.q_f16);
        const float f = pow2(shift);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
          const uint4 w = query_f16(v[j], a.q_f16, f);
          qf[j][r][0] = w.x, qf[j][r][1] = w.y, qf[j][r][2] = w.z, qf[j][r][3] = w.w;
        }
        factor[r] = pow2(-shift - 7) * a.scale_log2;
      }
    }

    // ---- the ring
    // a warp's parts: tokens [t_begin + 32 (warp + 4 i), + 32)
    const int parts = (t_end - t_begin + kTile - 1) / kTile;
    int page_next[2];
    auto page_load = [&](int i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = t_begin + (warp + kWarps * i) * kSub + 16 * j;
        page_next[j] = i < parts && t < t_end
                           ? a.table[static_cast<size_t>(b) * a.ld_table + div_u32(t >> 4, a.per_page)]
                           : -1;
      }
    };
    auto issue = [&](int i) {
      if (i < parts) {
        const uint32_t stage = base + (i % kStages) * (kWarps * L::kPart) + warp * L::kPart;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = t_begin + (warp + kWarps * i) * kSub + 16 * j;
          const bool here = t < t_end && page_next[j] >= 0 && page_next[j] < a.pages;
          if (t < t_end && !here && lane == 0) atomicOr(a.status, kStatusBadInput);
          const uint32_t place = ((t >> 4) - div_u32(t >> 4, a.per_page) * (a.page_size >> 4)) << 4;
          const size_t row = here ? static_cast<size_t>(un.head) * a.page_size + place : 0;
          const size_t page = here ? page_next[j] : 0;
#pragma unroll
          for (int sd = 0; sd < L::kSides; ++sd) {
            const uint8_t* codes = (sd ? a.v + page * a.v_page : a.k + page * a.k_page) + row * (D / 2);
            const uint8_t* scales =
                (sd ? a.v_scales + page * a.v_scale_page : a.k_scales + page * a.k_scale_page) + row * kBlocks;
            const uint32_t to = stage + sd * (L::kCodes + L::kRaw);
#pragma unroll
            for (int x = 0; x < kBlocks / 2; ++x) {  // 16 rows of kBlocks chunks
              const int e = lane + 32 * x, r = e / kBlocks, ch = e % kBlocks;
              cp_async_16(to + (16 * j + r) * (D / 2) + ((ch ^ flip<D>(r)) << 4), codes + e * 16,
                          here && t + r < t_end ? 16u : 0u);
            }
            if (lane < kBlocks) cp_async_16(to + L::kCodes + j * 16 * kBlocks + lane * 16, scales + lane * 16, here ? 16u : 0u);
          }
        }
      }
      cp_async_commit();
    };

    float acc[kChunks][8][4];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, u[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    page_load(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      issue(i);
      page_load(i + 1);
    }

    for (int i = 0; i < parts; ++i) {
      cp_async_wait<kStages - 2>();
      if constexpr (kCoop)
        __syncthreads();
      else
        __syncwarp();
      issue(i + kStages - 1);
      page_load(i + kStages);
      const uint32_t stage_all = base + (i % kStages) * (kWarps * L::kPart);
      const uint32_t stage = stage_all + warp * L::kPart;
      const int t0 = t_begin + (warp + kWarps * i) * kSub;

      // ---- scales of token `lane`: fp16 relative to the row's largest, and that one
      bool nan_value = false;
      {
        const bool here = t0 + lane < t_end;
        float2 tok = make_float2(0.f, 0.f);
#pragma unroll
        for (int sd = 0; sd < L::kSides; ++sd) {
          uint32_t w[(kBlocks + 3) / 4];
          const uint32_t from = stage + sd * (L::kCodes + L::kRaw) + L::kCodes + lane * kBlocks;
          if constexpr (kBlocks == 2) {
            asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(w[0]) : "r"(from));
          } else if constexpr (kBlocks == 4) {
            w[0] = lds32(from);
          } else if constexpr (kBlocks == 8) {
            const uint2 v = lds64(from);
            w[0] = v.x, w[1] = v.y;
          } else {
            const uint4 v = lds128(from);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          }
          int top = 0;
          bool nan = false;
#pragma unroll
          for (int k = 0; k < kBlocks; ++k) {
            const int x = (w[k / 4] >> (8 * (k % 4))) & 255;
            nan |= x == 255;
            top = max(top, x == 255 ? 0 : x);
          }
          const bool value = sd == 1 || kShared;
          if (value) nan_value = nan && here;
          // a NaN among values that not every row sees must not meet the others' zero
          // weights: it is added to its own rows below
          const bool quiet = value && masked;
          const uint32_t to = side0 + sd * L::kScales + (lane >> 4) * 32 + ((lane & 3) * 2 + ((lane >> 2) & 1)) * 4 +
                              ((lane >> 3) & 1) * 2;
#pragma unroll
          for (int k = 0; k < kBlocks; ++k) {
            const uint32_t x = (w[k / 4] >> (8 * (k % 4))) & 255;
            sts16(to + k * L::kScaleStride, !here || (quiet && x == 255u) ? 0u : scale_f16(x, top));
          }
          if (sd == 0) tok.x = __uint_as_float(max(static_cast<uint32_t>(top) << 23, 0x00400000u));
          if (value) tok.y = static_cast<float>(top - 127);
        }
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(tokens0 + lane * 8), "f"(tok.x), "f"(tok.y) : "memory");
      }
      __syncwarp();

      // ---- scores of this warp's tokens
      float x[2][2][4];  // [group][n tile][row, token c + 4 n (+ 8)]
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[j][n][e] = 0.f;
      {
        // column n of the first (second) n tile is token n / 2 (+ 4) + 8 (n & 1)
        const uint32_t row = (g >> 1) + 8 * (g & 1);
        const uint32_t pick = (g & 1) ? 0x3232u : 0x1010u;
#pragma unroll(kCoop ? 4 : kBlocks)
        for (int k = 0; k < kBlocks; ++k) {
          uint32_t qa[2][4];  // [kstep]
          if constexpr (kCoop) {
            const uint4 q0 = lds128(base + L::kOffQ + (k * 64 + lane) * 16);
            const uint4 q1 = lds128(base + L::kOffQ + (k * 64 + 32 + lane) * 16);
            qa[0][0] = q0.x, qa[0][1] = q1.x, qa[0][2] = q0.y, qa[0][3] = q1.y;
            qa[1][0] = q0.z, qa[1][1] = q1.z, qa[1][2] = q0.w, qa[1][3] = q1.w;
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              qa[h][0] = qf[k][0][2 * h], qa[h][1] = qf[k][1][2 * h];
              qa[h][2] = qf[k][0][2 * h + 1], qa[h][3] = qf[k][1][2 * h + 1];
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 sc = lds64(side0 + k * L::kScaleStride + j * 32 + (g >> 1) * 8);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t t = row + 4 * n;
              const uint32_t w = lds32(stage + (16 * j + t) * (D / 2) + ((k ^ flip<D>(t)) << 4) + 4 * c);
              const uint32_t scale = __byte_perm(n ? sc.y : sc.x, 0, pick);
              uint32_t r[4];
              codes_f16(w, r);
#pragma unroll
              for (int e = 0; e < 4; ++e) r[e] = mul_f16x2(r[e], scale);
              mma_f16(x[j][n], qa[0], r[0], r[1]);
              mma_f16(x[j][n], qa[1], r[2], r[3]);
            }
          }
        }
      }

      // ---- weights
      float vs[2][2][2];  // S_v of the tokens
      float mx[2] = {-INFINITY, -INFINITY}, ux[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tl = 16 * j + c + 4 * n + 8 * e;
            const uint2 tk = lds64(tokens0 + tl * 8);
            const float kf = __uint_as_float(tk.x);
            vs[j][n][e] = __uint_as_float(tk.y);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& v = x[j][n][2 * r + e];
              v = v * kf * factor[r];
              const int t = t0 + tl;
              if (t >= min(hi[r], t_end) || t < lo[r]) v = -INFINITY;
              mx[r] = fmaxf(mx[r], v);
              ux[r] = fmaxf(ux[r], v + vs[j][n][e]);
            }
          }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 1));
        ux[r] = fmaxf(ux[r], __shfl_xor_sync(kFull, ux[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 2));
        ux[r] = fmaxf(ux[r], __shfl_xor_sync(kFull, ux[r], 2));
      }
      if constexpr (kCoop) {
        if (c == 0) {
          rows_sh[warp * kAttendRows + g] = make_float2(mx[0], ux[0]);
          rows_sh[warp * kAttendRows + g + 8] = make_float2(mx[1], ux[1]);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 v = rows_sh[w * kAttendRows + g + 8 * r];
            mx[r] = fmaxf(mx[r], v.x);
            ux[r] = fmaxf(ux[r], v.y);
          }
      }
      float shrink[2], mr[2], ur[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], m[r]);
        ux[r] = fmaxf(ux[r], u[r]);
        // a row that has seen nothing yet has no maximum to subtract
        mr[r] = mx[r] == -INFINITY ? 0.f : mx[r];
        ur[r] = ux[r] == -INFINITY ? 0.f : ux[r];
        l[r] *= exp2_fast(m[r] - mr[r]);
        shrink[r] = exp2_fast(u[r] - ur[r]);
        m[r] = mx[r];
        u[r] = ux[r];
        ur[r] -= kWeightBits;
      }
      uint32_t p[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v0 = x[j][n][2 * r], v1 = x[j][n][2 * r + 1];
            l[r] += exp2_fast(v0 - mr[r]) + exp2_fast(v1 - mr[r]);
            p[j][2 * n + r] = pack_f16(exp2_fast(v0 + vs[j][n][0] - ur[r]), exp2_fast(v1 + vs[j][n][1] - ur[r]));
          }
      if constexpr (kCoop) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          sts128(base + L::kOffP + ((warp * 2 + j) * 32 + lane) * 16, make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]));
        __syncthreads();
      }
      if (__any_sync(kFull, shrink[0] != 1.f || shrink[1] != 1.f)) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][n][e] *= shrink[e >> 1];
      }

      // ---- weighted sums of the values
      constexpr int kGroups = kCoop ? kTile / 16 : 2;
#pragma unroll(kCoop ? 2 : kGroups)
      for (int j = 0; j < kGroups; ++j) {
        uint32_t pa[4];
        uint32_t from, sc_from;
        if constexpr (kCoop) {
          const uint4 v = lds128(base + L::kOffP + (j * 32 + lane) * 16);
          pa[0] = v.x, pa[1] = v.y, pa[2] = v.z, pa[3] = v.w;
          from = stage_all + (j >> 1) * L::kPart + (j & 1) * 8 * D;
          sc_from = base + L::kOffSide + (j >> 1) * L::kSide + (j & 1) * 32;
        } else {
          pa[0] = p[j][0], pa[1] = p[j][1], pa[2] = p[j][2], pa[3] = p[j][3];
          from = stage + j * 8 * D;
          sc_from = side0 + j * 32;
        }
        if constexpr (!kShared) {
          from += L::kCodes + L::kRaw;
          sc_from += L::kScales;
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int chunk = kCoop ? warp * kChunks + k : k;  // of 64 dimensions
          const uint32_t ch = 2 * chunk + (g >> 2);          // the 32-block of this thread's eight
          const uint2 sc = lds64(sc_from + ch * L::kScaleStride + c * 8);
          uint32_t w[4];  // tokens c, c + 8, c + 4, c + 12
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t t = c + 8 * (e & 1) + 4 * (e >> 1);
            w[e] = lds32(from + t * (D / 2) + ((ch ^ flip<D>(t)) << 4) + 4 * (g & 3));
          }
          // a byte of one code of each of two tokens, codes 2 i and 2 i + 1
          uint32_t ev[2][4], od[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_f16((w[2 * h] & 0x0F0F0F0Fu) | ((w[2 * h + 1] << 4) & 0xF0F0F0F0u), ev[h]);
            codes_f16(((w[2 * h] >> 4) & 0x0F0F0F0Fu) | (w[2 * h + 1] & 0xF0F0F0F0u), od[h]);
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            mma_f16(acc[k][2 * n], pa, mul_f16x2(ev[0][n], sc.x), mul_f16x2(ev[1][n], sc.y));
            mma_f16(acc[k][2 * n + 1], pa, mul_f16x2(od[0][n], sc.x), mul_f16x2(od[1][n], sc.y));
          }
        }
      }
      // ---- NaN values that only some rows see
      if (masked) {
        bool any = __any_sync(kFull, nan_value);
        if constexpr (kCoop) any = __syncthreads_or(any);
        if (any) {
          for (int t = 0; t < (kCoop ? kTile : kSub); ++t) {
            const uint8_t* from = smem + ((kCoop ? stage_all + (t >> 5) * L::kPart : stage) - base) +
                                  (kShared ? 0 : L::kCodes + L::kRaw) + L::kCodes + (t & 31) * kBlocks;
            const int pos = kCoop ? t_begin + i * kTile + t : t0 + t;
            if (pos >= t_end) break;
            bool row_nan = false;  // a shared row is a key as well: its score is NaN
            if constexpr (kShared)
              for (int k = 0; k < kBlocks; ++k) row_nan |= from[k] == 255;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (pos < lo[r] || pos >= hi[r]) continue;
              if (row_nan) l[r] = NAN;
#pragma unroll
              for (int k = 0; k < kChunks; ++k) {
                const int chunk = kCoop ? warp * kChunks + k : k;
                if (!row_nan && from[2 * chunk + (c >> 1)] != 255) continue;
#pragma unroll
                for (int n = 0; n < 8; ++n) acc[k][n][2 * r] = acc[k][n][2 * r + 1] = NAN;
              }
            }
          }
        }
      }
    }
    cp_async_wait<0>();

    // ---- join the warps
    const bool whole = tile0 == 0 && tile1 == s.tiles;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(kFull, l[r], 1);
      l[r] += __shfl_xor_sync(kFull, l[r], 2);
    }
    float* part_out = a.partial + (static_cast<size_t>(blockIdx.x) * 2 + part) * kPartFloats<D>;
    if constexpr (kCoop) {
      __syncthreads();
      if (c == 0) {
        rows_sh[warp * kAttendRows + g] = make_float2(m[0], l[0]);
        rows_sh[warp * kAttendRows + g + 8] = make_float2(m[1], l[1]);
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += rows_sh[w * kAttendRows + g + 8 * r].y;
        // sums relative to 2^(u + 15) -> to 2^m
        const float f = u[r] == -INFINITY ? 0.f : exp2f(u[r] - (m[r] == -INFINITY ? 0.f : m[r]) - kSumBits);
        int token, q_head;
        const bool ok = un.row(a, s, g + 8 * r, token, q_head);
        if (whole) {
          if (!ok) continue;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          uint16_t* out = a.out + static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head;
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            float v[16];
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] = acc[k][n][2 * r] * f, v[8 + n] = acc[k][n][2 * r + 1] * f;
            uint4* to = reinterpret_cast<uint4*>(out + (warp * kChunks + k) * 64 + 16 * c);
            to[0] = pack_out8(v, inv, a.q_f16);
            to[1] = pack_out8(v + 8, inv, a.q_f16);
          }
          if (a.lse != nullptr && warp == 0 && c == 0)
            a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (m[r] + log2f(sum)) * 0.6931471805599453f;
        } else {
          if (warp == 0 && c == 0) {
            part_out[g + 8 * r] = m[r];
            part_out[kAttendRows + g + 8 * r] = sum;
          }
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            float4* to = reinterpret_cast<float4*>(part_out + 2 * kAttendRows + (g + 8 * r) * D +
                                                   (warp * kChunks + k) * 64 + 16 * c);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < 8; n += 4)
                to[h * 2 + n / 4] = make_float4(acc[k][n][2 * r + h] * f, acc[k][n + 1][2 * r + h] * f,
                                                acc[k][n + 2][2 * r + h] * f, acc[k][n + 3][2 * r + h] * f);
          }
        }
      }
    } else {
      __syncthreads();  // all parts of the ring are read
      if (c == 0) {
        rows_sh[warp * kAttendRows + g] = make_float2(m[0], l[0]);
        rows_sh[warp * kAttendRows + g + 8] = make_float2(m[1], l[1]);
      }
      float* dump = reinterpret_cast<float*>(smem) + warp * kAttendRows * (D + 4);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = u[r] == -INFINITY ? 0.f : exp2f(u[r] - (m[r] == -INFINITY ? 0.f : m[r]) - kSumBits);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          float4* to = reinterpret_cast<float4*>(dump + (g + 8 * r) * (D + 4) + k * 64 + 16 * c);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 8; n += 4)
              to[h * 2 + n / 4] = make_float4(acc[k][n][2 * r + h] * f, acc[k][n + 1][2 * r + h] * f,
                                              acc[k][n + 2][2 * r + h] * f, acc[k][n + 3][2 * r + h] * f);
        }
      }
      __syncthreads();
      // eight threads to a row, eight dimensions of 64 at a time
      const int r = threadIdx.x >> 3, e0 = (threadIdx.x & 7) * 8;
      float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, rows_sh[w * kAttendRows + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = rows_sh[w * kAttendRows + r];
        f[w] = v.x == -INFINITY ? (v.y != v.y ? v.y : 0.f) : exp2f(v.x - top);
        sum += v.y * f[w];
      }
      int token, q_head;
      const bool ok = un.row(a, s, r, token, q_head);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        float v[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4* from = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                               (w * kAttendRows + r) * (D + 4) + k * 64 + e0);
          const float4 y = from[0], z = from[1];
          v[0] += y.x * f[w], v[1] += y.y * f[w], v[2] += y.z * f[w], v[3] += y.w * f[w];
          v[4] += z.x * f[w], v[5] += z.y * f[w], v[6] += z.z * f[w], v[7] += z.w * f[w];
        }
        if (whole) {
          if (ok)
            *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(token) * a.ldo +
                                      static_cast<size_t>(q_head) * a.ldo_head + k * 64 + e0) =
                pack_out8(v, inv, a.q_f16);
        } else {
          float4* to = reinterpret_cast<float4*>(part_out + 2 * kAttendRows + r * D + k * 64 + e0);
          to[0] = make_float4(v[0], v[1], v[2], v[3]);
          to[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      if ((threadIdx.x & 7) == 0) {
        if (!whole) {
          part_out[r] = top;
          part_out[kAttendRows + r] = sum;
        } else if (ok && a.lse != nullptr) {
          a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (top + log2f(sum)) * 0.6931471805599453f;
        }
      }
      __syncthreads();  // the dump lies in the ring
    }
  }
  pdl_launch_dependents();
}

// ------------------------------------------------------------- joining
// Block (c, row): if the run of CTA c + 1 begins within a unit, and is the first that does,
// the parts of that unit are added up for one row, in the order of the runs.
template <int D>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a, int ctas) {
  __shared__ ScanShared scan;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = total_work(a, scan, false);
  const int64_t run = run_of(total, ctas);
  const int64_t cut = run * (blockIdx.x + 1);
  if (cut >= total) return;
  const Found found = find_work(a, scan, cut);
  const Seq s = seq_of(a, found.b);
  const int64_t in = cut - found.first;
  const int unit = static_cast<int>(in / s.tiles);
  const int64_t first = found.first + static_cast<int64_t>(unit) * s.tiles;
  if (first == cut || cut - run > first) return;
  Unit16 un;
  un.head = unit / s.row_tiles;
  un.row0 = (unit - un.head * s.row_tiles) * kAttendRows;
  un.rows = s.n * a.group;
  const int r = blockIdx.y;
  int token, q_head;
  if (!un.row(a, s, r, token, q_head)) return;
  const int c0 = static_cast<int>(first / run), c1 = static_cast<int>((first + s.tiles - 1) / run);
  auto part = [&](int c) {
    return a.partial + (static_cast<size_t>(c) * 2 + (c == c0 && first != run * c0 ? 1 : 0)) * kPartFloats<D>;
  };
  float top = -INFINITY;
  for (int c = c0; c <= c1; ++c) top = fmaxf(top, part(c)[r]);
  float sum = 0.f, v[(D + kThreads - 1) / kThreads] = {};
  for (int c = c0; c <= c1; ++c) {
    const float* p = part(c);
    const float m = p[r], l = p[kAttendRows + r];
    const float f = m == -INFINITY ? (l != l ? l : 0.f) : exp2f(m - top);
    sum += l * f;
#pragma unroll
    for (int i = 0; i < (D + kThreads - 1) / kThreads; ++i) {
      const int d = threadIdx.x + i * kThreads;
      if (d < D) v[i] += p[2 * kAttendRows + r * D + d] * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = a.out + static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head;
#pragma unroll
  for (int i = 0; i < (D + kThreads - 1) / kThreads; ++i) {
    const int d = threadIdx.x + i * kThreads;
    if (d < D) out[d] = static_cast<uint16_t>(pack_out(v[i] * inv, 0.f, a.q_f16));
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (top + log2f(sum)) * 0.6931471805599453f;
}

// f(kernel, join kernel, shared bytes) of a variant.
template <int D, bool kShared, typename F>
auto with_kernels(F&& f) {
  return f(attend_kernel<D, kShared>, attend_join_kernel<D>, Layout<D, kShared>::kBytes);
}
template <typename F>
auto with_variant(int v, F&& f) {
  switch (v) {
    case 0: return with_kernels<64, false>(f);
    case 1: return with_kernels<64, true>(f);
    case 2: return with_kernels<128, false>(f);
    case 3: return with_kernels<128, true>(f);
    case 4: return with_kernels<256, false>(f);
    case 5: return with_kernels<256, true>(f);
    case 6: return with_kernels<512, false>(f);
    default: return with_kernels<512, true>(f);
  }
}

}  // namespace

int attend_variant(int d, bool shared) {
  const int i = d == 64 ? 0 : d == 128 ? 1 : d == 256 ? 2 : d == 512 ? 3 : -1;
  return i < 0 ? -1 : 2 * i + (shared ? 1 : 0);
}

cudaError_t set_attend_attributes(int sm_count, int (&ctas)[kAttendVariants]) {
  for (int v = 0; v < kAttendVariants; ++v) {
    const cudaError_t e = with_variant(v, [&](auto kernel, auto, int bytes) {
      cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      int n = 0;
      if (rc == cudaSuccess) rc = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, bytes);
      ctas[v] = n * sm_count;
      return rc == cudaSuccess && n < 1 ? cudaErrorInvalidConfiguration : rc;
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t attend_bytes(int d, int ctas) { return static_cast<size_t>(ctas) * 2 * kAttendRows * (d + 2) * sizeof(float); }

cudaError_t launch_attend(const AttendArgs& a, int d, bool shared, int ctas, cudaStream_t stream) {
  return with_variant(attend_variant(d, shared), [&](auto kernel, auto join, int bytes) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess || ctas < 2) return e;
    cfg.gridDim = dim3(ctas - 1, kAttendRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join, a, ctas);
  });
}

}  // namespace mx
