// attend.cu - attention of few query rows over the MXFP4 cache.
//
//   out[r] = sum over visible t of softmax_t(scale q[r].k[t]) v[t]
//
// The rows of a kv head (its group of query heads, of each query token) are the 8 columns
// of mma.sync.m16n8k16, once or twice, and the cache is its 16 rows: tokens for the scores, dimensions
// for the sums. That operand comes from registers: the codes go from shared memory through
// cvt.f16x2.e2m1x2 and one multiplication by their scale straight into the products, without a
// stop in shared memory at 16 bits (for the 5th-generation tensor cores the dequantized
// tile would have to be written and read there: at d = 512 28 bytes of shared memory
// traffic for each byte of cache).
//
// In 16 bits. fp16 holds what is multiplied, under powers of two that keep all rounding
// out but where it says so:
//   keys    code * 2^(s - S + 13), s the block's scale and S the row's largest: exact down
//           to 2^-27 of the row's largest block, nothing below; the score takes 2^(S - 13)
//           back in float32. Values the same.
//   queries times the power of two that brings the row's largest into [2^14, 2^15):
//           exact down to 2^-31 of it.
//   weights p = exp2(x - m + S_v - u + 8) rounded to fp16 (11 bits, where a bf16 weight would
//           have 8): x the score, m the running maximum, S_v the value row's scale, u the running
//           maximum of x - m + S_v (of the difference, which is exact near 0: S_v would be lost in a large
//           score). So what is rounded, and below 2^-22 of the largest loses bits, is a
//           token's contribution, not its weight. The weights' sum is of float32 exponentials.
//
// m and u are only moved when a score goes beyond by 2^24, or a
// contribution by 2^7: then the sums are scaled anew, otherwise nothing is.
//
// Tokens go by in tiles of 128, an equal part to each of four warps, through a ring filled by bulk copies. Up to
// d = 128 a warp is on its own: it keeps the queries and its sums in registers, and four warps' results are
// joined at the end. Above, a warp computes the scores of its tokens, hands the weights on through shared
// memory, and sums its share of the dimensions over all 128, with one barrier a tile.
//
// Which element of a row is which column of an operand is free as long as both operands have
// it the same, so a thread loads 16 bytes of a key row (a whole block: one scale) and 8 of
// a value row at once. Place n of eight tokens is token n ^ (n / 2 & 1), which
// spreads the rows that a warp reads over the banks.
//
// The work of all sequences is cut into equal runs of tiles (and of a little for each unit), one for each
// resident CTA, whatever the lengths; a run may end within a sequence. What a CTA has of a unit
// (sequence, kv head, 8 or 16 rows) that is not all its own goes to a workspace, from which a
// second kernel adds it up in the order of the tokens.
//
// Conversion, scale and products of 256 codes take 6.8 cycles of an SM where nothing else runs, and its share of HBM
// brings that many in 6.2. 61 sequences of up to 16384 tokens, 32 heads on 8 of 128: 160 to 168 us, 3.5 TB/s (loads
// alone 117, all but the loads 143, conversions and products at that rate 98: the chain from one to the next is
// not filled by 16 warps, which issue 2.4 instructions a cycle of 4); 48 of up to 32768 latents, 16 heads: 123 to 132 us,
// 1.9 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attend.cuh"

namespace mx {
namespace {

constexpr int kTile = kAttendTile;
constexpr int kScaleBits = 13;           // 6 * 2^13 < 65504
constexpr float kWeightBits = 8.f;       // weights are up to 2^8 when u is the maximum,
constexpr float kLagU = 7.f;             // and 2^15 before it is moved
constexpr float kLagM = 24.f;
constexpr float kSumBits = kScaleBits + kWeightBits;

// ------------------------------------------------------------- pieces
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The 8 x 8 matrix of 16-bit elements that a warp holds, row lane / 4, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Place n of eight tokens, and the other way round.
__device__ __forceinline__ constexpr int place_of(int n) { return n ^ ((n >> 1) & 1); }

// fp16 bits of 2^(s - top + 13) for scale byte s <= top: 0 below 2^-14. NaN for byte 255.
__device__ __forceinline__ uint32_t scale_f16(uint32_t s, int top) {
  const uint32_t v = static_cast<uint32_t>(max(static_cast<int>(s) - top + 28, 0)) << 10;
  return s == 255u ? 0x7E00u : v;
}

template <int D, bool kShared, int kRows>
struct Layout {
  static constexpr bool kCoop = D > 128;
  static constexpr int kWarps = 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSub = kTile / kWarps;       // tokens of a warp's part of a tile: a thread to each
  static_assert(kSub == 32, "scales");
  static constexpr int kSides = kShared ? 1 : 2;
  static constexpr int kBlocks = D / 32;
  // (rows of whole 128 bytes that were copied one by one, 16 bytes further each, had fewer bank
  // conflicts, and arrived at 3.7 TB/s at most)
  static constexpr int kPitch = D / 2;
  static constexpr int kCodes = kSub * kPitch;      // bytes of a warp's part of a stage
  static constexpr int kRaw = kSub * kBlocks;       // scale bytes
  static constexpr int kPart = kSides * (kCodes + kRaw);
  static constexpr int kStages = kCoop ? 2 : kRows == 8 ? 3 : 4;
  static constexpr int kRing = kStages * kWarps * kPart;
  // Of each warp's tokens: the keys' fp16 scales [token][block, in the order 0 2 1 3]; the values' [block][group of
  // 16] in the order of the places, a pair of each half together, and 16 bytes more to a block, so that
  // neighbouring blocks lie in different banks; {2^(S_k - 127), S_v - 127} [place].
  static constexpr int kKeyScales = kSub * kBlocks * 2;
  static constexpr int kValueStride = 2 * kSub + 16;
  static constexpr int kValueScales = kBlocks * kValueStride;
  static constexpr int kTokens = kSub * 8;
  static constexpr int kBuffers = kCoop ? 2 : 1;    // of what other warps read
  static constexpr int kSide = kKeyScales + kTokens + kBuffers * kValueScales;
  static constexpr int kDump = kWarps * kRows * (D + 4) * 4;
  static constexpr int kQ = kCoop ? kRows * D * 2 : 0;
  static constexpr int kP = kCoop ? kTile / 16 * 32 * kRows : 0;
  static constexpr int kRingArea = !kCoop && kDump > kRing ? kDump : kRing;
  static constexpr int kOffSide = kRingArea;
  static constexpr int kOffQ = kOffSide + kWarps * kSide;
  static constexpr int kOffP = kOffQ + kQ;
  static constexpr int kOffRows = kOffP + kBuffers * kP;                 // [warp][row] {max x, max x + S_v}, or {m, l}
  static constexpr int kOffScale = kOffRows + kWarps * kRows * 8;  // [row] factors
  static constexpr int kBytes = kOffScale + kRows * 4;
  // (16 rows at d = 128: with one, 61 sequences of four tokens took 189 us, with two 148)
  static constexpr int kCtas = D == 512 && !kShared ? 1 : D >= 256 ? 2 : kRows == 8 ? 4 : D == 128 ? 2 : 3;  // of an SM, by shared memory
};

// ------------------------------------------------------------- the kernel
template <int D, bool kShared, int kRows>
__global__ void __launch_bounds__(Layout<D, kShared, kRows>::kThreads, Layout<D, kShared, kRows>::kCtas) attend_kernel(const AttendArgs a) {
  using L = Layout<D, kShared, kRows>;
  constexpr bool kCoop = L::kCoop;
  constexpr int kExtra = kUnitExtra<D>;
  constexpr int kBlocks = L::kBlocks;
  constexpr int kStages = L::kStages;
  constexpr int kWarps = L::kWarps, kSub = L::kSub, kOwn = kSub / 16;  // groups of 16 tokens of a warp
  constexpr int kSlices = D <= 128 ? 1 : D / 128;  // of the scores: a thread has 1, or half a, block of each
  constexpr int kKeyWords = D == 64 ? 2 : 4;       // words of a key row's slice
  constexpr int kWords = D == 64 || D == 256 ? 1 : 2;  // words of a value row: 8 dimensions each
  constexpr int kN = kRows / 8;                    // tiles of rows
  constexpr int kWide = 64 * kWords;               // dimensions of a warp's sums
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanShared scan;
  __shared__ uint64_t full[kWarps][kStages];
  const uint32_t base = smem_u32(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t keys0 = base + L::kOffSide + warp * L::kSide;  // this warp's
  const uint32_t tokens0 = keys0 + L::kKeyScales;
  constexpr int kValues0 = L::kOffSide + L::kKeyScales + L::kTokens;  // the first warp's
  float2* rows_sh = reinterpret_cast<float2*>(smem + L::kOffRows);
  float* factor_sh = reinterpret_cast<float*>(smem + L::kOffScale);
  // this warp's dimensions
  const int wide0 = kCoop ? warp * kWide : 0;

  pdl_launch_dependents();  // every CTA is resident: a dependent grid waits for none to start
  if (lane < kStages) mbar_init(smem_u32(&full[warp][lane]), 1);
  fence_mbar_init();
  pdl_wait();
  int64_t total;
  const Found found = find_run<kRows, kWarps>(a, scan, seq_work<D>, total);
  const int64_t run = run_of(total, gridDim.x);
  int64_t at = run * blockIdx.x;
  const int64_t stop = min(at + run, total);
  Cut* cuts = reinterpret_cast<Cut*>(a.partial);
  float* parts0 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.partial) + cut_bytes(gridDim.x));
  if (threadIdx.x == 0) cuts[blockIdx.x].last = -1;  // until the run is seen to begin within a unit
  if (at >= stop) return;
  int b = found.b;
  int64_t seq_first = found.first;
  Seq s = seq_of(a, b, kRows);
  uint32_t slot0 = 0;  // parts that this warp has taken through the ring
  bool failed = false;

  while (at < stop) {
    while (at >= seq_first + seq_work<D>(a, s)) {  // sequences without queries have no work
      seq_first += seq_work<D>(a, s);
      s = seq_of(a, ++b, kRows);
    }
    const int64_t in = at - seq_first;
    const int unit = static_cast<int>(in / (s.tiles + kExtra));
    const int place = static_cast<int>(in - static_cast<int64_t>(unit) * (s.tiles + kExtra));
    const int tile0 = max(place - kExtra, 0);
    at += max(kExtra - place, 0);
    if (at >= stop) break;
    const int tile1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), tile0 + (stop - at)));
    // a CTA has two parts of units at most: the one its run begins within, and a later one
    const bool begin = at == run * blockIdx.x;
    AttendUnit un;
    un.head = unit / s.row_tiles;
    un.row0 = (unit - un.head * s.row_tiles) * kRows;
    un.rows = s.n * a.group;
    if (begin && tile0 > 0 && threadIdx.x == 0) {
      Cut cut;
      const int64_t first = at - tile0;
      cut.first = static_cast<int>(first / run);
      cut.last = static_cast<int>((first + s.tiles - 1) / run);
      cut.later = first != run * cut.first;
      cut.head = un.head, cut.row0 = un.row0, cut.rows = un.rows, cut.q0 = s.q0;
      cuts[blockIdx.x] = cut;
    }
    at += tile1 - tile0;
    const int t_begin = s.start + tile0 * kTile;
    const int t_end = min(s.start + tile1 * kTile, s.len);
    const int parts = (t_end - t_begin + kTile - 1) / kTile;

    // ---- the ring: a warp's part i is tokens [t_begin + kSub (warp + kWarps i), + kSub)
    int page_next[kOwn];
    const int* pages_of = a.table + static_cast<size_t>(b) * a.ld_table;
    auto page_load = [&](int i) {
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int t = t_begin + (warp + kWarps * i) * kSub + 16 * j;
        page_next[j] = -1;
        if (t < t_end) page_next[j] = pages_of[div_u32(t >> 4, a.per_page)];
      }
    };
    const size_t head_row = static_cast<size_t>(un.head) * a.page_size;
    uint32_t live = 0;  // groups of 16 tokens that are there, two bits to a stage
    // Rows behind the last token, and of a page outside the cache, are whatever lies there: their
    // scales become 0, and any code is finite.
    auto issue = [&](int i) {
      if (i >= parts) return;
      const uint32_t slot = (slot0 + i) % kStages;
      const uint32_t to0 = base + (slot * kWarps + warp) * L::kPart, bar = smem_u32(&full[warp][slot]);
      uint32_t here = 0;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int t = t_begin + (warp + kWarps * i) * kSub + 16 * j;
        if (static_cast<uint32_t>(page_next[j]) < static_cast<uint32_t>(a.pages))
          here |= 1u << j;
        else if (t < t_end && lane == 0)
          atomicOr(a.status, kStatusBadInput);
      }
      live = (live & ~(3u << (2 * slot))) | here << (2 * slot);
      if (lane == 0) mbar_expect_tx(bar, __popc(here) * L::kSides * 16 * (D / 2 + kBlocks));
      __syncwarp();
      // a thread to each run of neighbouring rows: codes and scales of each side, of both groups at once
      // where they lie in one page (a copy takes about 20 cycles whatever its size)
      const int t = t_begin + (warp + kWarps * i) * kSub;
      const uint32_t group = static_cast<uint32_t>(t) >> 4, col = div_u32(group, a.per_page);
      const bool together = here == 3u && div_u32(group + 1, a.per_page) == col;
      const int j = lane & 1, sd = (lane >> 1) & (L::kSides - 1);
      if (lane < 4 * L::kSides && (here >> j & 1u) && !(together && j == 1)) {
        const uint32_t of_page = j == 0 ? col : div_u32(group + 1, a.per_page);
        const size_t row = head_row + ((group + j - of_page * (a.page_size >> 4)) << 4);
        const int64_t page = j ? page_next[1] : page_next[0];
        const uint32_t to = to0 + sd * (L::kCodes + L::kRaw), rows = together ? 32u : 16u;
        const uint64_t policy = policy_evict_first();
        if (lane < 2 * L::kSides)
          bulk_load(to + j * 16 * L::kPitch, (sd ? a.v + page * a.v_page : a.k + page * a.k_page) + row * (D / 2),
                    rows * (D / 2), bar, policy);
        else
          bulk_load(to + L::kCodes + j * 16 * kBlocks,
                    (sd ? a.v_scales + page * a.v_scale_page : a.k_scales + page * a.k_scale_page) + row * kBlocks,
                    rows * kBlocks, bar, policy);
      }
    };
    page_load(0);

    // ---- queries and what each row sees: this thread's score columns are rows 8 n + 2 c and the next
    int lo[kN][2], hi[kN][2], lo_most = 0, hi_least = s.len;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int token, q_head;
        const bool valid = un.row(a, s, 8 * n + 2 * c + e, token, q_head);
        const int pos = s.len - s.n + token - s.q0;
        hi[n][e] = !valid ? 0 : min(a.causal ? min(pos + 1, s.len) : s.len, t_end);
        lo[n][e] = a.window > 0 ? pos - a.window + 1 : 0;
        // rows that are none see nothing, and nobody looks at them
        if (valid) lo_most = max(lo_most, lo[n][e]), hi_least = min(hi_least, hi[n][e]);
      }
    // whether a tile may hold tokens that not every row sees
    const bool masked = a.window > 0 || (a.causal && s.n > 1);
    uint32_t qf[kCoop ? 1 : kKeyWords][kN][4];  // [word][row 8 n + g][two dimensions]
    float factor[kN][2];
    fence_proxy_async_smem();  // what lay in the ring meanwhile is written over by copies
    __syncthreads();           // the previous unit's queries are read, and its results
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      issue(i);
      page_load(i + 1);
    }
    if constexpr (kCoop) {
#pragma unroll
      for (int i = 0; i < kRows / kWarps; ++i) {
        const int r = warp * (kRows / kWarps) + i;
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
        most = __reduce_max_sync(kFull, most);
        const int shift = query_shift(most, a.q_f16);
        const float f = pow2(shift);
#pragma unroll
        for (int j = 0; j < D / 256; ++j) {
          const int ch = lane + 32 * j;  // eight dimensions: slice ch / 16, thread's block ch / 4 % 4, word ch % 4
          sts128(base + L::kOffQ + ((((ch >> 4) * 4 + (ch & 3)) * kN + (r >> 3)) * 32 + (r & 7) * 4 + ((ch >> 2) & 3)) * 16,
                 query_f16(v[j], a.q_f16, f));
        }
        if (lane == 0) factor_sh[r] = pow2(-shift - kScaleBits) * a.scale_log2;
      }
    } else {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        int token, q_head;
        const bool ok = un.row(a, s, 8 * n + g, token, q_head);
        const uint16_t* q = a.q + static_cast<size_t>(token) * a.ldq + static_cast<size_t>(q_head) * a.ldq_head;
        uint4 v[kKeyWords];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < kKeyWords; ++j) {
          v[j] = ok ? *reinterpret_cast<const uint4*>(q + (c * kKeyWords + j) * 8) : make_uint4(0, 0, 0, 0);
          most = max(most, max_bits(v[j]));
        }
        most = max(most, __shfl_xor_sync(kFull, most, 1));
        most = max(most, __shfl_xor_sync(kFull, most, 2));
        const int shift = query_shift(most, a.q_f16);
        const float f = pow2(shift);
#pragma unroll
        for (int j = 0; j < kKeyWords; ++j) {
          const uint4 w = query_f16(v[j], a.q_f16, f);
          qf[j][n][0] = w.x, qf[j][n][1] = w.y, qf[j][n][2] = w.z, qf[j][n][3] = w.w;
        }
        if (warp == 0 && c == 0) factor_sh[8 * n + g] = pow2(-shift - kScaleBits) * a.scale_log2;
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      factor[n][0] = factor_sh[8 * n + 2 * c];
      factor[n][1] = factor_sh[8 * n + 2 * c + 1];
    }

    // [rows' tile][16 dimensions: codes 2 t and 2 t + 1 of this thread's][code, row 2 c (+ 1)]
    float acc[kN][4 * kWords][4];
    float m[kN][2], u[kN][2], l[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int t = 0; t < 4 * kWords; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][t][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) m[n][e] = u[n][e] = -INFINITY, l[n][e] = 0.f;
    }

    for (int i = 0; i < parts; ++i) {
      const uint32_t slot = (slot0 + i) % kStages;
      if (!failed && !mbar_wait(smem_u32(&full[warp][slot]), ((slot0 + i) / kStages) & 1)) failed = true;
      if constexpr (!kCoop) {
        __syncwarp();  // the stage before is read
        issue(i + kStages - 1);
        page_load(i + kStages);
      }
      const uint32_t stage_all = base + slot * (kWarps * L::kPart);
      const uint32_t stage = stage_all + warp * L::kPart;
      const int t0 = t_begin + (warp + kWarps * i) * kSub;
      const uint32_t values_all = base + kValues0 + (kCoop ? (i & 1) * L::kValueScales : 0);

      // ---- scales of token `lane`: fp16 relative to the row's largest, and that one
      const int token = lane;
      bool nan_value = false;
      {
        const bool here = t0 + token < t_end && (live >> (2 * slot + (token >> 4)) & 1u);
        const int col = place_of(token & 7);  // (token & 24) + col: the token's place
        float2 tok = make_float2(0.f, 0.f);
#pragma unroll
        for (int sd = 0; sd < L::kSides; ++sd) {
          uint32_t w[(kBlocks + 3) / 4];
          const uint32_t from = stage + sd * (L::kCodes + L::kRaw) + L::kCodes + token * kBlocks;
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
          // Two bytes at a time, 16 bits to each: blocks 4 k and 4 k + 2 in one word, 4 k + 1 and
          // 4 k + 3 in the next; 255 (NaN) goes by apart.
          constexpr int kPairs = kBlocks / 2;
          uint32_t f[kPairs];
          uint32_t nan = 0;
#pragma unroll
          for (int k = 0; k < (kBlocks + 3) / 4; ++k) nan |= ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & w[k] & 0x80808080u;
          const bool value = sd == 1 || kShared;
          int top = 0;
          if (__any_sync(kFull, nan != 0)) {
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
              const int x = (w[k / 4] >> (8 * (k % 4))) & 255;
              top = max(top, x == 255 ? 0 : x);
            }
#pragma unroll
            for (int k = 0; k < kPairs; ++k) f[k] = 0;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
              const uint32_t x = (w[k / 4] >> (8 * (k % 4))) & 255;
              // a NaN among values that not every row sees must not meet the others' zero
              // weights: it is added to its own rows below
              const uint32_t v = value && masked && x == 255u ? 0u : scale_f16(x, top);
              f[kBlocks == 2 ? 0 : k / 4 * 2 + k % 2] |= v << (kBlocks == 2 ? 16 * k : k % 4 / 2 * 16);
            }
            if (value) nan_value = nan != 0 && here;
          } else {
            if constexpr (kBlocks == 2) {
              f[0] = (w[0] & 255u) | (w[0] & 0xFF00u) << 8;
            } else {
#pragma unroll
              for (int k = 0; k < kBlocks / 4; ++k) {
                f[2 * k] = w[k] & 0x00FF00FFu;
                f[2 * k + 1] = (w[k] >> 8) & 0x00FF00FFu;
              }
            }
            uint32_t most = f[0];
#pragma unroll
            for (int k = 1; k < kPairs; ++k) most = __vmaxu2(most, f[k]);
            top = static_cast<int>(max(most & 0xFFFFu, most >> 16));
            // 2^(s - top + 13) in fp16, 0 below 2^-14: exponent 28 less the distance
            const uint32_t top2 = static_cast<uint32_t>(top) * 0x10001u;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) f[k] = (0x001C001Cu - __vminu2(top2 - f[k], 0x001C001Cu)) << 10;
          }
          // The bytes of a token that is not there are an earlier stage's: with a page outside the cache it is
          // a row of zeros, whose scale may not raise a reference.
          if (!here) {
            top = 0;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) f[k] = 0u;
          }
          if (sd == 0) {
            const uint32_t to = keys0 + token * kBlocks * 2;
            if constexpr (kBlocks == 2)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(f[0]) : "memory");
            else if constexpr (kBlocks == 4)
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(f[0]), "r"(f[1]) : "memory");
            else
#pragma unroll
              for (int k = 0; k < kPairs; k += 4) sts128(to + k * 4, make_uint4(f[k], f[k + 1], f[k + 2], f[k + 3]));
            tok.x = __uint_as_float(max(static_cast<uint32_t>(top) << 23, 0x00400000u));
          }
          if (value) {
            const uint32_t to =
                values_all + warp * L::kSide + (token >> 4) * 32 + (col >> 1) * 8 + ((token >> 3) & 1) * 4 + (col & 1) * 2;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
              const int low = kBlocks == 2 ? 0 : k / 2 * 4 + k % 2;
              sts16(to + low * L::kValueStride, f[k]);
              sts16(to + (kBlocks == 2 ? 1 : low + 2) * L::kValueStride, f[k] >> 16);
            }
            tok.y = static_cast<float>(top - 127);
          }
        }
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(tokens0 + ((token & 24) + col) * 8), "f"(tok.x), "f"(tok.y)
                       : "memory");
      }
      __syncwarp();

      // ---- scores of this warp's tokens
      float x[kOwn][kN][4];  // [group][rows' tile][token g, g + 8; row 2 c (+ 1)]
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[j][n][e] = 0.f;
      const uint32_t key_at = stage + place_of(g) * L::kPitch + c * (kKeyWords * 4);
      // (blocks 0 2 1 3 of each four)
      const uint32_t scale_at = keys0 + place_of(g) * kBlocks * 2 + (D == 64 ? c >> 1 : (c & 1) * 2 + (c >> 1)) * 2;
      constexpr int kAtOnce = kCoop ? kOwn : 1;  // groups that share a load of the queries
#pragma unroll 1
      for (int k = 0; k < kSlices; ++k)
#pragma unroll
        for (int j0 = 0; j0 < kOwn; j0 += kAtOnce) {
          uint32_t w[kAtOnce][2][kKeyWords], sc[kAtOnce][2];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t from = key_at + (16 * (j0 + j) + 8 * h) * L::kPitch + k * 64;
              if constexpr (kKeyWords == 4) {
                const uint4 v = lds128(from);
                w[j][h][0] = v.x, w[j][h][1] = v.y, w[j][h][2] = v.z, w[j][h][3] = v.w;
              } else {
                const uint2 v = lds64(from);
                w[j][h][0] = v.x, w[j][h][1] = v.y;
              }
              uint32_t f;
              asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}"
                           : "=r"(f)
                           : "r"(scale_at + (16 * (j0 + j) + 8 * h) * kBlocks * 2 + k * 8));
              sc[j][h] = f * 0x10001u;
            }
#pragma unroll
          for (int i = 0; i < kKeyWords; ++i) {
            uint4 q[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              if constexpr (kCoop)
                q[n] = lds128(base + L::kOffQ + (((k * 4 + i) * kN + n) * 32 + lane) * 16);
              else
                q[n] = make_uint4(qf[i][n][0], qf[i][n][1], qf[i][n][2], qf[i][n][3]);
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              uint32_t r[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                codes_f16(w[j][h][i], r[h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[h][e] = mul_f16x2(r[h][e], sc[j][h]);
              }
#pragma unroll
              for (int n = 0; n < kN; ++n) {
                mma_f16(x[j0 + j][n], r[0][0], r[1][0], r[0][1], r[1][1], q[n].x, q[n].y);
                mma_f16(x[j0 + j][n], r[0][2], r[1][2], r[0][3], r[1][3], q[n].z, q[n].w);
              }
            }
          }
        }

      // ---- weights
      float vs[kOwn][2];  // S_v of tokens g and g + 8
      float mx[kN][2], ux[kN][2];
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 tk = lds64(tokens0 + (16 * j + 8 * h + g) * 8);
          vs[j][h] = __uint_as_float(tk.y);
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) x[j][n][2 * h + e] = __fmul_rn(x[j][n][2 * h + e], __uint_as_float(tk.x) * factor[n][e]);  // (never fused)
        }
      if (__any_sync(kFull, t0 < lo_most || t0 + kSub > hi_least)) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = t0 + 16 * j + 8 * h + place_of(g);
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (t >= hi[n][e] || t < lo[n][e]) x[j][n][2 * h + e] = -INFINITY;
          }
      }
      bool beyond = false;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = ux[n][e] = -INFINITY;
          const float mr = m[n][e] == -INFINITY ? 0.f : m[n][e];
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            mx[n][e] = fmaxf(mx[n][e], fmaxf(x[j][n][e], x[j][n][2 + e]));
            ux[n][e] = fmaxf(ux[n][e], fmaxf(x[j][n][e] - mr + vs[j][0], x[j][n][2 + e] - mr + vs[j][1]));
          }
          beyond |= mx[n][e] > m[n][e] + kLagM || ux[n][e] > u[n][e] + kLagU;
        }
      uint32_t p[kOwn][kN][2];  // [group][rows' tile][tokens 2 c, 2 c + 1 of row g, of the first and the second eight]
      float sum[kN][2];
      auto weights = [&] {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          float mr[2], ur[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a row that has seen nothing yet has no maximum to subtract
            mr[e] = m[n][e] == -INFINITY ? 0.f : m[n][e];
            ur[e] = (u[n][e] == -INFINITY ? 0.f : u[n][e]) - kWeightBits;
            sum[n][e] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kOwn; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v = x[j][n][2 * h + e] - mr[e];
                sum[n][e] += exp2_fast(v);
                w[e] = exp2_fast(v + (vs[j][h] - ur[e]));
              }
              p[j][n][h] = transposed(pack_f16(w[0], w[1]));
            }
        }
      };
      auto hand_on = [&] {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const uint32_t to = base + L::kOffP + (i & 1) * L::kP + ((warp * kOwn + j) * 32 + lane) * (8 * kN);
          if constexpr (kN == 2)
            sts128(to, make_uint4(p[j][0][0], p[j][0][1], p[j][1][0], p[j][1][1]));
          else
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(p[j][0][0]), "r"(p[j][0][1]) : "memory");
        }
      };
      weights();
      if constexpr (kCoop) {
        hand_on();
        beyond = __syncthreads_or(beyond || failed);
      } else {
        beyond = __any_sync(kFull, beyond);
      }
      if (beyond) {
        // all warps' largest of v, each row's in [0] or [1] of rows_sh
        auto largest = [&](float (&v)[kN][2], int word) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) v[n][e] = fmaxf(v[n][e], __shfl_xor_sync(kFull, v[n][e], o));
          if constexpr (kCoop) {
            float* words = reinterpret_cast<float*>(rows_sh) + word;
            if (g == 0)
#pragma unroll
              for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) words[2 * (warp * kRows + 8 * n + 2 * c + e)] = v[n][e];
            __syncthreads();
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v[n][e] = fmaxf(v[n][e], words[2 * (w * kRows + 8 * n + 2 * c + e)]);
          }
        };
        largest(mx, 0);
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[n][e] = fmaxf(mx[n][e], m[n][e]);
            const float mr = mx[n][e] == -INFINITY ? 0.f : mx[n][e];
            l[n][e] *= exp2_fast(m[n][e] - mr);
            u[n][e] += (m[n][e] == -INFINITY ? 0.f : m[n][e]) - mr;
            m[n][e] = mx[n][e];
            ux[n][e] = -INFINITY;
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
              ux[n][e] = fmaxf(ux[n][e], fmaxf(x[j][n][e] - mr + vs[j][0], x[j][n][2 + e] - mr + vs[j][1]));
          }
        largest(ux, 1);
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ux[n][e] = fmaxf(ux[n][e], u[n][e]);
            const float shrink = exp2_fast(u[n][e] - (ux[n][e] == -INFINITY ? 0.f : ux[n][e]));
            u[n][e] = ux[n][e];
#pragma unroll
            for (int t = 0; t < 4 * kWords; ++t) {
              acc[n][t][e] *= shrink;
              acc[n][t][2 + e] *= shrink;
            }
          }
        weights();
        if constexpr (kCoop) {
          hand_on();
          __syncthreads();
        }
      }
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        l[n][0] += sum[n][0];
        l[n][1] += sum[n][1];
      }
      if constexpr (kCoop) {  // every warp has left the sums of the other stage
        issue(i + 1);
        page_load(i + 2);
      }

      // ---- weighted sums of the values
      constexpr int kGroups = kCoop ? kTile / 16 : kOwn;
#pragma unroll(kCoop ? 2 : kGroups)
      for (int j = 0; j < kGroups; ++j) {
        uint32_t pb[kN][2];
        uint32_t from, sc_from;
        if constexpr (kCoop) {
          const uint32_t p_at = base + L::kOffP + (i & 1) * L::kP + (j * 32 + lane) * (8 * kN);
          if constexpr (kN == 2) {
            const uint4 v = lds128(p_at);
            pb[0][0] = v.x, pb[0][1] = v.y, pb[kN - 1][0] = v.z, pb[kN - 1][1] = v.w;
          } else {
            const uint2 v = lds64(p_at);
            pb[0][0] = v.x, pb[0][1] = v.y;
          }
          from = stage_all + j / kOwn * L::kPart + j % kOwn * 16 * L::kPitch;
          sc_from = values_all + j / kOwn * L::kSide + j % kOwn * 32;
        } else {
#pragma unroll
          for (int n = 0; n < kN; ++n) pb[n][0] = p[j][n][0], pb[n][1] = p[j][n][1];
          from = stage + j * 16 * L::kPitch;
          sc_from = values_all + warp * L::kSide + j * 32;
        }
        if constexpr (!kShared) from += L::kCodes + L::kRaw;
        // this thread's dimensions: 8 kWords g on
        const uint2 sc = lds64(sc_from + (wide0 / 32 + (kWords == 2 ? g >> 1 : g >> 2)) * L::kValueStride + c * 8);
        uint32_t w[4][kWords];  // places 2 c, 2 c + 1, and 8 on
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t row_at = from + (place_of(2 * c + (e & 1)) + 8 * (e >> 1)) * L::kPitch + wide0 / 2 + g * 4 * kWords;
          if constexpr (kWords == 2) {
            const uint2 v = lds64(row_at);
            w[e][0] = v.x, w[e][1] = v.y;
          } else {
            w[e][0] = lds32(row_at);
          }
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          // a byte of one code of each of two tokens, codes 2 t and 2 t + 1
          uint32_t ev[2][4], od[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            codes_f16((w[2 * h][k] & 0x0F0F0F0Fu) | ((w[2 * h + 1][k] << 4) & 0xF0F0F0F0u), ev[h]);
            codes_f16(((w[2 * h][k] >> 4) & 0x0F0F0F0Fu) | (w[2 * h + 1][k] & 0xF0F0F0F0u), od[h]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t a0 = mul_f16x2(ev[0][t], sc.x), a1 = mul_f16x2(od[0][t], sc.x);
            const uint32_t a2 = mul_f16x2(ev[1][t], sc.y), a3 = mul_f16x2(od[1][t], sc.y);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_f16(acc[n][4 * k + t], a0, a1, a2, a3, pb[n][0], pb[n][1]);
          }
        }
      }
      // ---- NaN values that only some rows see
      if (masked) {
        bool any = __any_sync(kFull, nan_value);
        if constexpr (kCoop) any = __syncthreads_or(any);
        if (any) {
          for (int t = 0; t < (kCoop ? kTile : kSub); ++t) {
            const uint8_t* from = smem + ((kCoop ? stage_all + t / kSub * L::kPart : stage) - base) +
                                  (kShared ? 0 : L::kCodes + L::kRaw) + L::kCodes + t % kSub * kBlocks;
            const int pos = kCoop ? t_begin + i * kTile + t : t0 + t;
            if (pos >= t_end) break;
            // (of a page outside the cache nothing was copied)
            if (static_cast<uint32_t>(pages_of[div_u32(static_cast<uint32_t>(pos) >> 4, a.per_page)]) >= static_cast<uint32_t>(a.pages))
              continue;
            bool row_nan = false;  // a shared row is a key as well: its score is NaN
            if constexpr (kShared)
              for (int k = 0; k < kBlocks; ++k) row_nan |= from[k] == 255;
            // the block of this thread's sums
            if (!row_nan && from[wide0 / 32 + (kWords == 2 ? g >> 1 : g >> 2)] != 255) continue;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (pos < lo[n][e] || pos >= hi[n][e]) continue;
                if (row_nan) l[n][e] = NAN;
#pragma unroll
                for (int x = 0; x < 4 * kWords; ++x) acc[n][x][e] = acc[n][x][2 + e] = NAN;
              }
          }
        }
      }
    }
    slot0 += parts;

    // ---- join the warps
    const bool whole = tile0 == 0 && tile1 == s.tiles;
    // this thread has, of each of its rows, dimensions wide0 + 8 kWords g on
    float to_m[kN][2];  // from sums relative to 2^(m + u + 21) to 2^m
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(kFull, l[n][e], o);
        to_m[n][e] = u[n][e] == -INFINITY ? 0.f : exp2f(u[n][e] - kSumBits);
      }
    float* part_out = parts0 + (static_cast<size_t>(blockIdx.x) * 2 + (begin ? 0 : 1)) * kPartFloats<D, kRows>;
    __syncthreads();  // all parts of the ring are read
    if (g == 0)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) rows_sh[warp * kRows + 8 * n + 2 * c + e] = make_float2(m[n][e], l[n][e]);
    if constexpr (kCoop) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * c + e;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += rows_sh[w * kRows + r].y;
          int token, q_head;
          const bool ok = un.row(a, s, r, token, q_head);
          float v[8 * kWords];
#pragma unroll
          for (int t = 0; t < 4 * kWords; ++t) v[2 * t] = acc[n][t][e] * to_m[n][e], v[2 * t + 1] = acc[n][t][2 + e] * to_m[n][e];
          if (whole) {
            if (!ok) continue;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint4* to = reinterpret_cast<uint4*>(a.out + static_cast<size_t>(token) * a.ldo +
                                                 static_cast<size_t>(q_head) * a.ldo_head + wide0 + 8 * kWords * g);
#pragma unroll
            for (int t = 0; t < kWords; ++t) to[t] = pack_out8(v + 8 * t, inv, a.q_f16);
            if (a.lse != nullptr && warp == 0 && g == 0)
              a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (m[n][e] + log2f(sum)) * 0.6931471805599453f;
          } else {
            if (warp == 0 && g == 0) {
              part_out[r] = m[n][e];
              part_out[kRows + r] = sum;
            }
            float4* to = reinterpret_cast<float4*>(part_out + 2 * kRows + r * D + wide0 + 8 * kWords * g);
#pragma unroll
            for (int t = 0; t < 2 * kWords; ++t) to[t] = make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
          }
        }
    } else {
      float* dump = reinterpret_cast<float*>(smem) + warp * kRows * (D + 4);
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float4* to = reinterpret_cast<float4*>(dump + (8 * n + 2 * c + e) * (D + 4) + 8 * kWords * g);
#pragma unroll
          for (int t = 0; t < 4 * kWords; t += 2)
            to[t / 2] = make_float4(acc[n][t][e] * to_m[n][e], acc[n][t][2 + e] * to_m[n][e], acc[n][t + 1][e] * to_m[n][e],
                                    acc[n][t + 1][2 + e] * to_m[n][e]);
        }
      __syncthreads();
      // so many threads to a row, eight dimensions of each at a time
      constexpr int kTeam = L::kThreads / kRows;
      const int r = threadIdx.x / kTeam, e0 = threadIdx.x % kTeam * 8;
      float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, rows_sh[w * kRows + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = rows_sh[w * kRows + r];
        f[w] = v.x == -INFINITY ? (v.y != v.y ? v.y : 0.f) : exp2f(v.x - top);
        sum += v.y * f[w];
      }
      int token, q_head;
      const bool ok = un.row(a, s, r, token, q_head);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int d = e0; d < D; d += kTeam * 8) {
        float v[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4* from = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (w * kRows + r) * (D + 4) + d);
          const float4 y = from[0], z = from[1];
          v[0] += y.x * f[w], v[1] += y.y * f[w], v[2] += y.z * f[w], v[3] += y.w * f[w];
          v[4] += z.x * f[w], v[5] += z.y * f[w], v[6] += z.z * f[w], v[7] += z.w * f[w];
        }
        if (whole) {
          if (ok)
            *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(token) * a.ldo +
                                      static_cast<size_t>(q_head) * a.ldo_head + d) = pack_out8(v, inv, a.q_f16);
        } else {
          float4* to = reinterpret_cast<float4*>(part_out + 2 * kRows + r * D + d);
          to[0] = make_float4(v[0], v[1], v[2], v[3]);
          to[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      if (threadIdx.x % kTeam == 0) {
        if (!whole) {
          part_out[r] = top;
          part_out[kRows + r] = sum;
        } else if (ok && a.lse != nullptr) {
          a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (top + log2f(sum)) * 0.6931471805599453f;
        }
      }
    }
  }
  if (failed) atomicOr(a.status, kStatusTimeout);
}

// f(kernel, join kernel, shared bytes, threads, rows of a unit) of a variant.
template <int D, bool kShared, typename F>
auto with_kernels(bool few, F&& f) {
  return few ? f(attend_kernel<D, kShared, 8>, launch_join<D, 8>, Layout<D, kShared, 8>::kBytes,
                 Layout<D, kShared, 8>::kThreads, 8, kUnitExtra<D>)
             : f(attend_kernel<D, kShared, 16>, launch_join<D, 16>, Layout<D, kShared, 16>::kBytes,
                 Layout<D, kShared, 16>::kThreads, 16, kUnitExtra<D>);
}
template <typename F>
auto with_variant(int v, F&& f) {
  const bool few = v >= kAttendVariants / 2;  // 8 rows
  switch (v % (kAttendVariants / 2)) {
    case 0: return with_kernels<64, false>(few, f);
    case 1: return with_kernels<64, true>(few, f);
    case 2: return with_kernels<128, false>(few, f);
    case 3: return with_kernels<128, true>(few, f);
    case 4: return with_kernels<256, false>(few, f);
    case 5: return with_kernels<256, true>(few, f);
    case 6: return with_kernels<512, false>(few, f);
    default: return with_kernels<512, true>(few, f);
  }
}

}  // namespace

int attend_variant(int d, bool shared) {
  const int i = d == 64 ? 0 : d == 128 ? 1 : d == 256 ? 2 : d == 512 ? 3 : -1;
  return i < 0 ? -1 : 2 * i + (shared ? 1 : 0);
}

cudaError_t set_attend_attributes(int sm_count, int (&ctas)[kAttendVariants]) {
  for (int v = 0; v < kAttendVariants; ++v) {
    const cudaError_t e = with_variant(v, [&](auto kernel, auto, int bytes, int threads, int, int) {
      cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      int n = 0;
      if (rc == cudaSuccess) rc = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, bytes);
      ctas[v] = n * sm_count;
      return rc == cudaSuccess && n < 1 ? cudaErrorInvalidConfiguration : rc;
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t attend_bytes(int d, int ctas, int rows) {
  return cut_bytes(ctas) + static_cast<size_t>(ctas) * 2 * rows * (d + 2) * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, int variant, int ctas, cudaStream_t stream) {
  return with_variant(variant, [&](auto kernel, auto join, int bytes, int threads, int rows, int extra) {
    ctas = attend_ctas(a, rows, extra, ctas);
    const cudaError_t e = launch_overlapping(kernel, dim3(ctas), threads, bytes, stream, a);
    if (e != cudaSuccess || ctas < 2) return e;
    return join(a, ctas, stream);
  });
}

}  // namespace mx
