// attend_rows.cu - attention of many query rows over the MXFP4 cache: prompts, drafts, wide
// groups of heads.
//
// As attend.cu, with the products on the 5th-generation tensor cores: 128 query rows x 128
// cached tokens at a time, S = Q K^T and O += P V, with both accumulators and the
// weights P in tensor memory. Keys and values are dequantized into shared memory as fp16, once
// for all rows of a CTA: two tiles of 128 rows up to d = 128 (so that one's softmax runs
// under the other's products), one at 256. A row of 64 dimensions of a token is 128
// bytes of the 128-byte swizzle: as an operand of S it is K-major, as one of O it
// is N-major, in the same place and layout.
//
// fp16 under powers of two, as in attend.cu, but of a whole tile: the codes are held as
// code * 2^(s - S + 13), S the largest scale of the tile's keys, or of all values so far,
// so a block is exact down to 2^-27 of that one. The weights are exp2(x - m + 7), rounded to fp16
// (2^-11 down to 2^-21 of the largest, 2^-32 of it below), where m is a maximum of the row's scores that is
// behind by 2^8 at most: O is only rescaled when a score goes beyond.
//
// What runs where: four warps to each tile of rows take S to P (a thread to a row), four
// dequantize, one issues the products. Bound by the tensor cores, then by the
// exponentials (half their time at d = 128). A pair of 128 x 128 tiles takes 1.82 us at d = 128, 1.58 at 64, 2.75
// (one of 256 dimensions) at 256, where the products alone are 1.15; a block of rows costs 12 us besides (launch, queries,
// first tiles, results). Three prompts (518 GFLOP) 494 us, 1049 TFLOP/s.
//
// A CTA to a block of rows, in splits of its tokens where the blocks are fewer than the SMs. (CTAs that
// stay, with equal runs of tiles, waste nothing on a last wave, 13 % of those prompts' time. But
// every role then carries its place in the run, a tile took 7 % longer, and 561 us were left.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attend.cuh"

namespace mx {
namespace {

constexpr int kTokens = 128;    // of a tile
constexpr int kRows = 128;      // of a tile of queries
constexpr float kLag = 8.f;     // a score may be 2^8 above the row's reference
constexpr float kTop = 7.f;     // 2^7 and 2^8: weights up to 2^15
constexpr int kCodeBits = 13;   // 6 * 2^13 < 65504

template <int D, bool kShared>
struct Plan {
  static constexpr int kTiles = D <= 128 ? 2 : 1;            // of queries
  static constexpr int kStages = D <= 128 || kShared ? 2 : 1;  // of dequantized tokens
  static constexpr int kSides = kShared ? 1 : 2;
  static constexpr int kBlocks = D / 32;
  static constexpr int kThreads = kTiles * 128 + 128 + 32;
  static constexpr int kTile = kTokens * D * 2;              // bytes of one side of a stage, or of a query tile
  static constexpr int kOffQ = 0;
  static constexpr int kOffStage = kTiles * kTile;
  static constexpr int kOffNan = kOffStage + kStages * kSides * kTile;  // [tile parity][token] blocks that are NaN
  static constexpr int kBytes = kOffNan + 2 * kTokens + 1024;     // and the alignment of the base
  // tensor memory: S (and P over it) of each tile, then O
  static constexpr int kColO = kTiles * kTokens;
  static constexpr int kCols = kColO + kTiles * D <= 256 ? 256 : 512;
};

__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&d);
}

struct Shared {
  uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], s_full[2], p_full[2][2], o_done[2];
  uint32_t tmem;
  int abort;
  int b, row_block;      // of this CTA; b < 0: none
  int top[2][4][2];      // largest scale bytes of each dequantizing warp's share: [tile parity][warp][side]
  // of the tile, by its parity
  float k_factor[2];     // 2^(S_k - 127 - 13)
  int v_ref[2];          // S_v
  int nan[2];            // the tile has NaN values
};

// (block of rows, sequence) of number `index` among all sequences' blocks, last block
// first; by one warp.
__device__ void find_block(const AttendArgs& a, int per_block, int index, Shared& sh) {
  const int lane = threadIdx.x & 31;
  auto blocks_of = [&](int b) { return b < a.B ? (seq_of(a, b, kRows).n * a.group + per_block - 1) / per_block : 0; };
  int sum = 0;
  for (int b = lane; b < a.B; b += 32) sum += blocks_of(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) sh.b = -1;
  __syncwarp();
  if (index >= sum) return;
  const int at = sum - 1 - index;
  int base = 0;
  for (int c = 0; c < a.B && base <= at; c += 32) {
    const int w = blocks_of(c + lane);
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (base + incl - w <= at && at < base + incl) {
      sh.b = c + lane;
      sh.row_block = at - (base + incl - w);
    }
    base += __shfl_sync(kFull, incl, 31);
  }
}

template <int D, bool kShared>
__global__ void __launch_bounds__(Plan<D, kShared>::kThreads, 1) attend_rows_kernel(const AttendArgs a, int splits) {
  using L = Plan<D, kShared>;
  constexpr int kTiles = L::kTiles, kStages = L::kStages, kBlocks = L::kBlocks;
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (base - smem_u32(raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kDequant = kTiles * 4, kIssue = kDequant + 4;  // first warps of these roles

  const uint32_t unit = blockIdx.x;
  const int split = unit % splits;
  const int head = unit / splits % a.heads;
  const int index = unit / (splits * a.heads);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), 4);
      mbar_init(smem_u32(&sh.v_full[i]), 4);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i][0]), 4);
      mbar_init(smem_u32(&sh.p_full[i][1]), 4);
      mbar_init(smem_u32(&sh.o_done[i]), 1);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssue) tmem_alloc(smem_u32(&sh.tmem), L::kCols);
  pdl_wait();
  if (warp == 0) {
    if (blockIdx.x == 0) {
      bool bad = false;
      for (int b = lane; b < a.B; b += 32) bad |= seq_of(a, b, kRows).bad;
      if (bad) atomicOr(a.status, kStatusBadInput);
    }
    find_block(a, kTiles * kRows, index, sh);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int b = sh.b;
  const bool work = b >= 0;
  Seq s = {};
  int row0 = 0, rows = 0, t_first = 0, tiles = 0;
  if (work) {
    s = seq_of(a, b, kRows);
    rows = s.n * a.group;
    row0 = sh.row_block * (kTiles * kRows);
    // tokens that any row of the block sees
    const int q_first = row0 / a.group, q_last = (min(row0 + kTiles * kRows, rows) - 1) / a.group;
    const int64_t from = static_cast<int64_t>(s.len) - s.n + q_first - a.window + 1;
    const int begin = a.window > 0 && from > 0 ? min(static_cast<int>(from), s.len) & ~15 : 0;
    const int end = a.causal ? max(min(s.len - s.n + q_last + 1, s.len), begin) : s.len;
    const int all = (end - begin + kTokens - 1) / kTokens;
    const int first = static_cast<int>(static_cast<int64_t>(all) * split / splits);
    tiles = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / splits) - first;
    t_first = begin + first * kTokens;
  }
  volatile int* abort = &sh.abort;
  auto wait = [&](uint64_t& bar, int n) {  // for the n-th completion
    if (mbar_wait_or(smem_u32(&bar), (n - 1) & 1, abort)) return true;
    if (*abort == 0) {
      *abort = 1;
      atomicOr(a.status, kStatusTimeout);
    }
    return false;
  };
  auto arrive_warp = [&](uint64_t& bar) {  // once for the warp (32 arrivals on a barrier go one by one)
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };
  // as wait, the same for the whole warp
  auto wait_warp = [&](uint64_t& bar, int n) { return __all_sync(kFull, wait(bar, n)) != 0; };

  // ---- queries: fp16, each row's largest brought into [2^14, 2^15)
  float row_factor = 0.f;
  int lo = 0, hi = 0, token = 0, q_head = 0;
  bool valid = false;
  const int tile = warp >> 2;
  constexpr int kLanes = D / 8, kEach = 32 / kLanes;
  // 16 bytes of one of this warp's rows, in the queries' place
  const uint32_t rows0 = base + L::kOffQ + tile * L::kTile + (warp & 3) * (32 * 128);
  auto rows_at = [&](int r, int i) { return rows0 + (i >> 3) * (kRows * 128) + r * 128 + (((i & 7) ^ (r & 7)) << 4); };
  if (work && warp < kDequant) {
    const int r = row0 + tile * kRows + (warp & 3) * 32 + lane;
    valid = r < rows;
    token = r / a.group;
    q_head = head * a.group + r - token * a.group;
    const int pos = s.len - s.n + token;
    token += s.q0;
    hi = !valid ? 0 : a.causal ? min(pos + 1, s.len) : s.len;
    lo = a.window > 0 ? pos - a.window + 1 : 0;
    // Rows come by whole lines, kLanes lanes to each (loaded by a thread to each row of its own, twice, they took
    // 10000 cycles, and the results 5700).
    const int64_t q_at = valid ? static_cast<int64_t>(token) * a.ldq + static_cast<int64_t>(q_head) * a.ldq_head : -1;
#pragma unroll 2
    for (int i = 0; i < kLanes; ++i) {
      const int r = i * kEach + lane / kLanes;
      const int64_t from = __shfl_sync(kFull, q_at, r);
      cp_async_16(rows_at(r, lane % kLanes), a.q + max(from, int64_t{0}) + lane % kLanes * 8, from >= 0 ? 16 : 0);
    }
    cp_async_wait_all();
    __syncwarp();
    uint32_t most = 0;
#pragma unroll 4
    for (int i = 0; i < kLanes; ++i) most = max(most, max_bits(lds128(rows_at(lane, i))));
    const int shift = query_shift(most, a.q_f16);
    // a negative scale turns the queries' sign: the factor of the scores is not negative
    const float f = a.scale_log2 < 0.f ? -pow2(shift) : pow2(shift);
    row_factor = pow2(-shift) * fabsf(a.scale_log2);
#pragma unroll 4
    for (int i = 0; i < kLanes; ++i) sts128(rows_at(lane, i), query_f16(lds128(rows_at(lane, i)), a.q_f16, f));
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (work && tiles > 0) {
    if (warp < kDequant) {
      // ================= softmax: a thread to a row
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + tile * kTokens, t_o = tmem + lanes + L::kColO + tile * D;
      float m = -INFINITY, l = 0.f;
      int v_ref = -1;
      uint32_t nan_blocks = 0;
      for (int j = 0; j < tiles; ++j) {
        const int t0 = t_first + j * kTokens;
        // the dequantizing warps' words are theirs to publish: through their own barrier
        if (!wait_warp(sh.s_full[tile], j + 1) || !wait_warp(sh.k_full[j % kStages], j / kStages + 1)) break;
        tc_fence_after();
        // not 0, as -inf times it has to stay; scores of 2^44 at most times 2^-100 are 0 all the same
        const float f = fmaxf(row_factor * sh.k_factor[j & 1], 0x1p-100f);
        const int vr = sh.v_ref[j & 1];
        if (sh.nan[j & 1]) {
          for (int t = 0; t < kTokens; ++t)
            if (t0 + t >= lo && t0 + t < hi) nan_blocks |= smem[L::kOffNan + (j & 1) * kTokens + t];
        }
        if (__any_sync(kFull, t0 < lo || t0 + kTokens > hi)) {
          // what a row does not see becomes -inf; tiles at the diagonal and the ends only
#pragma unroll 1
          for (int c = 0; c < kTokens; c += 32) {
            uint32_t r[32];
            tmem_ld32(t_s + c, r);
            tmem_ld_wait();
            const int from = lo - t0 - c, to = hi - t0 - c;
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = i >= from && i < to ? r[i] : 0xFF800000u;
            tmem_st32(t_s + c, r);
          }
          tmem_st_wait();
        }
        // (loops are not unrolled more than they have to be: twelve warps run different code, and
        // waited for instructions: 8500 cycles a pair of tiles)
        float top = -INFINITY;
        {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t r0[32], r1[32];
          tmem_ld32(t_s, r0);
#pragma unroll 1
          for (int c = 0; c < kTokens; c += 64) {
            tmem_ld_wait();
            tmem_ld32(t_s + c + 32, r1);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i & 3] = fmaxf(x[i & 3], __uint_as_float(r0[i]));
            tmem_ld_wait();
            if (c + 64 < kTokens) tmem_ld32(t_s + c + 64, r0);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i & 3] = fmaxf(x[i & 3], __uint_as_float(r1[i]));
          }
          top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * f;
        }
        // the reference: the row's maximum when one was first seen, or was exceeded by 2^8
        float scale_o = 1.f;
        if (top > m + kLag || m == -INFINITY) {
          const float keep = exp2_fast(m - (top == -INFINITY ? 0.f : top));  // m = -inf: 0
          l *= keep;
          scale_o = keep;
          m = top;
        }
        if (j > 0 && vr != v_ref) scale_o *= pow2(max(v_ref - vr, -126));
        const bool rescale = j > 0 && __any_sync(kFull, scale_o != 1.f);
        v_ref = vr;
        if (rescale) {
          if (!wait_warp(sh.o_done[tile], j)) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            tmem_ld32(t_o + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * scale_o);
            tmem_st32(t_o + c, r);
          }
        }
        const float sub = (m == -INFINITY ? 0.f : m) - kTop;
        float2 sum = make_float2(0.f, 0.f);
        {
          const float2 f2 = make_float2(f, f), sub2 = make_float2(-sub, -sub);
          auto weights = [&](auto exact, const uint32_t (&r)[32], int c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float2 x = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
              if constexpr (decltype(exact)::value)
                x = add_f32x2(make_float2(__fmul_rn(x.x, f), __fmul_rn(x.y, f)), sub2);
              else
                x = fma_f32x2(x, f2, sub2);
              x.x = exp2_fast(x.x);
              x.y = exp2_fast(x.y);
              sum = add_f32x2(sum, x);
              p[i / 2] = pack_f16(x.x, x.y);
            }
            // P lies over the S columns that this thread has read: 32 of them make 16 of P
            tmem_st16(t_s + c / 2, p);
          };
          auto all = [&](auto exact) {
            uint32_t r0[32], r1[32];
            tmem_ld32(t_s, r0);
#pragma unroll 1
            for (int c = 0; c < kTokens; c += 64) {
              tmem_ld_wait();
              tmem_ld32(t_s + c + 32, r1);
              weights(exact, r0, c);
              tmem_ld_wait();
              if (c + 64 < kTokens) tmem_ld32(t_s + c + 64, r0);
              weights(exact, r1, c + 32);
              // the sums over the first half of the tokens begin
              tmem_st_wait();
              tc_fence_before();
              arrive_warp(sh.p_full[tile][c / 64]);
            }
          };
          // Fused, a product is not rounded as the maximum's was. Its difference from that is off by up
          // to half a step of it, the same for a whole row: a quarter at 2^22, but 64 at 2^30, where a
          // weight would not be finite.
          if (__any_sync(kFull, fabsf(sub) > 0x1p22f))
            all(std::true_type{});
          else
            all(std::false_type{});
        }
        l += sum.x + sum.y;
      }
      // ---- the result
      if (wait_warp(sh.o_done[tile], tiles)) {
        tc_fence_after();
        if (kShared && nan_blocks) l = NAN;
        const bool whole = splits == 1;
        const float to_m = pow2(max(v_ref - 127 - kCodeBits, -126));
        const float inv = (whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f) * to_m;
        // parts of splits: [unit][row] {m, l} and the sums
        float* part = a.partial + static_cast<size_t>(unit) * (kTiles * kRows) * (D + 2);
        const int pr = tile * kRows + (warp & 3) * 32 + lane;
        const int64_t out_at = valid ? static_cast<int64_t>(token) * a.ldo + static_cast<int64_t>(q_head) * a.ldo_head : -1;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32(t_o + c, r);
          tmem_ld_wait();
          float v[32];
          const float x = !kShared && ((nan_blocks >> (c / 32)) & 1u) ? NAN : inv;
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (whole) {  // the products with the queries are done
#pragma unroll
            for (int i = 0; i < 4; ++i) sts128(rows_at(lane, c / 8 + i), pack_out8(v + 8 * i, x, a.q_f16));
          } else {
            float4* to = reinterpret_cast<float4*>(part + 2 * kTiles * kRows + static_cast<size_t>(pr) * D + c);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              to[i / 4] = make_float4(v[i] * x, v[i + 1] * x, v[i + 2] * x, v[i + 3] * x);
          }
        }
        if (!whole) {
          part[pr] = m - kTop;
          part[kTiles * kRows + pr] = l;
        } else {
          if (valid && a.lse != nullptr)
            a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (m - kTop + log2f(l)) * 0.6931471805599453f;
          __syncwarp();
#pragma unroll 2
          for (int i = 0; i < kLanes; ++i) {
            const int r = i * kEach + lane / kLanes;
            const int64_t to = __shfl_sync(kFull, out_at, r);
            const uint4 y = lds128(rows_at(r, lane % kLanes));
            if (to >= 0) *reinterpret_cast<uint4*>(a.out + to + lane % kLanes * 8) = y;
          }
        }
      }
    } else if (warp < kIssue) {
      // ================= dequantization
      const int tid = (warp - kDequant) * 32 + lane;
      // A thread has a token: one page, 16 kBlocks neighbouring bytes of each side. (A share of every
      // row to each thread, loads of whole lines, took four times the instructions for addresses and
      // 1300 of the 3800 cycles of a tile.) Eight neighbours store 16 bytes of eight rows: all banks.
      const int tok = tid;
      // Loads run ahead: the page number two tiles, rows one, where two tiles of them fit in the
      // registers; else a side's next rows are loaded when the present ones are converted.
      constexpr bool kAhead = L::kSides * kBlocks <= 8;
      struct Rows {
        uint4 code[kBlocks];
        uint32_t scale[(kBlocks + 3) / 4];
      };
      const int* pages_of = a.table + static_cast<size_t>(b) * a.ld_table;
      bool bad = false;  // a page outside the cache
      Rows now[L::kSides], next[kAhead ? L::kSides : 1];
      bool here, next_here;  // whether there is a token
      int page, place;       // the next row's
      const int t_stop = min(t_first + tiles * kTokens, s.len);
      auto load_page = [&](int j) {
        const int t = t_first + j * kTokens + tok;
        const uint32_t col = div_u32(static_cast<uint32_t>(t) >> 4, a.per_page);
        place = t - col * a.page_size;
        const int pg = pages_of[t < t_stop ? col : 0];
        page = t < t_stop ? pg : -1;
      };
      const size_t head_row = static_cast<size_t>(head) * a.page_size;
      const uint8_t* codes_of[2] = {a.k + head_row * (D / 2), a.v + head_row * (D / 2)};
      const uint8_t* scales_of[2] = {a.k_scales + head_row * kBlocks, a.v_scales + head_row * kBlocks};
      auto load = [&](int j, int sd, Rows& to, bool& is) {
        // what is not there is read from the first page, and not used
        is = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
        bad |= !is && t_first + j * kTokens + tok < t_stop;
        const int64_t pg = is ? page : 0;
        const int at = is ? place : 0;
        const uint8_t* codes = codes_of[sd] + pg * (sd ? a.v_page : a.k_page) + at * (D / 2);
        const uint8_t* scales = scales_of[sd] + pg * (sd ? a.v_scale_page : a.k_scale_page) + at * kBlocks;
        if constexpr (kBlocks == 2) {
          to.scale[0] = *reinterpret_cast<const uint16_t*>(scales);
        } else {
#pragma unroll
          for (int x = 0; x < kBlocks / 4; ++x) to.scale[x] = reinterpret_cast<const uint32_t*>(scales)[x];
        }
#pragma unroll
        for (int x = 0; x < kBlocks; ++x) to.code[x] = reinterpret_cast<const uint4*>(codes)[x];
      };
      load_page(0);
#pragma unroll
      for (int sd = 0; sd < L::kSides; ++sd) load(0, sd, now[sd], here);
      load_page(1);
      // no less than 2^-113: the factors are normal numbers
      int v_ref = 127 + kCodeBits - 126;
      bool ok = true;
      for (int j = 0; j < tiles; ++j) {
        const int st = j % kStages;
        if constexpr (kAhead) {
          uint32_t all = static_cast<uint32_t>(page);
#pragma unroll
          for (int sd = 0; sd < L::kSides; ++sd) {
            all ^= now[sd].scale[0];
#pragma unroll
            for (int x = 0; x < kBlocks; ++x) all ^= now[sd].code[x].x;
          }
          arrived(all);
#pragma unroll
          for (int sd = 0; sd < L::kSides; ++sd) load(j + 1, sd, next[sd], next_here);
          load_page(j + 2);
        }
        // the tile's largest scales, and which of the values' blocks are NaN
        int top[2] = {0, 0};
        uint32_t nan = 0;
#pragma unroll
        for (int sd = 0; sd < L::kSides; ++sd) {
#pragma unroll
          for (int x = 0; x < kBlocks; ++x) {
            const int sc = (now[sd].scale[x / 4] >> (8 * (x % 4))) & 255;
            if (sd == L::kSides - 1 && sc == 255) nan |= 1u << x;
            top[sd] = max(top[sd], sc < 255 ? sc : 0);
          }
          if (!here) top[sd] = 0, nan = 0;
        }
#pragma unroll
        for (int sd = 0; sd < L::kSides; ++sd) top[sd] = __reduce_max_sync(kFull, top[sd]);
        const bool any_nan = __any_sync(kFull, nan != 0);
        if (lane == 0) {
          sh.top[j & 1][warp - kDequant][0] = top[0];
          sh.top[j & 1][warp - kDequant][1] = (kShared ? top[0] : top[1]) | (any_nan ? 256 : 0);
        }
        // every thread comes here, also after a wait that ran out: all leave together
        if (named_barrier_or(1, 128, !ok)) break;
        int k_top = 127 + kCodeBits - 126;
        bool nans = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          k_top = max(k_top, sh.top[j & 1][w][0]);
          const int v = sh.top[j & 1][w][1];
          v_ref = max(v_ref, v & 255);
          nans |= v >= 256;
        }
        if constexpr (kShared) k_top = v_ref;  // one copy serves both
        // Stage and words are free: the scores of this stage's last tile are done, and with two stages
        // its sums, whose weights the softmax took from tile j - 2's words. (With one stage: the scores of
        // tile j - 1 were issued after those sums.)
        if (j >= kStages) {
          if (!kShared) ok = wait_warp(sh.k_empty[st], j / kStages);
          if (kShared || kStages > 1) ok = ok && wait_warp(sh.v_empty[st], j / kStages);
        }
        if (nans) {
          // one byte a token
          if (ok) smem[L::kOffNan + (j & 1) * kTokens + tid] = static_cast<uint8_t>(nan);
        }
        if (ok && tid == 0) {
          sh.k_factor[j & 1] = pow2(k_top - 127 - kCodeBits);
          sh.v_ref[j & 1] = v_ref;
          sh.nan[j & 1] = nans;
        }
#pragma unroll
        for (int sd = 0; sd < L::kSides; ++sd) {
          const int ref = sd ? v_ref : k_top;
          if (sd == 1 && kStages == 1 && j > 0) ok = ok && wait_warp(sh.v_empty[st], j);
          if (!ok) continue;
          const uint32_t to = base + L::kOffStage + (st * L::kSides + sd) * L::kTile + tok * 128;
#pragma unroll
          for (int x = 0; x < kBlocks; ++x) {
            const uint32_t sc = (now[sd].scale[x / 4] >> (8 * (x % 4))) & 255u;
            // biased exponent of fp16
            uint32_t f = static_cast<uint32_t>(max(static_cast<int>(sc) - ref + 15 + kCodeBits, 0)) * (0x10001u << 10);
            // a NaN value is 0 here and comes back in its rows' results; a NaN key is NaN
            if (sc == 255u) f = sd == L::kSides - 1 ? 0u : 0x7E007E00u;
            if (!here) f = 0u;
            const uint4 cw = now[sd].code[x];
            const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t r[4];
              codes_f16(w[i], r);
              sts128(to + (x >> 1) * (kTokens * 128) + (((((x & 1) << 2) + i) ^ (tok & 7)) << 4),
                     make_uint4(mul_f16x2(r[0], f), mul_f16x2(r[1], f), mul_f16x2(r[2], f), mul_f16x2(r[3], f)));
            }
          }
          fence_proxy_async_smem();
          // One stage: these keys may be there before the softmax has looked at the barrier for the tile before, and
          // it would take this phase for that one. Its first weights come after that look, and before these scores.
          if (kStages == 1 && sd == 0 && j > 0) ok = ok && wait_warp(sh.p_full[0][0], j);
          arrive_warp(sd == 0 ? sh.k_full[st] : sh.v_full[st]);
          if constexpr (!kAhead) load(j + 1, sd, now[sd], next_here);
        }
        if constexpr (kAhead) {
#pragma unroll
          for (int sd = 0; sd < L::kSides; ++sd) now[sd] = next[sd];
        } else {
          load_page(j + 2);
        }
        here = next_here;
      }
      if (bad) atomicOr(a.status, kStatusBadInput);
    } else if (warp == kIssue) {
      // ================= products: the warp goes along, one lane issues
      const uint32_t id_s = idesc_f16(kTokens, false), id_o = idesc_f16(D, true);
      const uint32_t d0 = __shfl_sync(kFull, tmem, 0);
      constexpr uint32_t kSide16 = L::kTile / 16;
      const uint32_t q_lo = sw128_lo(base + L::kOffQ), k_lo = sw128_lo(base + L::kOffStage),
                     v_lo = sw128_lo(base + L::kOffStage, kTokens * 128) + (L::kSides - 1) * kSide16;
      bool ok = true;
      auto sums = [&](int g, int j) {  // O_g += P_g V of tile j
        const int st = j % kStages;
        for (int half = 0; half < 2; ++half) {
          if (!wait_warp(sh.p_full[g][half], j + 1)) return false;
          if (!kShared && g == 0 && half == 0 && !wait_warp(sh.v_full[st], j / kStages + 1)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t v = v_lo + st * (L::kSides * kSide16) + half * 512;
#pragma unroll
            for (int k = 0; k < kTokens / 32; ++k)
              mma_ts(d0 + L::kColO + g * D, d0 + g * kTokens + half * 32 + k * 8, v + k * 128, kSw128Hi, id_o,
                     j > 0 || half > 0 || k > 0);
            if (half == 1) {
              tc_commit(smem_u32(&sh.o_done[g]));
              if (g == kTiles - 1) tc_commit(smem_u32(&sh.v_empty[st]));
            }
          }
          __syncwarp();
        }
        return true;
      };
      for (int j = 0; ok && j < tiles; ++j) {
        const int st = j % kStages;
        // (one stage: the keys come after the first weights of the tile before, its sums need not wait for them)
        static_assert(kStages > 1 || kTiles == 1, "one wait for a tile's keys");
        if (kStages > 1 && !wait_warp(sh.k_full[st], j / kStages + 1)) break;
        for (int g = 0; ok && g < kTiles; ++g) {
          if (j > 0) ok = sums(g, j - 1);
          if (kStages == 1) ok = ok && wait_warp(sh.k_full[st], j + 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t q0 = q_lo + g * kSide16, k0 = k_lo + st * (L::kSides * kSide16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(d0 + g * kTokens, q0 + (k >> 2) * 1024 + (k & 3) * 2, kSw128Hi, k0 + (k >> 2) * 1024 + (k & 3) * 2,
                     kSw128Hi, id_s, k > 0);
            tc_commit(smem_u32(&sh.s_full[g]));
            if (!kShared && g == kTiles - 1) tc_commit(smem_u32(&sh.k_empty[st]));
          }
          __syncwarp();
        }
      }
      for (int g = 0; ok && g < kTiles; ++g) ok = sums(g, tiles - 1);
    }
  } else if (work && warp < kDequant) {
    // no token in sight: zeros, or an empty part
    if (splits == 1) {
      if (valid) {
        uint16_t* out = a.out + static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head;
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr) a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = -INFINITY;
      }
    } else {
      float* part = a.partial + static_cast<size_t>(unit) * (kTiles * kRows) * (D + 2);
      const int pr = tile * kRows + (warp & 3) * 32 + lane;
      part[pr] = -INFINITY;
      part[kTiles * kRows + pr] = 0.f;
      for (int c = 0; c < D; c += 4)
        *reinterpret_cast<float4*>(part + 2 * kTiles * kRows + static_cast<size_t>(pr) * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_dealloc(tmem, L::kCols);
}

// The splits of each block of rows, added up in order: a warp to a row.
template <int D, int kRowsOfBlock>
__global__ void __launch_bounds__(256) attend_rows_join_kernel(const AttendArgs a, int splits) {
  __shared__ Shared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.heads, index = blockIdx.x / a.heads;
  if (warp == 0) find_block(a, kRowsOfBlock, index, sh);
  __syncthreads();
  if (sh.b < 0) return;
  const Seq s = seq_of(a, sh.b, kRows);
  const int rows = s.n * a.group;
  const int i = blockIdx.y * 8 + warp, r = sh.row_block * kRowsOfBlock + i;
  if (r >= rows) return;
  const float* first = a.partial + static_cast<size_t>(blockIdx.x) * splits * kRowsOfBlock * (D + 2);
  constexpr size_t kPart = static_cast<size_t>(kRowsOfBlock) * (D + 2);
  float top = -INFINITY;
  for (int p = 0; p < splits; ++p) top = fmaxf(top, first[p * kPart + i]);
  float sum = 0.f, v[D / 32] = {};
  for (int p = 0; p < splits; ++p) {
    const float* x = first + p * kPart;
    const float m = x[i], l = x[kRowsOfBlock + i];
    const float f = m == -INFINITY ? (l != l ? l : 0.f) : exp2f(m - top);
    sum += l * f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] += x[2 * kRowsOfBlock + static_cast<size_t>(i) * D + c * 32 + lane] * f;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int q_token = r / a.group, token = s.q0 + q_token, q_head = head * a.group + r - q_token * a.group;
  uint16_t* out = a.out + static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = static_cast<uint16_t>(pack_out(v[c] * inv, 0.f, a.q_f16));
  if (a.lse != nullptr && lane == 0)
    a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool kShared, typename F>
auto with_kernels(F&& f) {
  using L = Plan<D, kShared>;
  return f(attend_rows_kernel<D, kShared>, attend_rows_join_kernel<D, L::kTiles * kRows>, L::kBytes, L::kThreads,
           L::kTiles * kRows);
}
template <typename F>
auto with_variant(int v, F&& f) {
  switch (v) {
    case 0: return with_kernels<64, false>(f);
    case 1: return with_kernels<64, true>(f);
    case 2: return with_kernels<128, false>(f);
    case 3: return with_kernels<128, true>(f);
    case 4: return with_kernels<256, false>(f);
    default: return with_kernels<256, true>(f);
  }
}

}  // namespace

cudaError_t set_attend_rows_attributes() {
  for (int v = 0; v < kAttendRowsVariants; ++v) {
    const cudaError_t e = with_variant(v, [&](auto kernel, auto, int bytes, int, int) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

AttendRowsPlan plan_attend_rows(int d, bool shared, int B, int T, bool uniform, int heads, int group, int64_t most_tokens,
                                int sm_count) {
  AttendRowsPlan p = {};
  const int v = attend_variant(d, shared);
  if (v < 0 || v >= kAttendRowsVariants) return p;
  // blocks of rows: at most one beyond the full ones in each sequence
  const int per = with_variant(v, [](auto, auto, int, int, int rows) { return rows; });
  const int64_t most = static_cast<int64_t>(T) * group / per + std::min(B, T);
  const int64_t blocks = uniform ? (static_cast<int64_t>(T / B) * group + per - 1) / per * B : most;
  if (blocks * heads >= (int64_t{1} << 30)) return p;
  p.blocks = static_cast<int>(blocks);
  const int64_t tiles = (most_tokens + kTokens - 1) / kTokens;
  const int64_t units = static_cast<int64_t>(p.blocks) * heads;
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sm_count / units, tiles)));
  p.ok = true;
  return p;
}

// Parts of at most sm_count splits.
size_t attend_rows_bytes(int d, bool shared, int sm_count) {
  const int v = attend_variant(d, shared);
  if (v < 0 || v >= kAttendRowsVariants) return 0;
  const int per = with_variant(v, [](auto, auto, int, int, int rows) { return rows; });
  return static_cast<size_t>(sm_count) * per * (d + 2) * sizeof(float);
}

cudaError_t launch_attend_rows(const AttendArgs& a, int d, bool shared, const AttendRowsPlan& p, cudaStream_t stream) {
  return with_variant(attend_variant(d, shared), [&](auto kernel, auto join, int bytes, int threads, int rows) {
    const uint32_t blocks = static_cast<uint32_t>(p.blocks) * a.heads;
    const cudaError_t e = launch_overlapping(kernel, dim3(blocks * p.splits), threads, bytes, stream, a, p.splits);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_overlapping(join, dim3(blocks, rows / 8), 256, 0, stream, a, p.splits);
  });
}

}  // namespace mx
