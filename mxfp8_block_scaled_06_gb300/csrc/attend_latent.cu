// attend_latent.cu - attention over latents of 512 dimensions in the MXFP4 cache, which are keys and
// values in one: prompts, and drafts of many tokens.
//
// On the 5th-generation tensor cores with the cache as the products' rows: for 128 tokens
//   S^T[token, row] = sum_d latent[token, d] Q[row, d]    (128 x 64 x 512)
//   O^T[d, row]    += sum_t latent[t, d] P[t, row]        (4 times 128 x 64 x 128)
// for 64 query rows. The latents are dequantized once, to fp16 in shared memory, [8 chunks of 64
// dimensions][128 tokens][128 bytes in the 128-byte swizzle], and read from there by both: K-major
// for the scores, M-major for the sums. fp16 under powers of two as in attend_rows.cu: the codes
// relative to the largest scale so far, weights 2^7 above a reference that a score may exceed by 2^8.
//
// The fp16 tile fills the shared memory, so there is one, and its chunks change hands singly: while the sums
// of tile j go from one 128 dimensions to the next, the chunks behind them are written for tile
// j + 1, and its scores follow these. What bounds it is that chain: a tile takes 4.4 us, 9100 cycles (a block of 64
// rows on every SM over 2048 and 8192 tokens, 93 and 304 us; 22 us beside its tiles), of which 3400 are
// the 64 products (53 cycles each, shared memory's rate; 68 for 128 rows, which it has no room for),
// 3700 the weights between them, the rest the last chunk's way to the scores. Two prompts of up to
// 6000 tokens and 16 heads: 727 us, 488 TFLOP/s, against 1609 us with 16 rows at a time (attend.cu).
//
// Four warps have a token to a thread and turn S to P (rows' references and sums in shared memory),
// eight dequantize, one issues the products; one CTA to an SM, its run of tiles as in attend.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attend.cuh"

namespace mx {
namespace {

constexpr int kD = 512;
constexpr int kTokens = 128;
static_assert(kTokens == kAttendTile, "tiles of the sequences' work");
constexpr int kRows = 64;  // of queries
constexpr int kBlocks = kD / 32, kChunks = kD / 64;
constexpr int kSoftmax = 4, kDequant = 8, kWarpsAll = kSoftmax + kDequant + 1, kThreads = 32 * kWarpsAll;
constexpr float kLag = 8.f, kTop = 7.f;
constexpr int kCodeBits = 13;  // 6 * 2^13 < 65504

constexpr int kOffQ = kTokens * kD * 2;                 // [chunk][row][128 bytes]
constexpr int kOffP = kOffQ + kRows * kD * 2;           // [token][128 bytes]
constexpr int kBytes = kOffP + kTokens * 128 + 1024;
constexpr int kColO = kRows;                            // S^T, then O^T of each 128 dimensions
constexpr int kCols = 512;                              // 5 * kRows of them, and a power of two

// ------------------------------------------------------------- runs of what rows see
// Blocks of kRows rows whose first and last tokens differ: block r of R has the tiles of 128 tokens that any
// of its rows sees, one at least. Blocks r and R - 1 - r stand together, as causal ones have about the same number of
// tiles between them: places for so many, the most that two have; the last of them may be empty. A block has
// kExtra places more in front of its tiles, for its queries and results.
// (48 sequences of up to 8192 tokens and 64 query rows 121 us without, 101 with 2, 87 with 4, 87 with 6; of 8192 rows
// 12.2 ms, 8.0, 6.6, 6.8.)
constexpr int kExtra = 4;
struct Span {
  int begin, end;  // tokens
  int tiles;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Seq& s, int r) {
  const int rows = s.n * a.group;
  const int pos0 = s.len - s.n + r * kRows / a.group, pos1 = s.len - s.n + (min((r + 1) * kRows, rows) - 1) / a.group;
  const int64_t from = static_cast<int64_t>(pos0) - a.window + 1;
  Span p;
  p.begin = a.window > 0 && from > 0 ? min(static_cast<int>(from), s.len) & ~15 : 0;
  p.end = a.causal ? max(min(pos1 + 1, s.len), p.begin) : s.len;
  p.tiles = max((p.end - p.begin + kAttendTile - 1) / kAttendTile, 1);
  return p;
}
__device__ __forceinline__ int64_t pair_tiles(const AttendArgs& a, const Seq& s) {
  // the last block ends last; with a window, none is longer than that and its rows' tokens
  int64_t most = 2 * static_cast<int64_t>((s.len + kAttendTile - 1) / kAttendTile);
  if (a.causal && s.n <= s.len) {
    // the two ends are (r + 1) kRows / group and (R - r) kRows / group tokens behind the cached ones, at most
    const int64_t ends = 2 * (static_cast<int64_t>(s.len) - s.n) + (static_cast<int64_t>(s.row_tiles) + 1) * kRows / a.group + 2;
    most = min(most, (ends + 2 * (kAttendTile - 1)) / kAttendTile);
  }
  if (a.window > 0)
    most = min(most, 2 * ((static_cast<int64_t>(a.window) + kRows / a.group + 16 + kAttendTile) / kAttendTile));
  return max(most, int64_t{2}) + 2 * kExtra;
}
__device__ __forceinline__ int64_t head_tiles(const AttendArgs& a, const Seq& s) {
  return s.row_tiles / 2 * pair_tiles(a, s) +
         (s.row_tiles & 1 ? span_of(a, s, s.row_tiles / 2).tiles + kExtra : 0);
}

// Where a warp is in its CTA's run of parts of blocks: in shared memory, a copy for each warp, as it would take
// registers from the roles' loops.
struct Walk {
  int64_t at, stop, run;
  int64_t pair_first, block_first;  // numbers of the first tiles
  int b, head, pair, second;        // block `pair` from the front, or (second) from the back
  Seq s;
};
// A part of a block.
struct Part {
  AttendUnit un;
  int b, q0, n, len;      // of its sequence
  bool whole;             // all of the block
  bool begin;             // the run begins with it
  int t_begin, t_end;     // tokens
  int tiles;              // to take, of 128 tokens
  int hi_least, lo_most;  // tokens from lo_most to hi_least are seen by all rows
  __device__ __forceinline__ bool row(const AttendArgs& a, int i, int& token, int& q_head) const {
    const int r = un.row0 + i;
    token = r / a.group;
    q_head = un.head * a.group + r - token * a.group;
    token += q0;
    return r < un.rows;
  }
};
__device__ __forceinline__ void walk_start(const AttendArgs& a, const Found& f, int64_t total, Walk& walk) {
  Walk w = {};
  w.run = run_of(total, gridDim.x);
  w.at = w.run * blockIdx.x;
  w.stop = min(w.at + w.run, total);
  if (w.at < w.stop) {
    w.b = f.b;
    w.s = seq_of(a, f.b, kRows);
    const int64_t in = w.at - f.first, of_head = head_tiles(a, w.s), of_pair = pair_tiles(a, w.s);
    w.head = static_cast<int>(in / of_head);
    const int64_t in_head = in - w.head * of_head;
    w.pair = static_cast<int>(min(in_head / of_pair, static_cast<int64_t>(w.s.row_tiles / 2)));
    w.pair_first = w.block_first = f.first + w.head * of_head + w.pair * of_pair;
  }
  if ((threadIdx.x & 31) == 0) walk = w;
  __syncwarp();
}
// The next part, the same for all warps (code that the roles share). note: writes the CTA's cut where the run begins within a block.
__device__ __noinline__ bool walk_next(const AttendArgs& a, Walk& walk, Part& p, Cut* note = nullptr) {
  Walk w = walk;
  bool found = false;
  while (w.at < w.stop) {
    const int half = w.s.row_tiles / 2;
    const int r = w.second ? w.s.row_tiles - 1 - w.pair : w.pair;
    const Span span = span_of(a, w.s, r);
    const int64_t first = w.block_first + kExtra;
    w.at = max(w.at, first);
    if (w.at >= w.stop) break;
    const int64_t off = w.at - first;
    if (off < span.tiles) {
      const int tile0 = static_cast<int>(off), take = static_cast<int>(min(span.tiles - off, w.stop - w.at));
      const int rows = w.s.n * a.group;
      p.un = AttendUnit{w.head, r * kRows, rows};
      p.b = w.b, p.q0 = w.s.q0, p.n = w.s.n, p.len = w.s.len;
      p.whole = take == span.tiles;
      p.begin = w.at == w.run * blockIdx.x;
      p.t_begin = min(span.begin + tile0 * kAttendTile, span.end);
      p.t_end = min(span.begin + (tile0 + take) * kAttendTile, span.end);
      p.tiles = (p.t_end - p.t_begin + kAttendTile - 1) / kAttendTile;
      const int pos0 = w.s.len - w.s.n + r * kRows / a.group;
      const int pos1 = w.s.len - w.s.n + (min((r + 1) * kRows, rows) - 1) / a.group;
      p.hi_least = a.causal ? min(pos0 + 1, w.s.len) : w.s.len;
      p.lo_most = a.window > 0 ? pos1 - a.window + 1 : 0;
      if (note != nullptr && p.begin && tile0 > 0) {
        // others have parts of this block too
        Cut c;
        c.first = static_cast<int>(first / w.run);
        c.last = static_cast<int>((first + span.tiles - 1) / w.run);
        c.later = first != w.run * c.first;
        c.head = w.head, c.row0 = r * kRows, c.rows = rows, c.q0 = w.s.q0;
        *note = c;
      }
      w.at += take;
      found = true;
      break;
    }
    if (!w.second && w.pair < half) {
      w.second = 1;
      w.block_first += span.tiles + kExtra;
      continue;
    }
    w.pair_first += w.pair < half ? pair_tiles(a, w.s) : span.tiles + kExtra;
    w.block_first = w.pair_first;
    w.at = max(w.at, w.pair_first);  // places behind the second block are empty
    w.second = 0;
    if (w.at >= w.stop) break;
    if (++w.pair < half + (w.s.row_tiles & 1)) continue;
    w.pair = 0;
    if (++w.head < a.heads) continue;
    w.head = 0;
    do w.s = seq_of(a, ++w.b, kRows);
    while (w.s.row_tiles == 0);  // there is one with queries: the run goes on
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) walk = w;
  __syncwarp();
  return found;
}

struct Shared {
  uint64_t pair_full[4], sums_done[4], s_full, p_full, q_full;
  uint32_t tmem;
  int abort;
  ScanShared scan;
  Walk walk[kWarpsAll];
  int top[2][kDequant];      // largest scale bytes, + 256: with NaN
  int ref[2];                // of the tile, by its parity
  uint8_t nan[2][kTokens];   // tokens with a NaN
  int any_nan[2];
  // of the rows, the softmax's own
  // (sub, lim: what is subtracted from a score, and which one moves the reference)
  alignas(16) float factor[kRows], m[kRows], sub[kRows], lim[kRows], keep[kRows];
  int lo[kRows], hi[kRows];
  float part[kSoftmax][kRows];
  size_t to[kRows];  // places of the rows' results
};

// Over the warp's lanes, of 16 values in each: lane i has f of them all for value i / 2. 16 shuffles,
// where one value after the other takes 80.
template <typename F>
__device__ __forceinline__ float reduce16(const float (&x)[16], int lane, F f) {
  float a[8], b[4], c[2];
  const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4, h2 = lane & 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = f(h16 ? x[i + 8] : x[i], __shfl_xor_sync(kFull, h16 ? x[i] : x[i + 8], 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = f(h8 ? a[i + 4] : a[i], __shfl_xor_sync(kFull, h8 ? a[i] : a[i + 4], 8));
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = f(h4 ? b[i + 2] : b[i], __shfl_xor_sync(kFull, h4 ? b[i] : b[i + 2], 4));
  const float y = f(h2 ? c[1] : c[0], __shfl_xor_sync(kFull, h2 ? c[0] : c[1], 2));
  return f(y, __shfl_xor_sync(kFull, y, 1));
}

__global__ void __launch_bounds__(kThreads, 1) attend_latent_kernel(const AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kIssue = kSoftmax + kDequant;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.pair_full[i]), kDequant);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.sums_done[i]), 1);
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.p_full), kSoftmax);
    mbar_init(smem_u32(&sh.q_full), kSoftmax);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssue) tmem_alloc(smem_u32(&sh.tmem), kCols);
  pdl_wait();
  int64_t total;
  auto work = [](const AttendArgs& a, const Seq& s) { return a.heads * head_tiles(a, s); };
  const Found found = find_run<kRows, kWarpsAll>(a, sh.scan, work, total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // after the tensor memory is here: a dependent CTA may take what is left
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;
  auto wait = [&](uint64_t& bar, uint32_t n) {  // for the n-th completion
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
  auto wait_warp = [&](uint64_t& bar, uint32_t n) { return __all_sync(kFull, wait(bar, n)) != 0; };
  Walk& walk = sh.walk[warp];
  walk_start(a, found, total, walk);
  Part next;
  Cut* cuts = reinterpret_cast<Cut*>(a.partial);
  if (threadIdx.x == 0) cuts[blockIdx.x].last = -1;
  float* parts0 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.partial) + cut_bytes(gridDim.x));
  uint32_t done = 0;  // tiles taken

  if (warp < kSoftmax) {
    // ================= queries, weights, results: a thread to a token, or to a dimension of the sums
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int tid = threadIdx.x;
    bool ok = true;
    while (ok && walk_next(a, walk, next, tid == 0 ? cuts + blockIdx.x : nullptr)) {
      const Part w = next;
      // ---- queries to fp16, a warp to a row at a time: each row's largest into [2^14, 2^15)
      // (four rows' loads at a time)
#pragma unroll 1
      for (int r0 = warp; r0 < kRows; r0 += 4 * kSoftmax) {
        uint4 v[4][2];
        int pos[4];
        bool there[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int token, q_head;
          const bool valid = w.row(a, r0 + i * kSoftmax, token, q_head);
          const uint16_t* q = a.q + static_cast<size_t>(token) * a.ldq + static_cast<size_t>(q_head) * a.ldq_head;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            v[i][j] = valid ? *reinterpret_cast<const uint4*>(q + (lane + 32 * j) * 8) : make_uint4(0, 0, 0, 0);
          pos[i] = w.len - w.n + token - w.q0;
          there[i] = valid;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i * kSoftmax;
          const int shift = query_shift(__reduce_max_sync(kFull, max(max_bits(v[i][0]), max_bits(v[i][1]))), a.q_f16);
          const float f = a.scale_log2 < 0.f ? -pow2(shift) : pow2(shift);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int ch = lane + 32 * j;
            sts128(base + kOffQ + (ch >> 3) * (kRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                   query_f16(v[i][j], a.q_f16, f));
          }
          if (lane == 0) {
            sh.factor[r] = pow2(-shift) * fabsf(a.scale_log2);
            sh.m[r] = sh.lim[r] = -INFINITY;
            sh.sub[r] = -kTop;
            sh.hi[r] = !there[i] ? 0 : a.causal ? min(pos[i] + 1, w.len) : w.len;
            sh.lo[r] = a.window > 0 ? pos[i] - a.window + 1 : 0;
          }
        }
      }
      fence_proxy_async_smem();
      if (w.tiles > 0) arrive_warp(sh.q_full);
      named_barrier_sync(1, 32 * kSoftmax);
      float l[kRows / 16];  // of row 16 g + lane / 2, this warp's tokens
#pragma unroll
      for (int g = 0; g < kRows / 16; ++g) l[g] = 0.f;
      int ref = 0;
      for (int j = 0; j < w.tiles; ++j) {
        const uint32_t n = done + j + 1;
        // the dequantizing warps' words are published through the last chunk's barrier
        ok = ok && wait_warp(sh.s_full, n) && wait_warp(sh.pair_full[3], n);
        tc_fence_after();
        const int par = (n - 1) & 1;
        const int new_ref = sh.ref[par];
        const float kf = pow2(new_ref - 127 - kCodeBits);
        const bool nan = sh.any_nan[par] != 0 && sh.nan[par][tid] != 0;
        const int t0 = w.t_begin + j * kTokens, t = t0 + tid;
        // tokens that not every row sees, or NaN
        const bool special = t0 < w.lo_most || t0 + kTokens > w.hi_least || sh.any_nan[par] != 0;
        // scores of 16 rows of this token
        auto scores = [&](int r0, float (&x)[16]) {
          uint32_t v[16];
          tmem_ld_32x32b_x16_nowait(tmem + lanes + r0, v);
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(&f[i]) = *reinterpret_cast<const float4*>(&sh.factor[r0 + i]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__uint_as_float(v[i]), kf * f[i]);  // (never fused)
          if (special) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (nan) x[i] = NAN;
              if (t >= sh.hi[r0 + i] || t < sh.lo[r0 + i]) x[i] = -INFINITY;
            }
          }
        };
        // The weights, by the references as they are, and whether one has to move. (Loops are rolled: with a
        // thread's 64 rows in a row, the warps waited for instructions, and took 5300 cycles instead of
        // 3700.)
        float sum[kRows / 16];
        auto weights = [&] {
          bool beyond = false;
          float x[16];
#pragma unroll 1
          for (int g = 0; g < kRows / 16; ++g) {
            scores(16 * g, x);
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 sub4 = *reinterpret_cast<const float4*>(&sh.sub[16 * g + i]);
              const float4 lim4 = *reinterpret_cast<const float4*>(&sh.lim[16 * g + i]);
              const float sub[4] = {sub4.x, sub4.y, sub4.z, sub4.w}, lim[4] = {lim4.x, lim4.y, lim4.z, lim4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                beyond |= x[i + e] > lim[e];
                x[i + e] = exp2_fast(x[i + e] - sub[e]);
              }
              p[i / 2] = pack_f16(x[i], x[i + 1]);
              p[i / 2 + 1] = pack_f16(x[i + 2], x[i + 3]);
            }
            const uint32_t to = base + kOffP + tid * 128;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              sts128(to + (((2 * g + i) ^ (tid & 7)) << 4), make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]));
            const float y = reduce16(x, lane, [](float p, float q) { return p + q; });
#pragma unroll
            for (int k = 0; k < kRows / 16; ++k) sum[k] = g == k ? y : sum[k];
          }
          return beyond;
        };
        const bool beyond = weights() || (j > 0 && new_ref != ref);
        // a wait that ran out makes all four warps leave together
        const bool votes = named_barrier_or(1, 32 * kSoftmax, beyond || !ok);
        if (*abort != 0) ok = false;
        if (votes) {
          // the rows' references become their maxima
#pragma unroll 1
          for (int r0 = 0; r0 < kRows; r0 += 16) {
            float x[16];
            scores(r0, x);
            const float y = reduce16(x, lane, [](float p, float q) { return fmaxf(p, q); });
            if ((lane & 1) == 0) sh.part[warp][r0 + lane / 2] = y;
          }
          named_barrier_sync(1, 32 * kSoftmax);
          if (tid < kRows) {
            float top = sh.m[tid];
#pragma unroll
            for (int i = 0; i < kSoftmax; ++i) top = fmaxf(top, sh.part[i][tid]);
            sh.keep[tid] = exp2_fast(sh.m[tid] - (top == -INFINITY ? 0.f : top));  // m = -inf: 0
            sh.m[tid] = top;
            sh.sub[tid] = (top == -INFINITY ? 0.f : top) - kTop;
            sh.lim[tid] = top + kLag;
          }
          named_barrier_sync(1, 32 * kSoftmax);
#pragma unroll
          for (int g = 0; g < kRows / 16; ++g) l[g] *= sh.keep[16 * g + lane / 2];
          if (j > 0) {  // the sums of the tiles before are done: this tile's scores were issued behind them
            const float by = pow2(max(ref - new_ref, -126));
#pragma unroll 1
            for (int c = 0; c < 4 * kRows; c += 16) {
              uint32_t v[16];
              tmem_ld_32x32b_x16_nowait(tmem + lanes + kColO + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * (by * sh.keep[c % kRows + i]));
              tmem_st16(tmem + lanes + kColO + c, v);
            }
            tmem_st_wait();
          }
        }
        if (votes) weights();
        ref = new_ref;
#pragma unroll
        for (int g = 0; g < kRows / 16; ++g) l[g] += sum[g];
        fence_proxy_async_smem();
        tc_fence_before();
        arrive_warp(sh.p_full);
      }
      done += w.tiles;
      // ---- results
      if (w.tiles > 0) ok = ok && wait_warp(sh.sums_done[3], done);
      tc_fence_after();
      if ((lane & 1) == 0)
#pragma unroll
        for (int g = 0; g < kRows / 16; ++g) sh.part[warp][16 * g + lane / 2] = l[g];
      named_barrier_sync(1, 32 * kSoftmax);
      const bool whole = w.whole;
      float* part = parts0 + (static_cast<size_t>(blockIdx.x) * 2 + (w.begin ? 0 : 1)) * kPartFloats<kD, kRows>;
      if (tid < kRows) {
        int token, q_head;
        const bool valid = w.row(a, tid, token, q_head);
        const float sum = sh.part[0][tid] + sh.part[1][tid] + sh.part[2][tid] + sh.part[3][tid];
        sh.keep[tid] = sum == 0.f ? 0.f : 1.f / sum;
        sh.to[tid] = static_cast<size_t>(token) * a.ldo + static_cast<size_t>(q_head) * a.ldo_head;
        if (valid && !whole) {
          part[tid] = sh.m[tid] - kTop;
          part[kRows + tid] = sum;
        } else if (valid && a.lse != nullptr) {
          a.lse[static_cast<size_t>(token) * a.q_heads + q_head] = (sh.m[tid] - kTop + log2f(sum)) * 0.6931471805599453f;
        }
      }
      named_barrier_sync(1, 32 * kSoftmax);
      const float to_m = w.tiles > 0 ? pow2(max(ref - 127 - kCodeBits, -126)) : 0.f;
#pragma unroll 1
      for (int c = 0; c < 4 * kRows; c += 16) {
        uint32_t v[16];
        if (w.tiles > 0) {
          tmem_ld_32x32b_x16_nowait(tmem + lanes + kColO + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0u;
        }
        const int d = c / kRows * 128 + tid, r0 = c % kRows, rows = w.un.rows - w.un.row0 - r0;
        if (!whole) {
          float* to = part + 2 * kRows + r0 * kD + d;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i < rows) to[i * kD] = __uint_as_float(v[i]) * to_m;
          continue;
        }
        // the places and factors before the first store, which might be to them for all that is known
        size_t to[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          to[i] = sh.to[r0 + i];
          v[i] = pack_out(__uint_as_float(v[i]) * sh.keep[r0 + i] * to_m, 0.f, a.q_f16);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < rows) a.out[to[i] + d] = static_cast<uint16_t>(v[i]);
      }
      tc_fence_before();
      ok = !named_barrier_or(1, 32 * kSoftmax, !ok);  // the rows' words are read; all go on, or none
    }
  } else if (warp < kIssue) {
    // ================= dequantization: a thread has one half of every 64 dimensions of a token
    const int tid = threadIdx.x - 32 * kSoftmax;
    const int tok = (tid & 7) + 8 * (tid >> 4), half = (tid >> 3) & 1;
    bool ok = true, bad = false, leave = false;
    while (!leave && walk_next(a, walk, next)) {
      const Part w = next;
      const int* pages_of = a.table + static_cast<size_t>(w.b) * a.ld_table;
      const size_t head_row = static_cast<size_t>(w.un.head) * a.page_size;
      const uint8_t* codes_of = a.k + head_row * (kD / 2) + half * 16;
      const uint8_t* scales_of = a.k_scales + head_row * kBlocks;
      int page, place;
      auto load_page = [&](int j) {
        const int t = w.t_begin + j * kTokens + tok;
        const uint32_t col = div_u32(static_cast<uint32_t>(t) >> 4, a.per_page);
        place = t - col * a.page_size;
        const int pg = pages_of[t < w.t_end ? col : 0];
        page = t < w.t_end ? pg : -1;
      };
      uint4 code[kChunks], next[kChunks], scale, next_scale;
      bool here, next_here;
      auto load = [&](int j, uint4 (&to)[kChunks], uint4& sc, bool& is) {
        // what is not there is read from the first page, and not used
        is = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
        bad |= !is && w.t_begin + j * kTokens + tok < w.t_end;
        const int64_t pg = is ? page : 0, at = is ? place : 0;
        sc = *reinterpret_cast<const uint4*>(scales_of + pg * a.k_scale_page + at * kBlocks);
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          to[k] = *reinterpret_cast<const uint4*>(codes_of + pg * a.k_page + at * (kD / 2) + k * 32);
      };
      // no less than 2^-113: the factors are normal numbers
      int ref = 127 + kCodeBits - 126;
      {
        load_page(0);
        load(0, code, scale, here);
        load_page(1);
      }
      for (int j = 0; j < w.tiles; ++j) {
        const uint32_t n = done + j + 1;
        const int par = (n - 1) & 1;
        uint32_t all = folded(scale) ^ static_cast<uint32_t>(page);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) all ^= code[k].x;
        arrived(all);
        const uint32_t sw[4] = {scale.x, scale.y, scale.z, scale.w};
        int top = 0;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
          const int x = (sw[k / 4] >> (8 * (k % 4))) & 255;
          nan |= x == 255;
          top = max(top, x == 255 ? 0 : x);
        }
        nan = nan && here;
        top = here ? top : 0;
        top = __reduce_max_sync(kFull, top);
        const bool any = __any_sync(kFull, nan);
        if (lane == 0) sh.top[par][warp - kSoftmax] = top | (any ? 256 : 0);
        // every thread comes here, also after a wait that ran out: all leave together
        leave = named_barrier_or(2, 32 * kDequant, !ok);
        if (leave) break;
        load(j + 1, next, next_scale, next_here);
        load_page(j + 2);
        bool nans = false;
#pragma unroll
        for (int i = 0; i < kDequant; ++i) {
          const int x = sh.top[par][i];
          ref = max(ref, x & 255);
          nans |= x >= 256;
        }
        // the words of tile n - 2 are read: its weights went into sums that the first chunk's wait
        // for tile n - 1 has shown to be done
        if (half == 0) sh.nan[par][tok] = nan;
        if (tid == 0) sh.ref[par] = ref, sh.any_nan[par] = nans;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          // the chunk is free when the sums of its dimensions over the tile before are done
          if (k % 2 == 0 && n > 1) ok = ok && wait_warp(sh.sums_done[k / 2], n - 1);
          const uint32_t s8 = (sw[k / 2] >> (16 * (k & 1) + 8 * half)) & 255u;
          uint32_t f = static_cast<uint32_t>(max(static_cast<int>(s8) - ref + 15 + kCodeBits, 0)) * (0x10001u << 10);
          // a NaN is 0 here: its token's weights are NaN where they are seen
          if (!here || s8 == 255u) f = 0u;
          const uint32_t cw[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
          const uint32_t to = base + k * (kTokens * 128) + tok * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t r[4];
            codes_f16(cw[i], r);
            if (ok)
              sts128(to + (((half * 4 + i) ^ (tok & 7)) << 4),
                     make_uint4(mul_f16x2(r[0], f), mul_f16x2(r[1], f), mul_f16x2(r[2], f), mul_f16x2(r[3], f)));
          }
          if (k % 2 == 1) {
            fence_proxy_async_smem();
            arrive_warp(sh.pair_full[k / 2]);
          }
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) code[k] = next[k];
        scale = next_scale;
        here = next_here;
      }
      done += w.tiles;
    }
    if (bad) atomicOr(a.status, kStatusBadInput);
  } else {
    // ================= products: the warp goes along, one lane issues
    bool ok = true;
    uint32_t units = 0;
    const uint32_t id_s = idesc_f16(kRows, false), id_o = idesc_f16(kRows, true, true);
    const uint32_t d0 = __shfl_sync(kFull, tmem, 0);
    const uint32_t k_lo = sw128_lo(base), q_lo = sw128_lo(base + kOffQ), v_lo = sw128_lo(base, kTokens * 128),
                   p_lo = sw128_lo(base + kOffP);
    while (ok && walk_next(a, walk, next)) {
      const Part w = next;
      if (w.tiles == 0) continue;
      ++units;
      ok = wait_warp(sh.q_full, units);
      for (int j = 0; ok && j < w.tiles; ++j) {
        const uint32_t n = done + j + 1;
#pragma unroll 1
        for (int k = 0; ok && k < kChunks; k += 2) {
          ok = wait_warp(sh.pair_full[k / 2], n);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_ss(d0, k_lo + (k + i / 4) * (kTokens * 8) + i % 4 * 2, kSw128Hi,
                     q_lo + (k + i / 4) * (kRows * 8) + i % 4 * 2, kSw128Hi, id_s, k > 0 || i > 0);
            if (k == kChunks - 2) tc_commit(smem_u32(&sh.s_full));
          }
          __syncwarp();
        }
        ok = ok && wait_warp(sh.p_full, n);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kTokens / 16; ++i)
              mma_ss(d0 + kColO + m * kRows, v_lo + 2 * m * (kTokens * 8) + i * 128, kSw128Hi, p_lo + i * 128, kSw128Hi,
                     id_o, j > 0 || i > 0);
            tc_commit(smem_u32(&sh.sums_done[m]));
          }
          __syncwarp();
        }
      }
      done += w.tiles;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) tmem_dealloc(tmem, kCols);
}

}  // namespace

cudaError_t set_attend_latent_attributes() {
  return cudaFuncSetAttribute(attend_latent_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
}

size_t attend_latent_bytes(int sm_count) {
  return cut_bytes(sm_count) + static_cast<size_t>(sm_count) * 2 * kPartFloats<kD, kRows> * sizeof(float);
}

cudaError_t launch_attend_latent(const AttendArgs& a, int sm_count, cudaStream_t stream) {
  const int ctas = attend_ctas(a, kRows, kExtra, sm_count);
  const cudaError_t e = launch_overlapping(attend_latent_kernel, dim3(ctas), kThreads, kBytes, stream, a);
  if (e != cudaSuccess || ctas < 2) return e;
  return launch_join<kD, kRows>(a, ctas, stream);
}

}  // namespace mx
