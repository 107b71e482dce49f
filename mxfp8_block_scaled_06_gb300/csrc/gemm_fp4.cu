// gemm_fp4.cu - products with MXFP4 weights on tcgen05 (sm_103a): the experts'
// grouped product, and the plain product as its one-expert case.
//
// out[r, n] = sum over k of dequant(a)[row(r), k] dequant(w[e(r)])[n, k], fp32
// accumulate, bf16 out; optionally silu(column 2i) * column 2i + 1.
//
// Swap-AB as in gemm.cu: 128 weight rows are the MMA's M, a tile of up to nt
// tokens its N, so a few rows per expert cost a narrow MMA and the weights are read
// once. Persistent CTAs walk the tiles (expert, 128 weight rows, token tile) and the
// ring of operand stages runs on across tiles. Warps:
//   0     weight boxes (TMA) and their scale tiles (bulk copies)
//   1     tcgen05.cp of the scales and tcgen05.mma, by an elected lane
//   2     activation rows, where they are neighbours: a TMA box
//   3     activation scales: gathered with plain loads into 128x4 scale tiles (wide
//         tiles: with a second warp, 2 where that has no rows to load, else the last)
//   4-7   epilogue: TMEM -> bf16, while the next tile accumulates in the other half (wide
//         tiles: with four more warps)
//   8-11  activation rows gathered by index: 16-byte cp.async into the swizzled
//         tile (tile::gather4 copies, four rows each, came at 34 ns apiece: 1.9 us
//         for a stage of 224 rows, against 0.4 us that the MMAs of a stage take)
// A stage holds 128 bytes of K per operand row in the 128-byte swizzle: 128
// elements against MXFP8 activations (.kind::mxf8f6f4 wants E2M1 unpacked to a
// byte each, which the tensor map does on the way: HBM sees 4 bits), 256 elements
// with both operands packed (.kind::mxf4). Either way four MMAs of 32 bytes.
// Every mbarrier wait is bounded; on expiry the kernel records MX_ERR_TIMEOUT,
// stops, waits for its copies and frees its tensor memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256, kGatherThreads = 128;  // the latter on top, where rows are gathered
// warps that load the activation scales: a second one where token
// tiles are wide (one alone held an MXFP4 stage of 224 rows at 0.4 us; 8192 x 8192 x
// 5120 took 130 us, without its loads 96)
__host__ __device__ constexpr int scale_warps(int mode) { return mode == 1 ? 1 : 2; }
constexpr int kScaleBatch = 4;  // scale tiles that such a warp loads at once, and two take in turn
// Stages that the ring needs. A warp that leaves n stages to others (a scale warp the other
// one's batch, a gathering warp every other stage) waits for the stage behind them
// by its parity, which says whether the slot's last use is over only if the use before it is
// known to be: what the warp knows is that the stage a ring before its last own one is over,
// so the ring has to be n + 1 stages long. (With four, scale warps overran each other.)
__host__ __device__ constexpr int min_stages(int mode, bool a_fp4) {
  return scale_warps(mode) == 2 ? kScaleBatch / (a_fp4 ? 2 : 1) + 1 : 3;
}
// Epilogue warps: a second set of four, before that one, where token tiles are wide. With
// few elements along K, or a gate, four could not keep up. Measured with eight / four: 64
// experts of 4096 x 4096, 32744 MXFP4 rows, gated 259 / 324 us; 14 of 5888 x 512, 20818
// rows, gated 82 / 96; 4096 x 4096 x 512 14.4 / 16.4; 8192 x 8192 x 5120 100 / 100.
__host__ __device__ constexpr int epilogue_warps(int mode) { return mode == 1 ? 4 : 8; }
__host__ __device__ constexpr int threads(int mode, bool gather) {
  return kThreads + (epilogue_warps(mode) - 4) * 32 + (gather ? kGatherThreads : (scale_warps(mode) - 1) * 32);
}
constexpr uint32_t kWBytes = 128 * 128;  // weight box in shared memory
// bytes that an unpacking copy of it completes on its barrier: the packed ones
constexpr uint32_t kWBytesUnpacked = 128 * 64;
constexpr uint32_t kSfTile = 512;  // one 128x4 scale tile: 128 rows x 128 elements of K
constexpr int kMaxNt = 224;        // two accumulators of 224 columns leave 64 columns of TMEM for scales
// Token tiles up to kSmallNt run two CTAs to an SM: a stage of narrow MMAs takes its
// one issuing thread about 400 cycles whatever their width, and two CTAs issue side
// by side. Measured with 64 experts of 4096 x 2048, gated, MXFP8 rows, two CTAs / a
// pair of SMs: 48 rows to an expert 55 / 68 us, 72 rows 84 / 70 us (in tiles of 64).
constexpr int kSmallNt = 64;
enum Mode : int {
  kOne = 0,    // a CTA to an SM
  kSmall = 1,  // two CTAs to an SM, token tiles up to kSmallNt
  kPair = 2,   // two SMs share a tile of 256 weight rows: half the activation rows each
               // (8192 x 8192 x 5120, as first built: 155 us, a CTA to an SM 164)
};
__host__ __device__ constexpr int rows_round(int mode) { return mode == kPair ? 32 : 16; }  // MMA N's granule
constexpr int kMaxE = kRouteMaxExperts;
// Activations of more bytes than this go over the weights in bands of as many, so that a
// band stays in L2 however many rows there are. Measured, us without bands / of 64 / 32 / 16
// MB: 32744 x 4096 x 4096 423 / 364 / 348 / 348 (MXFP4 rows 208 / 209 / 191 / 187), 16384 x
// 1280 x 16384 255 / 230 / 225 / 222, 60000 x 1024 x 2048 109 / 101 / 96 / 95.
constexpr long kBandBytes = 16L << 20;
constexpr uint32_t kFull = 0xFFFFFFFFu;

// Shared memory of one CTA, from its 1024-aligned base.
struct Layout {
  uint32_t a_bytes, stage_bytes, sfw_stage, sfa_stage, sfw, sfa, bars, table, end;
  // a_rows: activation rows of a stage (nt, or half of it for a pair)
  __host__ __device__ Layout(int nt, int a_rows, int stages, int tiles_per_chunk, int E) {
    a_bytes = static_cast<uint32_t>(a_rows) * 128u;
    stage_bytes = kWBytes + a_bytes;
    sfw_stage = tiles_per_chunk * kSfTile;
    sfa_stage = tiles_per_chunk * ((nt + 127) / 128) * kSfTile;
    sfw = stages * stage_bytes;
    sfa = sfw + stages * sfw_stage;
    bars = sfa + stages * sfa_stage;
    table = bars + 8u * (2 * stages + 4) + 16u;
    end = table + 8u * (E + 1);
  }
  __host__ __device__ size_t total() const { return 1024 + end; }
};

struct Tile {
  int w_row;  // first weight row, of all experts
  int n0;     // first output column
  int row0, rows;
  int n;  // MMA N: rows rounded up (an expert's token tiles are balanced)
};

// The CTA's table of the experts: tile numbers before each one, first rows.
template <int kMode>
struct Table {
  const int* cum;
  const int* off;
  int E, nt, band;
  __device__ Tile at(int idx, int N, int rank) const {
    constexpr int kRound = rows_round(kMode) - 1;
    int e = 0;
    for (int step = kMaxE; step > 0; step >>= 1)
      if (e + step < E && cum[e + step] <= idx) e += step;
    const int count = off[e + 1] - off[e];
    const int tt = (count + nt - 1) / nt;
    const int local = idx - cum[e];
    // an expert's tiles: all token tiles of a band with one weight tile after the other
    int width = tt, r = local, ti = 0;
    if (tt > band) {
      const int whole = band * (N >> (kMode == kPair ? 8 : 7)), b = local / whole;
      r = local - b * whole;
      ti = b * band;
      width = min(band, tt - ti);
    }
    const int ni = r / width;
    ti += r - ni * width;
    const int per = ((count + tt - 1) / tt + kRound) & ~kRound;
    Tile t;
    t.n0 = kMode == kPair ? ni * 256 + rank * 128 : ni * 128;
    t.w_row = e * N + t.n0;
    t.row0 = off[e] + ti * per;
    t.rows = min(per, count - ti * per);
    t.n = (t.rows + kRound) & ~kRound;
    return t;
  }
};

// g / (1 + exp(-g)) as g h / (1 + h), h = exp(g) (from 30 on the quotient is 1): for g below -87
// exp(-g) would be beyond what __fdividef takes as a divisor (2^126).
__device__ __forceinline__ float silu(float g) {
  const float h = __expf(fminf(g, 30.f));
  return g * __fdividef(h, 1.f + h);
}

template <bool kA4, bool kGather, int kMode>
__global__ void __launch_bounds__(threads(kMode, kGather), kMode == kSmall ? 2 : 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ GemmFp4Args p) {
  constexpr int kTiles = kA4 ? 2 : 1;  // scale tiles (128 elements of K) per stage
  constexpr int kNt = kMode == kSmall ? kSmallNt : kMaxNt;
  constexpr bool kTwo = kMode == kPair;
  constexpr int kScaleWarps = scale_warps(kMode);
  constexpr int kEpilogue = epilogue_warps(kMode);
  constexpr int kEpilogue2 = (kThreads + (kGather ? kGatherThreads : 0)) / 32;  // the first of the second four
  constexpr int kScale2 = kGather ? 2 : kEpilogue2 + kEpilogue - 4;  // the second scale warp
  constexpr int kStageRows = kTwo ? kNt / 2 : kNt;  // activation rows of a stage, at most
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw_addr);
  // the shuffle tells the compiler that the warp's number is uniform: the MMA warp's
  // loop then runs on uniform registers (an MMA and a scale copy every 50 to 70 cycles
  // of its one issuing thread, which bounds the loop; without it 20 % more)
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int stages = p.stages;
  const int rank = kTwo ? static_cast<int>(cluster_rank()) : 0;
  const int first = kTwo ? blockIdx.x >> 1 : blockIdx.x, stride = kTwo ? gridDim.x >> 1 : gridDim.x;
  const Layout L(p.nt, kTwo ? p.nt / 2 : p.nt, stages, kTiles, p.E);
  const int units = p.K >> 7;                        // scale tiles along K
  const int chunks = (units + kTiles - 1) / kTiles;  // stages along K
  // Warps that share a gathered stage: two where K is long, as every thread's arrival takes
  // its time (6144 rows, K = 2048 65 us, with four 70), four where it is short (20818 rows, K
  // = 512 91 us, with two 98) or the tiles narrow.
  const int per = kMode == kSmall || chunks <= 6 ? 4 : 2;
  const uint32_t bars = base + L.bars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (stages + s); };
  const uint32_t acc_full = bars + 16u * stages, acc_empty = acc_full + 16u;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + L.bars + 8 * (2 * stages + 4));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* const cum = reinterpret_cast<int*>(base_ptr + L.table);
  int* const off = cum + p.E + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      // weights, activation scales, activations (gathered: every thread's copies); the
      // first CTA of a pair: the second one's
      mbar_init(full(s), 2 + (kGather ? per * 32 : 1) + (kTwo && rank == 0));
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, (kTwo ? 2 : 1) * kEpilogue);  // the epilogues' warps
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_a);
  }
  if (warp == 0) {
    if constexpr (kTwo)
      tmem_alloc_pair(smem_u32(tmem_slot), p.tmem_cols);
    else
      tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    // only now: a dependent that shares the SM and took tensor memory this CTA still waits for
    // would keep it, waiting in turn for this kernel to end
    pdl_launch_dependents();
  }
  if (warp == 1) {
    if (p.offsets != nullptr) pdl_wait();
    // the experts' rows, clamped to the output, and the tiles before each expert; none at all
    // where the offsets fall (experts would share rows, and the tiles pass 32 bits). The
    // offsets of kAhead times 32 experts are loaded together.
    constexpr int kAhead = 4;
    const int ntiles = kTwo ? p.N >> 8 : p.N >> 7;
    int run = 0, rise = 0;  // the least rise of the offsets, of this lane
    for (int e0 = 0; e0 < p.E; e0 += 32 * kAhead) {
      int from[kAhead], to[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int e = e0 + 32 * j + lane;
        const bool given = p.offsets != nullptr && e < p.E;
        from[j] = given ? p.offsets[e] : 0;
        to[j] = given ? p.offsets[e + 1] : p.R;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (e0 + 32 * j >= p.E) break;
        const int e = e0 + 32 * j + lane;
        const int lo = min(max(from[j], 0), p.R), hi = min(max(to[j], 0), p.R);
        if (e < p.E) rise = min(rise, hi - lo);
        const int own = e < p.E ? (max(hi - lo, 0) + p.nt - 1) / p.nt * ntiles : 0;
        int s = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(kFull, s, o);
          if (lane >= o) s += up;
        }
        if (e < p.E) {
          cum[e] = run + s - own;
          off[e] = lo;
          if (e == p.E - 1) off[p.E] = hi;
        }
        run += __shfl_sync(kFull, s, 31);
      }
    }
    if (__any_sync(kFull, rise < 0)) {
      run = 0;
      if (lane == 0) atomicOr(p.status, kStatusBadInput);
    }
    if (lane == 0) cum[p.E] = run;
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (kTwo)
    cluster_sync();  // the pair's barriers and tensor memory are ready
  else
    __syncthreads();
  tc_fence_after();
  // nothing that an earlier kernel may have written is read, and nothing written,
  // before the wait; with early_weights warp 0 starts on the weights without it
  if (warp != 0 || !p.early_weights) pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const Table<kMode> table{cum, off, p.E, p.nt, p.band};
  const int total = cum[p.E];
  // one wait for the whole warp; false (for all lanes) once it has expired anywhere
  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
    const bool ok = mbar_wait_or(bar, parity, abort_flag);
    if (__all_sync(kFull, ok)) return true;
    if (lane == 0) {
      atomicOr(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    return false;
  };

  if (warp == 0) {
    // ---------------- weights and their scales
    const uint64_t pol = policy_evict_normal();
    int s = 0, issuer = 0;
    uint32_t ph = 1;
    bool ok = true, early = !kGather && p.early_weights;  // gathered rows come with offsets
    for (int idx = first; ok && idx < total; idx += stride) {
      const Tile t = table.at(idx, p.N, rank);
      const uint8_t* const sf = p.w_scales + static_cast<size_t>(t.w_row >> 7) * units * kSfTile;
      for (int i = 0; i < chunks; ++i) {
        if (!(ok = warp_wait(empty(s), ph))) break;
        if (lane == issuer) {
          const uint32_t sf_bytes = min(kTiles, units - i * kTiles) * kSfTile;
          mbar_expect_tx(full(s), (kA4 ? kWBytes : kWBytesUnpacked) + sf_bytes);
          tma_load_2d(base + s * L.stage_bytes, &tm_w, full(s), i * 128, t.w_row, pol);
          bulk_load(base + L.sfw + s * L.sfw_stage, sf + static_cast<size_t>(i) * kTiles * kSfTile, sf_bytes, full(s),
                    pol);
        }
        __syncwarp();
        issuer = (issuer + 1) & 31;
        if (++s == stages) {
          s = 0, ph ^= 1u;
          // from here on the waits' limit counts: not while the previous kernel may still run
          if (early) pdl_wait();
          early = false;
        }
      }
    }
  } else if (!kGather && warp == 2) {
    // ---------------- activation rows from row0 on: rows past the tile belong to
    // other tiles and end in columns that are not stored; past the tensor: zeros
    const uint64_t pol = policy_evict_last();
    int s = 0, issuer = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int idx = first; ok && idx < total; idx += stride) {
      const Tile t = table.at(idx, p.N, rank);
      for (int i = 0; i < chunks; ++i) {
        if (!(ok = warp_wait(empty(s), ph))) break;
        if (lane == issuer) {
          mbar_expect_tx(full(s), L.a_bytes);
          tma_load_2d(base + s * L.stage_bytes + kWBytes, &tm_a, full(s), i * 128, t.row0 + rank * (t.n >> 1), pol);
        }
        __syncwarp();
        issuer = (issuer + 1) & 31;
        if (++s == stages) s = 0, ph ^= 1u;
      }
    }
  } else if (kGather && warp >= kThreads / 32 && warp < (kThreads + kGatherThreads) / 32) {
    // ---------------- gathered activation rows: eight threads a row, 16 bytes each.
    // `per` warps share a stage, the groups of them take the stages in turn. A stage's
    // copies report to its barrier as they land, and the MMA warp fences them, so these
    // warps wait for free stages only. Measured with the warps waiting for their copies
    // and fencing them (a stage a warp, handed over after the next one's issue) / with
    // this, us: 14 experts of 5888 rows, 20818 MXFP8 rows, K = 512 122 / 91, K = 2048 190 /
    // 175; 64 of 4096 x 2048, 6144 rows 73 / 65; 16 of 1920 x 1024, 8000 rows 122 / 26; 64
    // of 4096 x 4096, 32744 rows 415 / 395 (MXFP4 rows 264 / 250; rows that need no
    // gathering 350 and 206).
    auto gather = [&](auto per_c) {
      constexpr int kPer = decltype(per_c)::value, groups = 4 / kPer, apart = 4 * kPer;
      constexpr int kRows = kStageRows / apart;  // rows per thread, so far apart
      const int gw = warp - kThreads / 32;
      const int c = lane & 7, r0 = (gw & (kPer - 1)) * 4 + (lane >> 3);
      const uint32_t row_bytes = kA4 ? p.K >> 1 : p.K;
      // apart is 8 or 16: one swizzle for all of a thread's rows
      const uint32_t dst0 = base + kWBytes + r0 * 128 + ((c ^ (r0 & 7)) << 4);
      int s = gw / kPer;  // stages: at least as many as groups (the plan)
      uint32_t ph = 1;
      // the next stage's tile and place along K, and the same of the group's next tile
      int idx = first, chunk = s;
      auto find = [&](int& tile, int& place) {
        while (place >= chunks && tile < total) place -= chunks, tile += stride;
      };
      // row numbers are read a tile ahead; rows past the tile and tokens outside read as zero
      int row[kRows], ahead[kRows], mine = 0, mine_ahead = 0;
      auto fetch_rows = [&](int tile) {
        const Tile t = table.at(tile, p.N, rank);
        mine_ahead = kTwo ? t.n >> 1 : t.n;  // rows of the tile in this CTA
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int r = r0 + apart * j, i = r + rank * mine_ahead;
          ahead[j] = r < mine_ahead && i < t.rows ? p.tokens[t.row0 + i] : -1;
        }
      };
      find(idx, chunk);
      if (idx < total) fetch_rows(idx);
      bool ok = true;
      while (ok && idx < total) {
        mine = mine_ahead;
#pragma unroll
        for (int j = 0; j < kRows; ++j) row[j] = ahead[j];
        int next = idx, next_chunk = chunk + (chunks - chunk + groups - 1) / groups * groups;
        find(next, next_chunk);
        bool fetch = next < total;
        for (; chunk < chunks; chunk += groups) {
          if (!(ok = warp_wait(empty(s), ph))) break;
          const uint32_t dst = dst0 + s * L.stage_bytes;
          const uint32_t at = static_cast<uint32_t>(chunk) * 128u + c * 16u;
          const bool in_row = at < row_bytes;
          const uint8_t* const col = p.a + (in_row ? at : 0u);
#pragma unroll
          for (int j = 0; j < kRows; ++j) {
            const bool real = static_cast<uint32_t>(row[j]) < static_cast<uint32_t>(p.a_rows);
            if (apart * j < mine)
              cp_async_16(dst + apart * j * 128, col + static_cast<size_t>(real ? row[j] : 0) * row_bytes,
                          real && in_row ? 16u : 0u);
          }
          cp_async_arrive(full(s));
          s += groups;
          while (s >= stages) s -= stages, ph ^= 1u;
          if (fetch) fetch_rows(next);
          fetch = false;
        }
        idx = next;
        chunk = next_chunk;
      }
    };
    if (kMode == kSmall || per == 4)
      gather(std::integral_constant<int, 4>{});
    else
      gather(std::integral_constant<int, kMode == kSmall ? 4 : 2>{});
    cp_async_wait_all();
  } else if (warp == 3 || (kScaleWarps == 2 && warp == kScale2)) {
    // ---------------- activation scales: lane l serves rows l, l + 32, ... of the
    // tile, whose words (4 scale bytes) are one 16-byte store per 128 rows. A batch of
    // kBatch scale tiles is loaded at once, the next one while it is stored; with two
    // warps they take the batches in turn.
    constexpr int kRows = (kNt + 31) / 32, kBatch = kScaleBatch;  // rows per lane
    constexpr int kBatchStages = kBatch / kTiles;
    const int which = warp == 3 ? 0 : 1;
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    auto advance = [&](int n) {
      s += n;
      while (s >= stages) s -= stages, ph ^= 1u;
    };
    const int sfa_tiles = (p.nt + 127) >> 7;
    // plain scales of four tiles are 16 bytes of a row: one load, where rows start at
    // multiples of 16
    const bool vec = !p.a_swizzled && (units & 3) == 0;
    const int step = p.a_swizzled ? kSfTile : 4;
    int batch = 0;  // over all tiles
    for (int idx = first; ok && idx < total; idx += stride) {
      const Tile t = table.at(idx, p.N, rank);
      const uint8_t* src[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int i = lane + 32 * j;
        src[j] = nullptr;
        if (i < t.rows) {
          const int r = kGather ? p.tokens[t.row0 + i] : t.row0 + i;
          if (r < 0 || r >= p.a_rows) {
            atomicOr(p.status, kStatusBadInput);  // reads as zero
          } else if (p.a_swizzled) {
            src[j] = p.a_scales + static_cast<size_t>(r >> 7) * units * kSfTile + (r & 31) * 16 + ((r >> 5) & 3) * 4;
          } else {
            src[j] = p.a_scales + static_cast<size_t>(r) * units * 4;
          }
        }
      }
      uint32_t v[kBatch][kRows], next[kBatch][kRows];
      auto load = [&](int u0, uint32_t (&w)[kBatch][kRows]) {
        if (vec) {
#pragma unroll
          for (int j = 0; j < kRows; ++j) {
            const uint4 q = src[j] != nullptr && u0 < units ? ld_global(reinterpret_cast<const uint4*>(src[j] + u0 * 4))
                                                            : make_uint4(0, 0, 0, 0);
            w[0][j] = q.x;
            w[1][j] = q.y;
            w[2][j] = q.z;
            w[3][j] = q.w;
          }
          return;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
          for (int j = 0; j < kRows; ++j)
            w[b][j] = src[j] != nullptr && u0 + b < units
                          ? ld_global(reinterpret_cast<const uint32_t*>(src[j] + static_cast<size_t>(u0 + b) * step))
                          : 0u;
      };
      int u0 = 0;
      if (kScaleWarps == 2 && (batch & 1) != which) {  // this tile's first batch is the other warp's
        u0 = kBatch;
        advance(min(kBatchStages, chunks));
      }
      if (u0 < units) load(u0, next);
      for (; ok && u0 < units; u0 += kBatch * kScaleWarps) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
          for (int j = 0; j < kRows; ++j) v[b][j] = next[b][j];
        load(u0 + kBatch * kScaleWarps, next);
#pragma unroll
        for (int c = 0; c < kBatchStages; ++c) {
          if (u0 + c * kTiles >= units) break;
          if (!(ok = warp_wait(empty(s), ph))) break;
          uint8_t* const dst = base_ptr + L.sfa + s * L.sfa_stage + lane * 16;
#pragma unroll
          for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int rt = 0; rt < (kNt + 127) / 128; ++rt) {
              const int b = c * kTiles + h;
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = 4 * rt + j < kRows ? v[b][min(4 * rt + j, kRows - 1)] : 0u;
              if (rt * 128 < t.n)
                *reinterpret_cast<uint4*>(dst + (h * sfa_tiles + rt) * kSfTile) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full(s));
          advance(1);
        }
        // the other warp's batch
        if (kScaleWarps == 2) advance(max(0, min(kBatchStages, chunks - (u0 + kBatch) / kTiles)));
      }
      batch += (units + kBatch - 1) / kBatch;
    }
  } else if (kTwo && warp == 1 && rank != 0) {
    // ---------------- the second CTA of a pair: its stages' arrivals, passed on to
    // the first one, which issues the pair's MMAs. A stage's bytes lie in this SM's own
    // shared memory, complete (its barrier) and visible to the async proxy (the writers'
    // fences, or the one below) before the arrival, and it is this SM that reads them for the
    // pair's MMA; the arrival itself releases at CTA scope (ptx.cuh). Measured at cluster scope,
    // us: a release a stage 8192 x 8192 x 5120 with MXFP4 rows 275 (now 104), one for all stages
    // that have landed 148, gathered experts of 4093 tokens, MXFP8 rows, 520 (355); no
    // pairs at all 123 and 470.
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int idx = first; ok && idx < total; idx += stride) {
      for (int i = 0; i < chunks; ++i) {
        if (!(ok = warp_wait(full(s), ph))) break;
        if (kGather) fence_proxy_async_smem();
        if (lane == 0) mbar_arrive_remote(map_shared_rank(full(s), 0));
        __syncwarp();
        if (++s == stages) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ---------------- scales into TMEM, and the MMAs
    const uint64_t wd = sdesc_k_sw128(base), fd = sdesc_sf(base + L.sfw), gd = sdesc_sf(base + L.sfa);
    const uint32_t op_hi = static_cast<uint32_t>(wd >> 32), sf_hi = static_cast<uint32_t>(fd >> 32);
    const uint32_t w_lo0 = static_cast<uint32_t>(wd), f_lo0 = static_cast<uint32_t>(fd);
    const uint32_t g_lo0 = static_cast<uint32_t>(gd);
    const int sfa_tiles = (p.nt + 127) >> 7;
    // tcgen05.cp and tcgen05.mma of one thread run in order, so two sets of scale
    // columns are enough
    const uint32_t sf_col = tmem + 2 * p.nt, sf_cols = 4 * kTiles * (1 + sfa_tiles);
    constexpr uint32_t kSf = (1u << 4) | (1u << 29);  // the next scale byte, in both fields of the descriptor
    auto copy_scales = [&](uint32_t taddr, uint32_t lo) {
      if constexpr (kTwo)
        tmem_cp_32x128b_x4_pair_lh(taddr, lo, sf_hi);
      else
        tmem_cp_32x128b_x4_lh(taddr, lo, sf_hi);
    };
    auto commit = [&](uint32_t bar) {
      if constexpr (kTwo)
        tc_commit_pair(bar);
      else
        tc_commit(bar);
    };
    int s = 0, it = 0;
    uint32_t ph = 0;
    uint32_t w_lo = w_lo0, f_lo = f_lo0, g_lo = g_lo0, ta = sf_col;
    bool ok = true, landed = false;
    // one stage: its scales, its MMAs (kHave scale tiles of K, the second one's two
    // MMAs left out where K ends inside the stage) and the commits
    auto issue = [&](auto have_c, const uint32_t d, const uint32_t id0, const bool wide, const bool begins,
                     const bool ends, const int buf) {
      constexpr int kHave = decltype(have_c)::value;
      const uint32_t tb = ta + 4 * kTiles;
#pragma unroll
      for (int h = 0; h < kHave; ++h) {
        copy_scales(ta + 4 * h, f_lo + h * (kSfTile >> 4));
        copy_scales(tb + 4 * h * sfa_tiles, g_lo + h * sfa_tiles * (kSfTile >> 4));
        if (wide) copy_scales(tb + 4 * (h * sfa_tiles + 1), g_lo + (h * sfa_tiles + 1) * (kSfTile >> 4));
      }
      const uint32_t a_lo = w_lo + (kWBytes >> 4);
#pragma unroll
      for (int j = 0; j < (kA4 ? 2 * kHave : 4); ++j) {
        // .mxf8f6f4: scale byte j of the stage's one tile; .mxf4: bytes 2 (j % 2) and the next of tile j / 2
        const int h = kA4 ? j >> 1 : 0;
        const uint32_t id = id0 + (kA4 ? 2 * (j & 1) : j) * kSf, sfw = ta + 4 * h, sfa = tb + 4 * h * sfa_tiles;
        if constexpr (kTwo)
          mma_w4_pair_lh<kA4>(d, w_lo + 2 * j, op_hi, a_lo + 2 * j, op_hi, id, sfw, sfa, j != 0 || !begins);
        else
          mma_w4_lh<kA4>(d, w_lo + 2 * j, op_hi, a_lo + 2 * j, op_hi, id, sfw, sfa, j != 0 || !begins);
      }
      commit(empty(s));
      if (ends) commit(acc_full + 8 * buf);
    };
    for (int idx = first; ok && idx < total; idx += stride, ++it) {
      const Tile t = table.at(idx, p.N, rank);
      const int buf = it & 1;
      if (!(ok = warp_wait(acc_empty + 8 * buf, ((it >> 1) & 1) ^ 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * p.nt;
      const uint32_t id0 = idesc_w4<kA4>(t.n, 0, kTwo ? 256 : 128);
      const bool wide = t.n > 128;
      for (int i = 0; i < chunks; ++i) {
        if (!__all_sync(kFull, landed) && !(ok = warp_wait(full(s), ph))) break;
        if (kGather) fence_proxy_async_smem();  // the gathered rows came by the generic proxy
        tc_fence_after();
        if (elect_one()) {
          const bool ends = i == chunks - 1;
          if (kTiles == 1 || (units & 1) == 0 || !ends)
            issue(std::integral_constant<int, kTiles>{}, d, id0, wide, i == 0, ends, buf);
          else
            issue(std::integral_constant<int, 1>{}, d, id0, wide, i == 0, ends, buf);
        }
        __syncwarp();
        ta = ta == sf_col ? sf_col + sf_cols : sf_col;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
          w_lo = w_lo0;
          f_lo = f_lo0;
          g_lo = g_lo0;
        } else {
          w_lo += L.stage_bytes >> 4;
          f_lo += L.sfw_stage >> 4;
          g_lo += L.sfa_stage >> 4;
        }
        landed = mbar_test_wait(full(s), ph);  // the next stage, while the MMAs run
      }
    }
  } else if ((warp >= 4 && warp < 8) || (kEpilogue == 8 && warp >= kEpilogue2 && warp < kEpilogue2 + 4)) {
    // ---------------- epilogue: lane l of quarter q holds output column n0 + 32q + l
    const int q = warp & 3;
    const bool odd = lane & 1;
    int it = 0;
    bool ok = true;
    const size_t ldo = p.gated ? p.N >> 1 : p.N;
    for (int idx = first; ok && idx < total; idx += stride, ++it) {
      const Tile t = table.at(idx, p.N, rank);
      const int buf = it & 1;
      if (!(ok = warp_wait(acc_full + 8 * buf, (it >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * p.nt;
      // Plain: two neighbouring lanes trade two tokens, so that a lane stores two columns of
      // one; in narrow tiles four lanes four tokens. Measured, us, a column a lane / two /
      // four: 20818 rows of 14 experts, N = 5888, K = 512 96 / 92 / 97; 32744 of 64, N = 4096,
      // K = 1408 132 / 132 / 137; 7182 x 8192 x 768 51.5 / 50.6 / 52.3; narrow: 128 x 8192 x
      // 512 7.3 / 7.1 / 6.5, 8 x 8192 x 1536 5.1 / 5.0 / 4.6.
      // Gated: four neighbouring lanes trade the four tokens c0 + 4i .. + 3, first in
      // pairs, the even lane taking gate and up of tokens 0 and 2, the odd one of 1
      // and 3; then, the products in bf16, between the pairs, the first one taking
      // tokens 0 and 1. A lane stores two columns of one token.
      const int tok0 = p.gated || kMode == kSmall ? (lane & 2) + odd : odd;
      const int col = t.n0 + q * 32 + (p.gated || kMode == kSmall ? lane & ~3 : lane & ~1);
      __nv_bfloat16* out = p.out + (static_cast<size_t>(t.row0) + tok0) * ldo + (p.gated ? col >> 1 : col);
      constexpr int kStep = 16 * kEpilogue / 4;  // of eight warps, four take every other 16 tokens
      const int c_first = kEpilogue == 8 && warp >= 8 ? 16 : 0;
      out += c_first * ldo;
      for (int c0 = c_first; c0 < t.n; c0 += kStep) {
        float v[16];
        tmem_ld_32x32b_x16(acc + c0, v);
        if (!p.gated) {
          const bool all = c0 + 16 <= t.rows;
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            const uint32_t own = *reinterpret_cast<const uint32_t*>(&two);
            const uint32_t got = __shfl_xor_sync(kFull, own, 1);
            w[i] = odd ? __byte_perm(got, own, 0x7632) : __byte_perm(own, got, 0x5410);
          }
          if constexpr (kMode == kSmall) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t got = __shfl_xor_sync(kFull, lane & 2 ? w[2 * i] : w[2 * i + 1], 2);
              if (all || c0 + 4 * i + tok0 < t.rows)
                *reinterpret_cast<uint2*>(out + 4 * i * ldo) =
                    lane & 2 ? make_uint2(got, w[2 * i + 1]) : make_uint2(w[2 * i], got);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (all || c0 + 2 * i + tok0 < t.rows) *reinterpret_cast<uint32_t*>(out + 2 * i * ldo) = w[i];
          }
          out += kStep * ldo;
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float two[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float even = v[4 * i + 2 * j], other = v[4 * i + 2 * j + 1];
            const float got = __shfl_xor_sync(kFull, odd ? even : other, 1);
            two[j] = silu(odd ? got : even) * (odd ? other : got);
          }
          const float got = __shfl_xor_sync(kFull, lane & 2 ? two[0] : two[1], 2);
          if (c0 + 4 * i + tok0 < t.rows)
            *reinterpret_cast<__nv_bfloat162*>(out) =
                __floats2bfloat162_rn(lane & 2 ? got : two[0], lane & 2 ? two[1] : got);
          out += 4 * ldo;
        }
        out += (kStep - 16) * ldo;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kTwo)
          mbar_arrive_remote(map_shared_rank(acc_empty + 8 * buf, 0));
        else
          mbar_arrive(acc_empty + 8 * buf);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0 && threadIdx.x == 0) {
    // copies still in flight land within this time, whether or not their stage's
    // barrier completes (its other arrivals may be missing)
    for (int s = 0; s < stages; ++s) {
      mbar_wait(full(s), 0, 2000000);
      mbar_wait(full(s), 1, 2000000);
    }
  }
  __syncwarp();
  if constexpr (kTwo)
    cluster_sync();  // no CTA frees its tensor memory, or leaves, while its peer may still use the pair's
  else
    __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    if constexpr (kTwo)
      tmem_dealloc_pair(tmem, p.tmem_cols);
    else
      tmem_dealloc(tmem, p.tmem_cols);
  }
  __syncwarp();
  if constexpr (kTwo) cluster_sync();
}

}  // namespace

GemmFp4Plan plan_gemm_fp4(int E, int R, int N, int K, bool a_fp4, int sm_count) {
  GemmFp4Plan pl{};
  const int kt = a_fp4 ? 2 : 1;
  // Token tile. A plain product takes its rows in as few tiles of at most kMaxNt as
  // they take, balanced, or more and narrower ones where that saves time in its last
  // wave: a tile costs about its rows and 100 more. Several experts: a third more
  // than the mean (an expert with more rows takes several balanced tiles). With 64
  // experts of 4096 x 2048, gated, us with twice the mean / with this: 512 tokens to 6
  // each 68 / 55 (MXFP4 rows 60 / 50), 1024 76 / 73 (74 / 61).
  // One CTA to an SM, MXFP8 rows: 208 rows at most, which leave room for five stages (min_stages).
  const int most_nt = N % 256 == 0 || a_fp4 ? kMaxNt : 208;
  const long want = E == 1 ? R : std::min<long>({R, 4L * ((R + E - 1) / E) / 3, most_nt});
  long tt = (want + most_nt - 1) / most_nt;
  if (E == 1 && want > most_nt / 2) {
    const int at_once = N % 256 == 0 ? sm_count / 2 : sm_count;
    const long w_tiles = N % 256 == 0 ? N / 256 : N / 128;
    auto cost = [&](long k) { return (w_tiles * k + at_once - 1) / at_once * ((want + k - 1) / k + 100); };
    const long most = 3 * tt;
    for (long k = tt + 1; k <= most && (want + k - 1) / k > kSmallNt; ++k)
      if (cost(k) < cost(tt)) tt = k;
  }
  const int nt = static_cast<int>((want + tt - 1) / tt);
  pl.mode = nt <= kSmallNt ? kSmall : N % 256 == 0 ? kPair : kOne;
  pl.nt = std::min(most_nt, (nt + rows_round(pl.mode) - 1) & -rows_round(pl.mode));
  pl.a_rows = pl.mode == kPair ? pl.nt / 2 : pl.nt;
  pl.ctas_per_sm = pl.mode == kSmall ? 2 : 1;
  pl.min_stages = min_stages(pl.mode, a_fp4);
  const int cols = 2 * pl.nt + 2 * 4 * kt * (1 + (pl.nt + 127) / 128);
  pl.tmem_cols = 32;
  while (pl.tmem_cols < cols) pl.tmem_cols <<= 1;
  const size_t fixed = Layout(pl.nt, pl.a_rows, 0, kt, E).total();
  const size_t per = Layout(pl.nt, pl.a_rows, 1, kt, E).total() - fixed;
  const size_t room = pl.ctas_per_sm == 1 ? kMaxDynamicSmem : 233472 / 2 - 1024;  // 1 KB of each CTA's is reserved
  pl.stages = static_cast<int>(std::min<size_t>((room - fixed) / per, 12));
  // CTAs that share an SM share its tensor memory: take the shared memory that
  // keeps any more than fit from being resident
  pl.smem = std::max(Layout(pl.nt, pl.a_rows, pl.stages, kt, E).total(),
                     static_cast<size_t>(233472 / (pl.ctas_per_sm + 1) + 1));
  pl.band = static_cast<int>(std::clamp(kBandBytes / (static_cast<long>(pl.nt) * (a_fp4 ? K / 2 : K)), 1L, 1L << 24));
  const int ctas = pl.mode == kPair ? 2 : 1;  // of a tile
  const long tiles = static_cast<long>(N / (128 * ctas)) * std::min<long>((R + pl.nt - 1L) / pl.nt + E - 1, R);
  pl.grid = static_cast<int>(std::min<long>(tiles, static_cast<long>(sm_count) * pl.ctas_per_sm / ctas)) * ctas;
  return pl;
}

cudaError_t set_gemm_fp4_attributes() {
  const void* const kernels[] = {
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, false, kOne>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, true, kOne>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, false, kOne>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, true, kOne>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, false, kSmall>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, true, kSmall>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, false, kSmall>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, true, kSmall>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, false, kPair>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<false, true, kPair>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, false, kPair>),
      reinterpret_cast<const void*>(&gemm_fp4_kernel<true, true, kPair>)};
  for (const void* k : kernels) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxDynamicSmem));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_gemm_fp4(const CUtensorMap& tm_w, const CUtensorMap& tm_a, const GemmFp4Args& args,
                            const GemmFp4Plan& plan, bool a_fp4, cudaStream_t stream) {
  const bool gather = args.tokens != nullptr;
  if (plan.smem > kMaxDynamicSmem || plan.stages < plan.min_stages) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.grid);
    cfg.blockDim = dim3(threads(plan.mode, gather));
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = plan.mode == kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_a, args);
  };
  auto pick = [&](auto mode) {
    constexpr int S = decltype(mode)::value;
    if (a_fp4) return gather ? go(gemm_fp4_kernel<true, true, S>) : go(gemm_fp4_kernel<true, false, S>);
    return gather ? go(gemm_fp4_kernel<false, true, S>) : go(gemm_fp4_kernel<false, false, S>);
  };
  if (plan.mode == kPair) return pick(std::integral_constant<int, kPair>{});
  if (plan.mode == kSmall) return pick(std::integral_constant<int, kSmall>{});
  return pick(std::integral_constant<int, kOne>{});
}

}  // namespace mx
