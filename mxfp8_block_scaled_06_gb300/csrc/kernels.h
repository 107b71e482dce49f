// kernels.h - host-side launchers of the CUDA kernels (internal to libmx).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace mx {

// Largest dynamic shared memory one CTA may ask for on sm_103a.
constexpr size_t kMaxDynamicSmem = 232448;

// ------------------------------------------------------------ quantizer
// Inverse RoPE applied before quantizing (WO-A activation): rows are tokens of
// heads of head_dim, dims from d_nope on rotated by -pos * f; cos_sin null = none.
struct RopeArgs {
  const int64_t* positions;
  const float* cos_sin;  // [max_pos, 64]: 32 cos | 32 sin
  int max_pos, head_dim, d_nope;
  int* status;
};
cudaError_t launch_quantize_rows(const void* x, long ldx, int M, int K, void* q, void* scales,
                                 int swizzled, cudaStream_t stream,
                                 const RopeArgs& rope = RopeArgs{nullptr, nullptr, 0, 0, 0, nullptr});

// y = bf16(x / sqrt(mean(x^2) + eps) * gamma) per row (float32 arithmetic), then
// MX-quantized into q / scales; y may be null.
cudaError_t launch_rmsnorm_quantize_rows(const void* x, long ldx, int M, int K, const void* gamma,
                                         float eps, void* y, void* q, void* scales, int swizzled,
                                         cudaStream_t stream);

// One thread waits on an mbarrier nothing completes; after the bounded wait's
// limit it sets the timeout bit of *status and returns.
cudaError_t launch_wait_selftest(int* status, cudaStream_t stream);

// ------------------------------------------------------------ block-scaled GEMM
// Plan of one GEMM launch: activation tile (MMA N), K-splits per weight tile
// (a thread-block cluster along K), pipeline depth, TMEM columns, shared bytes.
// Plan overrides for tuning, read from the environment once per handle (at
// mx_create): MX_SPLITS (K-splits of every GEMM, 1..8), MX_STAGES (ring depth),
// MX_PLAN_AT ("NxK:splits[:stages],..." for listed weight shapes),
// MX_WOA_SPLITS (fused WO-A K-splits). Zero / empty = none.
struct PlanEnv {
  int splits;
  int stages;
  int woa_splits;
  int push_rows;  // the push reduction up to this many rows (0: the default)
  char plan_at[256];
  // clusters of 2..8 CTAs, one CTA to an SM, that the device holds at once (0: not known)
  int clusters[9];
};
PlanEnv read_plan_env();

// How the K-splits' fp32 partials are summed (every form in rank order):
// items = a warp sums 32-column items from the peers' shared memory; rows = a
// warp sums whole rows with 16-byte peer loads; push = every CTA stores the
// partials of the units another rank owns straight into that rank's shared
// memory (st.async, counted on its mbarrier) and sums its own units locally,
// with a receive slot per rank, or (compact) per peer; bulk (MXFP4 weights) = every
// CTA copies the rows that another rank owns, as one block, into that rank's shared memory.
enum Reduction : int { kReduceItems = 0, kReduceRows = 1, kReducePush = 2, kReducePushCompact = 3, kReduceBulk = 4 };
// Whether a plan may take the push reduction, and with which receive area.
enum PushMode : int { kPushNone = 0, kPushCompact = 1, kPushFull = 2 };

// 128-row tiles of block scales behind `rows` rows.
__host__ __device__ constexpr int scale_row_tiles(int rows) { return (rows + 127) / 128; }

struct GemmPlan {
  int mtile;
  int splits;
  int stages;
  int tmem_cols;
  int reduction;  // Reduction
  int slice, slices;  // rows of a cluster, and how many take all (MXFP4 weights: slices of 128 or 256)
  size_t smem;
};

// RMS norm of the bf16 activation rows before their quantization (in-kernel
// quantization only; gamma null = none): y = bf16(x * 1/sqrt(mean(x^2) + eps) *
// gamma), the mean over the row's K values. The sum of squares is read, not
// computed: ssq [M, K/32] holds each 32-block's sum of its squares (written by
// the previous GEMM's epilogue, ssq_out), added here in block order. Tile 0's
// CTAs also write, over their K-range, the normalized rows to y [M, K] and the
// MXFP8 activation to a_q [M, K] and its swizzled scales a_q_scales (each null =
// not written).
struct GemmNorm {
  const uint16_t* gamma;
  float eps;
  const float* ssq;
  uint16_t* y;
  uint8_t* a_q;
  uint8_t* a_q_scales;
};

struct GemmArgs {
  int M, N, K;
  int w_fmt;  // 0: MXFP8 weights, 1: MXFP4 weights and MXFP8 activations, 2: both MXFP4
  int mtile, stages, nchunks, tmem_cols;
  int slice;  // rows of a cluster (MXFP4 weights)
  const uint8_t* a_scales;  // MXFP8 activations' swizzled scales (unused when x is set)
  const uint8_t* w_scales;
  // bf16 activations [M, K] (row stride ldx elements) quantized inside the
  // kernel instead of MXFP8 activations through tm_a / a_scales; null = MXFP8 in
  const uint16_t* x;
  long ldx;
  GemmNorm norm;
  // Grouped activations (0 = not grouped): weight tile t belongs to group
  // g = t / group_tiles and contracts the group's K-slice [g K, (g + 1) K) of
  // a wider MXFP8 activation whose scale layout has a_sf_chunks 128-wide
  // column blocks per row tile (= K / 128 when not grouped).
  int group_tiles;
  int a_sf_chunks;
  void* out;          // bf16 [M, N] or null
  uint8_t* q;         // fused requantization of columns [0, q_cols): E4M3 [M, q_cols]
  uint8_t* q_scales;  // swizzled scales of q
  int q_cols;
  // per-32-block sums of squares of the bf16 output, columns [0, ssq_cols):
  // ssq_out[m * ssq_cols / 32 + c / 32], each the xor-shuffle tree over the
  // block's 32 values (null = not written)
  float* ssq_out;
  int ssq_cols;
  int* status;
#ifdef MX_TIMELINE
  unsigned long long* tl;  // kTimelineSlots %globaltimer stamps per CTA, or null
#endif
};

#ifdef MX_TIMELINE
// Timeline build only: stamps per CTA of one GEMM launch (see gemm.cu).
constexpr int kTimelineSlots = 20;
constexpr int kTimelineCtas = 512;
#endif

// fused_a: bf16 activations quantized in the kernel; norm: with the RMS norm;
// push_mode: whether the push reduction may be chosen, and its receive area;
// table_depth: the ring depth of the split table's row (false: as planned);
// w_fmt as in GemmArgs (MXFP4 weights: neither fused_a nor a compact push area).
GemmPlan plan_gemm(int M, int N, int K, int sm_count, const PlanEnv& env, bool fused_a = false,
                   bool norm = false, int push_mode = kPushFull, bool table_depth = true, int w_fmt = 0);
cudaError_t set_gemm_attributes();
// how many clusters of `size` CTAs of the GEMM, one CTA to an SM, the device holds at once
int gemm_max_clusters(int size);
cudaError_t launch_gemm(const CUtensorMap& tm_w, const CUtensorMap& tm_a, const GemmArgs& args,
                        const GemmPlan& plan, bool pdl, cudaStream_t stream);

// ------------------------------------------------------------ persistent chain
// The three projections of mx_gemm_chain in one persistent kernel (chain.cu):
// clusters of kChainCluster CTAs, one CTA per SM, every CTA resident at once.
constexpr int kChainCluster = 8;
constexpr int kChainMaxUnits = 8;      // (tile, K split) work units per CTA, all projections
constexpr int kChainCounters = 16384;  // 32-bit words of the handle's chain workspace

// One projection as the chain kernel sees it.
struct ChainProj {
  const uint8_t* w_scales;  // swizzled [n, k/32]
  const uint8_t* a_scales;  // swizzled scales of the activation [M, k]
  int n, k;
  int splits;               // CTAs (ranks of one cluster) sharing a weight tile's K-range
  void* out;                // bf16 [M, n], or null
  uint8_t* q;               // MX requantization of columns [0, q_cols): the next activation
  uint8_t* q_scales;
  int q_cols;
};

// Shared-memory and TMEM plan of the chain kernel (offsets from the CTA's
// 1024-aligned base); ok == false: the three-launch path serves the call.
struct ChainPlan {
  bool ok;
  int clusters, ring, tmem_cols;
  int act_chunks[3], max_units[3];
  uint32_t off_act[3], off_asf[3], off_staged, off_recv[3], recv_unit_bytes[3], off_bars;
  size_t smem;
};

struct ChainArgs {
  int M, mtile, nsfb;
  ChainProj proj[3];
  ChainPlan plan;
  // workspace: [0] calls completed, [1] CTAs finished in this call, [2] abort,
  // then one counter per weight tile of the first two projections (from
  // cnt_off), zero at the start of every call
  unsigned* counters;
  int cnt_off[2];
  int* status;
#ifdef MX_TIMELINE
  unsigned long long* tl;  // kTimelineSlots %globaltimer stamps per CTA, or null
#endif
};

ChainPlan plan_chain(int M, const ChainProj (&proj)[3], int clusters);
// Clusters of kChainCluster CTAs of the chain kernel that can be resident at once.
int chain_max_clusters();
cudaError_t set_chain_attributes();
cudaError_t launch_chain(const CUtensorMap (&maps)[6], const ChainArgs& args, cudaStream_t stream);

// ------------------------------------------------------------ grouped WO-A
struct WoaPlan {
  int mtile;
  int splits;
  int stages;
  int tmem_cols;
  bool push;  // the push split-K reduction (full receive area)
  size_t smem;
};

struct WoaArgs {
  int T, G, H, R, D;  // tokens, groups, heads per group, o_lora_rank, head dim (512)
  int mtile, stages, tmem_cols;
  const uint16_t* x;  // bf16 bits
  long ldx;
  const int64_t* positions;
  const float* cos_sin;
  int max_pos;
  const uint8_t* w_scales;
  uint8_t* q;
  uint8_t* q_scales;
  uint16_t* debug_z;
  uint8_t* debug_xq;
  uint8_t* debug_xs;
  int early_trigger;
  int* status;
#ifdef MX_TIMELINE
  unsigned long long* tl;  // kTimelineSlots %globaltimer stamps per CTA, or null
#endif
};

WoaPlan plan_wo_a(int T, int G, int H, int R, int sm_count, const PlanEnv& env);
cudaError_t set_wo_a_attributes();
cudaError_t launch_wo_a(const CUtensorMap& tm_w, const WoaArgs& args, const WoaPlan& plan,
                        cudaStream_t stream);

// ------------------------------------------------------------ MXFP4 quantizer
// Element types of the inputs that may have several (MX_TYPE_* of mx.h).
enum ElementType : int { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };

// Division of 32-bit numbers by a fixed one (quantize_fp4.cu).
struct FastDiv {
  uint32_t mul;
  int shift;  // -1: the divisor is 1
};
FastDiv fast_div(uint32_t d);

// M * K / 8 < 2^31; y (the codes' values in bf16 [M, K]) may be null.
cudaError_t launch_quantize_rows_fp4(const void* x, long ldx, int x_type, int M, int K, void* q, void* scales,
                                     int swizzled, void* y, cudaStream_t stream);

// ------------------------------------------------------------ MXFP4 products
// out = dequant(a) x dequant(w)^T for the rows of E experts (route.cu orders them;
// a plain product is one expert of M rows). Row r of expert e, offsets[e] <= r <
// offsets[e + 1], is row tokens[r] of a (r itself where tokens is null).
struct GemmFp4Args {
  int E, N, K;
  int R;                    // output rows
  int a_rows;               // rows of a
  const uint8_t* a;         // the activations, read directly where tokens is set
  int nt;                   // largest token tile (MMA N), a multiple of 16
  int band;                 // token tiles that go over all weight tiles together
  int stages, tmem_cols;
  const uint8_t* a_scales;  // plain [a_rows, K / 32], or (a_swizzled) the 128x4 layout
  int a_swizzled;
  const uint8_t* w_scales;  // 128x4 layout of each expert's [N, K], one after another
  const int* offsets;       // device, [E + 1]; null: one expert of R rows
  const int* tokens;        // device, [R], or null
  int gated;                // out [R, N / 2] = silu(column 2i) * column 2i + 1
  int early_weights;        // weights are read before the previous kernel has ended (offsets null)
  __nv_bfloat16* out;
  int* status;
};
struct GemmFp4Plan {
  int mode;    // how CTAs share SMs and tiles (gemm_fp4.cu)
  int a_rows;  // activation rows of a stage: the tensor map's box
  int nt, band, stages, min_stages, tmem_cols, ctas_per_sm, grid;
  size_t smem;
};
GemmFp4Plan plan_gemm_fp4(int E, int R, int N, int K, bool a_fp4, int sm_count);
cudaError_t set_gemm_fp4_attributes();
// tm_w: [E N, K] weights, tm_a: the activations (box plan.a_rows rows high; unused where tokens is set).
cudaError_t launch_gemm_fp4(const CUtensorMap& tm_w, const CUtensorMap& tm_a, const GemmFp4Args& args,
                            const GemmFp4Plan& plan, bool a_fp4, cudaStream_t stream);

// ------------------------------------------------------------ routing to experts
enum Scoring : int { kScoreSoftmax = 0, kScoreSigmoid = 1 };
constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTopK = 32;
// Chunks of tokens whose rows are counted apart: at most four blocks to each of 152 SMs, all
// of them at once (512 left a fifth of the SMs a block short: 8192 tokens of 256 experts
// 27.5 us, with 608 23.9; 16384 40.6 and 38.2).
constexpr int kRouteChunks = 608;
// Tokens that one block routes and orders in one launch, and chunks whose counts every
// block of the last kernel adds up itself, without a scan kernel. Measured with 8 of
// 256 experts, us: 8 tokens 6.8 in one launch; 16 tokens 10.9 in one launch, 8.0 in two,
// 9.7 in three; 128 tokens (16 chunks) 9.5 in two, 9.9 in three; 256 tokens 13.2 and 10.2.
constexpr int kRouteOneBlock = 8;
constexpr int kRouteDirectChunks = 16;
// the handle's workspace: rows per (expert, chunk), rows per expert
constexpr size_t kRouteWorkspace = sizeof(int) * (static_cast<size_t>(kRouteMaxExperts) * kRouteChunks + kRouteMaxExperts);

struct RouteArgs {
  int T, E, top_k;
  const void* logits;  // float32 or bf16 [T, E], row stride ldl
  long ldl;
  int bf16;
  const float* bias;  // [E] or null
  int scoring, n_groups, topk_groups, renormalize;
  float scale;
  float* weights;  // [T, top_k]
  int* experts;    // [T, top_k]
  int* offsets;    // [E + 1]
  int* tokens;     // [T top_k]: token of each row in expert order
  int* slots;      // [T, top_k]: the row of each (token, choice)
  int* counts;     // workspace [E][chunks]
  int* totals;     // workspace [E]
  // set by launch_route
  int chunk, chunks, group_parts, group_regs, shared_keys, direct;
  FastDiv per_group;
};
cudaError_t launch_route(RouteArgs args, cudaStream_t stream);

struct CombineArgs {
  int T, top_k, N, R;
  const __nv_bfloat16* y;  // [R, N], row stride ldy
  long ldy;
  const int* slots;
  const float* weights;
  const __nv_bfloat16* residual;  // [T, N] or null
  __nv_bfloat16* out;             // [T, N]
  int* status;
};
cudaError_t launch_combine(const CombineArgs& args, cudaStream_t stream);

// ------------------------------------------------------------ rotary positions
enum RopeScaling : int { kRopePlain = 0, kRopeLinear = 1, kRopeYarn = 2 };
constexpr int kRopeMaxDim = 512;
struct RopeTable {
  int max_pos, d_rope, scaling;
  double base, factor, beta_fast, beta_slow;
  int original;
  float magnitude;
};
cudaError_t launch_rope_table(const RopeTable& t, int sm_count, float* cos_sin, cudaStream_t stream);

// From this many chunks on a thread takes four heads of one, where there are four. (32 heads of 128, one head against
// four: 64 tokens 2.3 and 2.9 us, 256 2.7 and 3.2, 512 3.5 and 3.4, 4096 9.5 and 8.2, 16381 46.9 and 43.7; 4096
// tokens of one head of 512 3.1 and 3.9.)
constexpr int64_t kRopeManyUnits = 1 << 17;
struct RopeRows {
  int tokens, heads, d, first, d_rope;
  const void* x;
  long ldx, ldx_head;
  const int64_t* positions;
  const float* cos_sin;  // [max_pos, d_rope]
  int max_pos, interleaved, inverse;
  void* out;
  long ldo, ldo_head;
  int* status;
  // set by launch_rope
  uint32_t units, chunks, turned, head_groups;
  FastDiv per_row, per_token;
};
int rope_vec(const RopeRows& a, int size);
cudaError_t launch_rope(const RopeRows& a, int x_type, cudaStream_t stream);

// ------------------------------------------------------------ attention cache
// From this many 16-element units on a thread takes two (8 heads of 128, read, one against two: 4096 rows 5.0 us
// both, 16381 rows 14.0 and 13.3, 32749 rows 32.5 and 30.4; four: 5.6, 12.9, 28.5 and 7.9 instead of 7.2 at 8192).
constexpr uint32_t kCacheManyUnits = 1u << 19;
struct CacheSide {
  const void* x;  // write: [rows, heads, d], strides ldx and ldx_head elements
  long ldx, ldx_head;
  void* y;  // write: the values in bf16, or null; read: the output
  uint8_t* codes;
  uint8_t* scales;
  long page_stride, scale_page_stride;  // bytes
};
struct CacheRows {
  int rows, sides;
  uint32_t heads, head_units;  // head_units = d / 16
  uint32_t page_size;
  int64_t slot_count;  // pages * page_size, below 2^31
  const int64_t* slots;
  CacheSide side[2];
  int* status;
  // set by the launchers
  uint32_t units;
  FastDiv per_head, per_row, per_page;
};
cudaError_t launch_cache_write(const CacheRows& args, int x_type, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRows& args, int out_type, cudaStream_t stream);

// ------------------------------------------------------------ attention over the cache
struct AttendArgs {
  int B, T, q_heads, heads, group;  // group = q_heads / heads
  const uint16_t* q;  // bf16 or (q_f16) fp16 bits [T, q_heads, d], strides in elements
  long ldq, ldq_head;
  int q_f16;
  const int* q_offsets;  // [B + 1], or null: T / B query tokens of each sequence
  const int* table;      // [B, table_cols] pages, row stride ld_table
  long ld_table;
  int table_cols;
  const int* lengths;  // [B]
  const uint8_t* k;
  const uint8_t* k_scales;
  const uint8_t* v;  // keys' pools where values are shared
  const uint8_t* v_scales;
  long k_page, k_scale_page, v_page, v_scale_page;  // bytes between pages
  int pages, page_size;
  FastDiv per_page;  // by page_size / 16
  float scale_log2;  // scale * log2(e)
  int causal, window;
  uint16_t* out;  // of q's type [T, q_heads, d]
  long ldo, ldo_head;
  float* lse;  // [T, q_heads] or null
  float* partial;
  int* status;
};
// Kernel variants of few query rows: head dims 64, 128, 256, 512, values apart or shared, with units
// of 16 rows, then the same with 8.
constexpr int kAttendVariants = 16;
int attend_variant(int d, bool shared);  // the one of 16 rows; -1: no such head dim
cudaError_t set_attend_attributes(int sm_count, int (&ctas)[kAttendVariants]);
size_t attend_bytes(int d, int ctas, int rows);
cudaError_t launch_attend(const AttendArgs& args, int variant, int ctas, cudaStream_t stream);
// Latents of 512 dimensions that are keys and values in one, in units of 64 rows.
cudaError_t set_attend_latent_attributes();
size_t attend_latent_bytes(int sm_count);
cudaError_t launch_attend_latent(const AttendArgs& args, int sm_count, cudaStream_t stream);
// Many query rows (head dims up to 256): blocks of rows, and splits of their tokens.
constexpr int kAttendRowsVariants = 6;
struct AttendRowsPlan {
  bool ok;
  int blocks, splits;
};
cudaError_t set_attend_rows_attributes();
// uniform: T / B query tokens of every sequence; most_tokens: of a sequence at most.
AttendRowsPlan plan_attend_rows(int d, bool shared, int B, int T, bool uniform, int heads, int group, int64_t most_tokens,
                                int sm_count);
size_t attend_rows_bytes(int d, bool shared, int sm_count);
cudaError_t launch_attend_rows(const AttendArgs& args, int d, bool shared, const AttendRowsPlan& plan, cudaStream_t stream);

}  // namespace mx
