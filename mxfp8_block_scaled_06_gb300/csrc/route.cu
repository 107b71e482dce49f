// route.cu - routing tokens to experts, and the weighted sum of the experts' rows.
//
// mx_route: a token's scores s = softmax(x) or 1 / (1 + exp(-x)) over E logits,
// keys s + bias, the top_k largest keys among the chosen groups of experts (ties
// to the lowest index), weights s_j / sum s_j * scale, and the order of all
// (token, choice) rows by expert for a grouped product.
//
// One warp per token; lane l holds experts l, l + 32, ... in registers. A key is
// compared as an order-preserving 32-bit pattern, so one round of the selection
// is a scan over the lane's keys and two warp reductions (the largest key, then
// the lowest index that has it).
//
// The selection is the one that exact scores give. Without a bias the scores'
// order is the logits' order and the logits themselves are compared. With a bias
// the keys are float32 sums with a known error; whenever two neighbours of the
// selection, the last one taken and one left out, or the last chosen and the
// first rejected group are closer than their errors, the token is done again in
// float64. With 256 experts that is a few tokens in a thousand.
//
// Masked logits: -inf and NaN logits have score 0 and are chosen last; +inf
// counts as the largest float. When every chosen score is 0 so are the weights.
//
// Row order: the tokens are cut into at most kRouteChunks chunks; each chunk
// counts its rows per expert, one warp per expert turns the chunks' counts into
// starts, and each chunk places its rows in (token, choice) order, so the order is
// the stable one whatever the launch (integer sums only).
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kRouteWarps = 8;

// Order-preserving bits: a < b as floats <=> ord(a) < ord(b); never 0 for a number.
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float load_logit(const void* p, size_t i, int bf16) {
  const float f = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
  return isnan(f) ? -CUDART_INF_F : fminf(f, CUDART_MAX_NORMAL_F);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Keeps the two largest of (a1 >= a2) and (b1 >= b2) in a1, a2.
template <typename F>
__device__ __forceinline__ void merge_top2(F& a1, F& a2, F b1, F b2) {
  a2 = max(min(a1, b1), a1 >= b1 ? a2 : b2);
  a1 = max(a1, b1);
}

struct Token {
  float top;  // largest logit (softmax)
  float sum;  // sum of exp(x - top) (softmax)
};

__device__ __forceinline__ float score32(const RouteArgs& p, const Token& t, float x) {
  if (p.scoring == kScoreSigmoid) return 1.f / (1.f + expf(-x));
  return t.sum > 0.f ? expf(x - t.top) / t.sum : 0.f;
}

// Bound of |computed key - exact key| of score32(x) + bias in float32: expf is
// within 2 units in the last place, x - top is rounded once (an error that exp
// multiplies by the score), the sum of E <= 512 terms and the division add a few
// more, and the addition rounds the key once.
__device__ __forceinline__ float key_error(const RouteArgs& p, const Token& t, float x, float s, float key) {
  const float d = p.scoring == kScoreSigmoid ? 8.f : 24.f + (t.top - x);
  return (s > 0.f ? s * d * 1.2e-7f : 0.f) + fabsf(key) * 1.2e-7f + 1e-37f;
}

// Groups in the order of their best keys: a bit mask of the topk_groups first.
// keys: the warp's E keys in shared memory. best = the largest key of a group, or
// with a bias the sum of its two largest. Sets *close when the last group in and
// the first one out differ by no more than err.
template <typename F>
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& p, const volatile F* keys, F err, bool* close) {
  const int lane = threadIdx.x & 31;
  const int parts = p.group_parts;  // lanes per group, a power of two
  const int g = lane / parts, part = lane & (parts - 1);
  const int size = p.E / p.n_groups;
  F a1 = -CUDART_INF_F, a2 = -CUDART_INF_F;
  if (g < p.n_groups)
    for (int e = part; e < size; e += parts) merge_top2<F>(a1, a2, keys[g * size + e], -CUDART_INF_F);
  for (int o = 1; o < parts; o <<= 1) {
    const F b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    merge_top2<F>(a1, a2, b1, b2);
  }
  const F best = p.bias == nullptr || size == 1 ? a1 : a1 + a2;
  int rank = 0;
  for (int j = 0; j < p.n_groups; ++j) {
    const F b = __shfl_sync(kFull, best, j * parts);
    rank += b > best || (b == best && j < g);
  }
  const bool mine = g < p.n_groups && part == 0;
  const uint32_t in = __ballot_sync(kFull, mine && rank < p.topk_groups);
  const uint32_t last = __ballot_sync(kFull, mine && rank == p.topk_groups - 1);
  const uint32_t next = __ballot_sync(kFull, mine && rank == p.topk_groups);
  if (next != 0) {
    const F x = __shfl_sync(kFull, best, __ffs(last) - 1), y = __shfl_sync(kFull, best, __ffs(next) - 1);
    if (y > -CUDART_INF_F && !(x - y > err)) *close = true;
  }
  uint32_t mask = 0;
  for (int j = 0; j < p.n_groups; ++j) mask |= (in >> (j * parts) & 1u) << j;
  return mask;
}

// The token's selection in float64, for keys too close for float32: lane j < top_k
// returns the j-th expert. keys: the warp's shared memory.
__device__ __noinline__ int select64(const RouteArgs& p, size_t token, volatile double* keys) {
  const int lane = threadIdx.x & 31;
  const size_t base = token * static_cast<size_t>(p.ldl);
  double top = -CUDART_INF, sum = 0;
  for (int e = lane; e < p.E; e += 32) top = fmax(top, static_cast<double>(load_logit(p.logits, base + e, p.bf16)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
  if (p.scoring == kScoreSoftmax && top > -CUDART_INF) {
    for (int e = lane; e < p.E; e += 32) sum += exp(static_cast<double>(load_logit(p.logits, base + e, p.bf16)) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) {
    const double x = load_logit(p.logits, base + e, p.bf16);
    const double s = p.scoring == kScoreSigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum;
    keys[e] = x == -CUDART_INF || isnan(p.bias[e]) ? -CUDART_INF : s + static_cast<double>(p.bias[e]);
  }
  __syncwarp();
  uint32_t open = kFull;
  bool close = false;
  if (p.n_groups > 1) open = choose_groups<double>(p, keys, 0.0, &close);
  const int size = p.E / p.n_groups;
  int mine = 0;
  // each round takes the largest (key, then lowest index) after the last one taken
  double last = CUDART_INF;
  int last_e = -1;
  for (int j = 0; j < p.top_k; ++j) {
    double k = -CUDART_INF;
    int at = p.E;
    for (int e = lane; e < p.E; e += 32) {
      const double v = keys[e];
      if (p.n_groups > 1 && !(open >> (e / size) & 1u)) continue;
      if (v > last || (v == last && e <= last_e)) continue;
      if (at == p.E || v > k) k = v, at = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ok = __shfl_xor_sync(kFull, k, o);
      const int oa = __shfl_xor_sync(kFull, at, o);
      if (oa < p.E && (at == p.E || ok > k || (ok == k && oa < at))) k = ok, at = oa;
    }
    if (lane == j) mine = at;
    last = k;
    last_e = at;
  }
  return mine;
}

// The selection of one token: lane j < top_k returns the j-th expert and its weight.
template <int V>  // keys per lane
__device__ __forceinline__ void route_token(const RouteArgs& p, size_t token, const float (&bias)[V],
                                            const int (&group)[V], double* shared, int* expert, float* weight) {
  const int lane = threadIdx.x & 31;
  const size_t base = token * static_cast<size_t>(p.ldl);
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < p.E ? load_logit(p.logits, base + e, p.bf16) : -CUDART_INF_F;
  }
  Token t{0.f, 1.f};
  if (p.scoring == kScoreSoftmax) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
    // order-preserving bits, so that one reduction takes signs too
    t.top = unord32(__reduce_max_sync(kFull, ord32(top)));
    float sum = 0.f;
    if (t.top > -CUDART_INF_F) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(x[i] - t.top);
    }
    t.sum = warp_sum(sum);
  }
  uint32_t key[V];
  float far = 0.f;  // the largest error of the token's keys
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float k = x[i];
    if (p.bias != nullptr && k > -CUDART_INF_F) {
      const float s = score32(p, t, x[i]);
      k = isnan(bias[i]) ? -CUDART_INF_F : s + bias[i];
      if (k > -CUDART_INF_F) far = fmaxf(far, key_error(p, t, x[i], s, k));
    }
    key[i] = lane + 32 * i < p.E ? ord32(k + 0.f) : 0u;  // + 0: -0 and 0 are the same key
  }
  far = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(far)));
  bool close = false;
  if (p.n_groups > 1) {
    volatile float* const keys = reinterpret_cast<volatile float*>(shared);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < p.E) keys[lane + 32 * i] = unord32(key[i]);
    __syncwarp();
    // a group's sum has at most twice the largest error, and rounds once more;
    // without a bias the keys are exact
    const uint32_t open = choose_groups<float>(p, keys, p.bias == nullptr ? -1.f : 6.f * far, &close);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(open >> group[i] & 1u)) key[i] = 0u;  // no round takes a closed expert
  }
  int mine = 0;
  uint32_t last = 0;  // the previous round's key; its expert
  int last_e = 0;
  for (int j = 0; j < p.top_k && !close; ++j) {
    uint32_t k = key[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > k) k = key[i], at = lane + 32 * i;
    const uint32_t best = __reduce_max_sync(kFull, k);
    const int e = static_cast<int>(__reduce_min_sync(kFull, k == best ? static_cast<uint32_t>(at) : 0xFFFFu));
    // neighbours of the selection that float32 cannot tell apart, unless they are a
    // true tie (the same logit and bias), which the lowest index has won
    if (p.bias != nullptr && j > 0 && best > ord32(-CUDART_INF_F) && !(unord32(last) - unord32(best) > 2.f * far))
      close = load_logit(p.logits, base + last_e, p.bf16) != load_logit(p.logits, base + e, p.bf16) ||
              p.bias[last_e] != p.bias[e];
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i == e) key[i] = 0u;
    last = best;
    last_e = e;
  }
  if (p.bias != nullptr && last > ord32(-CUDART_INF_F)) {
    // and whatever was left out that may belong before the last one taken
    const float least = unord32(last) - 2.f * far;
    const float xl = load_logit(p.logits, base + last_e, p.bf16), bl = p.bias[last_e];
    bool near = false;
#pragma unroll
    for (int i = 0; i < V; ++i) near |= key[i] != 0u && !(unord32(key[i]) < least) && (x[i] != xl || bias[i] != bl);
    close |= __any_sync(kFull, near) != 0;
  }
  if (close) mine = select64(p, token, shared);
  float w = 0.f;
  if (lane < p.top_k) {
    const float xm = load_logit(p.logits, base + mine, p.bf16);
    w = xm > -CUDART_INF_F ? score32(p, t, xm) : 0.f;
  }
  if (p.renormalize) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  *expert = mine;
  *weight = w * p.scale;
}

// v[0..n) become the sums of the values before each, by one warp; returns the sum of all.
__device__ __forceinline__ int exclusive_scan(int* v, int n) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int e0 = 0; e0 < n; e0 += 32) {
    const int own = e0 + lane < n ? v[e0 + lane] : 0;
    int s = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += up;
    }
    if (e0 + lane < n) v[e0 + lane] = run + s - own;
    run += __shfl_sync(kFull, s, 31);
  }
  __syncwarp();
  return run;
}

// Places the rows [r0, r1) in (token, choice) order, by one warp; base[e] (shared
// memory) is the next free row of expert e.
__device__ __forceinline__ void place_rows(const RouteArgs& p, int r0, int r1, int* base) {
  const int lane = threadIdx.x & 31;
  for (int r = r0; r < r1; r += 32) {
    const bool in = r + lane < r1;
    const int e = in ? p.experts[r + lane] : -1;
    const uint32_t peers = __match_any_sync(kFull, e);
    const int before = __popc(peers & ((1u << lane) - 1));
    const int at = in ? base[e] + before : 0;
    __syncwarp();
    if (in && before == 0) base[e] = at + __popc(peers);
    __syncwarp();
    if (in) {
      p.slots[r + lane] = at;
      p.tokens[at] = (r + lane) / p.top_k;
    }
  }
}

// One block per chunk of tokens: the selection, and the chunk's rows per expert
// (counts[e][chunk]). With a single chunk the block also orders the rows.
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ RouteArgs p) {
  extern __shared__ double route_smem[];
  int* const hist = reinterpret_cast<int*>(route_smem + (p.shared_keys ? kRouteWarps * p.E : 0));
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double* const keys = route_smem + (p.shared_keys ? warp * p.E : 0);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  pdl_wait();
  float bias[V];
  int group[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    bias[i] = p.bias != nullptr && e < p.E ? p.bias[e] : 0.f;
    group[i] = p.n_groups > 1 && e < p.E ? e / (p.E / p.n_groups) : 0;
  }
  __syncthreads();
  const int t1 = min(p.T, static_cast<int>(blockIdx.x + 1) * p.chunk);
  for (int t = blockIdx.x * p.chunk + warp; t < t1; t += kRouteWarps) {
    int e;
    float w;
    route_token<V>(p, t, bias, group, keys, &e, &w);
    if (lane < p.top_k) {
      const size_t r = static_cast<size_t>(t) * p.top_k + lane;
      p.experts[r] = e;
      p.weights[r] = w;
      atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.counts[e * p.chunks + blockIdx.x] = hist[e];
    return;
  }
  if (warp == 0) {
    const int rows = exclusive_scan(hist, p.E);
    for (int e = lane; e < p.E; e += 32) p.offsets[e] = hist[e];
    if (lane == 0) p.offsets[p.E] = rows;
    __syncwarp();
    place_rows(p, 0, rows, hist);
  }
}

// One warp per expert: counts[e][chunk] become the rows of the chunks before, and
// totals[e] the expert's rows.
__global__ void __launch_bounds__(kRouteWarps * 32) route_scan_kernel(const __grid_constant__ RouteArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  const int e = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (e >= p.E) return;
  const int total = exclusive_scan(p.counts + static_cast<size_t>(e) * p.chunks, p.chunks);
  if ((threadIdx.x & 31) == 0) p.totals[e] = total;
}

// One warp per chunk: its rows into expert order.
__global__ void __launch_bounds__(32) route_place_kernel(const __grid_constant__ RouteArgs p) {
  extern __shared__ double route_smem[];
  int* const base = reinterpret_cast<int*>(route_smem);
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x;
  for (int e = lane; e < p.E; e += 32) base[e] = p.totals[e];
  __syncwarp();
  const int rows = exclusive_scan(base, p.E);
  if (blockIdx.x == 0) {
    for (int e = lane; e < p.E; e += 32) p.offsets[e] = base[e];
    if (lane == 0) p.offsets[p.E] = rows;
  }
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) base[e] += p.counts[static_cast<size_t>(e) * p.chunks + blockIdx.x];
  __syncwarp();
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  place_rows(p, t0 * p.top_k, t1 * p.top_k, base);
}

// out[t] = sum over j of weights[t][j] y[slots[t][j]] (+ residual[t]) in float32,
// in the order of j. A thread owns eight columns of a token; the rows' loads of
// four choices are in flight together.
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ CombineArgs p) {
  pdl_launch_dependents();
  const int c = blockIdx.y * kCombineThreads + threadIdx.x;
  const size_t t = blockIdx.x;
  pdl_wait();
  if (c * 8 >= p.N) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](const uint4& v, float w) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xFFFF0000u), acc[2 * i + 1]);
    }
  };
  const int* const slots = p.slots + t * p.top_k;
  const float* const weights = p.weights + t * p.top_k;
  uint4 res = make_uint4(0, 0, 0, 0);
  if (p.residual != nullptr) res = reinterpret_cast<const uint4*>(p.residual + t * p.N)[c];
  for (int j0 = 0; j0 < p.top_k; j0 += 4) {
    uint4 v[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i;
      const int s = j < p.top_k ? slots[j] : 0;
      const bool ok = s >= 0 && s < p.R;
      if (!ok && c == 0) atomicOr(p.status, kStatusBadInput);
      w[i] = ok && j < p.top_k ? weights[j] : 0.f;
      // a slot out of range reads nothing and adds nothing
      v[i] = ok && j < p.top_k ? __ldg(reinterpret_cast<const uint4*>(p.y + static_cast<size_t>(s) * p.ldy) + c)
                               : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < p.top_k) add(v[i], w[i]);
  }
  if (p.residual != nullptr) add(res, 1.f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i])) |
           static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i + 1]))) << 16;
  reinterpret_cast<uint4*>(p.out + t * p.N)[c] = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename Args>
cudaError_t launch_pdl(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace

cudaError_t launch_route(RouteArgs p, cudaStream_t stream) {
  // tokens per chunk: at least kRouteMinChunk (one block then does everything up
  // to that many tokens), at most kRouteChunks chunks
  p.chunk = std::max(kRouteMinChunk, (p.T + kRouteChunks - 1) / kRouteChunks);
  p.chunks = (p.T + p.chunk - 1) / p.chunk;
  p.group_parts = 32;
  while (p.group_parts * p.n_groups > 32) p.group_parts >>= 1;
  p.shared_keys = p.n_groups > 1 || p.bias != nullptr;
  const size_t smem = (p.shared_keys ? sizeof(double) * kRouteWarps * p.E : 0) + sizeof(int) * p.E;
  const dim3 grid(p.chunks);
  const int threads = kRouteWarps * 32;
  cudaError_t e;
  if (p.E <= 32) e = launch_pdl(route_kernel<1>, grid, threads, smem, stream, p);
  else if (p.E <= 64) e = launch_pdl(route_kernel<2>, grid, threads, smem, stream, p);
  else if (p.E <= 128) e = launch_pdl(route_kernel<4>, grid, threads, smem, stream, p);
  else if (p.E <= 256) e = launch_pdl(route_kernel<8>, grid, threads, smem, stream, p);
  else e = launch_pdl(route_kernel<16>, grid, threads, smem, stream, p);
  if (e != cudaSuccess || p.chunks == 1) return e;
  e = launch_pdl(route_scan_kernel, dim3((p.E + kRouteWarps - 1) / kRouteWarps), threads, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(route_place_kernel, grid, 32, sizeof(int) * p.E, stream, p);
}

cudaError_t launch_combine(const CombineArgs& p, cudaStream_t stream) {
  const dim3 grid(p.T, (p.N / 8 + kCombineThreads - 1) / kCombineThreads);
  return launch_pdl(combine_kernel, grid, kCombineThreads, 0, stream, p);
}

}  // namespace mx
