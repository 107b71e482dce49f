// route.cu - routing tokens to experts, and the weighted sum of the experts' rows.
//
// mx_route: a token's scores s = softmax(x) or 1 / (1 + exp(-x)) over E logits,
// keys s + bias, the top_k largest keys among the chosen groups of experts (ties
// to the lowest index), weights s_j / sum s_j * scale, and the order of all
// (token, choice) rows by expert for a grouped product.
//
// One warp per token; lane l holds experts l, l + 32, ... in registers, their keys as
// order-preserving 32-bit patterns. The top_k-th largest of the lanes' largest keys
// bounds the selection from below; the few keys at or above it (with a bias: or
// within the keys' error of it) are gathered one to a lane and ranked by counting.
// Rounds of a scan over each lane's keys and two warp reductions, one round for
// each choice, took twice the instructions (1945 against about 1000 a token with 256
// experts, eight groups and a bias; 60 % of the issue slots were busy).
//
// The selection is the one that exact scores give. Without a bias the scores'
// order is the logits' order and the logits themselves are compared. With a bias
// the keys are float32 sums with a known error; whenever two neighbours of the
// selection, the last one taken and one left out, or the last chosen and the
// first rejected group are closer than their errors, the keys in question are
// computed again in float64. With 256 experts that is a few tokens in a thousand.
//
// Masked logits: -inf and NaN logits have score 0 and are chosen last; +inf
// counts as the largest float, and so does a bias of +inf (keys and their errors stay
// finite). When every chosen score is 0 so are the weights.
//
// Row order: the tokens are cut into at most kRouteChunks chunks; each chunk
// counts its rows per expert and numbers them in (token, choice) order, one warp per
// expert turns the chunks' counts into starts, and a third kernel adds the two, so
// the order is the stable one whatever the launch (integer sums only).
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kRouteWarps = 8;
constexpr uint32_t kMasked = 0x007FFFFFu;  // ord32(-inf)

// Order-preserving bits: a < b as floats <=> ord(a) < ord(b); never 0 for a number.
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float load_logit(const void* p, size_t i, int bf16) {
  const float f = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
  return isnan(f) ? -CUDART_INF_F : fminf(f, CUDART_MAX_NORMAL_F);
}

// An expert's bias: NaN counts as -inf, +inf as the largest float.
__device__ __forceinline__ float bias_value(float b) {
  return isnan(b) ? -CUDART_INF_F : fminf(b, CUDART_MAX_NORMAL_F);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// n / d for the d that f was made for (fast_div).
__device__ __forceinline__ uint32_t div_u32(uint32_t n, FastDiv f) {
  const uint32_t t = __umulhi(f.mul, n);
  return f.shift < 0 ? n : (t + ((n - t) >> 1)) >> f.shift;
}

// Renormalized weights of scores (lane j: of logit x, -inf where it has no choice) whose sum is
// so small that some of them may be float32 subnormals or 0: in float64; 0 where the sum is 0
// there too. With the sum at kSmallSum or more such a score's weight is below 2^-106.
constexpr float kSmallSum = 1.f / (1 << 20);
__device__ __noinline__ float small_weights(const RouteArgs& p, float x, float top) {
  double s = 0.0;
  if (x > -CUDART_INF_F)
    s = p.scoring == kScoreSigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x))) : exp(static_cast<double>(x) - top);
  double sum = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum > 0.0 ? static_cast<float>(s / sum) : 0.f;
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
  // far below 0 exp(-x) overflows, and the score is exp(x) to within exp(x) of itself
  if (p.scoring == kScoreSigmoid) return x < -80.f ? expf(x) : 1.f / (1.f + expf(-x));
  return t.sum > 0.f ? expf(x - t.top) / t.sum : 0.f;
}

// The keys' score: approximate exp and reciprocal, a few units in the last place.
__device__ __forceinline__ float quick_sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Bound of |computed score - exact score| of the token's keys, in units of 2^-23.
// __expf(y) is within 2 + 1.18 |y| units (2 ulp and its argument's rounding),
// __fdividef within 2, an addition or division within 0.5.
//   sigmoid: s = 1 / D, D = 1 + exp(-x): relative (1 - s)(2 + 1.18 |x|) + 0.5 + 2, so
//            absolute at most 0.63 + 2.5 (s (1 - s)(2 + 1.18 |x|) peaks at 0.627).
//   softmax: u = top - x is rounded once: a term is off by 2 + 1.68 u, the sum of E <=
//            512 terms (a softmax's mean u is at most ln E) by 12.6 + 21 roundings, the
//            quotient by 1 more: s is off by s (26.1 + 1.68 u) <= 26.2 s_top.
__device__ __forceinline__ float scores_error(const RouteArgs& p, const Token& t) {
  const float s = p.scoring == kScoreSigmoid ? 3.2f : t.sum > 0.f ? 26.2f / t.sum : 0.f;
  return s * 1.2e-7f + 1e-37f;
}

// Bound of |computed key - exact key|: the score's, and half a unit of the sum with the bias,
// taken twice to leave room for the roundings of what is computed with it. It is the
// key's own, so a large bias elsewhere (-1e9 for a masked expert) brings no other key
// into question. k + key_error and k - key_error grow with k, so keys sorted by k that
// are further apart than their errors from neighbour to neighbour are so altogether.
__device__ __forceinline__ float key_error(float score_error, float k) { return score_error + 1.2e-7f * fabsf(k); }

// The parts of a token's selection in float64, for keys that float32 cannot tell
// apart; out of line, as few tokens come here. float64 is slow on this GPU (a warp
// instruction takes about 16 cycles), so only the keys in question are computed,
// one to a lane.

// Sum of exp(x - top) over the token's experts in float64 (softmax; 1 otherwise).
__device__ __noinline__ double sum64(const RouteArgs& p, size_t base, float top) {
  if (p.scoring == kScoreSigmoid) return 1.0;
  double sum = 0;
  for (int e = threadIdx.x & 31; e < p.E; e += 32)
    sum += exp(static_cast<double>(load_logit(p.logits, base + e, p.bf16)) - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum;
}

__device__ __forceinline__ double key64(const RouteArgs& p, size_t base, int e, float top, double sum) {
  const double x = load_logit(p.logits, base + e, p.bf16);
  const float b = bias_value(p.bias[e]);
  if (x == -CUDART_INF) return -CUDART_INF;
  return (p.scoring == kScoreSigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum) + static_cast<double>(b);
}

// Lane i < n holds one of n candidates (expert e): the candidate of rank lane by
// (key, then lowest index) to every lane < n.
__device__ __noinline__ int order64(const RouteArgs& p, size_t base, int e, int n, float top, volatile int* list) {
  const int lane = threadIdx.x & 31;
  const double sum = sum64(p, base, top);
  const double k = lane < n ? key64(p, base, e, top, sum) : 0.0;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double kj = __shfl_sync(kFull, k, j);
    const int ej = __shfl_sync(kFull, e, j);
    rank += kj > k || (kj == k && ej < e);
  }
  __syncwarp();
  if (lane < n) list[rank] = e;
  __syncwarp();
  return list[lane < n ? lane : 0];
}

// The whole token in float64, where more than 32 keys are in question: lane j <
// top_k returns the j-th expert of the open groups. keys: the warp's shared memory.
__device__ __noinline__ int select64(const RouteArgs& p, size_t base, float top, uint32_t open, volatile double* keys) {
  const int lane = threadIdx.x & 31;
  const double sum = sum64(p, base, top);
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) keys[e] = key64(p, base, e, top, sum);
  __syncwarp();
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
      if (!(open >> (e / size) & 1u)) continue;
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

// The selection by rounds where more than 32 keys are at or above the bound (many
// equal ones) and the float32 keys are exact. keys: the warp's shared memory; a key
// of 0 is not taken.
__device__ __noinline__ int select32(const RouteArgs& p, volatile uint32_t* keys) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t k = 0u, at = 0xFFFFu;
    for (int e = lane; e < p.E; e += 32)
      if (keys[e] > k) k = keys[e], at = e;
    const uint32_t best = __reduce_max_sync(kFull, k);
    const uint32_t e = __reduce_min_sync(kFull, k == best ? at : 0xFFFFu);
    if (static_cast<uint32_t>(lane) == (e & 31)) keys[e] = 0u;
    if (lane == j) mine = e;
  }
  return mine;
}

// The chosen groups when the float32 sums of `contended` groups (a bit mask) are too
// close: `in` of the groups outside it are chosen already. With each contended
// group's keys that may be among its two largest (at least `floor`, float32) in
// float64, its exact sum; the largest sums fill the places left.
__device__ __noinline__ uint32_t groups64(const RouteArgs& p, size_t base, float top, uint32_t in, uint32_t contended,
                                          const volatile float* keys32, float score_error) {
  const int lane = threadIdx.x & 31;
  const int size = p.E / p.n_groups;
  const double sum = sum64(p, base, top);
  double best = -CUDART_INF;  // lane g: the sum of contended group g
  for (uint32_t left = contended; left != 0; left &= left - 1) {
    const int g = __ffs(left) - 1;
    float a1 = -CUDART_INF_F, a2 = -CUDART_INF_F;
    for (int e = lane; e < size; e += 32) merge_top2<float>(a1, a2, keys32[g * size + e], -CUDART_INF_F);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
      merge_top2<float>(a1, a2, b1, b2);
    }
    const float second = size == 1 ? a1 : a2, floor = second - 2.f * key_error(score_error, second);
    double d1 = -CUDART_INF, d2 = -CUDART_INF;
    for (int e = lane; e < size; e += 32)
      if (!(keys32[g * size + e] < floor))
        merge_top2<double>(d1, d2, key64(p, base, g * size + e, top, sum), -CUDART_INF);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double b1 = __shfl_xor_sync(kFull, d1, o), b2 = __shfl_xor_sync(kFull, d2, o);
      merge_top2<double>(d1, d2, b1, b2);
    }
    if (lane == g) best = size == 1 ? d1 : d1 + d2;
  }
  int rank = 0;
  for (uint32_t left = contended; left != 0; left &= left - 1) {
    const int j = __ffs(left) - 1;
    const double b = __shfl_sync(kFull, best, j);
    rank += b > best || (b == best && j < lane);
  }
  return in | __ballot_sync(kFull, (contended >> lane & 1u) && rank < p.topk_groups - __popc(in));
}

// A group's two largest keys (without a bias and in groups of one expert the second is 0).
struct Best {
  float k1, k2;
};
// What ranks the groups: their largest keys, or with a bias the sum of their two largest; beyond
// float's range its end, -inf where the second is masked.
__device__ __forceinline__ float group_sum(Best b) {
  const float sum = fmaxf(fminf(b.k1 + b.k2, CUDART_MAX_NORMAL_F), -CUDART_MAX_NORMAL_F);
  return fminf(b.k1, b.k2) > -CUDART_INF_F ? sum : -CUDART_INF_F;
}

// Each group's two largest keys, in lane g; for groups of whole registers of the warp (32, 64, ... experts): two warp reductions a
// group, where the keys in shared memory took 387 instructions a token in all.
template <int V>
__device__ __forceinline__ Best best_of_registers(const RouteArgs& p, const uint32_t (&key)[V]) {
  const int lane = threadIdx.x & 31;
  uint32_t k1 = 0, k2 = 0, best1 = 0, best2 = 0;
  int g = 0, left = p.group_regs;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    k2 = max(k2, min(k1, key[i]));
    k1 = max(k1, key[i]);
    if (--left == 0) {
      const uint32_t w1 = __reduce_max_sync(kFull, k1);
      const uint32_t owner = __ffs(__ballot_sync(kFull, k1 == w1)) - 1;
      const uint32_t w2 = __reduce_max_sync(kFull, static_cast<uint32_t>(lane) == owner ? k2 : k1);
      if (lane == g) best1 = w1, best2 = w2;
      k1 = k2 = 0;
      left = p.group_regs;
      ++g;
    }
  }
  return {unord32(best1), p.bias == nullptr ? 0.f : unord32(best2)};
}

// The same for any groups, from the warp's E keys in shared memory.
__device__ __forceinline__ Best best_of_shared(const RouteArgs& p, const volatile float* keys) {
  const int lane = threadIdx.x & 31;
  const int parts = p.group_parts;  // lanes per group, a power of two
  const int g = lane / parts, part = lane & (parts - 1);
  const int size = p.E / p.n_groups;
  float a1 = -CUDART_INF_F, a2 = -CUDART_INF_F;
  if (g < p.n_groups)
    for (int e = part; e < size; e += parts) merge_top2<float>(a1, a2, keys[g * size + e], -CUDART_INF_F);
  for (int o = 1; o < parts; o <<= 1) {
    const float b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    merge_top2<float>(a1, a2, b1, b2);
  }
  const int from = lane < p.n_groups ? lane * parts : 0;
  a2 = p.bias == nullptr || size == 1 ? 0.f : a2;
  return {__shfl_sync(kFull, a1, from), __shfl_sync(kFull, a2, from)};
}

// The groups (a bit mask) that float32 cannot rank where it matters, each by its own error: a
// wide one may belong to any group, those of a sum far below among them.
__device__ __noinline__ uint32_t groups_in_question(Best best, float score_error, bool chosen, bool left) {
  const float sum = group_sum(best);
  const float err = sum > -CUDART_INF_F ? fminf(key_error(score_error, best.k1) + key_error(score_error, best.k2) +
                                                    1.2e-7f * fabsf(best.k1 + best.k2),
                                                CUDART_MAX_NORMAL_F)
                                        : 0.f;
  // how low the chosen ones may be, and how high the ones left out
  const float low = sum - err, high = sum + err;
  const float least = unord32(__reduce_min_sync(kFull, chosen ? ord32(low) : ord32(CUDART_INF_F)));
  const float most = unord32(__reduce_max_sync(kFull, left ? ord32(high) : kMasked));
  if (least > most) return 0u;
  return __ballot_sync(kFull, (chosen && !(low > most)) || (left && !(high < least)));
}

// The topk_groups groups of the largest sums (lane g: group g's), as a bit mask.
// *contended: the groups that float32 cannot rank where it matters, of which none is in
// the mask; 0 if there are none.
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& p, Best best, float score_error,
                                                  uint32_t* contended) {
  const int lane = threadIdx.x & 31;
  const float sum = group_sum(best);
  int rank = 0;
  for (int j = 0; j < p.n_groups; ++j) {
    const float b = __shfl_sync(kFull, sum, j);
    rank += b > sum || (b == sum && j < lane);
  }
  const bool mine = lane < p.n_groups;
  const uint32_t in = __ballot_sync(kFull, mine && rank < p.topk_groups);
  const uint32_t next = __ballot_sync(kFull, mine && rank == p.topk_groups);
  *contended = 0;
  if (p.bias == nullptr || next == 0) return in;
  // the last one in and the first one out, further apart than twice the error of any sum
  const uint32_t last = __ballot_sync(kFull, mine && rank == p.topk_groups - 1);
  const float x = __shfl_sync(kFull, sum, __ffs(last) - 1), y = __shfl_sync(kFull, sum, __ffs(next) - 1);
  const float size = mine && sum > -CUDART_INF_F ? fmaxf(fabsf(best.k1), fabsf(best.k2)) : 0.f;
  const float largest = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)));
  if (!(y > -CUDART_INF_F) || x - y > 4.f * score_error + 1e-6f * largest) return in;
  *contended = groups_in_question(best, score_error, mine && rank < p.topk_groups, mine && rank >= p.topk_groups);
  return in & ~*contended;
}

// The selection of one token: lane j < top_k returns the j-th expert and its weight.
// groups: the lane's keys' groups, five bits each. shared: the warp's shared memory.
template <int V>  // keys per lane
__device__ __forceinline__ void route_token(const RouteArgs& p, size_t token, const float (&bias)[V],
                                            const uint32_t (&groups)[(V + 5) / 6],
                                            double* shared, int* expert, float* weight) {
  const int lane = threadIdx.x & 31;
  const size_t base = token * static_cast<size_t>(p.ldl);
  float x[V];
  if (p.bf16) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = lane + 32 * i < p.E ? load_logit(p.logits, base + lane + 32 * i, 1) : -CUDART_INF_F;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = lane + 32 * i < p.E ? load_logit(p.logits, base + lane + 32 * i, 0) : -CUDART_INF_F;
  }
  Token t{0.f, 1.f};
  uint32_t key[V];
  float score_error = 0.f;
  if (p.scoring == kScoreSoftmax) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
    // order-preserving bits, so that one reduction takes signs too
    t.top = unord32(__reduce_max_sync(kFull, ord32(top)));
    float sum = 0.f;
    if (t.top > -CUDART_INF_F) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += __expf(x[i] - t.top);
    }
    t.sum = warp_sum(sum);
  }
  if (p.bias != nullptr) {
    score_error = scores_error(p, t);
    const float inv = p.scoring == kScoreSoftmax && t.sum > 0.f ? 1.f / t.sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = p.scoring == kScoreSigmoid ? quick_sigmoid(x[i]) : __expf(x[i] - t.top) * inv;
      if (x[i] > -CUDART_INF_F) x[i] = s + bias[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < p.E ? ord32(x[i] + 0.f) : 0u;  // + 0: -0 and 0 are the same key
  uint32_t open = kFull;
  if (p.n_groups > 1) {
    volatile float* const keys = reinterpret_cast<volatile float*>(shared);
    auto share_keys = [&]() {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < p.E) keys[lane + 32 * i] = x[i];
      __syncwarp();
    };
    Best best;
    if (p.group_regs > 0) {
      best = best_of_registers<V>(p, key);
    } else {
      share_keys();
      best = best_of_shared(p, keys);
    }
    uint32_t contended;
    open = choose_groups(p, best, score_error, &contended);
    if (contended != 0) {
      share_keys();
      open = groups64(p, base, t.top, open, contended, keys, score_error);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(open >> (groups[i / 6] >> (5 * (i % 6)) & 31u) & 1u)) key[i] = 0u;  // no closed expert is taken
  }
  // at least top_k keys are at or above the top_k-th largest of the lanes' largest
  auto bound = [&]() {
    uint32_t most = key[0], least = 0;
#pragma unroll
    for (int i = 1; i < V; ++i) most = max(most, key[i]);
    for (int j = 0; j < p.top_k; ++j) {
      least = __reduce_max_sync(kFull, most);
      if (most == least) most = 0;
    }
    return least;
  };
  uint32_t least = bound();
  if (least <= kMasked) {
    // Masked experts may have to be taken, the lowest index first: below the key of -inf
    // there are no other keys, so theirs can say that order. (Left equal, more than 32
    // of them went by rounds; a few padding tokens then took 17 of 29 us.)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] == kMasked) key[i] -= lane + 32 * i;
    least = bound();
  }
  if (p.bias != nullptr && least > kMasked)
    least = ord32(unord32(least) - 2.f * key_error(score_error, unord32(least)));
  least = max(least, 1u);
  // gathered in the order of their indices
  volatile uint2* const list = reinterpret_cast<volatile uint2*>(shared);
  int n = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t m = __ballot_sync(kFull, key[i] >= least);
    const int at = n + __popc(m & ((1u << lane) - 1));
    if (key[i] >= least && at < 32) {
      list[at].x = key[i];
      list[at].y = lane + 32 * i;
    }
    n += __popc(m);
  }
  __syncwarp();
  int mine;
  if (n <= 32) {
    uint32_t k = lane < n ? list[lane].x : 0u, e = lane < n ? list[lane].y : 0u;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t kj = __shfl_sync(kFull, k, j);
      rank += kj > k || (kj == k && j < lane);
    }
    __syncwarp();
    if (lane < n) {
      list[rank].x = k;
      list[rank].y = e;
    }
    __syncwarp();
    if (lane < n) k = list[lane].x, e = list[lane].y;
    mine = e;
    if (p.bias != nullptr) {
      // neighbours of the selection, or the last one taken and one left out, that
      // float32 cannot tell apart, unless they are a true tie (the same logit and bias)
      const int other = lane < p.top_k ? max(lane - 1, 0) : p.top_k - 1;
      const uint32_t ko = __shfl_sync(kFull, k, other), eo = __shfl_sync(kFull, e, other);
      bool close = false;
      if (lane > 0 && lane < n && k > kMasked &&
          !(unord32(ko) - unord32(k) > key_error(score_error, unord32(ko)) + key_error(score_error, unord32(k))))
        close = load_logit(p.logits, base + eo, p.bf16) != load_logit(p.logits, base + e, p.bf16) ||
                bias_value(p.bias[eo]) != bias_value(p.bias[e]);
      if (__any_sync(kFull, close)) mine = order64(p, base, e, n, t.top, reinterpret_cast<volatile int*>(shared));
    }
  } else if (p.bias != nullptr) {
    mine = select64(p, base, t.top, open, shared);
  } else {
    volatile uint32_t* const keys = reinterpret_cast<volatile uint32_t*>(shared);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < p.E) keys[lane + 32 * i] = key[i];
    __syncwarp();
    mine = select32(p, keys);
  }
  float w = 0.f, xm = -CUDART_INF_F;
  if (lane < p.top_k) {
    xm = load_logit(p.logits, base + mine, p.bf16);
    w = xm > -CUDART_INF_F ? score32(p, t, xm) : 0.f;
  }
  if (p.renormalize) {
    const float sum = warp_sum(w);
    w = sum < kSmallSum ? small_weights(p, xm, t.top) : w / sum;
  }
  *expert = mine;
  *weight = w * p.scale;
}

// v[0..n) become the sums of the values before each, by one warp; returns the sum of
// all. n <= 608; the loads are issued together.
__device__ __forceinline__ int exclusive_scan(int* v, int n) {
  const int lane = threadIdx.x & 31;
  constexpr int kOwn = std::max(kRouteChunks, kRouteMaxExperts) / 32;
  int own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) own[i] = 32 * i + lane < n ? v[32 * i + lane] : 0;
  int run = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    if (32 * i >= n) break;
    int s = own[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += up;
    }
    if (32 * i + lane < n) v[32 * i + lane] = run + s - own[i];
    run += __shfl_sync(kFull, s, 31);
  }
  __syncwarp();
  return run;
}

// The places of the rows [r0, r1) in (token, choice) order, by one warp: slots[r] =
// base[its expert]++ (base in shared memory); with tokens also the token behind each place.
__device__ __forceinline__ void place_rows(const RouteArgs& p, int r0, int r1, int* base, bool tokens) {
  const int lane = threadIdx.x & 31;
  constexpr int kAhead = 8;
  for (int b = r0; b < r1; b += 32 * kAhead) {
    int expert[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) expert[i] = b + 32 * i + lane < r1 ? p.experts[b + 32 * i + lane] : -1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = b + 32 * i + lane, e = expert[i];
      if (b + 32 * i >= r1) break;
      const uint32_t peers = __match_any_sync(kFull, e);
      const int before = __popc(peers & ((1u << lane) - 1));
      const int at = e >= 0 ? base[e] + before : 0;
      __syncwarp();
      if (e >= 0 && before == 0) base[e] = at + __popc(peers);
      __syncwarp();
      if (e >= 0) {
        p.slots[r] = at;
        if (tokens) p.tokens[at] = r / p.top_k;
      }
    }
  }
}

// One block per chunk of tokens: the selection, the chunk's rows per expert
// (counts[e][chunk]) and each row's place among the chunk's rows of its expert
// (slots). With a single chunk that place is the row's.
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32, 4) route_kernel(const __grid_constant__ RouteArgs p) {
  extern __shared__ double route_smem[];
  int* const hist = reinterpret_cast<int*>(route_smem + kRouteWarps * p.shared_keys);
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  pdl_wait();
  float bias[V];
  uint32_t groups[(V + 5) / 6] = {};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    bias[i] = bias_value(p.bias != nullptr && e < p.E ? p.bias[e] : 0.f);
    if (e < p.E) groups[i / 6] |= div_u32(e, p.per_group) << (5 * (i % 6));
  }
  __syncthreads();
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  for (int t = t0 + warp; t < t1; t += kRouteWarps) {
    int e;
    float w;
    route_token<V>(p, t, bias, groups, route_smem + warp * p.shared_keys, &e, &w);
    if (lane < p.top_k) {
      const size_t r = static_cast<size_t>(t) * p.top_k + lane;
      p.experts[r] = e;
      p.weights[r] = w;
      atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      p.counts[e * p.chunks + blockIdx.x] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
    if (warp == 0) place_rows(p, t0 * p.top_k, t1 * p.top_k, hist, false);
  } else if (warp == 0) {
    const int rows = exclusive_scan(hist, p.E);
    for (int e = lane; e < p.E; e += 32) p.offsets[e] = hist[e];
    if (lane == 0) p.offsets[p.E] = rows;
    __syncwarp();
    place_rows(p, 0, rows, hist, true);
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

// One block per chunk: its rows' places among all rows. With few chunks (p.direct) each
// block adds up the chunks' counts itself and no scan kernel runs before it.
__global__ void __launch_bounds__(kRouteWarps * 32) route_place_kernel(const __grid_constant__ RouteArgs p) {
  extern __shared__ double route_smem[];
  int* const base = reinterpret_cast<int*>(route_smem);
  pdl_launch_dependents();
  pdl_wait();
  int before[kRouteMaxExperts / (kRouteWarps * 32)];  // rows of this thread's experts in earlier chunks
#pragma unroll
  for (int i = 0; i < kRouteMaxExperts / (kRouteWarps * 32); ++i) {
    const int e = threadIdx.x + i * kRouteWarps * 32;
    before[i] = 0;
    if (e >= p.E) continue;
    const int* const counts = p.counts + static_cast<size_t>(e) * p.chunks;
    if (p.direct) {
      int total = 0;
#pragma unroll 8
      for (int c = 0; c < p.chunks; ++c) {
        const int n = counts[c];
        total += n;
        before[i] += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
      base[e] = total;
    } else {
      base[e] = p.totals[e];
      before[i] = counts[blockIdx.x];
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int rows = exclusive_scan(base, p.E);
    if (blockIdx.x == 0) {
      for (int e = threadIdx.x; e < p.E; e += 32) p.offsets[e] = base[e];
      if (threadIdx.x == 0) p.offsets[p.E] = rows;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRouteMaxExperts / (kRouteWarps * 32); ++i) {
    const int e = threadIdx.x + i * kRouteWarps * 32;
    if (e < p.E) base[e] += before[i];
  }
  __syncthreads();
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  for (int r = t0 * p.top_k + threadIdx.x; r < t1 * p.top_k; r += blockDim.x) {
    const int at = base[p.experts[r]] + p.slots[r];
    p.slots[r] = at;
    p.tokens[at] = r / p.top_k;
  }
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
      v[i] = ok && j < p.top_k ? reinterpret_cast<const uint4*>(p.y + static_cast<size_t>(s) * p.ldy)[c]
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
  // tokens per chunk: one block does everything up to kRouteOneBlock tokens; beyond,
  // a token to a warp, and at most kRouteChunks chunks
  p.chunk = p.T <= kRouteOneBlock ? p.T : std::max(kRouteWarps, (p.T + kRouteChunks - 1) / kRouteChunks);
  p.chunks = (p.T + p.chunk - 1) / p.chunk;
  p.direct = p.chunks <= kRouteDirectChunks;
  p.group_parts = 32;
  while (p.group_parts * p.n_groups > 32) p.group_parts >>= 1;
  p.per_group = fast_div(p.E / p.n_groups);
  p.group_regs = p.E / p.n_groups % 32 == 0 ? p.E / p.n_groups / 32 : 0;
  p.shared_keys = std::max(p.E, 32);  // per warp: its keys, or 32 candidates
  const size_t smem = sizeof(double) * kRouteWarps * p.shared_keys + sizeof(int) * p.E;
  const dim3 grid(p.chunks);
  const int threads = kRouteWarps * 32;
  cudaError_t e;
  if (p.E <= 32) e = launch_pdl(route_kernel<1>, grid, threads, smem, stream, p);
  else if (p.E <= 64) e = launch_pdl(route_kernel<2>, grid, threads, smem, stream, p);
  else if (p.E <= 128) e = launch_pdl(route_kernel<4>, grid, threads, smem, stream, p);
  else if (p.E <= 256) e = launch_pdl(route_kernel<8>, grid, threads, smem, stream, p);
  else e = launch_pdl(route_kernel<16>, grid, threads, smem, stream, p);
  if (e != cudaSuccess || p.chunks == 1) return e;
  if (!p.direct) {
    e = launch_pdl(route_scan_kernel, dim3((p.E + kRouteWarps - 1) / kRouteWarps), threads, 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(route_place_kernel, grid, threads, sizeof(int) * p.E, stream, p);
}

cudaError_t launch_combine(const CombineArgs& p, cudaStream_t stream) {
  const dim3 grid(p.T, (p.N / 8 + kCombineThreads - 1) / kCombineThreads);
  return launch_pdl(combine_kernel, grid, kCombineThreads, 0, stream, p);
}

}  // namespace mx
