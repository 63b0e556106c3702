// route.hip -- a mixture-of-experts router's choice and the map that sorts
// it, and the weighted sum that brings the experts' answers back.
//
// Routing.  Token t has logits l[t][0..E).  Its choice is the top_k largest
// keys, ties to the lower expert:
//   key = l                           (no selection bias: softmax and sigmoid
//                                      are monotonic, so the logits decide)
//   key = score(l) + bias[e]          (in fp64: the choice is a comparison of
//                                      sums of rounded terms, and fp32 would
//                                      turn near ties over)
// An expert whose logit is -inf (or NaN) is masked and never chosen; a token
// with fewer than top_k live experts gets id -1, weight 0, slot -1 there.
//   softmax  w = exp(l - max) / sum      over the chosen (renorm) or all experts
//   sigmoid  w = 1 / (1 + exp(-l)),      over the sum of the chosen if renorm
//                                        (0 if all of them are 0 in fp32)
// times `scale`.  With experts in groups only those of the token's best groups
// can be chosen: a group is rated by its experts' best key or by the sum of
// its two best (scores, in fp64).  The pairs (t, j) sorted by expert, then token, are the
// slots of the grouped products: offsets[e] .. offsets[e + 1) are expert e's
// and rows[slot] = t.
//
// Sorting without atomics that change the order: a workgroup takes 32
// tokens, and since a token names an expert at most once, expert e's tokens
// in the group are one 32-bit mask.  Bits are set with an OR (any order, the
// same word); a token's place among the group's is the number of set bits
// below its own, the group's count the number of all.  Above 32 tokens a
// second launch adds the groups before its own to each expert's offset.
//
// A row of 16 lanes takes a token of up to 256 experts and 16 choices, so a
// wave's step of the choice serves four tokens and needs no lane reads
// (8192 tokens, 8 of 128 experts: 11.6 us with a wave to a token, 5.5 with a
// row; then 4.1 for the places, which wait for two rounds of loads out of L2
// and two scans).  Both calls are bound by their chains of latencies: the
// 2.2 MB they move take under 1 us.
//
// Combination.  out[t][c] = bf16( sum_j w[t][j] * y[slots[t][j]][c] ), fp32,
// j ascending: one pass over the chosen rows, bound by HBM.  8 rows of 2048
// columns for each of 8192 tokens: 64.7 us with the rows' loads behind a test
// of each slot, 60.0 with eight of them leaving at once, 51.5 (5.8 TB/s) with
// non-temporal loads and stores, since no row is read twice.  Columns that are
// no multiple of 8 go one at a time: 1024 tokens, 8 rows of 2040 / 2047 / 2048,
// 7.9 / 11.1 / 7.6 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "fp8w.h"
#include "internal.hpp"

namespace fp8w {
namespace {

constexpr int kRouteTokens = 32;     // tokens of a workgroup: one mask word per expert
constexpr int kRouteThreads = 512;   // 8 waves, 4 tokens each
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kRouteMaxE = 1024;
constexpr int kRouteMaxK = 64;       // a lane holds one choice
constexpr float kLeastScore = -103.972077f;   // -150 ln 2: e^x rounds to zero in fp32 from here down
static_assert(kRouteMaxE == FP8W_MAX_EXPERTS && kRouteMaxK == FP8W_MAX_TOP_K, "what the entry points check");

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp_mov(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ float pick_max(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double pick_max(double a, double b) { return __builtin_fmax(a, b); }
template <int CTRL>
__device__ __forceinline__ int dpp_min(int v) {
  const int o = __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
  return v < o ? v : o;
}

// Reductions over L = 16 or 64 neighbouring lanes, the result in each of
// them: four steps within rows of 16, then the four rows' values by lane
// reads.
template <int L, typename T>
__device__ __forceinline__ T group_max(T v) {
  v = pick_max(v, dpp_mov<0xB1>(v));    // quad_perm [1,0,3,2]
  v = pick_max(v, dpp_mov<0x4E>(v));    // quad_perm [2,3,0,1]
  v = pick_max(v, dpp_mov<0x141>(v));   // row_half_mirror
  v = pick_max(v, dpp_mov<0x140>(v));   // row_mirror
  if constexpr (L == 16) return v;
  return pick_max(pick_max(lane_value(v, 0), lane_value(v, 16)), pick_max(lane_value(v, 32), lane_value(v, 48)));
}
template <int L, typename T>
__device__ __forceinline__ T group_total(T v) {
  v += dpp_mov<0xB1>(v);
  v += dpp_mov<0x4E>(v);
  v += dpp_mov<0x141>(v);
  v += dpp_mov<0x140>(v);
  if constexpr (L == 16) return v;
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
  v = dpp_min<0xB1>(v);
  v = dpp_min<0x4E>(v);
  v = dpp_min<0x141>(v);
  v = dpp_min<0x140>(v);
  if constexpr (L == 16) return v;
  const int a = min(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
  const int b = min(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48));
  return min(a, b);
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* slots;
  int32_t* rows;
  int32_t* offsets;
  uint8_t* counts;       // [groups][pad4(E)]: tokens of each group that chose e
  int64_t stride;        // logits row stride, elements
  float scale;
  int32_t tokens, experts, top_k, score, renorm;
  int32_t groups, top_groups, top2;   // groups 1: none
  int32_t log_lanes;                  // a group's lanes are 2^log_lanes
};

template <typename T>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  if constexpr (sizeof(T) == 4) return ld_global<float>(p, (size_t)at * 4);
  return bf16_lo(ld_global<uint16_t>(p, (size_t)at * 2));
}

// The experts' scores in fp64 (softmax: not yet divided by their sum; +inf is
// taken as 2^200, far above all others, so that it has a difference from itself
// and a score of 1).  Of few
// experts a lane by one copy of the exponential, with the registers moved on
// under it: a lone token's time is that of fetching the code.
template <int R>
__device__ __forceinline__ void scores(const RouteArgs& a, const float (&x)[R], float top, double (&score)[R]) {
  const double best = __builtin_fmin((double)top, 0x1p200);
  const auto of = [&](float v) {
    const double e = exp(a.score == 0 ? __builtin_fmin((double)v, 0x1p200) - best : -(double)v);
    return a.score == 0 ? e : 1.0 / (1.0 + e);
  };
  if constexpr (R > 4) {
#pragma unroll
    for (int r = 0; r < R; ++r) score[r] = of(x[r]);
    return;
  }
  float v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = x[r];
#pragma unroll 1
  for (int n = 0; n < R; ++n) {
    const double s = of(v[0]);
#pragma unroll
    for (int r = 0; r + 1 < R; ++r) {
      v[r] = v[r + 1];
      score[r] = score[r + 1];
    }
    score[R - 1] = s;
  }
}

// Shuts the groups that are not among the token's best: their experts' keys
// become -inf.  2^log_lanes neighbouring lanes hold a group's experts (lanes
// past the last group hold none), so a group's two best keys meet in steps of
// lane exchanges, and its rank is the number of groups that beat it.  The
// ratings are of the scores in fp64 where two keys are added, since sums of
// logits would be another order.  One token, 256 experts: 1.7 us (two best 3.2:
// the exponentials); through LDS exchanges alone 2.2 and 4.
template <typename Key, int L, int R>
__device__ __forceinline__ void shut_groups(const RouteArgs& a, const float (&x)[R], float top, Key (&key)[R]) {
  const int lane = threadIdx.x & (L - 1), mine = lane >> a.log_lanes;
  const double ninf = -(double)__builtin_inff();
  double first = ninf, second = ninf;
  const auto meet = [&](double f, double s) {
    second = pick_max(pick_max(second, s), first < f ? first : f);
    first = pick_max(first, f);
  };
  if (sizeof(Key) == 4 && a.top2) {
    double score[R];
    scores<R>(a, x, top, score);
#pragma unroll
    for (int r = 0; r < R; ++r) meet(x[r] > -__builtin_inff() ? score[r] : ninf, ninf);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) meet((double)key[r], ninf);
  }
  // Lanes that have met hold the same, so that a mirrored row or half of one
  // brings the other half's.
  if (a.log_lanes > 0) meet(dpp_mov<0xB1>(first), dpp_mov<0xB1>(second));
  if (a.log_lanes > 1) meet(dpp_mov<0x4E>(first), dpp_mov<0x4E>(second));
  if (a.log_lanes > 2) meet(dpp_mov<0x141>(first), dpp_mov<0x141>(second));
  if (a.log_lanes > 3) meet(dpp_mov<0x140>(first), dpp_mov<0x140>(second));
  for (int off = 16; off < 1 << a.log_lanes; off <<= 1) meet(__shfl_xor(first, off), __shfl_xor(second, off));
  const double rating = a.top2 && second > ninf ? first + second : first;
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    double other;
    if constexpr (L == kWave)
      other = lane_value(rating, g << a.log_lanes);
    else
      other = __shfl(rating, g << a.log_lanes, L);
    better += other > rating || (other == rating && g < mine) ? 1 : 0;
  }
  if (better >= a.top_groups) {
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = -(Key)__builtin_inff();
  }
}

// A token's choice by L lanes with R experts each (expert r * L + lane of
// the group of lanes; with groups of experts, a group's experts go round its own
// lanes): lane j ends with the j-th expert (-1: none) and its weight.  A step
// takes the largest key left, and among its equals the lowest expert.
template <typename T, typename Key, int L, int R, bool GROUPS>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int& my_id, float& my_w) {
  constexpr bool kBias = sizeof(Key) == 8;
  const int lane = threadIdx.x & (L - 1);
  const float ninf = -__builtin_inff();
  // past the experts there are, or past its group's: none
  const int size = GROUPS ? a.experts / a.groups : 0, part = GROUPS ? lane >> a.log_lanes : 0;
  const auto expert = [&](int r) {
    if (!GROUPS) return r * L + lane;
    const int in = (r << a.log_lanes) + (lane & ((1 << a.log_lanes) - 1));
    return part < a.groups && in < size ? part * size + in : kRouteMaxE;
  };
  float x[R], bias[kBias ? R : 1];
  Key key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = expert(r);
    const float v = load_logit<T>(a.logits, (int64_t)t * a.stride + (e < a.experts ? e : 0));
    x[r] = v == v && e < a.experts ? v : ninf;
    if constexpr (kBias) bias[r] = ld_global<float>(a.bias, (size_t)(e < a.experts ? e : 0) * 4);
  }
  float top = x[0];
#pragma unroll
  for (int r = 1; r < R; ++r) top = __builtin_fmaxf(top, x[r]);
  top = group_max<L>(top);
  float z = 0.0f;   // of all experts' terms
  if (a.score == 0 && !a.renorm) {
#pragma unroll
    for (int r = 0; r < R; ++r) z += x[r] > ninf ? expf(x[r] - top) : 0.0f;
    z = group_total<L>(z);
  }
  if constexpr (kBias) {
    scores<R>(a, x, top, key);
    if (a.score == 0) {
      double zd = 0.0;
#pragma unroll
      for (int r = 0; r < R; ++r) zd += x[r] > ninf ? key[r] : 0.0;
      zd = group_total<L>(zd);
#pragma unroll
      for (int r = 0; r < R; ++r) key[r] = key[r] / zd;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const double k = key[r] + (double)bias[r];
      key[r] = x[r] > ninf && k == k ? k : (double)ninf;
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = x[r];
  }
  if constexpr (GROUPS) shut_groups<Key, L, R>(a, x, top, key);

  my_id = -1;
  float my_x = ninf;
  for (int j = 0; j < a.top_k; ++j) {
    Key best = key[0];
#pragma unroll
    for (int r = 1; r < R; ++r) best = pick_max(best, key[r]);
    best = group_max<L>(best);
    const bool live = best > (Key)ninf;
    if (!__ballot(live)) break;   // no token of the wave has an expert left
    int first = kRouteMaxE;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) first = key[r] == best ? expert(r) : first;
    const int id = group_min<L>(first);
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = expert(r) == id ? (Key)ninf : key[r];
    if (live && lane == j) {
      my_id = id;
      if constexpr (!kBias) my_x = (float)best;
    }
  }

  const bool live = my_id >= 0;
  if constexpr (kBias) {
    if (live) my_x = load_logit<T>(a.logits, (int64_t)t * a.stride + my_id);
  }
  float w;
  if (a.score == 0) {
    // Of the chosen alone, their own largest: under a bias, or in a group that
    // is shut, the row's may not be among them, and terms taken from it could all be zero.
    if constexpr (kBias || GROUPS) {
      if (a.renorm) top = group_max<L>(my_x);
    }
    w = live ? expf(my_x - top) : 0.0f;
    if (a.renorm) z = group_total<L>(w);
    w = live ? w / z : 0.0f;
  } else {
    // e^x / (1 + e^x) below zero: 1 + e^-x overflows where the score is still
    // a number.  To be divided by their sum the chosen scores are taken times
    // e^-best, since most of an fp32's bits are gone before the ratio is.
    const float best = a.renorm ? group_max<L>(my_x) : 0.0f;
    const float t = expf(-__builtin_fabsf(my_x));
    const float up = a.renorm && best < 0.0f ? expf(my_x - best) : my_x < 0.0f ? t : 1.0f;
    w = live ? up / (1.0f + t) : 0.0f;
    if (a.renorm) {
      const float sum = group_total<L>(w);
      w = live && best > kLeastScore ? w / sum : 0.0f;   // every chosen score is zero in fp32: no weight
    }
  }
  my_w = w * a.scale;
}

// Exclusive prefix sums of count[0..E) in place, E <= 1024, by the whole
// workgroup (512 threads, two experts each); returns the total.
__device__ __forceinline__ int scan_experts(int* count, int experts, int* wave_sums) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
  const int e0 = 2 * tid, e1 = 2 * tid + 1;
  const int c0 = e0 < experts ? count[e0] : 0, c1 = e1 < experts ? count[e1] : 0;
  int s = c0 + c1;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int up = __shfl_up(s, off);
    if (lane >= off) s += up;
  }
  if (lane == kWave - 1) wave_sums[w] = s;
  __syncthreads();
  int before = s - c0 - c1, total = 0;
#pragma unroll
  for (int i = 0; i < kRouteWaves; ++i) {
    if (i < w) before += wave_sums[i];
    total += wave_sums[i];
  }
  if (e0 < experts) count[e0] = before;
  if (e1 < experts) count[e1] = before + c0;
  __syncthreads();
  return total;
}

// The choice of 32 tokens, and their places among them.  ONE: this group is
// the whole call, so the map is finished here.
template <typename T, typename Key, int L, int R, bool GROUPS, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void k_route_choose(RouteArgs a) {
  __shared__ uint32_t mask[kRouteMaxE];
  __shared__ int16_t chosen_id[kRouteTokens * kRouteMaxK];
  __shared__ int count[ONE ? kRouteMaxE : 1];
  __shared__ int wave_sums[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & (L - 1);
  const int t0 = blockIdx.x * kRouteTokens;
  const int nt = min(kRouteTokens, a.tokens - t0);
  for (int e = tid; e < a.experts; e += kRouteThreads) mask[e] = 0;
  __syncthreads();
#pragma unroll 1
  for (int first = 0; first < nt; first += kRouteThreads / L) {
    const int i = first + tid / L;
    if (L == kWave ? i >= nt : i - i % (kWave / L) >= nt) break;   // a wave's lanes stay together
    int id;
    float w;
    route_token<T, Key, L, R, GROUPS>(a, t0 + min(i, nt - 1), id, w);
    if (i < nt && lane < a.top_k) {
      const int64_t at = (int64_t)(t0 + i) * a.top_k + lane;
      a.ids[at] = id;
      a.weights[at] = w;
      chosen_id[i * kRouteMaxK + lane] = (int16_t)id;
      if (id >= 0) atomicOr(&mask[id], 1u << i);
    }
  }
  __syncthreads();
  if constexpr (ONE) {
    for (int e = tid; e < a.experts; e += kRouteThreads) count[e] = __popc(mask[e]);
    __syncthreads();
    const int total = scan_experts(count, a.experts, wave_sums);
    for (int e = tid; e < a.experts; e += kRouteThreads) a.offsets[e] = count[e];
    if (tid == 0) a.offsets[a.experts] = total;
    for (int i = total + tid; i < a.tokens * a.top_k; i += kRouteThreads) a.rows[i] = -1;
  } else {
    const int pad = (a.experts + 3) & ~3;
    for (int e = tid; e < pad; e += kRouteThreads)
      a.counts[(size_t)blockIdx.x * pad + e] = e < a.experts ? (uint8_t)__popc(mask[e]) : 0;
  }
  for (int i = tid; i < nt * a.top_k; i += kRouteThreads) {
    const int t = i / a.top_k, j = i - t * a.top_k;
    const int id = chosen_id[t * kRouteMaxK + j];
    int slot = -1;
    if (id >= 0) {
      slot = __popc(mask[id] & ((1u << t) - 1u));
      if constexpr (ONE) {
        slot += count[id];
        a.rows[slot] = t0 + t;
      }
    }
    a.slots[(int64_t)t0 * a.top_k + i] = slot;
  }
}

// Group b's tokens from their places in the group to their slots: expert e's
// base is its offset plus the counts of the groups before b.  Every group
// sums the whole count table (a byte per group and expert, out of L2), which
// grows with the tokens' square: both launches, 8 of 128 experts, 10.3 us for
// 8192 tokens, 32 us for 32768, 257 us for 131072 (8 of 256: 12.5, 50, 487).
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a, int groups) {
  __shared__ int all[kRouteMaxE];
  __shared__ int before[kRouteMaxE];
  __shared__ int wave_sums[kRouteWaves];
  const int tid = threadIdx.x, b = blockIdx.x;
  const int pad = (a.experts + 3) & ~3, cols = pad / 4;   // cols <= 256: two rows at least
  for (int e = tid; e < pad; e += kRouteThreads) all[e] = before[e] = 0;
  __syncthreads();
  const int per = kRouteThreads / cols;
  const int col = tid % cols, part = tid / cols;
  if (part < per) {
    int s[4] = {0, 0, 0, 0}, f[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int g = part; g < groups; g += per) {
      const uint32_t v = ld_global<uint32_t>(a.counts, (size_t)g * pad + 4 * col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (v >> (8 * i)) & 0xFF;
        s[i] += c;
        f[i] += g < b ? c : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // integer sums: the same in any order
      atomicAdd(&all[4 * col + i], s[i]);
      atomicAdd(&before[4 * col + i], f[i]);
    }
  }
  __syncthreads();
  const int total = scan_experts(all, a.experts, wave_sums);
  if (b == 0) {
    for (int e = tid; e < a.experts; e += kRouteThreads) a.offsets[e] = all[e];
    if (tid == 0) a.offsets[a.experts] = total;
  }
  const int64_t pairs = (int64_t)a.tokens * a.top_k;
  for (int64_t i = total + (int64_t)b * kRouteThreads + tid; i < pairs; i += (int64_t)groups * kRouteThreads)
    a.rows[i] = -1;
  const int t0 = b * kRouteTokens;
  const int n = min(kRouteTokens, a.tokens - t0) * a.top_k;
  for (int i = tid; i < n; i += kRouteThreads) {
    const int64_t at = (int64_t)t0 * a.top_k + i;
    const int place = a.slots[at];
    if (place < 0) continue;
    const int id = a.ids[at];
    const int slot = all[id] + before[id] + place;
    a.slots[at] = slot;
    a.rows[slot] = t0 + i / a.top_k;
  }
}

// No token: every expert's range is empty.
__global__ void k_route_empty(int32_t* offsets, int experts) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e <= experts) offsets[e] = 0;
}

template <typename T, typename Key, int L, int R, bool GROUPS = false>
hipError_t route_launch(const RouteArgs& a, hipStream_t stream) {
  const int groups = (a.tokens + kRouteTokens - 1) / kRouteTokens;
  if (groups == 1) {
    k_route_choose<T, Key, L, R, GROUPS, true><<<1, kRouteThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  k_route_choose<T, Key, L, R, GROUPS, false><<<groups, kRouteThreads, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_route_place<<<groups, kRouteThreads, 0, stream>>>(a, groups);
  return hipGetLastError();
}

// A row of 16 lanes to a token where a lane can hold its experts and one
// choice of it: four tokens share a wave's instructions, and no value has to
// cross rows.
template <typename T, typename Key>
hipError_t route_by_experts(RouteArgs a, hipStream_t stream) {
  if (a.groups > 1) {
    // Lanes of a group: as many as 16 or 64 lanes have for the next power of
    // two groups, and enough registers for its experts.
    int parts = 2;
    while (parts < a.groups) parts *= 2;
    const int size = a.experts / a.groups;
    const auto lanes = [&](int l) {
      a.log_lanes = 0;
      while (parts << (a.log_lanes + 1) <= l) ++a.log_lanes;
      return parts <= l ? (size + (1 << a.log_lanes) - 1) >> a.log_lanes : kRouteMaxE;   // experts of a lane
    };
    if (a.top_k <= 16 && lanes(16) <= 16) return route_launch<T, Key, 16, 16, true>(a, stream);
    if (lanes(64) <= 8) return route_launch<T, Key, 64, 8, true>(a, stream);
    // Up to 1024 / groups over 64 / parts >= 32 / groups lanes.  32 experts a lane
    // spill (with a bias 114 registers): 8 of 1024 experts in 16 groups 51-61 us
    // without a bias and 107-156 with one for 32 ... 4096 tokens; 512 experts in 8
    // groups, the form above, 22-27 and 32-38.
    return route_launch<T, Key, 64, 32, true>(a, stream);
  }
  if (a.top_k <= 16) {
    if (a.experts <= 64) return route_launch<T, Key, 16, 4>(a, stream);
    if (a.experts <= 128) return route_launch<T, Key, 16, 8>(a, stream);
    if (a.experts <= 256) return route_launch<T, Key, 16, 16>(a, stream);
  }
  if (a.experts <= 256) return route_launch<T, Key, 64, 4>(a, stream);
  return route_launch<T, Key, 64, 16>(a, stream);
}

// out = sum of a token's chosen rows: a wave takes 64 * VEC columns of one
// token.  Its lanes hold the token's slots and weights, and the rows' loads
// leave eight at a time.
template <int VEC>
struct CombineSum {
  const uint16_t* y;
  int64_t slot_rows;
  int n, c, slot;      // this lane's column, and slot `lane`
  float weight;
  float acc[VEC];

  template <int N>
  __device__ __forceinline__ void rows(int j) {
    uint4 v[N];
    float w[N];
    bool valid[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = __builtin_amdgcn_readlane(slot, j + i);
      valid[i] = s >= 0 && s < slot_rows;
      const size_t from = ((size_t)(valid[i] ? s : 0) * n + c) * 2;   // row 0 is there: checked by the caller
      if constexpr (VEC == 8)
        v[i] = ld_stream_u4(y, from);
      else
        v[i].x = ld_global<uint16_t>(y, from);
      w[i] = valid[i] ? lane_value(weight, j + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t d[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int q = 0; q < (VEC + 1) / 2; ++q) {
        const uint32_t pair = valid[i] ? d[q] : 0;
        acc[2 * q] = __builtin_fmaf(w[i], bf16_lo(pair), acc[2 * q]);
        if constexpr (VEC > 1) acc[2 * q + 1] = __builtin_fmaf(w[i], bf16_hi(pair), acc[2 * q + 1]);
      }
    }
  }
};

template <int VEC>
__global__ __launch_bounds__(256) void k_combine(const uint16_t* y, int64_t slot_rows, const float* weights,
                                                 const int32_t* slots, uint32_t pieces, uint32_t per_token, int top_k,
                                                 int n, uint16_t* out) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint32_t piece = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + threadIdx.x / kWave);
  if (piece >= pieces) return;
  const uint32_t t = piece / per_token;
  const uint32_t c = ((piece - t * per_token) * kWave + lane) * VEC;   // may pass n, and 2^31 with it
  const bool inside = c < (uint32_t)n;
  CombineSum<VEC> sum{y, slot_rows, n, inside ? (int)c : 0, -1, 0.0f, {}};
  if (lane < top_k) {
    sum.slot = ld_global<int32_t>(slots, ((size_t)t * top_k + lane) * 4);
    sum.weight = ld_global<float>(weights, ((size_t)t * top_k + lane) * 4);
  }
  if (slot_rows > 0) {
    int j = 0;
    for (; j + 8 <= top_k; j += 8) sum.template rows<8>(j);
    if (j + 4 <= top_k) {
      sum.template rows<4>(j);
      j += 4;
    }
    for (; j < top_k; ++j) sum.template rows<1>(j);
  }
  if (!inside) return;
  const size_t to = ((size_t)t * n + c) * 2;
  if constexpr (VEC == 8) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_pair(sum.acc[2 * i], sum.acc[2 * i + 1]);
    st_stream_u4(out, to, v);
  } else {
    st_global<uint16_t>(out, to, (uint16_t)f32_to_bf16_rne(sum.acc[0]));
  }
}

}  // namespace

int64_t route_workspace_bytes(int64_t tokens, int64_t experts) {
  if (tokens <= kRouteTokens) return 0;
  return (tokens + kRouteTokens - 1) / kRouteTokens * ((experts + 3) & ~(int64_t)3);
}

hipError_t launch_route_experts(const RouteCall& c, hipStream_t stream) {
  if (c.tokens == 0) {
    k_route_empty<<<(c.experts + 256) / 256, 256, 0, stream>>>(c.offsets, c.experts);
    return hipGetLastError();
  }
  const RouteArgs a{c.logits, c.bias, c.ids, c.weights, c.slots, c.rows, c.offsets, static_cast<uint8_t*>(c.workspace),
                    c.stride, c.scale, c.tokens, c.experts, c.top_k, c.score, c.renorm, c.groups, c.top_groups,
                    c.group_top2, 0};
  if (c.f32) return c.bias ? route_by_experts<float, double>(a, stream) : route_by_experts<float, float>(a, stream);
  return c.bias ? route_by_experts<uint16_t, double>(a, stream) : route_by_experts<uint16_t, float>(a, stream);
}

int64_t combine_blocks(int64_t tokens, int64_t n, bool vec) {
  const int64_t columns = kWave * (vec ? 8 : 1);
  return (tokens * ((n + columns - 1) / columns) + 3) / 4;
}

hipError_t launch_combine_experts(const uint16_t* y, int64_t slot_rows, const float* weights, const int32_t* slots,
                                  int64_t tokens, int64_t top_k, int64_t n, uint16_t* out, bool vec,
                                  hipStream_t stream) {
  const unsigned blocks = (unsigned)combine_blocks(tokens, n, vec);
  const int64_t columns = kWave * (vec ? 8 : 1), per_token = (n + columns - 1) / columns;
  const uint32_t pieces = (uint32_t)(tokens * per_token);
  if (vec)
    k_combine<8><<<blocks, 256, 0, stream>>>(y, slot_rows, weights, slots, pieces, (uint32_t)per_token, (int)top_k,
                                             (int)n, out);
  else
    k_combine<1><<<blocks, 256, 0, stream>>>(y, slot_rows, weights, slots, pieces, (uint32_t)per_token, (int)top_k,
                                             (int)n, out);
  return hipGetLastError();
}

}  // namespace fp8w
