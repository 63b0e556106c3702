// logprobs.hip -- log probabilities of given tokens, entropy and the top
// alternatives of rows of logits, in one pass over the row.
//
// With m = max x, z = sum 2^((x - m) log2 e) and u = sum of the same terms
// times their exponents (x - m) log2 e,
//   log p(i) = (x_i - m) - ln z,      entropy = ln z - ln 2 * u / z.
// Each thread keeps (m, z, u) of what it has read and moves them to a new
// maximum once per 16 values; u is taken relative to m, so logits far from
// zero lose nothing.  A masked logit (-inf) has its exponent clamped at
// -300, where the term is zero, so 0 * inf never appears.
//
// Top alternatives ride on the same pass.  A value and its place make one
// 64-bit key (the value's ordered bits, then the complement of the place):
// larger keys are larger values, lower places first among equals, and no
// two are equal, so any correct selection gives the same answer.  Each wave
// lists the keys above a threshold that is never above the top-th key of the
// row: with w waves, every wave publishes its r-th largest value so far, r =
// ceil(top / w), and at least `top` values reach the ceil(top / r)-th largest
// of those.  It follows the row closely (5 of 152 k values: 7 to 20 reach it)
// and costs a wave a few lane maxima when it finds a larger value.  (Larger r
// bounds more tightly but takes longer to find: r = ceil(top / 5), twenty of
// 152 k, 2048 rows, 149 us against 142; the smallest of the published values,
// five, 125 us against 123, one, 127 against 118.)  A wave looks at single
// values only where a lane's maximum reaches the threshold: the values of
// four such lanes at a time go through LDS to one lane each, so that the wave
// tests 64 values of interest at once and a step without any pays one
// comparison a lane.  A list that fills up all the same (ties, masks) is cut
// to its largest keys, which gives a second threshold.
//
// Rows are cut into segments where there are too few of them to fill the
// chip, and a second launch joins the segments.
//
// Measured, vocabulary 151936, bf16: 2048 rows 106 us without alternatives
// (5.9 TB/s, which is what one pass of loads reaches), 118 with one, 123 with
// five (5.1), 142 with twenty; 4 rows 6.8, 10.4, 11.3 and 13.7 us, of which 6
// are the two launches and the chain of one load, one join.  1024 rows of
// fp32: 100 us, and 106 with five.  Without alternatives bound by HBM, with
// them by the VALU: 12 instructions a value, 8 of them for the statistics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "fp8w.h"
#include "internal.hpp"

namespace fp8w {
namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWaves = kLpThreads / kWave;
constexpr int kLpBlock = 1024;        // values of one wave step: 16 per lane
constexpr int kLpMaxTop = 64;
static_assert(kLpMaxTop == FP8W_MAX_TOP, "what the entry points check");
constexpr int kLpCap = 256;           // keys a wave's list holds (4 per lane)
constexpr int kLpMaxSegs = 64;
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMinExp = -300.0f;    // 2^-300 is zero in fp32

// Value bits whose unsigned order is the values' order (-0 equal to +0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (uint32_t)(((int32_t)b >> 31) | 0x80000000);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint64_t kFirstKey = (uint64_t)(0x007FFFFFu + 1) << 32;   // above every key of -inf

struct LpStats {
  float m, z, u;
};

__device__ __forceinline__ LpStats lp_join(LpStats a, LpStats b) {
  const float m = __builtin_elementwise_maximum(a.m, b.m);   // NaN stays
  const float da = __builtin_fmaxf((a.m - m) * kLog2E, kMinExp), db = __builtin_fmaxf((b.m - m) * kLog2E, kMinExp);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  return LpStats{m, a.z * fa + b.z * fb, fa * __builtin_fmaf(da, a.z, a.u) + fb * __builtin_fmaf(db, b.z, b.u)};
}

struct LpArgs {
  const void* logits;
  const int32_t* targets;    // may be null (with logprob)
  float* logprob;            // may be null
  float* entropy;            // may be null
  int32_t* top_ids;
  float* top_logprobs;
  LpStats* seg_stats;        // [tokens][segs], segs > 1
  uint64_t* seg_keys;        // [tokens][segs][top]
  int64_t stride;            // elements
  int32_t tokens, vocab, top, segs, seg_values;
};

// What a row's statistics give; the row holding NaN or +inf has no
// distribution and gets NaN, the row masked throughout log p = -inf and
// entropy 0.
struct LpRow {
  float m, ln_z;
  bool bad, empty;
  __device__ __forceinline__ explicit LpRow(const LpStats& s) {
    m = s.m;
    bad = !(s.m < __builtin_inff());
    empty = s.m == -__builtin_inff();
    ln_z = __builtin_amdgcn_logf(s.z) * kLn2;
  }
  __device__ __forceinline__ float logp(float x) const {
    if (bad) return __builtin_nanf("");
    if (empty) return -__builtin_inff();
    return (x - m) - ln_z;
  }
};

template <typename T>
__device__ __forceinline__ float lp_load(const void* p, int64_t at) {
  if constexpr (sizeof(T) == 4) return ld_global<float>(p, (size_t)at * 4);
  return bf16_lo(ld_global<uint16_t>(p, (size_t)at * 2));
}

// The given token's logit (any value if there is none, or it is outside).
template <typename T>
__device__ __forceinline__ float lp_target(const LpArgs& a, int t) {
  if (!a.logprob) return 0.0f;
  const int id = a.targets[t];
  return id >= 0 && id < a.vocab ? lp_load<T>(a.logits, (int64_t)t * a.stride + id) : __builtin_nanf("");
}

// How many of the keys (LDS) are larger.
__device__ __forceinline__ int lp_rank(const uint64_t* keys, int count, uint64_t key) {
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < count; ++j) rank += keys[j] > key ? 1 : 0;
  return rank;
}

// Target, entropy and top alternatives of row t from its statistics, its
// given token's logit (thread 0) and the `count` keys of its candidates
// (every live logit, if fewer than top), by the whole workgroup.
__device__ __forceinline__ void lp_finish(const LpArgs& a, int t, const LpStats& s, float target, const uint64_t* keys,
                                          int count) {
  const LpRow row(s);
  const int tid = threadIdx.x;
  if (tid == 0) {
    if (a.entropy)
      a.entropy[t] = row.bad ? __builtin_nanf("") : row.empty ? 0.0f : row.ln_z - kLn2 * (s.u / s.z);
    if (a.logprob) a.logprob[t] = target == target ? row.logp(target) : __builtin_nanf("");
  }
  for (int i = tid; i < count; i += blockDim.x) {
    const uint64_t key = keys[i];
    const int rank = lp_rank(keys, count, key);
    if (rank < a.top) {
      const int64_t at = (int64_t)t * a.top + rank;
      a.top_ids[at] = (int32_t)~(uint32_t)key;
      a.top_logprobs[at] = row.logp(unordered((uint32_t)(key >> 32)));
    }
  }
  // Fewer live logits than alternatives: the rest are masked tokens, lowest first.
  if (count < a.top && tid == 0) {
    int filled = count;
    for (int id = 0; filled < a.top; ++id) {
      bool live = false;
      for (int j = 0; j < count; ++j) live |= (int32_t)~(uint32_t)keys[j] == id;
      if (!live) {
        const int64_t at = (int64_t)t * a.top + filled++;
        a.top_ids[at] = id;
        a.top_logprobs[at] = row.logp(-__builtin_inff());
      }
    }
  }
}

// The largest of a lane's values where some are NaN, as ordered bits (rows
// with NaN still rank the others).
__device__ __forceinline__ uint32_t lp_nan_max(const float (&x)[16]) {
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t o = x[i] == x[i] ? ordered(x[i]) : 0;
    best = o > best ? o : best;
  }
  return best;
}

// A threshold that at least `want` of the wave's keys reach (0 if there are
// fewer), built from the top bit down until no more than `enough` reach it.
// Keys: PER a lane.
template <typename K, int PER>
__device__ __forceinline__ K wave_threshold(const K (&key)[PER], int want, int enough) {
  K thr = 0;
  for (int bit = 8 * (int)sizeof(K) - 1; bit >= 0; --bit) {
    const K cand = thr | ((K)1 << bit);
    int reach = 0;
#pragma unroll
    for (int r = 0; r < PER; ++r) reach += __builtin_popcountll(__ballot(key[r] >= cand));
    if (reach >= want) {
      thr = cand;
      if (reach <= enough) break;
    }
  }
  return thr;
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ uint32_t pick_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t pick_larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Largest value of the wave, in every lane.
__device__ __forceinline__ uint32_t wave_largest(uint32_t v) {
  v = pick_max(v, lane_move<0xB1>(v));    // quad_perm [1,0,3,2]
  v = pick_max(v, lane_move<0x4E>(v));    // quad_perm [2,3,0,1]
  v = pick_max(v, lane_move<0x141>(v));   // row_half_mirror
  v = pick_max(v, lane_move<0x140>(v));   // row_mirror
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return pick_max(pick_max(a, b), pick_max(c, d));
}

// The largest values that a wave has seen, the r-th in lane r.
struct LpBest {
  uint32_t mine = 0;

  // Takes in a value a lane (0: none); returns the `want`-th largest (0: not
  // that many yet).
  __device__ __forceinline__ uint32_t take(uint32_t v, int want) {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t kept = 0, last = 0;
    for (int r = 0; r < want; ++r) {
      last = wave_largest(pick_max(v, mine));
      if (last == 0) break;
      const int l = __builtin_ctzll(__ballot(pick_max(v, mine) == last));
      if (lane == l) {   // one of the lane's two is used up
        if (v == last)
          v = 0;
        else
          mine = 0;
      }
      if (lane == r) kept = last;
    }
    mine = kept;
    return last;
  }
};

// The m-th largest of what the waves have published, as a threshold: lane l
// compares wave l % 8's value with wave l / 8's.
__device__ __forceinline__ uint64_t published_bound(const uint32_t* published, int m) {
  static_assert(kLpWaves == 8, "a pair of waves a lane");
  int lane = threadIdx.x & (kWave - 1);
  asm volatile("" : "+v"(lane)::"memory");   // what depends on it is not kept in registers from call to call
  const volatile uint32_t* p = published;
  const uint32_t mine = p[lane & 7], other = p[lane >> 3];
  const uint64_t reach = __ballot(other >= mine) & 0x0101010101010101ull << (lane & 7);
  uint32_t v = __builtin_popcountll(reach) >= m ? mine : 0;
  v = pick_max(v, lane_move<0xB1>(v));
  v = pick_max(v, lane_move<0x4E>(v));
  v = pick_max(v, lane_move<0x141>(v));
  return (uint64_t)__builtin_amdgcn_readfirstlane(v) << 32;
}

// A wave's list of candidates.
struct LpList {
  uint64_t* keys;              // LDS, kLpCap words of this wave
  uint64_t* shared_tau;        // LDS, of the workgroup
  uint64_t tau;                // keys below it cannot be in the answer
  int count;

  // Cut the list down to its largest keys: `top` at least, `enough` at most.
  __device__ __forceinline__ void cut(int top, int enough) {
    const int lane = threadIdx.x & (kWave - 1);
    uint64_t k[kLpCap / kWave];
#pragma unroll
    for (int r = 0; r < kLpCap / kWave; ++r) k[r] = r * kWave + lane < count ? keys[r * kWave + lane] : 0;
    const uint64_t thr = wave_threshold(k, top, enough);
    keep(k, thr);
    raise(thr);
  }
  // Drop the keys below the threshold.
  __device__ __forceinline__ void sweep() {
    const int lane = threadIdx.x & (kWave - 1);
    uint64_t k[kLpCap / kWave];
#pragma unroll
    for (int r = 0; r < kLpCap / kWave; ++r) k[r] = r * kWave + lane < count ? keys[r * kWave + lane] : 0;
    keep(k, tau);
  }
  __device__ __forceinline__ void keep(const uint64_t (&k)[kLpCap / kWave], uint64_t thr) {
    const int lane = threadIdx.x & (kWave - 1);
    int kept = 0;
#pragma unroll
    for (int r = 0; r < kLpCap / kWave; ++r) {
      const bool stay = k[r] >= thr && k[r] != 0;
      const uint64_t who = __ballot(stay);
      if (stay) keys[kept + __builtin_popcountll(who & ((1ull << lane) - 1))] = k[r];
      kept += __builtin_popcountll(who);
    }
    __builtin_amdgcn_wave_barrier();
    count = kept;
  }
  __device__ __forceinline__ void raise(uint64_t t) {
    if (t > tau) {
      tau = t;
      if ((threadIdx.x & (kWave - 1)) == 0) atomicMax(reinterpret_cast<unsigned long long*>(shared_tau), (unsigned long long)t);
    }
  }
  __device__ __forceinline__ void add(bool want, uint64_t key, int top) {
    const uint64_t who = __ballot(want);
    if (!who) return;
    if (count > kLpCap - kWave) sweep();
    if (count > kLpCap - kWave) {
      cut(top, kLpCap / 4 > top + 8 ? kLpCap / 4 : top + 8);
      want = want && key >= tau;
    }
    const uint64_t now = __ballot(want);
    const int lane = threadIdx.x & (kWave - 1);
    if (want) keys[count + __builtin_popcountll(now & ((1ull << lane) - 1))] = key;
    __builtin_amdgcn_wave_barrier();
    count += __builtin_popcountll(now);
  }
};

// One workgroup per row segment.  With alternatives six waves a SIMD: asked
// for eight, the lists' state spills to scratch (five of 152 k, 2048 rows:
// 141 us against 132; fp32, 1024 rows: 168 against 108).
template <typename T, bool TOP>
__global__ __launch_bounds__(kLpThreads, TOP ? 6 : 8) void k_logprobs(LpArgs a) {
  constexpr int kVec = 16 / sizeof(T);       // values of one 16-byte load
  constexpr int kLoads = 16 / kVec;
  __shared__ uint64_t lists[TOP ? kLpWaves * kLpCap : 1];
  __shared__ __attribute__((aligned(16))) float picked[TOP ? kLpWaves : 1][kWave];   // 16 values of four lanes
  __shared__ int picked_lane[TOP ? kLpWaves : 1][4];
  __shared__ uint64_t shared_tau;
  __shared__ uint32_t published[kLpWaves];
  __shared__ LpStats wave_stats[kLpWaves];
  __shared__ int kept;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int t = blockIdx.x / a.segs, seg = blockIdx.x - t * a.segs;
  if (tid == 0) {
    shared_tau = kFirstKey;
    kept = 0;
  }

  // Places are counted from the 16-byte boundary at or below the row's
  // start, so that every load of whole 16 bytes is aligned; `skew` values
  // there belong to what lies before the row and are never read.
  const char* row = static_cast<const char*>(a.logits) + (size_t)t * a.stride * sizeof(T);
  const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const char* base = row - skew * sizeof(T);
  const int64_t end = (int64_t)a.vocab + skew;
  const int64_t lo = (int64_t)seg * a.seg_values;
  const int64_t hi = lo + a.seg_values < end && seg + 1 < a.segs ? lo + a.seg_values : end;

  LpStats s{-__builtin_inff(), 0.0f, 0.0f};
  LpList list{lists + wave * kLpCap, &shared_tau, kFirstKey, 0};
  // each wave that has values publishes its `want`-th largest, and m of them
  // bound the answer
  const int64_t blocks = (hi - lo + kLpBlock - 1) / kLpBlock;
  const int active = blocks < kLpWaves ? (int)blocks : kLpWaves;
  const int want = TOP ? (a.top + active - 1) / active : 1, m = (a.top + want - 1) / want;
  LpBest best;
  const auto lane_largest = [&](const float (&x)[16], float top) __attribute__((always_inline)) {
    const uint32_t o = top == top ? ordered(top) : lp_nan_max(x);
    return o > (uint32_t)((kFirstKey >> 32) - 1) ? o : 0;   // 0: nothing live
  };
  const auto largest = [](const float (&x)[16]) __attribute__((always_inline)) {   // NaN if there is one
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = __builtin_elementwise_maximum(top, x[i]);
    return top;
  };
  // 1024 values from `at` on, 16 a lane: load v holds those of place (v * 64 + lane) * kVec.
  const auto consume = [&](const float (&x)[16], int64_t at) __attribute__((always_inline)) {
    uint64_t cut = 0;
    if constexpr (TOP) cut = *(volatile uint64_t*)&shared_tau;   // read ahead of its use
    const float top = largest(x);
    const float mx = __builtin_elementwise_maximum(s.m, top);
    const float down = __builtin_fmaxf((s.m - mx) * kLog2E, kMinExp), f = __builtin_amdgcn_exp2f(down);
    float z = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float e = __builtin_fmaxf((x[i] - mx) * kLog2E, kMinExp);   // the difference first: m log2 e can overflow
      const float p = __builtin_amdgcn_exp2f(e);
      z += p;
      u = __builtin_fmaf(e, p, u);
    }
    s = LpStats{mx, __builtin_fmaf(s.z, f, z), __builtin_fmaf(f, __builtin_fmaf(down, s.z, s.u), u)};

    if constexpr (TOP) {
      cut = uniform64(cut);
      if (cut > list.tau) list.tau = cut;
      // not below the threshold's value (NaN too: there may be others beside it)
      uint64_t hit = __ballot(!(top < unordered((uint32_t)(list.tau >> 32))));
      if (hit) {
        const uint32_t mine = lane_largest(x, top);
        hit = __ballot(mine >= (uint32_t)(list.tau >> 32));
        const uint32_t old = published[wave];
        if (__ballot(mine > old)) {   // a lane's largest stands for all its values: a bound either way
          const uint32_t now = best.take(mine, want);
          if (now > old) {
            if (lane == 0) published[wave] = now;
            list.raise(published_bound(published, m));
          }
        }
      }
      while (hit) {
        const int r = __builtin_popcountll(hit & ((1ull << lane) - 1));
        if ((hit >> lane & 1) && r < 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(&picked[wave][16 * r + 4 * i]) = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
          picked_lane[wave][r] = lane;
        }
        const int n = __builtin_popcountll(hit);
        asm volatile("" ::: "memory");
        const float v = picked[wave][lane];
        const int from = picked_lane[wave][lane >> 4], i = lane & 15;
        asm volatile("" ::: "memory");
        const int64_t p = at + ((i / kVec) * kWave + from) * kVec + i % kVec;
        const uint64_t key = ((uint64_t)ordered(v) << 32) | (uint32_t)~(uint32_t)(p - skew);
        list.add(lane >> 4 < n && v == v && key >= list.tau, key, a.top);
#pragma unroll
        for (int j = 0; j < 4; ++j) hit &= hit - 1;
      }
    }
  };

  // Whole blocks by 16-byte loads, the next one's on their way while one is
  // consumed; the row's edges value by value.
  constexpr int kStride = kLpWaves * kLpBlock;
  const auto whole = [&](int64_t at) { return at >= skew && at + kLpBlock <= hi; };
  const int64_t mine0 = lo + wave * kLpBlock;
  const int64_t safe = whole(mine0) ? mine0 : mine0 + kStride;   // a whole block of this wave, if it has one
  uint4 raw[kLoads];
  const auto request = [&](int64_t at) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < kLoads; ++v) raw[v] = ld_stream_u4(base, (size_t)(at + (v * kWave + lane) * kVec) * sizeof(T));
  };
  const auto widened = [&](float (&x)[16]) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < kLoads; ++v) {
      const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          x[v * kVec + 2 * i] = bf16_lo(w[i]);
          x[v * kVec + 2 * i + 1] = bf16_hi(w[i]);
        } else {
          x[v * kVec + i] = __uint_as_float(w[i]);
        }
      }
    }
  };
  const auto edge = [&](float (&x)[16], int64_t at) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < kLoads; ++v)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t p = at + (v * kWave + lane) * kVec + i;
        x[v * kVec + i] = p >= skew && p < hi ? lp_load<T>(base, p) : -__builtin_inff();
      }
  };
  const bool has_whole = whole(safe);
  if (has_whole) request(safe);
  if constexpr (TOP) {
    // every wave's first values give the first threshold
    uint32_t now = 0;   // reaches no bound
    if (wave < blocks) {
      float x[16];
      if (has_whole)
        widened(x);
      else
        edge(x, mine0);
      LpBest first;
      now = first.take(lane_largest(x, largest(x)), want);
    }
    if (lane == 0) published[wave] = now;
    __syncthreads();
    list.raise(published_bound(published, m));
  }
#pragma unroll 1
  for (int64_t at = safe; has_whole && whole(at); at += kStride) {
    float x[16];
    widened(x);
    request(whole(at + kStride) ? at + kStride : at);   // the last round asks for its block again: no branch
    consume(x, at);
  }
#pragma unroll 1
  for (int64_t at = mine0; at < hi; at += kStride) {
    if (whole(at)) {   // on to the edge behind the whole blocks
      at += (hi - kLpBlock - at) / kStride * kStride;
      continue;
    }
    float x[16];
    edge(x, at);
    consume(x, at);
  }

  // The given token's logit is on its way while the statistics are joined:
  // the wave's, then the workgroup's.
  const float target = tid == 0 && a.segs == 1 ? lp_target<T>(a, t) : 0.0f;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const LpStats o{__shfl_xor(s.m, off), __shfl_xor(s.z, off), __shfl_xor(s.u, off)};
    s = lp_join(s, o);
  }
  if (lane == 0) wave_stats[wave] = s;
  __syncthreads();
  if constexpr (TOP) {   // the final threshold, the same in every wave
    list.tau = pick_larger(shared_tau, published_bound(published, m));
    list.sweep();
    if (list.count > kWave) list.cut(a.top, kWave);   // at most 64: one key a lane
  }
  s = wave_stats[0];
#pragma unroll
  for (int w = 1; w < kLpWaves; ++w) s = lp_join(s, wave_stats[w]);
  int count = 0;
  uint64_t* joined = lists;
  if constexpr (TOP) {
    const uint64_t key = lane < list.count ? list.keys[lane] : 0;
    __syncthreads();
    const bool keep = key >= shared_tau && key != 0;
    if (keep) joined[atomicAdd(&kept, 1)] = key;
    __syncthreads();
    count = kept;
  }
  if (a.segs == 1) {
    lp_finish(a, t, s, target, joined, count);
    return;
  }
  const size_t cell = (size_t)blockIdx.x;
  if (tid == 0) a.seg_stats[cell] = s;
  if constexpr (TOP) {
    uint64_t* out = a.seg_keys + cell * a.top;
    for (int i = tid; i < count; i += kLpThreads) {
      const uint64_t key = joined[i];
      const int rank = lp_rank(joined, count, key);
      if (rank < a.top) out[rank] = key;
    }
    for (int i = count + tid; i < a.top; i += kLpThreads) out[i] = 0;
  }
}

// Segments of a row joined, one workgroup per row: lane i of every wave takes
// segment i's statistics.
template <typename T>
__global__ __launch_bounds__(256) void k_logprobs_join(LpArgs a) {
  __shared__ uint64_t keys[kLpMaxSegs * kLpMaxTop];
  __shared__ uint64_t marks[kWave];
  __shared__ uint64_t tau;
  __shared__ int kept;
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  static_assert(kLpMaxSegs == kWave, "a lane a segment");
  // Everything that is read, at once: the first two keys of a thread, and
  // each segment's r-th.  The m-th largest of those, m = ceil(top / r), is
  // reached by m * r keys, `top` at least; r = ceil(top / segments) lets the
  // fewest keys through (20 of 19 segments: about 32 on average, where the
  // largest of the segments' last keys lets 230 of 380 through and costs 6 us
  // in ranks).
  const int r = max((a.top + a.segs - 1) / a.segs, 1), m = (a.top + r - 1) / r;
  const int cells = a.segs * a.top;
  const uint64_t* k = a.seg_keys + (size_t)t * cells;
  LpStats s{-__builtin_inff(), 0.0f, 0.0f};
  uint64_t mark = 0, key[2] = {0, 0};
  if (lane < a.segs) s = a.seg_stats[(size_t)t * a.segs + lane];
  if (tid < a.segs && a.top > 0) mark = k[(size_t)tid * a.top + r - 1];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (tid + 256 * j < cells) key[j] = k[tid + 256 * j];
  const float target = tid == 0 ? lp_target<T>(a, t) : 0.0f;
  if (tid == 0) {
    kept = 0;
    tau = 1;
  }
  if (tid < kWave) marks[tid] = mark;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const LpStats o{__shfl_xor(s.m, off), __shfl_xor(s.z, off), __shfl_xor(s.u, off)};
    s = lp_join(s, o);
  }
  __syncthreads();
  // no two live keys are equal; a mark of 0 (fewer live than r) leaves tau at 1
  if (mark != 0 && lp_rank(marks, a.segs, mark) == m - 1) tau = mark;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (key[j] >= tau) keys[atomicAdd(&kept, 1)] = key[j];
  for (int i = tid + 512; i < cells; i += 256) {
    const uint64_t more = k[i];
    if (more >= tau) keys[atomicAdd(&kept, 1)] = more;
  }
  __syncthreads();
  lp_finish(a, t, s, target, keys, kept);
}

template <typename T>
hipError_t lp_launch(const LpArgs& a, hipStream_t stream) {
  const unsigned blocks = (unsigned)((int64_t)a.tokens * a.segs);
  if (a.top > 0)
    k_logprobs<T, true><<<blocks, kLpThreads, 0, stream>>>(a);
  else
    k_logprobs<T, false><<<blocks, kLpThreads, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.segs == 1) return e;
  k_logprobs_join<T><<<a.tokens, 256, 0, stream>>>(a);
  return hipGetLastError();
}

// Values of a segment: whole steps of all the workgroup's waves.
constexpr int64_t kLpSegUnit = kLpBlock * kLpWaves;

// Counted from the row's values alone: the last segment, which always has
// some, also takes what a row that is not aligned moves up by (7 places at
// most).
int64_t lp_units(int64_t vocab) { return (vocab + kLpSegUnit - 1) / kLpSegUnit; }

}  // namespace

int logprobs_segments(int64_t tokens, int64_t vocab) {
  if (tokens < 1) return 1;
  const int64_t units = lp_units(vocab);
  // Four workgroups a CU, which is what fits without alternatives; with them
  // it is three.  A sweep (bf16; rows x vocabulary: us at 512 / 768 / 1024 /
  // 2048 workgroups):
  //   top 5   4 x 151936: 11.3 everywhere    64 x 151936: 16.5 17.1 17.3 21.2
  //           256 x 32000: 15.2 15.1 21.7 21.9    256 x 151936: 28.2 27.5 31.8 37.2
  //           600 x 14500: 13.9 25.4 25.4 25.4    1000 x 32000: 27.2 27.4 37.0 37.3
  //   none    64 x 151936: 10.4 11.0 11.1 13.0    600 x 14500: 9.1 15.2 15.2 15.2
  // so fewer would serve some hundred rows better, up to twofold.
  int64_t want = (1024 + tokens - 1) / tokens;
  if (want > units) want = units;
  if (want > kLpMaxSegs) want = kLpMaxSegs;
  if (want <= 1) return 1;
  const int64_t per = (units + want - 1) / want;
  return (int)((units + per - 1) / per);
}

int64_t logprobs_workspace_bytes(int64_t tokens, int64_t vocab, int64_t top) {
  const int64_t segs = logprobs_segments(tokens, vocab);
  return segs <= 1 ? 0 : tokens * segs * (8 * top + (int64_t)sizeof(LpStats));
}

hipError_t launch_logprobs(const LogprobsCall& c, hipStream_t stream) {
  const int segs = logprobs_segments(c.tokens, c.vocab);
  const int64_t per = (lp_units(c.vocab) + segs - 1) / segs * kLpSegUnit;
  LpArgs a{c.logits, c.targets, c.logprob, c.entropy, c.top_ids, c.top_logprobs, nullptr, nullptr, c.stride,
           c.tokens, c.vocab, c.top, segs, segs == 1 ? 0 : (int32_t)per};
  if (segs > 1) {   // the keys first: 8-byte words
    a.seg_keys = static_cast<uint64_t*>(c.workspace);
    a.seg_stats = reinterpret_cast<LpStats*>(a.seg_keys + (size_t)c.tokens * segs * c.top);
  }
  return c.f32 ? lp_launch<float>(a, stream) : lp_launch<uint16_t>(a, stream);
}

}  // namespace fp8w
