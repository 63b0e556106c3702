// sample.hip -- a token drawn from each row of logits under a temperature,
// top-k, top-p and min-p, by one given random number.
//
// With the row's tokens in order (larger logits first, lower tokens first
// among equals) and weights w_j = exp((x_j - x_0) / T), every filter keeps the
// first so many of them:
//   top-k   n <= k
//   top-p   n <= the smallest n with C(n) >= p C(k),   C(n) = w_0 + ... + w_(n-1)
//   min-p   n <= the number of j with (x_j - x_0) / T >= ln(min_p)
// and the token drawn with u is the first whose C exceeds u C(n).  So
// nothing needs the whole order: each of these asks for one place in it, by
// count, by weight or by value.
//
// Weights are whole numbers, 2^S w rounded (S = 62 - ceil(log2 vocab), at most
// 50), from fp64 exponentials: their sums are the same in any order, so that
// atomics may add them up, and a choice between two tokens changes with the
// 2^-45 of a weight's rounding alone.  fp32 would turn over one of some
// thousand choices among 10^5 tokens.  (fp64 multiply-adds run at the rate of fp32's.)
//
// A workgroup takes a row in passes over it (out of L2 from the second on):
// its largest and smallest logit; a histogram of the distance from the
// largest, counts and weights; and the tokens of the bins that matter, into
// LDS, where they are sorted.  Bins that hold more than that has room for are
// divided again by the values' bits, down to a single value, whose tokens
// differ by their place alone.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "internal.hpp"

namespace fp8w {
namespace {

constexpr int kSmThreads = 1024;
constexpr int kSmWaves = kSmThreads / kWave;
constexpr int kSmBins = kSmThreads;   // a thread a bin
constexpr int kSmCap = 2048;          // tokens of a sorted list
constexpr uint32_t kFirstLive = 0x00800000u;   // the ordered bits of the lowest value; -inf is one below

// Value bits whose unsigned order is the values' order (-0 equal to +0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (uint32_t)(((int32_t)b >> 31) | 0x80000000);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct SampleArgs {
  const void* logits;
  const float* uniforms;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* ids;
  float* logprob;
  int32_t* kept;
  int64_t stride;
  int32_t tokens, vocab, bits;   // bits: S
};

// What turns a row's logits into weights and bins.
struct RowScale {
  float m;           // the largest logit
  double per;        // log2 e / T
  float inv;         // bins for each unit of distance
  int bits;

  // 2^bits exp((x - m) / T), rounded to nearest: exp2 of a whole part and a
  // polynomial (Taylor, to 2^-42 of the value) of what is left, |f| <= 1/2.
  __device__ __forceinline__ uint64_t weight(float x) const {
    const double d = x == m ? 0.0 : (double)x - (double)m;
    const double t = __builtin_fmax(d * per, -128.0);   // NaN (inf / inf) too
    const double n = __builtin_rint(t), f = t - n;
    double p = 7.054911620801121e-09;                   // ln2^k / k!, k = 10 ... 0
    p = __builtin_fma(p, f, 1.0178086009239696e-07);
    p = __builtin_fma(p, f, 1.3215486790144305e-06);
    p = __builtin_fma(p, f, 1.5252733804059838e-05);
    p = __builtin_fma(p, f, 1.5403530393381606e-04);
    p = __builtin_fma(p, f, 1.3333558146428441e-03);
    p = __builtin_fma(p, f, 9.618129107628477e-03);
    p = __builtin_fma(p, f, 5.550410866482158e-02);
    p = __builtin_fma(p, f, 2.402265069591007e-01);
    p = __builtin_fma(p, f, 6.931471805599453e-01);
    p = __builtin_fma(p, f, 1.0);
    const double w = __builtin_ldexp(p, (int)n + bits);
    return (uint64_t)__double_as_longlong(w + 4503599627370496.0) & ((1ull << 52) - 1);   // + 2^52: the units' place is the last bit
  }
  // Bin 0 holds the largest; a larger logit is never in a later bin.
  __device__ __forceinline__ uint32_t bin(float x) const {
    const float d = x == m ? 0.0f : __builtin_fminf(m - x, 3.4e38f);
    const uint32_t b = (uint32_t)(d * inv);
    return b < kSmBins ? b : kSmBins - 1;
  }
};

// Every token of the row once: f(logit, token).
template <typename T, typename F>
__device__ __forceinline__ void walk(const SampleArgs& a, int t, const F& f) {
  constexpr int kVec = 16 / sizeof(T);
  // Places are counted from the 16-byte boundary at or below the row's start;
  // only 16 bytes that lie in the row are loaded whole.
  const char* row = static_cast<const char*>(a.logits) + (size_t)t * a.stride * sizeof(T);
  const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const char* base = row - skew * sizeof(T);
  const int64_t end = (int64_t)a.vocab + skew;
  const int64_t v0 = skew ? 1 : 0, v1 = end / kVec;
  const int tid = threadIdx.x;
  const auto value = [&](int64_t at) {
    float x;
    if constexpr (sizeof(T) == 4)
      x = ld_global<float>(base, (size_t)at * 4);
    else
      x = bf16_lo(ld_global<uint16_t>(base, (size_t)at * 2));
    f(x, (int)(at - skew));
  };
#pragma unroll 4
  for (int64_t v = v0 + tid; v < v1; v += kSmThreads) {
    const uint4 r = ld_global_u4(base, (size_t)v * 16);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    const int at = (int)(v * kVec - skew);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f(__uint_as_float(w[i]), at + i);
      } else {
        f(bf16_lo(w[i]), at + 2 * i);
        f(bf16_hi(w[i]), at + 2 * i + 1);
      }
    }
  }
  if (tid < kVec) {   // the row's two ends
    if (v0 == 1 && tid >= skew && tid < end) value(tid);
    const int64_t at = (v1 > v0 ? v1 : v0) * kVec + tid;
    if (at < end) value(at);
  }
}

struct Shared {
  uint64_t list[kSmCap];        // ordered bits, then the token's complement
  uint64_t list_mass[kSmCap];   // weights of the list up to and with each
  uint64_t mass[2][kSmBins];    // of the whole row's bins, of one bin's parts
  uint32_t count[2][kSmBins];
  uint64_t wave_mass[kSmWaves];
  uint32_t wave_count[kSmWaves];
  float wave_max[kSmWaves], wave_min[kSmWaves];
  int length;
  uint64_t found_mass;
  uint32_t found, found_count;
};

// Sums up to and with each thread's; the total in `total`.
template <typename V>
__device__ __forceinline__ V block_prefix(V v, V* waves, V& total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const V up = __shfl_up(v, off);
    if (lane >= off) v += up;
  }
  __syncthreads();   // the last sums have been read
  if (lane == kWave - 1) waves[w] = v;
  __syncthreads();
  V before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSmWaves; ++i) {
    if (i < w) before += waves[i];
    total += waves[i];
  }
  return v + before;
}

// The place in the row's order that is looked for: the smallest n with n >=
// goal or C(n) >= goal, or the number of tokens whose bits are >= goal.
enum class By { kCount, kMass, kKey };

// A place: n, C(n), and the n-th token's bits.
struct Place {
  uint32_t n;
  uint64_t mass;
  uint32_t key;
  int32_t id;
};

// One workgroup's view of its row.
template <typename T>
struct Row {
  const SampleArgs& a;
  const int t;
  Shared& s;
  RowScale scale;
  uint32_t top;             // ordered bits of the largest
  // what s.list holds: the tokens of these bits, and what stands before them
  uint32_t lo = 1, hi = 0, before = 0, length = 0;
  uint64_t before_mass = 0, mass = 0;

  // The smallest bits whose bin is b or an earlier one: 64 places of the
  // range at a time, the same in every wave.
  __device__ uint32_t first_key(uint32_t b) const {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t from = kFirstLive, to = top;   // bin(to) <= b
    while (from < to) {
      const uint32_t step = (to - from) / kWave + 1;
      const uint64_t at = (uint64_t)from + (uint64_t)step * lane;
      const uint64_t yes = __ballot(at >= to || scale.bin(unordered((uint32_t)at)) <= b);
      if (yes == 0) {
        from += step * (kWave - 1) + 1;
        continue;
      }
      const int l = __builtin_ctzll(yes);
      const uint64_t next = (uint64_t)from + (uint64_t)step * l;
      if (next < to) to = (uint32_t)next;
      if (l > 0) from += step * (l - 1) + 1;
    }
    return to;
  }

  // Counts, and weights if they are wanted, by `where` (a bin, or none for
  // kSmBins and above) of the tokens, up to and with each bin.
  template <typename Where>
  __device__ void histogram(int at, bool weights, const Where& where) {
    const int tid = threadIdx.x;
    __syncthreads();
    s.count[at][tid] = 0;
    s.mass[at][tid] = 0;
    __syncthreads();
    walk<T>(a, t, [&](float x, int) {
      if (!(x > -__builtin_inff())) return;
      const uint32_t b = where(x);
      if (b >= kSmBins) return;
      atomicAdd(&s.count[at][b], 1u);
      if (weights) {
        const uint64_t q = scale.weight(x);
        if (q) atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[at][b]), (unsigned long long)q);
      }
    });
    __syncthreads();
    uint32_t all;
    uint64_t all_mass;
    const uint32_t n = block_prefix(s.count[at][tid], s.wave_count, all);
    const uint64_t m = block_prefix(s.mass[at][tid], s.wave_mass, all_mass);
    s.count[at][tid] = n;
    s.mass[at][tid] = m;
    __syncthreads();
  }

  // The first bin that reaches the goal, with `n0` and `m0` before them all.
  __device__ uint32_t bin_of(int at, By by, uint64_t goal, uint32_t n0, uint64_t m0) {
    const int tid = threadIdx.x;
    const uint64_t upto = by == By::kCount ? n0 + s.count[at][tid] : m0 + s.mass[at][tid];
    const uint64_t less = tid == 0 ? (by == By::kCount ? n0 : m0) : by == By::kCount ? n0 + s.count[at][tid - 1] : m0 + s.mass[at][tid - 1];
    if (tid == 0) s.found = kSmBins - 1;
    __syncthreads();
    if (less < goal && upto >= goal) s.found = tid;
    __syncthreads();
    const uint32_t b = s.found;
    __syncthreads();
    return b;
  }

  // The tokens of these bits (no more than the list holds) into the list, in order.
  __device__ void load(uint32_t from, uint32_t to, uint32_t n0, uint64_t m0) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) s.length = 0;
    __syncthreads();
    walk<T>(a, t, [&](float x, int id) {
      const uint32_t k = ordered(x);
      if (!(x > -__builtin_inff()) || k < from || k > to) return;
      const int at = atomicAdd(&s.length, 1);
      if (at < kSmCap) s.list[at] = ((uint64_t)k << 32) | (uint32_t)~id;
    });
    __syncthreads();
    const int n = min(s.length, kSmCap);
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kSmThreads) s.list[i] = 0;
    __syncthreads();
    // bitonic, larger first; keys are unique but for the filling
    for (int k = 2; k <= size; k *= 2) {
      for (int j = k / 2; j > 0; j /= 2) {
        if (tid < size / 2) {
          const int i = 2 * tid - (tid & (j - 1));   // bit j clear
          const uint64_t x = s.list[i], y = s.list[i + j];
          if ((x < y) == ((i & k) == 0)) {
            s.list[i] = y;
            s.list[i + j] = x;
          }
        }
        __syncthreads();
      }
    }
    const int i0 = 2 * tid, i1 = 2 * tid + 1;
    const uint64_t q0 = i0 < n ? scale.weight(unordered((uint32_t)(s.list[i0] >> 32))) : 0;
    const uint64_t q1 = i1 < n ? scale.weight(unordered((uint32_t)(s.list[i1] >> 32))) : 0;
    uint64_t all;
    const uint64_t upto = block_prefix(q0 + q1, s.wave_mass, all);
    if (i0 < n) s.list_mass[i0] = m0 + upto - q1;
    if (i1 < n) s.list_mass[i1] = m0 + upto;
    __syncthreads();
    lo = from;
    hi = to;
    before = n0;
    before_mass = m0;
    length = (uint32_t)n;
    mass = all;
  }

  __device__ bool listed(By by, uint64_t goal) const {
    switch (by) {
      case By::kCount: return goal > before && goal <= (uint64_t)before + length;
      case By::kMass: return goal > before_mass && goal <= before_mass + mass;
      default: return lo <= hi && goal >= lo && goal <= hi;
    }
  }

  // The goal's place within the list.
  __device__ Place in_list(By by, uint64_t goal) {
    const int tid = threadIdx.x;
    if (tid == 0) s.found = by == By::kKey ? 0 : length;
    __syncthreads();
    for (uint32_t i = tid; i < length; i += kSmThreads) {
      if (by == By::kKey) {
        const bool here = (s.list[i] >> 32) >= goal, next = i + 1 < length && (s.list[i + 1] >> 32) >= goal;
        if (here && !next) s.found = i + 1;
      } else if (by == By::kMass) {
        if (s.list_mass[i] >= goal && (i == 0 || s.list_mass[i - 1] < goal)) s.found = i + 1;
      }
    }
    __syncthreads();
    const uint32_t n = by == By::kCount ? (uint32_t)goal - before : s.found;
    __syncthreads();
    if (n == 0) return Place{before, before_mass, top, -1};
    const uint64_t e = s.list[n - 1];
    return Place{before + n, s.list_mass[n - 1], (uint32_t)(e >> 32), (int32_t)~(uint32_t)e};
  }

  // The n-th token, by place in the row, of those with these bits.
  __device__ int32_t nth_equal(uint32_t key, uint32_t n) {
    const int tid = threadIdx.x;
    const int per = (a.vocab + kSmThreads - 1) / kSmThreads;
    const int64_t first = (int64_t)tid * per, last = min(first + per, (int64_t)a.vocab);
    const char* row = static_cast<const char*>(a.logits) + (size_t)t * a.stride * sizeof(T);
    const auto is = [&](int64_t i) {
      float x;
      if constexpr (sizeof(T) == 4)
        x = ld_global<float>(row, (size_t)i * 4);
      else
        x = bf16_lo(ld_global<uint16_t>(row, (size_t)i * 2));
      return x == x && ordered(x) == key;
    };
    uint32_t mine = 0, all;
    for (int64_t i = first; i < last; ++i) mine += is(i) ? 1 : 0;
    const uint32_t upto = block_prefix(mine, s.wave_count, all);
    if (tid == 0) s.found = 0;
    __syncthreads();
    if (mine && upto - mine < n && upto >= n) {
      uint32_t left = n - (upto - mine);
      int64_t i = first;
      for (; i < last; ++i)
        if (is(i) && --left == 0) break;
      s.found = (uint32_t)i;
    }
    __syncthreads();
    const int32_t id = (int32_t)s.found;
    __syncthreads();
    return id;
  }

  // The goal's place, which the row has.  The histogram holds weights if
  // `goal` may lie past the list's.
  __device__ Place find(By by, uint64_t goal) {
    if (listed(by, goal)) return in_list(by, goal);
    uint32_t b = by == By::kKey ? scale.bin(unordered((uint32_t)goal)) : bin_of(0, by, goal, 0, 0);
    uint32_t n0 = b ? s.count[0][b - 1] : 0, n = s.count[0][b] - n0;
    uint64_t m0 = b ? s.mass[0][b - 1] : 0;
    uint32_t from = first_key(b), to = b ? first_key(b - 1) - 1 : top;
    if (n0 + n <= kSmCap) {   // all that stands before it too: the next goal is likely among them
      load(from, top, 0, 0);
      return in_list(by, goal);
    }
    while (n > kSmCap && from < to) {   // too many: by their bits
      int shift = 0;
      while ((to - from) >> shift >= kSmBins) ++shift;
      histogram(1, true, [&](float x) {
        const uint32_t k = ordered(x);
        return k < from || k > to ? kSmBins : (to - k) >> shift;
      });
      b = by == By::kKey ? (to - (uint32_t)goal) >> shift : bin_of(1, by, goal, n0, m0);
      const uint32_t nb = b ? s.count[1][b - 1] : 0;
      n = s.count[1][b] - nb;
      n0 += nb;
      m0 += b ? s.mass[1][b - 1] : 0;
      to -= b << shift;
      from = to - from < (1u << shift) ? from : to - (1u << shift) + 1;
    }
    if (n <= kSmCap) {
      load(from, to, n0, m0);
      return in_list(by, goal);
    }
    const uint64_t q = scale.weight(unordered(to));   // n tokens of one value
    const uint32_t r = by == By::kCount ? (uint32_t)goal - n0 : by == By::kKey ? n : (uint32_t)((goal - m0 + q - 1) / q);
    return Place{n0 + r, m0 + r * q, to, nth_equal(to, r)};
  }
};

template <typename T>
__global__ __launch_bounds__(kSmThreads) void k_sample(SampleArgs a) {
  __shared__ Shared s;
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  const float inf = __builtin_inff();
  float most = -inf, least = inf;
  walk<T>(a, t, [&](float x, int) {
    most = __builtin_fmaxf(most, x);   // NaN passes by
    if (x > -inf) least = __builtin_fminf(least, x);
  });
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    most = __builtin_fmaxf(most, __shfl_xor(most, off));
    least = __builtin_fminf(least, __shfl_xor(least, off));
  }
  if (lane == 0) {
    s.wave_max[tid / kWave] = most;
    s.wave_min[tid / kWave] = least;
  }
  __syncthreads();
  for (int w = 0; w < kSmWaves; ++w) {
    most = __builtin_fmaxf(most, s.wave_max[w]);
    least = __builtin_fminf(least, s.wave_min[w]);
  }
  if (most == -inf) {   // masked throughout
    if (tid == 0) {
      a.ids[t] = -1;
      if (a.logprob) a.logprob[t] = -inf;
      if (a.kept) a.kept[t] = 0;
    }
    return;
  }

  float temp = a.temperature ? a.temperature[t] : 1.0f;
  int64_t k = a.top_k ? a.top_k[t] : 0;
  float p = a.top_p ? a.top_p[t] : 1.0f, low = a.min_p ? a.min_p[t] : 0.0f;
  if (!(temp > 0.0f)) {
    temp = 1.0f;
    k = 1;
    p = 1.0f;
    low = 0.0f;
  }
  // Bins reach to where weights are zero, or as far as the row does.
  const float far = __builtin_fminf(temp * (float)((a.bits + 1) * 0.6931472), most - least);
  Row<T> row{a, t, s, RowScale{most, 1.4426950408889634 / (double)temp, far > 0.0f ? __builtin_fminf(kSmBins / far, 3.0e38f) : 0.0f, a.bits},
             ordered(most)};
  // A few tokens alone are asked for: no weight is needed but theirs.
  const bool few = k > 0 && k <= kSmCap / 2;
  row.histogram(0, !few, [&](float x) { return row.scale.bin(x); });
  const uint32_t live = s.count[0][kSmBins - 1];
  if (few) {
    const uint32_t want = k < live ? (uint32_t)k : live;
    if (s.count[0][row.bin_of(0, By::kCount, want, 0, 0)] > kSmCap)
      row.histogram(0, true, [&](float x) { return row.scale.bin(x); });
    else
      row.find(By::kCount, want);
  }
  Place cut{live, s.mass[0][kSmBins - 1], ordered(least), -1};
  if (k > 0 && k < live) cut = row.find(By::kCount, (uint64_t)k);
  else if (few) cut = row.find(By::kCount, live);
  if (p < 1.0f) {
    const double goal = __builtin_ceil((double)p * (double)cut.mass);
    cut = row.find(By::kMass, goal < 1.0 ? 1 : goal >= (double)cut.mass ? cut.mass : (uint64_t)goal);
  }
  if (low > 0.0f) {
    // The least bits that pass: found from the bound's own value, 64 at a time
    // as first_key does.
    const double bound = log((double)low);
    const auto passes = [&](uint32_t key) {
      const float x = unordered(key);
      return x == most || ((double)x - (double)most) / (double)temp >= bound;
    };
    uint32_t from = kFirstLive, to = row.top;
    while (from < to) {
      const uint32_t step = (to - from) / kWave + 1;
      const uint64_t at = (uint64_t)from + (uint64_t)step * lane;
      const uint64_t yes = __ballot(at >= to || passes((uint32_t)at));
      if (yes == 0) {
        from += step * (kWave - 1) + 1;
        continue;
      }
      const int l = __builtin_ctzll(yes);
      const uint64_t next = (uint64_t)from + (uint64_t)step * l;
      if (next < to) to = (uint32_t)next;
      if (l > 0) from += step * (l - 1) + 1;
    }
    if (cut.key < to) cut = row.find(By::kKey, to);
  }
  const float u = a.uniforms[t];
  const double at = __builtin_floor((double)u * (double)cut.mass);
  const uint64_t goal = !(at > 0.0) ? 0 : at >= (double)cut.mass ? cut.mass - 1 : (uint64_t)at;
  const Place drawn = row.find(By::kMass, (goal < cut.mass ? goal : cut.mass - 1) + 1);
  if (tid == 0) {
    a.ids[t] = drawn.id;
    if (a.kept) a.kept[t] = (int32_t)cut.n;
    if (a.logprob) {
      const float x = unordered(drawn.key);
      const double d = x == most ? 0.0 : ((double)x - (double)most) / (double)temp;
      a.logprob[t] = (float)(d - (log((double)cut.mass) - a.bits * 0.6931471805599453));
    }
  }
}

}  // namespace

int sample_segments(int64_t, int64_t) { return 1; }
int64_t sample_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleCall& c, hipStream_t stream) {
  int log = 0;
  while (((int64_t)1 << log) < c.vocab) ++log;
  const SampleArgs a{c.logits, c.uniforms, c.temperature, c.top_k, c.top_p, c.min_p, c.ids, c.logprob, c.kept,
                     c.stride, c.tokens, c.vocab, log > 12 ? 62 - log : 50};
  if (c.f32)
    k_sample<float><<<c.tokens, kSmThreads, 0, stream>>>(a);
  else
    k_sample<uint16_t><<<c.tokens, kSmThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp8w
