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
// atomics may add them up.  Those of a whole bin are known to 2^-31 of their sum
// (2^-19 for 2^24 tokens), as RowScale says, and half a unit of each of its
// tokens.  fp32 sums would turn over one choice of some thousand among 10^5
// tokens.  (fp64 multiply-adds run at the rate of fp32's.)
//
// A row is taken in passes: its largest and smallest logit; a histogram of the
// distance from the largest, counts and weights; and the tokens of the bins
// that matter, into LDS, where they are sorted.  Bins that hold more than that
// has room for are divided again by the values' bits, down to a single value,
// whose tokens differ by their place alone.
//
// With rows enough one workgroup does all of it, and finds the row in the
// caches again from pass to pass.  With fewer the first two passes are
// launches of their own over pieces of rows, and a third adds the pieces'
// histograms.
//
// What bounds it is a chain of latencies: 4 x 151936 bf16 under top-k and top-p
// takes 27 us, of which the range 3, the histogram 6 and the choice 18 (code
// that runs but once, and is fetched as it runs; some twenty barriers a place
// that is looked for).  512 x 32000 44 us (0.75 TB/s): two rounds of the same.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "internal.hpp"

namespace fp8w {
namespace {

constexpr int kSmThreads = 512;       // of a workgroup that has a row, or a piece of one, to itself
constexpr int kSmMany = 1024;         // of one that takes up a row from its pieces
constexpr int kSmBins = 1024;
constexpr int kSmCap = 2048;          // tokens of a sorted list
constexpr int kSmSmall = 256;         // of one that is ranked by counting
constexpr int kSmPieces = 16;         // of a row, at most
constexpr uint32_t kFirstLive = 0x00800000u;   // the ordered bits of the lowest value; -inf is one below

// Value bits whose unsigned order is the values' order (-0 equal to +0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (uint32_t)(((int32_t)b >> 31) | 0x80000000);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A value that all threads have alike, taken into scalar registers.
__device__ __forceinline__ uint32_t alike(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int32_t alike(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t alike(uint64_t v) {
  return (uint64_t)alike((uint32_t)(v >> 32)) << 32 | alike((uint32_t)v);
}
__device__ __forceinline__ float alike(float v) { return __uint_as_float(alike(__float_as_uint(v))); }
__device__ __forceinline__ double alike(double v) {
  return __longlong_as_double((int64_t)alike((uint64_t)__double_as_longlong(v)));
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
  int32_t shift, fraction;       // of the histogram's words (RowScale)
  int32_t segs, per;             // pieces of a row, and places of a piece
  // of the pieces, where there is more than one
  float2* ranges;                // [tokens][segs]: largest and smallest logit
  uint64_t* words;               // [tokens][segs][bins]
};

// What turns a row's logits into weights and bins.  Bins are of equal width, and
// reach to where weights are zero, or as far as the row does.
//
// The histogram adds, for each token, one to its bin's count and to the same
// word the weight relative to that of the bin's middle, less one: |e| < 2^-5
// (a bin is no wider than 62/1023 powers of two), as a whole number of
// 2^-fraction, so that a bin's weight is that of its middle times (count + sum
// of e).  Half a unit's rounding and the term left out, |ln2 wide/2|^5 / 120 <
// 2^-34, make 2^-31 of a weight (and that of the middle is a whole number, half a
// unit off) for up to 2^18 tokens, whose counts leave 31 bits of fraction; above,
// count and sum each take one of these for each doubling.  The sum of e +
// 2^-5 stays below 2^(fraction - 4) times the count, and so below 2^shift.  An
// exponential for every token would take twice as long, a second atomic as well.
struct RowScale {
  double m;            // the largest logit (2^200 for infinity)
  double per;          // log2 e / T
  double inv, unit;    // bins for each unit of distance, and the distance of one
  double wide;         // log2 of a bin's weights' ratio
  double c1, c2, c3, c4;   // e of a place in the bin, times 2^fraction
  int bits, shift, fraction;
  uint32_t bias;           // added to e, so that it is positive: 2^-5

  static constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: a sum's low word is its whole part, rounded

  __device__ __forceinline__ RowScale(float most, float least, float temperature, const SampleArgs& a) {
    m = above(most);
    per = 1.4426950408889634 / (double)temperature;
    bits = a.bits;
    shift = a.shift;
    fraction = a.fraction;
    bias = 1u << (fraction - 5);
    const double far = __builtin_fmin((double)temperature * ((bits + 12) * 0.6931471805599453), m - above(least));
    inv = far > 0.0 ? __builtin_fmin((kSmBins - 1) / far, 1e300) : 0.0;
    unit = inv > 0.0 ? 1.0 / inv : 0.0;
    wide = per * unit;
    const double w = wide * 0.6931471805599453, one = __builtin_ldexp(1.0, fraction);
    c1 = -w * one;
    c2 = w * w * (one / 2);
    c3 = -w * w * w * (one / 6);
    c4 = w * w * w * w * (one / 24);
    m = alike(m), per = alike(per), inv = alike(inv), unit = alike(unit), wide = alike(wide);
    c1 = alike(c1), c2 = alike(c2), c3 = alike(c3), c4 = alike(c4);
  }
  static __device__ __forceinline__ double above(float x) { return __builtin_fmin((double)x, 0x1p200); }

  // 2^bits 2^t, t <= 0, rounded to nearest: a whole part and a polynomial
  // (Taylor, to 2^-42 of the value) of what is left, |f| <= 1/2.
  __device__ __forceinline__ uint64_t power(double t) const {
    t = __builtin_fmax(t, -128.0);
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
    return whole(__builtin_ldexp(p, (int)n + bits));
  }
  static __device__ __forceinline__ uint64_t whole(double v) {   // below 2^52, rounded
    return (uint64_t)__double_as_longlong(v + 4503599627370496.0) & ((1ull << 52) - 1);
  }
  __device__ __forceinline__ uint64_t weight(float x) const { return power((above(x) - m) * per); }

  // Bin 0 holds the largest; a larger logit is never in a later bin.  `at` is
  // its place, in bins, and `middle` the bin's.
  __device__ __forceinline__ uint32_t bin(float x, double& at, double& middle) const {
    at = __builtin_fmin((m - above(x)) * inv, (double)(kSmBins - 1));
    const double y = at + kMagic;
    middle = y - kMagic;
    return (uint32_t)__double_as_longlong(y);
  }
  __device__ __forceinline__ uint32_t bin(float x) const {
    double at, middle;
    return bin(x, at, middle);
  }
  // What a token adds to its bin's word, without weight and with.
  __device__ __forceinline__ uint64_t one() const { return 1ull << shift; }
  __device__ __forceinline__ uint64_t one(double at, double middle) const {
    const double d = at - middle;
    double e = __builtin_fma(c4, d, c3);
    e = __builtin_fma(e, d, c2);
    e = __builtin_fma(e, d, c1);
    const uint32_t low = (uint32_t)__double_as_longlong(__builtin_fma(e, d, kMagic)) + bias;
    return one() + low;
  }
  // A word's count and, of tokens around the middle of bin b, their weight.
  __device__ __forceinline__ uint32_t count_of(uint64_t word) const { return (uint32_t)(word >> shift); }
  __device__ __forceinline__ uint64_t mass_of(uint64_t word, uint32_t b) const {
    const double count = (double)count_of(word);
    const double e = (double)(word & (one() - 1)) - count * (double)bias;
    const double all = __builtin_fma(e, __builtin_ldexp(1.0, -fraction), count);
    const double w = (double)power(-(double)b * wide);
    return (uint64_t)(all * w);
  }
};

// A row's logits, or those of one piece of it, as a workgroup of N threads
// reads them, 16 bytes at a time.  (Rows of up to 64 KB kept in registers from
// pass to pass were no faster than the caches: 56.4 us for 512 x 32000 both.)
//
// A pass's code runs but once or a few times a wave, so its time is that of
// fetching it: what is done for each value is written out for two values of a
// load, with the registers moved on under it, not for each of eight (32 copies
// of the exponential, and a place of the order looked for in five copies,
// took 50 us where the row had 5000 tokens).
template <typename T, int N>
struct Logits {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kBatch = 4;   // loads that leave at once
  // Places are counted from the 16-byte boundary at or below the row's start;
  // only 16 bytes that lie in the row are loaded whole.
  const char* base;
  int skew;
  int64_t v0, v1, end, tail;   // whole 16 bytes, and the values behind them

  __device__ __forceinline__ Logits(const SampleArgs& a, int t, int seg) {
    const char* row = static_cast<const char*>(a.logits) + (size_t)t * a.stride * sizeof(T);
    skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    base = row - skew * sizeof(T);
    end = (int64_t)a.vocab + skew;
    v0 = skew ? 1 : 0;
    v1 = end / kVec;
    tail = (v1 > v0 ? v1 : v0) * kVec;
    if (a.segs > 1 && seg >= 0) {   // a piece: whole units of 16 bytes
      const int64_t lo = (int64_t)seg * (a.per / kVec), hi = lo + a.per / kVec;
      if (seg + 1 < a.segs) {
        v1 = hi < v1 ? hi : v1;
        end = 0;   // its end is not the row's
      }
      if (seg > 0) {
        v0 = lo > v0 ? lo : v0;
        skew |= 0x40000000;   // nor its start
      }
    }
  }
  // Nothing to see in what is not there: NaN.
  __device__ __forceinline__ uint4 load(int64_t v) const {
    constexpr uint32_t kNan = 0xFFFFFFFFu;
    return v < v1 ? ld_global_u4(base, (size_t)v * 16) : make_uint4(kNan, kNan, kNan, kNan);
  }
  __device__ __forceinline__ float value(int64_t at) const {
    if constexpr (sizeof(T) == 4) return ld_global<float>(base, (size_t)at * 4);
    return bf16_lo(ld_global<uint16_t>(base, (size_t)at * 2));
  }
  // The row's two ends: f(logit, token) of what its whole 16 bytes leave.
  template <typename F>
  __device__ __forceinline__ void ends(const F& f) const {
    const int tid = threadIdx.x;
    if (tid >= 2 * kVec) return;
    const int64_t at = tid < kVec ? tid : tail + tid - kVec;
    const bool there = tid < kVec ? skew > 0 && skew < kVec && tid >= skew && (end == 0 || tid < end) : at < end;
    if (there) f(value(at), (int)at - (skew & 0xFF));
  }
  // The kVec values of 16 bytes in one expression each.
  template <typename F>
  static __device__ __forceinline__ void values(const uint4& r, const F& f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f(__uint_as_float(w[i]));
      } else {
        f(bf16_lo(w[i]));
        f(bf16_hi(w[i]));
      }
    }
  }
  // 16 bytes at a time, a few at once: g(16 bytes, which of the row's).
  template <typename G>
  __device__ __forceinline__ void loads(const G& g) const {
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int64_t v = v0 + tid; v < v1; v += kBatch * N) {
      uint4 r[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) r[i] = load(v + i * N);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) g(r[i], (int)(v + i * N));
    }
  }
  __device__ __forceinline__ int first_token(int v) const { return v * kVec - (skew & 0xFF); }
  // Whether one of 16 bytes' values may lie in [lo, hi], by their bits: on one
  // side of zero these are in order, and a difference and a minimum for each
  // value (two of bf16's at once) tell.
  struct Band {
    float lo, hi;
    bool bits;             // both on one side of zero
    uint32_t first, width;
    __device__ __forceinline__ Band(float l, float h) : lo(l), hi(h), bits(l > 0.0f || h < 0.0f) {
      const uint32_t near = __float_as_uint(l > 0.0f ? l : h), far = __float_as_uint(l > 0.0f ? h : l);
      constexpr int kShift = sizeof(T) == 4 ? 0 : 16;
      first = near >> kShift;
      width = (far >> kShift) - first;
    }
    __device__ __forceinline__ bool has(const uint4& r) const {
      if (!bits) {
        bool any = false;
        values(r, [&](float x) __attribute__((always_inline)) { any |= x >= lo && x <= hi; });
        return any;
      }
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
      if constexpr (sizeof(T) == 4) {
        uint32_t least = w[0] - first;
#pragma unroll
        for (int i = 1; i < 4; ++i) least = min(least, w[i] - first);
        return least <= width;
      } else {
        const u16x2 down = {(uint16_t)first, (uint16_t)first};
        u16x2 least = __builtin_bit_cast(u16x2, w[0]) - down;
#pragma unroll
        for (int i = 1; i < 4; ++i) least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, w[i]) - down);
        return least[0] <= width || least[1] <= width;
      }
    }
  };
  // Each of 16 bytes' values, f(logit, token), two copies of f.
  template <typename F>
  static __device__ __forceinline__ void one_by_one(uint4 r, int id, const F& f) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f(__uint_as_float(r.x), id + i);
      } else {
        f(bf16_lo(r.x), id + 2 * i);
        f(bf16_hi(r.x), id + 2 * i + 1);
      }
      r.x = r.y;
      r.y = r.z;
      r.z = r.w;
    }
  }
  // Every token once, for what takes long: f(logit, token).
  template <typename F>
  __device__ __forceinline__ void walk(const F& f) const {
    loads([&](const uint4& r, int v) __attribute__((always_inline)) {
      if (v < v1) one_by_one(r, first_token(v), f);
    });
    ends(f);
  }
};

// The words of the tokens by `where(logit, bin)` (none: kSmBins and above).
template <typename T, int N, typename Where>
__device__ __forceinline__ void fill(const Logits<T, N>& logits, const RowScale& scale, uint64_t* words, bool weights,
                                     const Where& where) {
  __syncthreads();
  for (int b = threadIdx.x; b < kSmBins; b += N) words[b] = 0;
  __syncthreads();
  logits.walk([&](float x, int) __attribute__((always_inline)) {
    if (!(x > -__builtin_inff())) return;
    double place, middle;
    const uint32_t b = where(x, scale.bin(x, place, middle));
    if (b >= kSmBins) return;
    const uint64_t word = weights ? scale.one(place, middle) : scale.one();
    atomicAdd(reinterpret_cast<unsigned long long*>(&words[b]), (unsigned long long)word);
  });
  __syncthreads();
}

template <int N>
struct Shared {
  uint64_t list[kSmCap];        // ordered bits, then the token's complement
  uint64_t list_mass[kSmCap];   // weights of the list up to and with each
  uint64_t mass[2][kSmBins];    // of the whole row's bins, of one bin's parts
  uint32_t count[2][kSmBins];
  int rank[N / kSmSmall][kSmSmall];
  uint64_t wave_mass[N / kWave];
  uint32_t wave_count[N / kWave];
  float2 wave_range[N / kWave];
  int length, queued;
  uint32_t found[2];
};

// A value from the lane n places below in its row of 16 (0 from none).
template <int N>
__device__ __forceinline__ uint32_t lanes_below(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x110 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ uint64_t lanes_below(uint64_t v) {
  return (uint64_t)lanes_below<N>((uint32_t)(v >> 32)) << 32 | lanes_below<N>((uint32_t)v);
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ uint64_t of_lane(uint64_t v, int l) {
  return (uint64_t)of_lane((uint32_t)(v >> 32), l) << 32 | of_lane((uint32_t)v, l);
}

// Sums up to and with each lane's, of its row of 16.
template <typename V>
__device__ __forceinline__ V row_prefix(V v) {
  v += lanes_below<1>(v);
  v += lanes_below<2>(v);
  v += lanes_below<4>(v);
  v += lanes_below<8>(v);
  return v;
}

// Sums up to and with each thread's; the total in `total`.
template <int N, typename V>
__device__ __forceinline__ V block_prefix(V v, V* waves, V& total) {
  constexpr int kWaves = N / kWave;
  static_assert(kWaves <= 16, "a row of lanes adds up the waves");
  const int lane = threadIdx.x & (kWave - 1), w = alike((int)threadIdx.x / kWave);
  v = row_prefix(v);
  const V a = of_lane(v, 15), b = a + of_lane(v, 31), c = b + of_lane(v, 47), all = c + of_lane(v, 63);
  const int row = lane >> 4;
  v += row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c;
  __syncthreads();   // the last sums have been read
  if (lane == 0) waves[w] = all;
  __syncthreads();
  const V upto = row_prefix(waves[lane & (kWaves - 1)]);
  total = of_lane(upto, kWaves - 1);
  return v + (w > 0 ? of_lane(upto, w - 1) : 0);
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
template <typename T, int N>
struct Row {
  static constexpr int kPer = kSmBins / N;   // neighbouring bins of a thread
  const SampleArgs& a;
  const int t;
  Shared<N>& s;
  const Logits<T, N>& logits;
  RowScale scale;
  uint32_t top;             // ordered bits of the largest
  // what s.list holds: the tokens of these bits and these bins, and what
  // stands before them
  uint32_t lo = 1, hi = 0, bin0 = 0, bin1 = 0, before = 0, length = 0;
  uint64_t before_mass = 0, mass = 0;
  // what all bins, and all parts of one, hold
  uint32_t all_count[2] = {0, 0};
  uint64_t all_mass[2] = {0, 0};

  // The smallest bits for which `yes` holds, as it does for the largest logit's
  // and for all above the answer: 64 places of the range at a time, the same
  // in every wave.
  template <typename Yes>
  __device__ uint32_t least_key(const Yes& yes) const {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t from = kFirstLive, to = top;
    while (from < to) {
      const uint32_t step = (to - from) / kWave + 1;
      const uint64_t at = (uint64_t)from + (uint64_t)step * lane;
      const uint64_t holds = __ballot(at >= to || yes((uint32_t)at));
      if (holds == 0) {
        from += step * (kWave - 1) + 1;
        continue;
      }
      const int l = __builtin_ctzll(holds);
      const uint64_t next = (uint64_t)from + (uint64_t)step * l;
      if (next < to) to = (uint32_t)next;
      if (l > 0) from += step * (l - 1) + 1;
    }
    return to;
  }
  // The smallest bits whose bin is b or an earlier one.
  __device__ uint32_t first_key(uint32_t b) const {
    return least_key([&](uint32_t k) { return scale.bin(unordered(k)) <= b; });
  }

  // Words into counts and weights up to and with each bin.  The tokens are
  // those of bin `only`, or each of the bin that its place names.
  __device__ __forceinline__ void sum_up(int at, bool weights, uint32_t only = kSmBins) {
    const int tid = threadIdx.x;
    uint32_t n[kPer], count = 0;
    uint64_t m[kPer], mass = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int b = tid * kPer + j;
      const uint64_t word = s.mass[at][b];
      count += n[j] = scale.count_of(word);
      mass += m[j] = weights ? scale.mass_of(word, only < kSmBins ? only : b) : 0;
    }
    count = block_prefix<N>(count, s.wave_count, all_count[at]);
    all_mass[at] = 0;
    if (weights) mass = block_prefix<N>(mass, s.wave_mass, all_mass[at]);
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j) {
      const int b = tid * kPer + j;
      s.count[at][b] = count;
      s.mass[at][b] = mass;
      count -= n[j];
      mass -= m[j];
    }
    __syncthreads();
  }

  // One of the words by which a thread tells the others what it found: in
  // turn, so that a barrier lies between the last look at it and its next use.
  int turn = 0;
  __device__ __forceinline__ uint32_t& answer() { return s.found[turn ^= 1]; }

  // The first bin that reaches the goal, with `n0` and `m0` before them all.
  // Where none does, the last that holds a token: a goal may come from sums that
  // were rounded otherwise, as those of a bin's parts and of the bin are.
  __device__ __forceinline__ uint32_t bin_of(int at, By by, uint64_t goal, uint32_t n0, uint64_t m0) {
    const int first = threadIdx.x * kPer;
    uint32_t& found = answer();
    if (by == By::kMass && goal > m0 + all_mass[at]) {
      by = By::kCount;
      goal = n0 + all_count[at];
    }
    const auto upto = [&](int b) { return b < 0 ? (by == By::kCount ? n0 : m0) : by == By::kCount ? n0 + s.count[at][b] : m0 + s.mass[at][b]; };
    uint64_t less = upto(first - 1);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint64_t now = upto(first + j);
      if (less < goal && now >= goal) found = first + j;
      less = now;
    }
    __syncthreads();
    return alike(found);
  }

  // The list in order, larger first: each key's place is the number of larger
  // ones, counted by a few threads.
  __device__ __forceinline__ void rank_list(int n) {
    constexpr int kParts = N / kSmSmall;
    const int tid = threadIdx.x, e = tid % kSmSmall, part = tid / kSmSmall;
    const uint64_t key = e < n ? s.list[e] : 0;
    const int per = (n + kParts - 1) / kParts, last = min((part + 1) * per, n);
    int rank = 0;
#pragma unroll 8
    for (int j = part * per; j < last; ++j) rank += s.list[j] > key ? 1 : 0;
    s.rank[part][e] = rank;
    __syncthreads();
    if (part == 0 && e < n) {
#pragma unroll
      for (int i = 1; i < kParts; ++i) rank += s.rank[i][e];
      s.list[rank] = key;
    }
    __syncthreads();
  }

  // The same for more of them, bitonic: keys are unique but for the filling.
  // Steps of up to 64 places stay within a wave's own 128.
  __device__ void sort_list(int n) {
    const int tid = threadIdx.x;
    int size = 2 * kSmSmall;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += N) s.list[i] = 0;
    __syncthreads();
    const auto step = [&](int k, int j) {
#pragma unroll 1
      for (int p = tid; p < size / 2; p += N) {
        const int i = 2 * p - (p & (j - 1));   // bit j clear
        const uint64_t x = s.list[i], y = s.list[i + j];
        if ((x < y) == ((i & k) == 0)) {
          s.list[i] = y;
          s.list[i + j] = x;
        }
      }
    };
    for (int k = 2; k <= size; k *= 2) {
      int j = k / 2;
      for (; j > kWave; j /= 2) {
        step(k, j);
        __syncthreads();
      }
      for (; j > 0; j /= 2) {
        step(k, j);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
      }
      __syncthreads();
    }
  }

  // Values that no logit of bin b is below, or above: the bin's edges with
  // room for the roundings of a place.
  __device__ __forceinline__ float floor_of(uint32_t b) const {
    if (b + 1 >= kSmBins || !(scale.inv > 0.0) || scale.m > 1e50) return -3.4028234e38f;
    const double d = ((double)b + 0.5) * scale.unit, x = scale.m - d - (__builtin_fabs(scale.m) + d) * 0x1p-20;
    return x > -3.4e38 ? (float)x : -3.4028234e38f;
  }
  __device__ __forceinline__ float ceiling_of(uint32_t b) const {
    if (b == 0 || !(scale.inv > 0.0) || scale.m > 1e50) return unordered(top);
    const double d = ((double)b - 0.5) * scale.unit, x = scale.m - d + (__builtin_fabs(scale.m) + d) * 0x1p-20;
    return __builtin_fminf(x < 3.4e38 ? (float)x : __builtin_inff(), unordered(top));
  }

  // The tokens of these bits and bins (no more than the list holds) into the
  // list, in order.  What may hold one is noted first, 16 bytes at a time, and
  // looked at again by all threads together.
  __device__ void load(uint32_t from, uint32_t to, uint32_t b0, uint32_t b1, uint32_t n0, uint64_t m0) {
    const int tid = threadIdx.x;
    int* const queue = reinterpret_cast<int*>(s.list_mass);
    constexpr int kQueue = kSmCap * 2;
    __syncthreads();
    if (tid == 0) s.length = s.queued = 0;
    __syncthreads();
    const typename Logits<T, N>::Band band(alike(__builtin_fmaxf(unordered(from), floor_of(b1))),
                                              alike(__builtin_fminf(unordered(to), ceiling_of(b0))));
    const auto take = [&](float x, int id) __attribute__((always_inline)) {
      if (!(x >= band.lo && x <= band.hi)) return;   // NaN and -inf too
      const uint32_t k = ordered(x), b = scale.bin(x);
      if (k < from || k > to || b < b0 || b > b1) return;
      const int at = atomicAdd(&s.length, 1);
      if (at < kSmCap) s.list[at] = ((uint64_t)k << 32) | (uint32_t)~id;
    };
    logits.loads([&](const uint4& r, int v) __attribute__((always_inline)) {
      if (!band.has(r) || v >= logits.v1) return;
      const int at = atomicAdd(&s.queued, 1);
      if (at < kQueue) queue[at] = v;
    });
    __syncthreads();
    if (s.queued <= kQueue) {
      logits.ends(take);
#pragma unroll 1
      for (int e = tid; e < s.queued; e += N) logits.one_by_one(logits.load(queue[e]), logits.first_token(queue[e]), take);
    } else {   // more that may than room to note it
      logits.walk(take);
    }
    __syncthreads();
    const int n = alike(min(s.length, kSmCap));
    if (n <= kSmSmall)
      rank_list(n);
    else
      sort_list(n);
    // weights up to and with each token: a thread takes some neighbours
    constexpr int kSome = kSmCap / N;
    const int some = n <= N ? 1 : kSome, first = tid * some;
    uint64_t mine = 0, all;
#pragma unroll 1
    for (int j = 0; j < some; ++j)
      if (first + j < n) {
        mine += scale.weight(unordered((uint32_t)(s.list[first + j] >> 32)));
        s.list_mass[first + j] = mine;
      }
    const uint64_t less = m0 + block_prefix<N>(mine, s.wave_mass, all) - mine;
#pragma unroll 1
    for (int j = 0; j < some; ++j)
      if (first + j < n) s.list_mass[first + j] += less;
    __syncthreads();
    lo = from;
    hi = to;
    bin0 = b0;
    bin1 = b1;
    before = n0;
    before_mass = m0;
    length = (uint32_t)n;
    mass = alike(all);
  }

  __device__ bool listed(By by, uint64_t goal) const {
    switch (by) {
      case By::kCount: return goal > before && goal <= (uint64_t)before + length;
      case By::kMass: return goal > before_mass && goal <= before_mass + mass;
      default: {
        const uint32_t b = scale.bin(unordered((uint32_t)goal));
        return lo <= hi && goal >= lo && goal <= hi && b >= bin0 && b <= bin1;
      }
    }
  }

  // The goal's place within the list (its last token's, where sums that were
  // rounded otherwise fall short of the goal).
  __device__ __forceinline__ Place in_list(By by, uint64_t goal) {
    const int tid = threadIdx.x;
    uint32_t n = (uint32_t)goal - before;
    if (by != By::kCount) {
      uint32_t& found = answer();
      if (tid == 0 && length == 0) found = 0;
#pragma unroll 1
      for (uint32_t i = tid; i < length; i += N) {
        const bool last = i + 1 == length;
        if (by == By::kKey) {
          const bool here = (s.list[i] >> 32) >= goal;
          if (here && (last || (s.list[i + 1] >> 32) < goal)) found = i + 1;
          if (i == 0 && !here) found = 0;
        } else {
          const bool reached = s.list_mass[i] >= goal;
          if ((reached || last) && (i == 0 || s.list_mass[i - 1] < goal)) found = i + 1;
        }
      }
      __syncthreads();
      n = alike(found);
    }
    if (n == 0) return Place{before, before_mass, (uint32_t)goal, -1};   // bits that none of these has
    const uint64_t e = alike(s.list[n - 1]);
    return Place{before + n, alike(s.list_mass[n - 1]), (uint32_t)(e >> 32), (int32_t)~(uint32_t)e};
  }

  // The n-th token, by place in the row, of those with these bits.
  __device__ int32_t nth_equal(uint32_t key, uint32_t n) {
    const int tid = threadIdx.x;
    const int per = (a.vocab + N - 1) / N;
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
    const uint32_t upto = block_prefix<N>(mine, s.wave_count, all);
    uint32_t& found = answer();
    if (mine && upto - mine < n && upto >= n) {
      uint32_t left = n - (upto - mine);
      int64_t i = first;
      for (; i < last; ++i)
        if (is(i) && --left == 0) break;
      found = (uint32_t)i;
    }
    __syncthreads();
    return (int32_t)alike(found);
  }

  // The goal's place, which the row has.  The histogram holds weights if
  // `goal` may lie past the list's.
  __device__ Place find(By by, uint64_t goal) {
    if (listed(by, goal)) return in_list(by, goal);
    uint32_t b = by == By::kKey ? scale.bin(unordered((uint32_t)goal)) : bin_of(0, by, goal, 0, 0);
    uint32_t n0 = b ? alike(s.count[0][b - 1]) : 0, n = alike(s.count[0][b]) - n0;
    uint64_t m0 = b ? alike(s.mass[0][b - 1]) : 0;
    const uint32_t first = b;
    uint32_t from = kFirstLive, to = top, b0 = b;
    if (n0 + n <= kSmSmall || (n0 + n <= kSmCap && all_mass[0] == 0)) {
      // all that stands before it too: the next goal is likely among them, and
      // is where no weights were counted
      b0 = 0;
      n += n0;
      n0 = 0;
      m0 = 0;
    }
    if (n > kSmCap) {
      from = first_key(b);
      to = b ? first_key(b - 1) - 1 : top;
    }
    while (n > kSmCap && from < to) {   // too many: by their bits
      int shift = 0;
      while ((to - from) >> shift >= kSmBins) ++shift;
      fill(logits, scale, s.mass[1], true, [&](float x, uint32_t in) __attribute__((always_inline)) {
        const uint32_t k = ordered(x);
        return in != first || k < from || k > to ? kSmBins : (to - k) >> shift;
      });
      sum_up(1, true, first);
      b = by == By::kKey ? (to - (uint32_t)goal) >> shift : bin_of(1, by, goal, n0, m0);
      const uint32_t nb = b ? alike(s.count[1][b - 1]) : 0;
      n = alike(s.count[1][b]) - nb;
      n0 += nb;
      m0 += b ? alike(s.mass[1][b - 1]) : 0;
      to -= b << shift;
      from = to - from < (1u << shift) ? from : to - (1u << shift) + 1;
    }
    if (n <= kSmCap) {
      load(from, to, b0, first, n0, m0);
      return in_list(by, goal);
    }
    const uint64_t q = scale.weight(unordered(to));   // n tokens of one value
    const uint64_t by_mass = q ? (goal - m0 + q - 1) / q : n;
    const uint32_t r = by == By::kCount ? (uint32_t)goal - n0 : by == By::kKey || by_mass > n ? n : by_mass ? (uint32_t)by_mass : 1;
    return Place{n0 + r, m0 + r * q, to, nth_equal(to, r)};
  }
};

// A row's settings, with those that are off in numbers that keep all.
struct Settings {
  float temperature, p, low;
  int64_t k;
  bool few;   // a few tokens alone are asked for: no weight is needed but theirs
  __device__ __forceinline__ Settings(const SampleArgs& a, int t)
      : temperature(a.temperature ? a.temperature[t] : 1.0f), p(a.top_p ? a.top_p[t] : 1.0f),
        low(a.min_p ? a.min_p[t] : 0.0f), k(a.top_k ? a.top_k[t] : 0) {
    if (!(temperature > 0.0f) || low > 1.0f) {   // the first alone (above 1 not even its equals stay)
      temperature = 1.0f;
      k = 1;
      p = 1.0f;
      low = 0.0f;
    }
    few = k > 0 && k <= kSmCap / 2;
  }
  // Beside a logit of +inf no other has weight, at no temperature.
  __device__ __forceinline__ void beside(float most) {
    if (most > 3.4028234e38f) temperature = __builtin_fminf(temperature, 3.4028234e38f);
  }
};

// The largest and smallest live logit, in every thread.
template <typename T, int N>
__device__ __forceinline__ float2 range_of(const Logits<T, N>& logits, float2* waves) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  float most = -__builtin_inff(), least = __builtin_inff();
  const auto take = [&](float x) __attribute__((always_inline)) {
    most = __builtin_fmaxf(most, x);   // NaN passes by
    least = __builtin_fminf(least, x > -__builtin_inff() ? x : __builtin_inff());
  };
  logits.loads([&](const uint4& r, int) __attribute__((always_inline)) { logits.values(r, take); });
  logits.ends([&](float x, int) __attribute__((always_inline)) { take(x); });
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    most = __builtin_fmaxf(most, __shfl_xor(most, off));
    least = __builtin_fminf(least, __shfl_xor(least, off));
  }
  if (lane == 0) waves[tid / kWave] = make_float2(most, least);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < N / kWave; ++w) {
    most = __builtin_fmaxf(most, waves[w].x);
    least = __builtin_fminf(least, waves[w].y);
  }
  return make_float2(alike(most), alike(least));
}

// The same of a row whose pieces' are known: a lane asks for one of them, and
// they meet once something else is on its way too.
__device__ __forceinline__ float2 piece_range(const SampleArgs& a, int t) {
  const int lane = threadIdx.x & (kSmPieces - 1);
  return a.ranges[(size_t)t * a.segs + (lane < a.segs ? lane : 0)];
}
__device__ __forceinline__ float2 joined_range(float2 r) {
#pragma unroll
  for (int off = 1; off < kSmPieces; off <<= 1) {
    r.x = __builtin_fmaxf(r.x, __shfl_xor(r.x, off));
    r.y = __builtin_fminf(r.y, __shfl_xor(r.y, off));
  }
  return make_float2(alike(r.x), alike(r.y));
}

template <typename T>
__global__ __launch_bounds__(kSmThreads) void k_sample_range(SampleArgs a) {
  __shared__ float2 waves[kSmThreads / kWave];
  const int t = blockIdx.x / a.segs, seg = blockIdx.x - t * a.segs;
  const Logits<T, kSmThreads> logits(a, t, seg);
  const float2 r = range_of(logits, waves);
  if (threadIdx.x == 0) a.ranges[blockIdx.x] = r;
}

template <typename T>
__global__ __launch_bounds__(kSmThreads) void k_sample_bins(SampleArgs a) {
  __shared__ uint64_t words[kSmBins];
  const int t = blockIdx.x / a.segs, seg = blockIdx.x - t * a.segs;
  const float2 piece = piece_range(a, t);
  Settings set(a, t);
  const Logits<T, kSmThreads> logits(a, t, seg);
  const float2 range = joined_range(piece);
  if (range.x == -__builtin_inff()) return;
  set.beside(range.x);
  const RowScale scale(range.x, range.y, set.temperature, a);
  fill(logits, scale, words, !set.few, [](float, uint32_t b) { return b; });
  for (int b = threadIdx.x; b < kSmBins; b += kSmThreads) a.words[(size_t)blockIdx.x * kSmBins + b] = words[b];
}

// The choice.  PIECES: the pieces' histograms are there, and the rows are few.
// Whole rows are taken by two workgroups a CU, of which one computes while the
// other waits (1024 x 32000 fp32 93 us, 118 with one of twice the threads);
// few rows by one of many threads (64 x 151936 40 us, 46 with half of them).
template <typename T, int N, bool PIECES>
__global__ __launch_bounds__(N, 4) void k_sample(SampleArgs a) {
  constexpr int kPer = kSmBins / N;
  __shared__ Shared<N> s;
  const int t = blockIdx.x, tid = threadIdx.x;
  const Logits<T, N> logits(a, t, -1);
  // All that is known beforehand is asked for at once: each is a way to memory.
  float2 range;
  uint64_t words[PIECES ? kPer : 1][kSmPieces];
  if constexpr (PIECES) {
    range = piece_range(a, t);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int i = 0; i < kSmPieces; ++i)
        words[j][i] = a.words[((size_t)t * a.segs + (i < a.segs ? i : 0)) * kSmBins + tid + j * N];
  }
  Settings set(a, t);
  const float u = a.uniforms[t];
  if constexpr (PIECES)
    range = joined_range(range);
  else
    range = range_of(logits, s.wave_range);
  const float most = range.x, least = range.y;
  if (most == -__builtin_inff()) {   // masked throughout
    if (tid == 0) {
      a.ids[t] = -1;
      if (a.logprob) a.logprob[t] = -__builtin_inff();
      if (a.kept) a.kept[t] = 0;
    }
    return;
  }
  set.beside(most);
  Row<T, N> row{a, t, s, logits, RowScale(most, least, set.temperature, a), ordered(most)};
  bool weights = !set.few;
  uint32_t live = 0;
  if constexpr (PIECES) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      uint64_t word = 0;
#pragma unroll
      for (int i = 0; i < kSmPieces; ++i) word += i < a.segs ? words[j][i] : 0;
      s.mass[0][tid + j * N] = word;
    }
    __syncthreads();
  } else {
    fill(logits, row.scale, s.mass[0], weights, [](float, uint32_t b) { return b; });
  }
#pragma unroll 1
  for (;;) {
    row.sum_up(0, weights);
    live = row.all_count[0];
    if (weights) break;
    // more equal ones than the list holds: weights after all
    const uint32_t want = set.k < live ? (uint32_t)set.k : live;
    if (alike(s.count[0][row.bin_of(0, By::kCount, want, 0, 0)]) <= kSmCap) break;
    weights = true;
    fill(logits, row.scale, s.mass[0], true, [](float, uint32_t b) { return b; });
  }
  const int64_t k = set.k;
  // The places that cut the order, then the one that is drawn, by one copy of
  // the search.  Sums of the same tokens may differ by their roundings (a bin's
  // and its parts', a crowd's of equal ones): no place behind a cut is taken for
  // what is before it.  A uniform of 1 or more leaves no room for them and goes by
  // counts, to the last kept token whose weight is not zero.  (What long
  // functions need is taken before: the compiler would keep their constants in
  // registers throughout.)
  double bound = -(double)__builtin_inff();   // at an infinite temperature all are as likely
  if (set.low > 0.0f && set.temperature < __builtin_inff()) bound = log((double)set.low) * (double)set.temperature;
  Place cut{live, row.all_mass[0], ordered(least), -1}, drawn = cut;
  // The steps: top-k, top-p, min-p, the draw; and seldom, by counts, the last
  // place with weight, and the place that is drawn.
  uint32_t end = 0;
  int steps = alike((int)(u >= 1.0f)) ? 6 : 4;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    By by = By::kMass;
    uint64_t goal = 0;   // none
    if (step == 0 && (set.few || (k > 0 && k < live))) {
      by = By::kCount;
      goal = k < live ? (uint64_t)k : live;
    } else if (step == 1 && set.p < 1.0f) {
      const double at = __builtin_ceil((double)set.p * (double)cut.mass);
      goal = at < 1.0 ? 1 : at >= (double)cut.mass ? cut.mass : (uint64_t)at;
    } else if ((step == 2 && set.low > 0.0f) || step == 4) {
      const double low = step == 2 ? bound : -(a.bits + 1) * 0.6931471805599453 * (double)set.temperature;   // half a unit
      const uint32_t key = row.least_key([&](uint32_t key) __attribute__((always_inline)) {
        const float x = unordered(key);
        return x == most || RowScale::above(x) - row.scale.m >= low;
      });
      by = By::kKey;
      goal = cut.key < key ? key : step == 4 ? cut.key : 0;
    } else if (step == 3) {
      const double at = __builtin_floor((double)u * (double)cut.mass);
      const uint64_t below = !(at > 0.0) ? 0 : at >= (double)cut.mass ? cut.mass - 1 : (uint64_t)at;
      goal = (below < cut.mass ? below : cut.mass - 1) + 1;
    } else if (step == 5) {
      by = By::kCount;
      goal = end;
    }
    if (goal == 0) continue;
    drawn = row.find(by, goal);
    if (step < 3) {
      if (drawn.n <= cut.n) cut = drawn;
    } else if (__builtin_expect(step < 5 && (step == 4 || drawn.n > cut.n), 0)) {
      end = min(drawn.n, cut.n);
      if (steps == 4) {
        step = 4;
        steps = 6;
      }
    }
  }
  if (tid == 0) {
    a.ids[t] = drawn.id;
    if (a.kept) a.kept[t] = (int32_t)cut.n;
    if (a.logprob) {
      const float x = unordered(drawn.key);
      const double d = (RowScale::above(x) - row.scale.m) / (double)set.temperature;
      a.logprob[t] = (float)(d - log(__builtin_ldexp((double)cut.mass, -a.bits)));   // of one token 0, exactly
    }
  }
}

// Pieces of a row: four workgroups a CU for the whole call, where rows are few
// and long.  Three launches take longer than they save on rows of 32000 (1 row
// 22.3 us in pieces, 21.2 whole; 256 rows 42.6 and 33.0) and save on 65536 (1
// row 23.2 and 31.4); more than a row a CU is work enough (256 x 151936: 122 us
// in pieces, 131 whole; 500 x 151936: 188 and 145).
int64_t pieces_of(int64_t tokens, int64_t vocab) {
  if (tokens >= 350 || vocab < 49152) return 1;
  int64_t segs = 1024 / (tokens > 0 ? tokens : 1);
  if (segs > kSmPieces) segs = kSmPieces;
  return segs > vocab / 8192 ? vocab / 8192 : segs;
}

template <typename T>
hipError_t sample_launch(const SampleArgs& a, hipStream_t stream) {
  if (a.segs > 1) {
    k_sample_range<T><<<a.tokens * a.segs, kSmThreads, 0, stream>>>(a);
    k_sample_bins<T><<<a.tokens * a.segs, kSmThreads, 0, stream>>>(a);
    k_sample<T, kSmMany, true><<<a.tokens, kSmMany, 0, stream>>>(a);
  } else {
    k_sample<T, kSmThreads, false><<<a.tokens, kSmThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

int sample_segments(int64_t tokens, int64_t vocab) { return (int)pieces_of(tokens, vocab); }

int64_t sample_workspace_bytes(int64_t tokens, int64_t vocab) {
  const int64_t segs = pieces_of(tokens, vocab);
  return segs == 1 ? 0 : tokens * segs * (int64_t)(sizeof(float2) + kSmBins * sizeof(uint64_t));
}

hipError_t launch_sample(const SampleCall& c, hipStream_t stream) {
  int log = 0;
  while (((int64_t)1 << log) < c.vocab) ++log;
  const int segs = (int)pieces_of(c.tokens, c.vocab);
  SampleArgs a{c.logits, c.uniforms, c.temperature, c.top_k, c.top_p, c.min_p, c.ids, c.logprob, c.kept,
               c.stride, c.tokens, c.vocab, log > 12 ? 62 - log : 50, log > 18 ? 63 - log : 45,
               log > 18 ? 67 - 2 * log : 31, segs, 0, nullptr, nullptr};
  if (segs > 1) {
    a.per = (int32_t)(((c.vocab + 7) / segs + 8) & ~7);   // a piece starts at a multiple of 16 bytes
    a.words = static_cast<uint64_t*>(c.workspace);
    a.ranges = reinterpret_cast<float2*>(a.words + (size_t)c.tokens * segs * kSmBins);
  }
  return c.f32 ? sample_launch<float>(a, stream) : sample_launch<uint16_t>(a, stream);
}

}  // namespace fp8w
