// linear.hip -- a dense layer's product on fp8 weights with its epilogue:
//
//   y = act(x . deq(W)^T + bias) + residual
//
// for any number of rows of x; bf16 x, fp32 sums, one rounding at the end.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act.hpp"
#include "device.hpp"
#include "internal.hpp"

namespace fp8w {
namespace {

// bias of weight row n (0 without)
__device__ __forceinline__ float bias_of(const LinearCall& c, int n) {
  if (!c.bias) return 0.0f;
  return c.bias_f32 ? ld_global<float>(c.bias, (size_t)n * 4) : bf16_lo(ld_global<uint16_t>(c.bias, (size_t)n * 2));
}

// Output (i, n): the residual added, rounded to y's type.
__device__ __forceinline__ void store_one(const LinearCall& c, int i, int n, float v) {
  if (c.residual) v += bf16_lo(ld_global<uint16_t>(c.residual, ((size_t)i * c.residual_stride + n) * 2));
  const size_t at = (size_t)i * c.y_stride + n;
  if (c.y_f32)
    st_global<float>(c.y, at * 4, v);
  else
    st_global<uint16_t>(c.y, at * 2, (uint16_t)f32_to_bf16_rne(v));
}

// MX weights of up to three groups a row, of which the others read four
// exponents at a time: one wave takes 16 weight rows (gated: 16 of each half)
// against 16 rows of x, operands straight from memory.
template <bool GATED>
__global__ __launch_bounds__(256) void k_linear_simple(LinearCall c, int n_groups) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int n_out = GATED ? c.n / 2 : c.n;
  const int m0 = (int)(blockIdx.x / (unsigned)n_groups) * 16;
  const int n0 = ((int)(blockIdx.x % (unsigned)n_groups) * 4 + wave) * 16;
  if (n0 >= n_out) return;
  const int i = lane & 15, g = lane >> 4;
  const int row = min(m0 + i, c.m - 1);
  f32x4 acc[2] = {};
  const int ng = (c.k + 31) / 32;
  for (int first = 0; first < c.k; first += 64) {
    const int col = first + 16 * g;
    const bool in = col < c.k;   // all lanes take part in a product, those past k with zeros
    uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
    if (in) {
      b0 = ld_global_u4(c.x, ((size_t)row * c.x_stride + col) * 2);
      b1 = ld_global_u4(c.x, ((size_t)row * c.x_stride + col) * 2 + 16);
    }
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      const int n = min(n0 + i, n_out - 1) + q * n_out;
      uint4 w = make_uint4(0, 0, 0, 0);
      float s = 1.0f;
      if (in) {
        w = ld_global_u4(c.codes, (size_t)n * c.k + col);
        s = mx_scale(ld_global<uint8_t>(c.scales, (size_t)n * ng + col / 32));
      }
      bf16x8 a0, a1;
      a_operands<true>(w, s, a0, a1);
      acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, b0), acc[q], 0, 0, 0);
      acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, b1), acc[q], 0, 0, 0);
    }
  }
  if (m0 + i >= c.m) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int n = n0 + 4 * g + v;
    if (n >= n_out) continue;
    float r[2];
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) r[q] = acc[q][v] + bias_of(c, n + q * n_out);
    store_one(c, m0 + i, n, GATED ? gated(c.act, r[0], r[1]) : c.act == kActGelu ? gelu(r[0]) : activated(c.act, r[0]));
  }
}

// Four neighbouring outputs of a row: what they take besides their sums
// (gated: g's and u's), asked for ahead of its use and kept as it comes (a
// conversion next to its load would wait for it), and the end.
template <int FMT, bool GATED>
struct FourOutputs {
  static constexpr int kHalves = GATED ? 2 : 1;
  f32x4 scale[kHalves];
  uint32_t bias[kHalves][4], residual[4];
  int row, n, n_out;

  __device__ __forceinline__ FourOutputs(const LinearCall& c, int r, int at) : row(r), n(at), n_out(GATED ? c.n / 2 : c.n) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int w = min(n + j, n_out - 1) + h * n_out;
        scale[h][j] = FMT == kFmtRow ? ld_global<float>(c.scales, (size_t)w * 4) : FMT == kFmtTensor ? ld_global<float>(c.scales, 0) : 1.0f;
        bias[h][j] = 0;
      }
    if (c.bias) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int w = min(n + j, n_out - 1) + h * n_out;
          bias[h][j] = c.bias_f32 ? ld_global<uint32_t>(c.bias, (size_t)w * 4) : ld_global<uint16_t>(c.bias, (size_t)w * 2);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) residual[j] = 0;
    if (c.residual) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        residual[j] = ld_global<uint16_t>(c.residual, ((size_t)row * c.residual_stride + min(n + j, n_out - 1)) * 2);
    }
  }
  __device__ __forceinline__ float biased(const LinearCall& c, int h, int j, float sum) const {
    return __builtin_fmaf(scale[h][j], sum, __uint_as_float(c.bias_f32 ? bias[h][j] : bias[h][j] << 16));
  }
  __device__ __forceinline__ void finish(const LinearCall& c, f32x4 v, f32x4 u) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = biased(c, 0, j, v[j]);
      if constexpr (GATED) v[j] = gated(c.act, v[j], biased(c, 1, j, u[j]));
    }
    if constexpr (!GATED) {
      if (c.act == kActGelu) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = gelu(v[j]);
      } else if (c.act != kActNone) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = activated(c.act, v[j]);
      }
    }
    if (c.residual) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += bf16_lo(residual[j]);
    }
    const size_t to = (size_t)row * c.y_stride + n;
    if (n + 4 <= n_out && c.y_stride % 4 == 0 && reinterpret_cast<uintptr_t>(c.y) % 16 == 0) {
      if (c.y_f32)
        st_global<f32x4>(c.y, to * 4, v);
      else
        st_global<u32x2>(c.y, to * 2, u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= n_out) break;
      if (c.y_f32)
        st_global<float>(c.y, (to + j) * 4, v[j]);
      else
        st_global<uint16_t>(c.y, (to + j) * 2, (uint16_t)f32_to_bf16_rne(v[j]));
    }
  }
};

// 16 bytes a lane from memory to LDS at `to` + 16 * lane (`to` uniform).
__device__ __forceinline__ void stage16(const void* from, unsigned char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Block scale `at` (uniform), by a scalar load: there are none of two bytes, and
// a vector load would be waited for with all that left before it.  For a bf16
// scale the aligned word it lies in is read: at either end of the buffer that may
// be two bytes outside it, in the same page, whose value is dropped.
template <int FMT>
__device__ __forceinline__ float scalar_scale(const char* scales, int at) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(scales) + (size_t)at * (FMT == kFmtBlock ? 4 : 2);
  if constexpr (FMT == kFmtBlock) return *reinterpret_cast<const __attribute__((address_space(4))) float*>(p);
  const uint32_t both = *reinterpret_cast<const __attribute__((address_space(4))) uint32_t*>(p & ~(uintptr_t)3);
  return __uint_as_float(p & 2 ? both & 0xFFFF0000u : both << 16);
}

// What x holds past its columns.
__device__ const uint4 kNoColumns = {0, 0, 0, 0};

// s_waitcnt vmcnt(n) lgkmcnt(0), n < 64, then the workgroup's barrier.  The
// LDS reads before it have returned, so that what they read may be
// overwritten after it; and all but the wave's last n loads have landed.
template <int N>
__device__ __forceinline__ void land_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// These 16 values are computed here, not where the compiler would rather.
__device__ __forceinline__ void settle(float (&v)[16]) {
  asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]),
               "+v"(v[8]), "+v"(v[9]), "+v"(v[10]), "+v"(v[11]), "+v"(v[12]), "+v"(v[13]), "+v"(v[14]), "+v"(v[15]));
}

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32_unaligned __attribute__((aligned(1)));

// A wave's number among the four that share a tile's columns.
__device__ __forceinline__ int wave_of_four() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave % 4); }

// Where a workgroup works: a tile of x's rows and of outputs, and a slice of
// k's 128-column blocks.
struct LinearTile {
  int m0, count, group, kb0, kb1;
  int turn;   // how far into its columns it starts: XCDs do not all read the same ones
};

// How the tiles of a call are laid out.  Workgroups go round the 8 XCDs in
// turn, and each XCD has its own L2: it gets one contiguous eighth of the
// tiles, the tiles of one group of weight rows next to each other.
struct LinearGrid {
  int tiles_m, groups, splits;
  __device__ __forceinline__ bool at(int height, int m, int nkb, LinearTile& t, int64_t& id) const {
    const int64_t total = (int64_t)tiles_m * groups * splits, share = (total + 7) / 8;
    id = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= share || id >= total) return false;
    const uint32_t pair = (uint32_t)id / (uint32_t)tiles_m;
    t.m0 = (int)((uint32_t)id - pair * (uint32_t)tiles_m) * height;
    t.count = min(height, m - t.m0);
    const uint32_t split = pair / (uint32_t)groups;
    t.group = (int)(pair - split * (uint32_t)groups);
    t.kb0 = (int)((int64_t)nkb * split / splits);
    t.kb1 = (int)((int64_t)nkb * (split + 1) / splits);
    t.turn = (int)(blockIdx.x & 7);
    return true;
  }
};

// The tiled kernels' wave: 32 * TW weight rows (gated: half of them of each
// half of W) against 32 * MT rows of x.
template <bool GATED, int TW>
struct WaveRows {
  static constexpr int kRows = 32 * TW;
  static constexpr int kCols = GATED ? kRows / 2 : kRows;   // outputs of a row
  int n0, n_out;
  __device__ __forceinline__ WaveRows(const LinearCall& c, int group, int wave)
      : n0((group * 4 + wave) * kCols), n_out(GATED ? c.n / 2 : c.n) {}
  // Row r of the wave's (r may be uniform or a lane's): output out_row(r),
  // weight row half(r) further on.
  __device__ __forceinline__ int out_row(int r) const { return n0 + r % kCols; }
  __device__ __forceinline__ int half(int r) const { return r >= kCols ? n_out : 0; }
};

// The end of a tile.  A lane holds x's row 32q + l%32 and, for each v4, weight
// rows 8 v4 + 4 (l / 32) .. + 3 of each tile of 32: sums are scaled, and the
// bias added, where they are; 32 rows at a time then go through the wave's own
// LDS in fp32 (16-byte units swizzled), so that the residual is read and the
// results written as whole lines.
template <int FMT, bool GATED, int MT, int TW, typename Acc>
__device__ __forceinline__ void finish_tile(const LinearCall& c, const LinearTile& at, Acc (&acc)[TW][MT], unsigned char* wl) {
  using Rows = WaveRows<GATED, TW>;
  constexpr int kCols = Rows::kCols, kUnits = kCols / 4;   // 16-byte units of a row of results
  const int lane = threadIdx.x & (kWave - 1), wave = wave_of_four();
  const int i = lane & 31, hh = lane >> 5;
  const Rows w(c, at.group, wave);
  if (FMT == kFmtRow || FMT == kFmtTensor || c.bias) {
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = 32 * t + 8 * (v >> 2) + 4 * hh + (v & 3), n = min(w.out_row(r), w.n_out - 1) + w.half(r);
        const float s = FMT == kFmtRow ? ld_global<float>(c.scales, (size_t)n * 4) : FMT == kFmtTensor ? ld_global<float>(c.scales, 0) : 1.0f;
        const float b = bias_of(c, n);
#pragma unroll
        for (int q = 0; q < MT; ++q) acc[t][q][v] = __builtin_fmaf(s, acc[t][q][v], b);
      }
  }
  if (!GATED && (c.act == kActSilu || c.act == kActGeluTanh || c.act == kActRelu)) {
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[t][q][v] = activated(c.act, acc[t][q][v]);
  }
  const bool vec = c.y_stride % 8 == 0 && reinterpret_cast<uintptr_t>(c.y) % 16 == 0 &&
                   (!c.residual || (c.residual_stride % 8 == 0 && reinterpret_cast<uintptr_t>(c.residual) % 16 == 0));
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    if (32 * q >= at.count) break;
#pragma unroll
    for (int u = 0; u < kCols / 8; ++u) {   // outputs 8u + 4 (l / 32) .. + 3 of the wave's
      const auto sum = [&](int r, int v) { return acc[r / 32][q][r % 32 / 2 + v]; };   // of row r + 4 (l / 32) + v
      f32x4 r;
#pragma unroll
      for (int v = 0; v < 4; ++v) r[v] = GATED ? gated(c.act, sum(8 * u, v), sum(8 * u + kCols, v)) : sum(8 * u, v);
      *reinterpret_cast<f32x4*>(wl + i * 4 * kCols + 16 * ((2 * u + hh) ^ (i & (kUnits - 1)))) = r;
    }
    asm volatile("" ::: "memory");
    if (!GATED && c.act == kActGelu) {   // erfc is long: once in the code, not for every sum
#pragma unroll 1
      for (int j = 0; j < kCols / 8; ++j) {
        f32x4* at4 = reinterpret_cast<f32x4*>(wl + 16 * (j * kWave + lane));
        f32x4 r = *at4;
#pragma unroll
        for (int v = 0; v < 4; ++v) r[v] = gelu(r[v]);
        *at4 = r;
      }
      asm volatile("" ::: "memory");
    }
    if (!vec) {   // rows that start anywhere: an output a lane
      const int col = lane % kCols, n = w.n0 + col;
#pragma unroll 4
      for (int r = lane / kCols; r < min(32, at.count - 32 * q); r += kWave / kCols) {
        const float v = *reinterpret_cast<const float*>(wl + r * 4 * kCols + 16 * ((col >> 2) ^ (r & (kUnits - 1))) + 4 * (col & 3));
        if (n < w.n_out) store_one(c, at.m0 + 32 * q + r, n, v);
      }
      asm volatile("" ::: "memory");
      continue;
    }
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j) {   // 8 outputs a lane
      constexpr int kLanes = kCols / 8;      // lanes of a row
      const int r = j * (kWave / kLanes) + lane / kLanes, u = lane % kLanes, n = w.n0 + 8 * u;
      const f32x4 v0 = *reinterpret_cast<const f32x4*>(wl + r * 4 * kCols + 16 * ((2 * u) ^ (r & (kUnits - 1))));
      const f32x4 v1 = *reinterpret_cast<const f32x4*>(wl + r * 4 * kCols + 16 * ((2 * u + 1) ^ (r & (kUnits - 1))));
      if (32 * q + r >= at.count || n >= w.n_out) continue;
      const int row = at.m0 + 32 * q + r;
      float o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = v0[e];
        o[4 + e] = v1[e];
      }
      if (n + 8 > w.n_out) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < w.n_out) store_one(c, row, n + e, o[e]);
        continue;
      }
      if (c.residual) {
        const uint4 x = ld_global_u4(c.residual, ((size_t)row * c.residual_stride + n) * 2);
        const uint32_t d[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] += bf16_lo(d[e]);
          o[2 * e + 1] += bf16_hi(d[e]);
        }
      }
      const size_t to = (size_t)row * c.y_stride + n;
      if (c.y_f32) {
        st_global<f32x4>(c.y, to * 4, f32x4{o[0], o[1], o[2], o[3]});
        st_global<f32x4>(c.y, to * 4 + 16, f32x4{o[4], o[5], o[6], o[7]});
      } else {
        st_global<u32x4>(c.y, to * 2, u32x4{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]), bf16_pair(o[4], o[5]), bf16_pair(o[6], o[7])});
      }
    }
    asm volatile("" ::: "memory");
  }
}

// A slice's sums to the workspace as the lanes hold them, and back: whole
// lines either way.
template <int MT, int TW, typename Acc, typename F>
__device__ __forceinline__ void each_sum(Acc (&acc)[TW][MT], const F& f) {
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int a = 0; a < 4; ++a) f(((t * MT + q) * 4 + a) * 4096, &acc[t][q], 4 * a);
}
template <int MT, int TW>
constexpr int64_t slice_bytes() { return (int64_t)TW * MT * 4 * 4096; }

// The tiled kernel: 128 * TW weight rows against 32 * MT rows of x on the
// 32x32x16 MFMA, four waves of 32 * TW rows (gated: half of them of each half
// of W), two (TW = 2) or four workgroups a CU.
//
// Everything reaches LDS by loads that write it directly, in whole 128-byte
// lines.
//   * Weights: a wave's rows of a 128-column block are its own 4 * TW KB.  At
//     the start of a block it takes them into registers in the A layout and
//     asks for the next block at once: a block's time to arrive.
//   * x: half of the columns of the block (64-row tiles of four waves: half of
//     the rows) for all four waves, three buffers, asked for two steps ahead;
//     one barrier a step.
// Eight waves (a CU has one such workgroup) have room for two blocks of each,
// weights two blocks ahead and one barrier a block: 203 x 6144 x 4096 MX 26.9
// us, 28.9 without on the same card; 64 x 24576 x 4096 29.0 and 32.5; 512 x 4096
// x 12288 64 and 69.5; with few rounds it gives nothing (384 x 4096 x 4096 25.7).
// The waits name how many younger loads may still be on their way; a wait
// for everything would put the memory's latency into every step.
//
// A lane's 16 bytes of codes are two MFMA steps of 8 columns each, so step
// (p, s) takes columns 32p + 16(l/32) + 8s of the block, for weights and x
// alike.  LDS rows are 128 or 256 bytes, their 16-byte units XOR-swizzled by
// row / 2 or the row, so that any 16 consecutive rows fall into 16 different
// bank groups.
//
// A block scale multiplies a step's sums of 32 rows at a time (sums of all rows
// would need as many registers as the accumulators).  With half of the rows a
// step that is once for 128 columns instead of twice: 512 x 6144 x 4096 44 us,
// 46 otherwise; 128-row tiles have no registers for it (a block's operands are
// 64 of them), and spilled 300.  As they are they spill 93 with block scales and
// gates and 11 with block scales alone, before and after the loop over blocks,
// which has none.  MX scales multiply the codes as they become bf16 (exact); row
// and tensor scales the results.
//
// Measured: 2048 x 24576 x 4096 gated 400-410 us with block scales (1010 TFLOP/s),
// 335 with row scales (1230; the library's bf16 product of dequantized weights
// 320); 1777 x 4096 x 12288 row scales 172 (1040; 158).  There a wave's
// products of a block take 2048 clocks, and its VALU 2000 (block) or 900 (row):
// what is missing is their overlap at two waves a SIMD.  203 x 6144 x 4096 MX
// 24-28 us by card: 192 tiles' 16 rounds of loads, products and barriers, 1.6 us
// each.  32 x 24576 x 4096 gated 25.9 us: HBM, 3.9 TB/s.
template <int FMT, bool GATED, int MT, int TW, int KW, bool BORDER>
__device__ __forceinline__ void linear_run(const LinearCall& c, const LinearTile& at, float* partial, unsigned char* ws,
                                           unsigned char* xs0, unsigned char* xs1, unsigned char* xs2,
                                           unsigned char* xs3, unsigned char* ws1) {
  constexpr bool kBlock = FMT == kFmtBlock || FMT == kFmtBlockBf16;
  constexpr bool kMx = FMT == kFmtMx;
  using Rows = WaveRows<GATED, TW>;
  constexpr int kRows = Rows::kRows;
  constexpr int kXLoads = MT;          // x loads of a wave and step (1 KB each)
  constexpr int kWLoads = 4 * TW;      // weight loads of a wave and block
  constexpr bool kDeep = KW == 2;      // two blocks of weights and of x at a time
  constexpr bool kTall = MT == 2 && KW == 1;   // a step is half of the rows, else half of the columns
  constexpr int kStepQ = kTall ? MT / 2 : MT, kStepU = kTall ? 8 : 4;   // rows / 32, columns / 16
  constexpr int kUnits = 2 * kStepU, kPerLoad = kWave / kUnits;        // 16 bytes of a row, rows of a load
  const int lane = threadIdx.x & (kWave - 1), wave = wave_of_four();
  const int i = lane & 31, hh = lane >> 5;
  const int k = c.k, nkb = (k + 127) / 128, ng = (k + 31) / 32;
  const Rows w(c, at.group, wave);
  const int n_out = w.n_out;
  // Of KW groups of four waves each takes a part of the columns, as many blocks
  // as the others (their barriers are the workgroup's); what is past the slice
  // becomes past k, where all is zeros.
  const int part = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / 256);
  const int blocks = (at.kb1 - at.kb0 + KW - 1) / KW, first_block = at.kb0 + part * blocks;
  int turned = at.turn % blocks, here = turned;
  const auto block_now = [&]() {
    const int b = first_block + turned;
    return KW == 1 || b < at.kb1 ? b : nkb;
  };
  int kb = block_now();   // the block in hand
  const auto next_block = [&]() {
    turned = turned + 1 < blocks ? turned + 1 : 0;
    return block_now();
  };
  // (By the wave's number in the workgroup: as a part's four waves' the compiler
  // takes what is on its way to x's LDS to be on its way here.)
  unsigned char* const wl = ws + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * kRows * 128;
  unsigned char* const wl1 = ws1 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * kRows * 128;   // (kDeep)

  // Load j of a wave's weights brings rows 8j + l/8; LDS place l%8 of a row
  // holds its unit (l%8) ^ (row / 2 % 8), so j odd the unit of j even ^ 4.
  // Rows past the end are the last one, columns past it the last ones (zeroed
  // by take_w, and in x by no_columns, so that no infinity of a column that is
  // read in their place meets them).  No branches: a load that two paths share is
  // one the compiler takes to write any of the arrays.  Offsets pass through
  // an empty asm statement where they are used: the addresses of all loads
  // would otherwise be kept in registers throughout.
  const int wu = (lane & 7) ^ (lane >> 4);
  uint32_t wrow = (uint32_t)(lane >> 3) * (uint32_t)k;
  int wcol = 16 * wu;
  const auto load_w = [&](int kb, int j, unsigned char* to) __attribute__((always_inline)) {
    asm volatile("" : "+v"(wrow), "+v"(wcol)::"memory");
    const uint32_t c0 = (uint32_t)kb * 128 + (uint32_t)(wcol ^ (j & 1) * 64);
    const int row = min(w.out_row(8 * j), n_out - 1);
    const uint32_t within = (uint32_t)min(n_out - 1 - row, 7) * (uint32_t)k;
    stage16(c.codes + (size_t)(row + w.half(8 * j)) * k + (min(wrow, within) + min(c0, (uint32_t)k - 16)), to + j * 1024);
    asm volatile("" ::: "memory");
  };
  const auto request_w = [&](int kb, unsigned char* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) load_w(kb, j, to);
  };
  // x rows a wave stages: kPerLoad (MT * wave + j) + l / kUnits of the step's,
  // place l % kUnits with unit (l % kUnits) ^ row % 16 (of 8: row / 2 % 8 = 4
  // (row / 8 % 2) + l / 16).  Offsets within a load's rows have 32 bits.
  const uint32_t x_row = 2 * (uint32_t)c.x_stride;
  uint32_t xrow = (uint32_t)(lane / kUnits) * x_row;
  int xcol = kTall ? 8 * ((lane & 15) ^ (lane >> 4) ^ (kXLoads * wave & 3) * 4) : 8 * (wu ^ (kXLoads * wave & 1) * 4);
  const auto load_x = [&](int kb, int h, int j, unsigned char* to) __attribute__((always_inline)) {
    asm volatile("" : "+v"(xcol), "+v"(xrow)::"memory");
    const uint32_t c0 = (uint32_t)kb * 128 + (kTall ? 0 : 64 * h) + (uint32_t)(xcol ^ (j & (kTall ? 3 : 1)) * 32);
    const int row = min(kPerLoad * (kXLoads * wave + j) + (kTall ? 16 * MT * h : 0), at.count - 1);
    const uint32_t within = (uint32_t)min(at.count - 1 - row, kPerLoad - 1) * x_row;
    stage16(reinterpret_cast<const char*>(c.x) + (size_t)(at.m0 + row) * x_row + (min(xrow, within) + 2 * min(c0, (uint32_t)k - 8)),
            to + (kXLoads * wave + j) * 1024);
    asm volatile("" ::: "memory");
  };
  const auto request_x = [&](int kb, int h, unsigned char* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) load_x(kb, h, j, to);
  };

  // scales of the next block: a float a run of rows that lie in one scale
  // block (a half's, or a 32-row tile; scalar loads), or two where the second
  // half's blocks begin anywhere (BORDER); or the four MX exponents of the
  // lane's row in each tile
  static_assert(!BORDER || (kBlock && GATED && TW == 1), "runs of 16 rows");
  constexpr int kScales = kMx ? TW : GATED ? 2 : TW;
  const auto scale_of = [](int t, int v) { return GATED && TW == 1 ? v >> 3 : t; };   // of sum v of tile t
  const char* sp[kScales];
  float sc[kScales], after[BORDER ? kScales : 1];
  int border[BORDER ? kScales : 1], down[BORDER ? kScales : 1];
  uint32_t ex[kScales];
#pragma unroll
  for (int t = 0; t < kScales; ++t) {
    const int first = t * (kRows / kScales);
    const char* scales = static_cast<const char*>(c.scales);
    if constexpr (BORDER) {
      const int row = min(w.out_row(first), n_out - 1) + w.half(first);
      border[t] = 128 - row % 128;
      down[t] = row / 128 < (c.n - 1) / 128 ? nkb : 0;
    }
    if (kBlock) sp[t] = scales + (size_t)((min(w.out_row(first), n_out - 1) + w.half(first)) / 128) * nkb * (FMT == kFmtBlock ? 4 : 2);
    if (kMx) sp[t] = scales + (size_t)(min(w.out_row(32 * t + i), n_out - 1) + w.half(32 * t + i)) * ng;
  }
  const auto request_s = [&](int b) __attribute__((always_inline)) {
    const int kb = KW == 1 ? b : min(b, nkb - 1);
#pragma unroll
    for (int t = 0; t < kScales; ++t) {
      const auto scale = [&](int at) {
        return scalar_scale<FMT>(sp[t], at);
      };
      if (kBlock) sc[t] = scale(kb);
      if constexpr (BORDER) after[t] = scale(kb + down[t]);
      // four bytes that end with the row's last, where the block has fewer
      if (kMx) ex[t] = ld_global<u32_unaligned>(sp[t], (size_t)min(4 * kb, ng - 4));
    }
  };

  // the sums: single registers where scales are applied to them, else the
  // MFMA's own
  std::conditional_t<kBlock, float[16], f32x16> acc[TW][MT];
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[t][q][v] = 0.0f;

  uint4 wr[TW][4];                 // tile, 32-column pair of the block
  bf16x8 a[TW][kStepU];            // the same as operands
  float s[kScales], s_after[BORDER ? kScales : 1];
  uint32_t e[TW];
  const auto scale_now = [&](int t, int v) {   // of sum v of tile t
    const int run = scale_of(t, v);
    if constexpr (BORDER) return 8 * (v >> 2 & 1) + 4 * hh + (v & 3) < border[run] ? s[run] : s_after[run];
    return s[run];
  };
  const auto take_w = [&](int kb, int next, const unsigned char* wl) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        wr[t][p] = *reinterpret_cast<const uint4*>(&wl[(32 * t + i) * 128 + 16 * ((2 * p + hh) ^ (i >> 1 & 7))]);
    if ((uint32_t)kb * 128 + 128 > (uint32_t)k) {
      const uint32_t from = (uint32_t)kb * 128 + 16 * (lane_fresh() >> 5);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int t = 0; t < TW; ++t)
          if (from + 32 * p >= (uint32_t)k) wr[t][p] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < kScales; ++t) {
      if (kBlock) s[t] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sc[t])));   // stays scalar
      if constexpr (BORDER) s_after[t] = after[t];
      if (kMx) e[t] = ex[t] >> (8 * (4 * kb - min(4 * kb, ng - 4)) & 31);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): the codes are in registers
    request_s(next);
    __builtin_amdgcn_sched_barrier(0);
  };
  // A step.  Scaled sums are settled after every 32 rows: left alone the
  // compiler starts all products first, each with sums of its own, and spills.
  const auto step = [&](int h, const unsigned char* xb, const auto& load) __attribute__((always_inline)) {
    const auto read_b = [&](int n) __attribute__((always_inline)) {
      const int q = n / kStepU, u = n % kStepU;
      return *reinterpret_cast<const bf16x8*>(
          &xb[(32 * q + i) * 16 * kUnits + 16 * ((4 * (u >> 1) + 2 * hh + (u & 1)) ^ (kTall ? i & 15 : i >> 1 & 7))]);
    };
    const auto operands = [&](int p, int from) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < TW; ++t)
        a_operands<kMx>(wr[t][from], kMx ? mx_scale((uint8_t)(e[t] >> 8 * from)) : 1.0f, a[t][2 * p], a[t][2 * p + 1]);
    };
    bf16x8 b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) b[u] = read_b(u);
    if (!kTall || h == 0) {
#pragma unroll
      for (int p = 0; p < kStepU / 2; ++p) operands(p, kTall ? p : 2 * h + p);
    }
#pragma unroll
    for (int q = 0; q < kStepQ; ++q) {
      const int rows = kTall ? h * kStepQ + q : q;
      f32x16 part[TW];
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        if constexpr (kBlock) {
#pragma unroll
          for (int v = 0; v < 16; ++v) part[t][v] = 0.0f;
        } else {
          part[t] = acc[t][rows];
        }
      }
#pragma unroll
      for (int u = 0; u < kStepU; ++u) {
        const int n = q * kStepU + u;
#pragma unroll
        for (int t = 0; t < TW; ++t) part[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[t][u], b[u & 3], part[t], 0, 0, 0);
        // the operand's register is free: what is four products on into it
        if (n + 4 < kStepQ * kStepU) b[u & 3] = read_b(n + 4);
        if (TW == 2) load(n);
        if (n + 1 < kStepQ * kStepU) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        if constexpr (kBlock) {
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[t][rows][v] = __builtin_fmaf(scale_now(t, v), part[t][v], acc[t][rows][v]);
          settle(acc[t][rows]);
        } else {
          acc[t][rows] = part[t];
        }
      }
    }
  };
  // Where a block of any of the groups reaches past k (the last one, or one past
  // the slice), x's columns there become zeros once they have landed.
  const auto no_columns = [&](int h, unsigned char* xb) __attribute__((always_inline)) {
    bool any = false;
#pragma unroll
    for (int p = 0; p < KW; ++p) {
      const int b = at.kb0 + p * blocks + here;
      any |= b >= at.kb1 || (uint32_t)b * 128 + 128 > (uint32_t)k;
    }
    if (__builtin_expect(!any, 1)) return;
    const int from = (int)min((uint32_t)k - min((uint32_t)kb * 128, (uint32_t)k), 128u) - (kTall ? 0 : 64 * h);   // columns there are
#pragma unroll 1
    for (int u = wave * kWave + lane_fresh(); u < 256 * MT; u += 256) {
      const int row = u / kUnits, unit = u % kUnits ^ (kTall ? row & 15 : row >> 1 & 7);
      if (8 * unit >= from) *reinterpret_cast<uint4*>(xb + 16 * u) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  };
  // A block of 128 columns: its two steps' x are in x0 and x1, and
  // the two after them go to x2 and x0.
  const auto block = [&](unsigned char* x0, unsigned char* x1, unsigned char* x2) __attribute__((always_inline)) {
    here = turned;
    const int next = next_block();   // the last block asks for one nobody takes
    take_w(kb, next, wl);
    const auto first = [&](int n) __attribute__((always_inline)) {   // 4 MT places for 8 + MT loads
      const int to = (n + 1) * (kWLoads + kXLoads) / (4 * MT);
#pragma unroll
      for (int j = n * (kWLoads + kXLoads) / (4 * MT); j < to; ++j) {
        if (j < kWLoads)
          load_w(next, j, wl);
        else
          load_x(next, 0, j - kWLoads, x2);
      }
    };
    const auto second = [&](int n) __attribute__((always_inline)) {
      if (n % 4 == 0) load_x(next, 1, n / 4, x0);
    };
    if (TW == 1) {
      request_w(next, wl);
      request_x(next, 0, x2);
      __builtin_amdgcn_sched_barrier(0);
    }
    no_columns(0, x0);
    step(0, x0, first);
    land_and_meet<kWLoads + kXLoads>();           // younger than x1's: weights and x2's
    if (TW == 1) request_x(next, 1, x0);
    no_columns(1, x1);
    step(1, x1, second);
    land_and_meet<kXLoads>();                     // the weights and x2's have landed
    kb = next;
  };

  // The same with room for two: its steps' x are in x0 and x1, the next block's
  // go to y0 and y1 and the second next's weights where its own are, so that
  // weights have two blocks' time to arrive, and one barrier does.
  const auto deep_block = [&](unsigned char* x0, unsigned char* x1, unsigned char* y0, unsigned char* y1,
                              unsigned char* w) __attribute__((always_inline)) {
    const auto none = [](int) {};
    here = turned;
    const int next = next_block(), after_next = turned + 1 < blocks ? turned + 1 : 0;
    take_w(kb, next, w);
    request_x(next, 0, y0);
    request_x(next, 1, y1);
    request_w(first_block + after_next < at.kb1 ? first_block + after_next : nkb, w);
    __builtin_amdgcn_sched_barrier(0);
    no_columns(0, x0);
    no_columns(1, x1);
    step(0, x0, none);
    step(1, x1, none);
    land_and_meet<kWLoads>();                     // all but the weights just asked for
    kb = next;
  };

  request_s(kb);
  request_w(kb, wl);
  request_x(kb, 0, xs0);
  request_x(kb, 1, xs1);
  int left = blocks;
  if constexpr (kDeep) {
    const int second = turned + 1 < blocks ? turned + 1 : 0;
    request_w(first_block + second < at.kb1 ? first_block + second : nkb, wl1);
    land_and_meet<kWLoads>();
#pragma unroll 1
    for (; left > 1; left -= 2) {
      deep_block(xs0, xs1, xs2, xs3, wl);
      deep_block(xs2, xs3, xs0, xs1, wl1);
    }
    if (left > 0) deep_block(xs0, xs1, xs2, xs3, wl);
  } else {
    land_and_meet<kXLoads>();
#pragma unroll 1
    for (; left > 2; left -= 3) {
      block(xs0, xs1, xs2);
      block(xs2, xs0, xs1);
      block(xs1, xs2, xs0);
    }
    if (left > 0) block(xs0, xs1, xs2);
    if (left > 1) block(xs2, xs0, xs1);
  }
  vm_wait_all();   // nothing may land in LDS that is no longer ours

  if constexpr (KW > 1) {   // the groups' sums meet in the first's registers, in their order
    static_assert((KW - 1) * MT <= KW, "they have the weights' LDS");
    __syncthreads();
    if (part > 0)
      each_sum<MT, TW>(acc, [&](int off, auto* from, int a) {
        *reinterpret_cast<f32x4*>(ws + (part - 1) * slice_bytes<MT, TW>() + off + (threadIdx.x & 255) * 16) =
            f32x4{(*from)[a], (*from)[a + 1], (*from)[a + 2], (*from)[a + 3]};
      });
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int p = 0; p < KW - 1; ++p)
        each_sum<MT, TW>(acc, [&](int off, auto* to, int a) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(ws + p * slice_bytes<MT, TW>() + off + threadIdx.x * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) (*to)[a + e] += v[e];
        });
    }
    __syncthreads();   // the tile's end writes over them
    if (part > 0) return;
  }
  if (partial) {
    each_sum<MT, TW>(acc, [&](int off, auto* sums, int a) {
      st_global<f32x4>(partial, (size_t)off + threadIdx.x * 16, f32x4{(*sums)[a], (*sums)[a + 1], (*sums)[a + 2], (*sums)[a + 3]});
    });
    return;
  }
  finish_tile<FMT, GATED, MT, TW>(c, at, acc, wl);
}

template <int FMT, bool GATED, int MT, int TW, int KW, bool BORDER>
__global__ __launch_bounds__(256 * KW, TW == 2 || KW == 2 || BORDER ? 2 : 4) void k_linear_tile(LinearCall c, LinearGrid grid) {
  // separate arrays: the compiler then knows that reads of one need not wait
  // for what is on its way into another
  __shared__ __attribute__((aligned(16))) unsigned char ws[KW * 4 * 32 * TW * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs0[KW * 32 * MT * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs1[KW * 32 * MT * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs2[KW * 32 * MT * 128];
  // (KW = 2 alone)
  __shared__ __attribute__((aligned(16))) unsigned char xs3[KW * 32 * MT * 128];
  __shared__ __attribute__((aligned(16))) unsigned char ws1[KW * 4 * 32 * TW * 128];
  const int part = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / 256);
  LinearTile at;
  int64_t id;
  if (!grid.at(32 * MT, c.m, (c.k + 127) / 128, at, id)) return;
  float* partial = grid.splits == 1 ? nullptr
                                    : reinterpret_cast<float*>(static_cast<char*>(c.workspace) + id * slice_bytes<MT, TW>());
  linear_run<FMT, GATED, MT, TW, KW, BORDER>(c, at, partial, ws, xs0 + part * 32 * MT * 128,
                                     xs1 + part * 32 * MT * 128, xs2 + part * 32 * MT * 128,
                                     KW == 2 ? xs3 + part * 32 * MT * 128 : xs0, KW == 2 ? ws1 : ws);
}

// The slices' sums added, in their order, and the tile's end.
template <int FMT, bool GATED, int MT, int TW>
__global__ __launch_bounds__(256) void k_linear_join(LinearCall c, LinearGrid grid) {
  __shared__ __attribute__((aligned(16))) unsigned char ws[4 * 32 * TW * 128];
  const int splits = grid.splits;
  grid.splits = 1;
  LinearTile at;
  int64_t id;
  if (!grid.at(32 * MT, c.m, 1, at, id)) return;
  const int64_t stride = (int64_t)grid.tiles_m * grid.groups * slice_bytes<MT, TW>();
  float acc[TW][MT][16];
  each_sum<MT, TW>(acc, [&](int off, auto* sums, int a) {
    f32x4 v = ld_global<f32x4>(c.workspace, (size_t)(id * slice_bytes<MT, TW>() + off) + threadIdx.x * 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) (*sums)[a + e] = v[e];
  });
  for (int p = 1; p < splits; ++p)
    each_sum<MT, TW>(acc, [&](int off, auto* sums, int a) {
      f32x4 v = ld_global<f32x4>(c.workspace, (size_t)(p * stride + id * slice_bytes<MT, TW>() + off) + threadIdx.x * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) (*sums)[a + e] += v[e];
    });
  finish_tile<FMT, GATED, MT, TW>(c, at, acc, ws + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * 32 * TW * 128);
}

// The streaming kernel, for few rows of x: 16 * NT weight rows (gated: half of
// them of each half of W) against 16 * MT rows of x, bound by the weights' way
// from HBM.
//
// The NW waves share k: wave w takes the 128-column blocks w, w + NW, ...
// (each workgroup from another one on), so that a workgroup reads NW * 128
// bytes of each row at about the same time.  A wave asks for its weights (2 KB
// a 16-row tile, in whole lines) and its operands of x D blocks ahead, into
// registers; weights pass through LDS of the wave's own into the A layout.
// Nothing is shared between waves until their sums meet in LDS at the end.
// There is no branch between the loads, whose number the compiler must know
// to wait for one block alone: blocks past a wave's last one are zeros.
// (Weights straight to LDS: the compiler then waits for every load before it
// uses one of x's.)
//
// Bound by HBM and, where weights are few, by launch, first loads and the join:
// 1 x 6144 x 4096 8.2 us (3.1 TB/s; a bare read of as much 5.7), 16 x 4096 x
// 12288 13.9 and 2 for the second launch, 8 x 151936 x 2048 52.6 (5.9 TB/s).
// Non-temporal loads and workgroups that start at different columns are worth
// a quarter: a bare read of 24576 x 4096 took 21.9 us without, 16.9 with both.
template <int FMT, bool GATED, int NT, int MT, int NW, int D>
__global__ __launch_bounds__(NW * kWave) void k_linear_stream(LinearCall c) {
  constexpr bool kBlock = FMT == kFmtBlock || FMT == kFmtBlockBf16;
  constexpr bool kMx = FMT == kFmtMx;
  constexpr int kOut = GATED ? NT / 2 : NT;        // 16-row tiles of outputs
  __shared__ __attribute__((aligned(16))) unsigned char ws[NW * NT * 2048];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x, split = blockIdx.y, splits = gridDim.y;
  const int n_out = GATED ? c.n / 2 : c.n;
  const int k = c.k, nkb = (k + 127) / 128, ng = (k + 31) / 32;
  int kb0 = 0, blocks = nkb;
  if (splits > 1) {   // nkb <= 2^21, splits <= kFill = 256: 32 bits hold the product
    kb0 = nkb * split / splits;
    blocks = nkb * (split + 1) / splits - kb0;
  }
  // where the workgroup starts: not all at the same columns
  const int turn = (int)((uint32_t)tile * NW & ((1u << (31 - __builtin_clz((uint32_t)blocks))) - 1));
  const int n0 = tile * 16 * kOut;
  const auto out_row = [&](int t) { return n0 + 16 * (t % kOut); };
  const auto half = [&](int t) { return t >= kOut ? n_out : 0; };
  unsigned char* const wl = ws + wave * NT * 2048;
  const uint64_t zeros = reinterpret_cast<uint64_t>(&kNoColumns);

  // Load j of a block brings rows 8j + l/8 (tile j / 2), unit l%8, which goes
  // to the row's LDS place (l%8) ^ (row / 2 % 8).  Rows past the end are the
  // last one; past k weights and x are zeros.
  uint64_t wp[2 * NT];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j)
    wp[j] = reinterpret_cast<uint64_t>(c.codes) +
            (uint64_t)(min(out_row(j >> 1) + 8 * (j & 1) + (lane >> 3), n_out - 1) + half(j >> 1)) * (uint32_t)k;
  const int place = (lane & 7) ^ (lane >> 4);   // j odd: ^ 4
  uint64_t xp[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) xp[q] = reinterpret_cast<uint64_t>(c.x) + (uint64_t)min(16 * q + i, c.m - 1) * (2 * (uint32_t)c.x_stride);
  // A tile's 16 rows lie in one scale block, or in two from row `border` on
  // (halves that start anywhere).
  const char* sp[NT];
  int border[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int first = min(out_row(t), n_out - 1) + half(t);
    border[t] = 128 - first % 128;
    if (kBlock) sp[t] = static_cast<const char*>(c.scales) + (size_t)(first / 128) * nkb * (FMT == kFmtBlock ? 4 : 2);
    if (kMx) sp[t] = static_cast<const char*>(c.scales) + (size_t)(min(out_row(t) + i, n_out - 1) + half(t)) * ng;
  }
  const bool two = kBlock && GATED && n_out % 16 != 0;
  const int last_block = (c.n - 1) / 128;

  struct Slot {
    uint4 w[2 * NT], x[MT][4];
    float s[NT][2];
    uint32_t ex[NT];
  };
  const auto block_at = [&](int p) {
    const int b = p < blocks ? p + turn : 0;
    return kb0 + (b < blocks ? b : b - blocks);
  };
  const auto request = [&](int p, Slot& slot) __attribute__((always_inline)) {
    const int kb = block_at(p), from = p < blocks ? kb * 128 : 1 << 29;   // past every column
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int col = from + 16 * (lane & 7);
      slot.w[j] = ld_stream_u4(reinterpret_cast<const void*>(col < k ? wp[j] + (uint32_t)col : zeros), 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (kBlock) {
        const auto scale = [&](int down) {
          return scalar_scale<FMT>(sp[t], down * nkb + kb);
        };
        slot.s[t][0] = scale(0);
        if (GATED) slot.s[t][1] = scale(two && (min(out_row(t), n_out - 1) + half(t)) / 128 < last_block ? 1 : 0);
      }
      // four bytes that end with the row's last, where the block has fewer
      if (kMx) slot.ex[t] = ld_global<u32_unaligned>(sp[t], (size_t)min(4 * kb, ng - 4));
    }
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = from + 64 * (u >> 1) + 16 * g + 8 * (u & 1);
        slot.x[q][u] = ld_global_u4(reinterpret_cast<const void*>(col < k ? xp[q] + (uint32_t)(2 * col) : zeros), 0);
      }
    asm volatile("" ::: "memory");
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < MT; ++q) acc[t][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const auto consume = [&](int p, Slot& slot) __attribute__((always_inline)) {
    const int kb = block_at(p);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
      *reinterpret_cast<uint4*>(wl + j * 1024 + (lane >> 3) * 128 + 16 * (place ^ (j & 1) * 4)) = slot.w[j];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 part[MT] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = *reinterpret_cast<const uint4*>(wl + (16 * t + i) * 128 + 16 * ((4 * h + g) ^ (i >> 1)));
        bf16x8 a0, a1;
        a_operands<kMx>(w, kMx ? mx_scale((uint8_t)(slot.ex[t] >> 8 * (4 * kb - min(4 * kb, ng - 4)) >> 8 * (2 * h + (g >> 1)))) : 1.0f, a0, a1);
#pragma unroll
        for (int q = 0; q < MT; ++q) {
          part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, slot.x[q][2 * h]), part[q], 0, 0, 0);
          part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, slot.x[q][2 * h + 1]), part[q], 0, 0, 0);
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float s = 1.0f;
        if (kBlock) s = GATED && 4 * g + v >= border[t] ? slot.s[t][1] : slot.s[t][0];
#pragma unroll
        for (int q = 0; q < MT; ++q) acc[t][q][v] = __builtin_fmaf(s, part[q][v], acc[t][q][v]);
      }
    }
    asm volatile("" ::: "memory");
  };
  Slot slot[D];
#pragma unroll
  for (int d = 0; d < D; ++d) request(wave + d * NW, slot[d]);
  // what a thread's four outputs take besides their sums
  const int mt = MT == 1 ? 0 : threadIdx.x / kWave % MT, ml = threadIdx.x % kWave, mo = threadIdx.x / (MT * kWave);
  static_assert(NT * MT <= NW, "a thread finishes no more than four outputs");
  const bool mine = mo < (splits > 1 ? NT : kOut) && 16 * mt + (ml & 15) < c.m && out_row(mo) + 4 * (ml >> 4) < n_out;
  FourOutputs<FMT, GATED> four(c, min(16 * mt + (ml & 15), c.m - 1), min(out_row(mo) + 4 * (ml >> 4), n_out - 1));
#pragma unroll 1
  for (int p = wave; p - wave < blocks; p += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      consume(p + d * NW, slot[d]);
      request(p + (D + d) * NW, slot[d]);
    }
  }

  // the waves' sums meet, each in its own part of LDS
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < MT; ++q) *reinterpret_cast<f32x4*>(wl + ((t * MT + q) * kWave + lane) * 16) = acc[t][q];
  __syncthreads();
  if (!mine) return;
  const auto total = [&](int t) {
    f32x4 v = *reinterpret_cast<const f32x4*>(ws + ((t * MT + mt) * kWave + ml) * 16);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(ws + w * NT * 2048 + ((t * MT + mt) * kWave + ml) * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += o[j];
    }
    return v;
  };
  const f32x4 v = total(mo);
  if (splits > 1) {   // rows of n sums (padded to four) for each slice
    const size_t stride = (size_t)(GATED ? 2 : 1) * ((n_out + 3) & ~3);
    st_global<f32x4>(c.workspace, (((size_t)split * c.m + four.row) * stride + (mo >= kOut ? stride / 2 : 0) + four.n) * 4, v);
  } else if constexpr (GATED) {
    four.finish(c, v, total(mo + kOut));
  } else {
    four.finish(c, v, v);
  }
}

// The slices' sums of the streaming kernel added, in their order: a thread
// takes four outputs of a row.
template <int FMT, bool GATED>
__global__ __launch_bounds__(256) void k_linear_rows(LinearCall c, int splits) {
  const int n_out = GATED ? c.n / 2 : c.n, quads = (n_out + 3) / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(e / quads), n = 4 * (int)(e - (int64_t)row * quads);
  if (row >= c.m) return;
  const size_t stride = (size_t)(GATED ? 2 : 1) * 4 * quads;
  f32x4 v[2] = {};
  for (int p = 0; p < splits; ++p)
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
      const f32x4 o = ld_global<f32x4>(c.workspace, (((size_t)p * c.m + row) * stride + h * (stride / 2) + n) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[h][j] += o[j];
    }
  FourOutputs<FMT, GATED>(c, row, n).finish(c, v[0], v[1]);
}

bool is_gated(int act) { return act == kActSwiglu || act == kActGeglu; }

constexpr int kStreamRows = 16;   // x's rows that the streaming kernel takes
constexpr int kFill = 256;        // workgroups: one a CU

// The kernel of a call, by its sizes.
struct LinearPlan {
  enum Kind { kSimple, kStream, kTile } kind;
  int height, width;   // x's rows and outputs of a tile
  int nt;              // the streaming kernel's
  int mt, tw, kw;      // the tiled kernel's
  bool border;
  LinearGrid grid;
  int64_t slice;       // workspace of one tile and slice
};

// Times are of weights that come from HBM, in us.
//
// Up to 16 rows of x the streaming kernel: 16 nt weight rows a workgroup, four
// waves that share k (nt = 1: eight).
//   nt = 1 where 32 rows a workgroup left CUs without one, and k is short:
//     1 x 4096 x 4096 6.4, 7.6 with nt = 2; 1 x 6144 x 4096 8.2 with either.
//     Long k is cut in slices instead, and x read half as often:
//     16 x 4096 x 12288 15.2, 17.8 with nt = 1.
//   nt = 4 where there are workgroups enough all the same, and the reads of x
//     weigh: 8 x 151936 x 2048 54, 60 with nt = 2; 16 x 16384 x 4096 18 and 21;
//     but 1 x 24576 x 4096 23 and 21.
// Above, the tiled kernel of 128 weight rows (mt = 4: 256) by 32 mt rows of x.
//   mt = 2 up to 512 rows (300 x 24576 x 4096 88, 124 with mt = 4; 512 x 6144
//     x 4096 44 and 52; 512 x 4096 x 12288 69 and 65), and above while tiles of
//     mt = 4 were fewer than 160 (1000 x 4096 x 4096 46 and 61; 1000 x 6144 x
//     4096, which has 192, 68 and 60).  mt = 4 also needs halves of whole 32 rows.
//   mt = 1 up to 32 rows, and where its tiles fill the CUs once and twice as
//     high ones did not: 128 x 6144 x 4096 17.7, 21 with mt = 2 and two slices.
//   While there is no more than a tile a CU, eight waves share its k: 203 x
//     6144 x 4096 25, 29 with four, 30 with four and two slices; 64 x 24576 x
//     4096 30 and 34; 512 x 6144 x 4096 (384 tiles) 44 with either.  With mt = 1
//     and 96 tiles or more sixteen waves: 32 x 24576 x 4096 25.9, 27.3 with
//     eight, 32 x 12288 x 4096 20 and 21; 17 x 6144 x 4096 (48) 14.4 and 13.9.
// Fewer tiles than CUs are cut in slices of k, of eight blocks (streaming: 32)
// at least, and a second launch adds these up: 64 x 4096 x 12288 with eight
// slices 24.6, four 28; 32 x 4096 x 12288 with eight 20.5, one 35.  More than
// one workgroup a CU does not pay: 1777 x 4096 x 12288 (224 tiles) 170, with
// two slices 178.
LinearPlan linear_plan(int64_t m, int64_t n, int64_t k, int format, int act) {
  const bool gate = is_gated(act), block = format == kFmtBlock || format == kFmtBlockBf16;
  const int outputs = gate ? 1 : 2;   // of two weight rows
  const int64_t n_out = gate ? n / 2 : n, nkb = (k + 127) / 128;
  const int64_t second = gate && block ? n_out : 0;   // where the second half's scale blocks start
  LinearPlan p{LinearPlan::kSimple, 16, 64, 0, 0, 0, 1, false, {1, 1, 1}, 0};
  int64_t least = 8;   // blocks of a slice
  const int64_t groups = (n_out + 64 * outputs - 1) / (64 * outputs);
  if (format == kFmtMx && k <= 96) {
    // rows of fewer than four exponents, which the others read at a time
  } else if (m <= kStreamRows) {
    p.kind = LinearPlan::kStream;
    p.nt = n >= 65536 || (m > 8 && n >= 64 * kFill) ? 4 : n <= 16 * kFill && nkb < 64 && !gate ? 1 : 2;
    p.height = kStreamRows;
    p.width = 8 * p.nt * outputs;
    least = 32;
  } else {
    p.kind = LinearPlan::kTile;
    const int64_t flat = (m + 31) / 32 * groups;
    const int64_t wide = (m + 127) / 128 * ((groups + 1) / 2);
    p.mt = m <= 32 || (flat > 128 && flat <= kFill) ? 1 : m <= 512 || wide < 160 || second % 32 != 0 ? 2 : 4;
    p.tw = p.mt == 4 ? 2 : 1;
    const int64_t tiles = (m + 32 * p.mt - 1) / (32 * p.mt) * groups;
    p.kw = p.mt == 4 || tiles > kFill ? 1 : p.mt == 1 && tiles >= 96 ? 4 : 2;
    p.border = second % 16 != 0;
    p.height = 32 * p.mt;
    p.width = 64 * p.tw * outputs;
    p.slice = (int64_t)p.mt * p.tw * 4 * 4096;
  }
  p.grid.tiles_m = (int)((m + p.height - 1) / p.height);
  p.grid.groups = (int)((n_out + p.width - 1) / p.width);
  if (p.kind == LinearPlan::kSimple) return p;
  int64_t splits = kFill / ((int64_t)p.grid.tiles_m * p.grid.groups);
  if (splits > nkb / least) splits = nkb / least;
  p.grid.splits = splits < 1 ? 1 : (int)splits;
  return p;
}

template <int FMT, bool GATED>
hipError_t launch_stream(const LinearCall& c, const LinearPlan& p, hipStream_t stream) {
  const dim3 grid(p.grid.groups, p.grid.splits);
  if (p.nt == 4) {
    k_linear_stream<FMT, GATED, 4, 1, 4, 2><<<grid, 4 * kWave, 0, stream>>>(c);
  } else if (p.nt == 2) {
    k_linear_stream<FMT, GATED, 2, 1, 4, 2><<<grid, 4 * kWave, 0, stream>>>(c);
  } else if constexpr (!GATED) {
    k_linear_stream<FMT, GATED, 1, 1, 8, 2><<<grid, 8 * kWave, 0, stream>>>(c);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.grid.splits == 1) return e;
  const int64_t quads = (int64_t)c.m * (((GATED ? c.n / 2 : c.n) + 3) / 4);
  k_linear_rows<FMT, GATED><<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(c, p.grid.splits);
  return hipGetLastError();
}

template <int FMT, bool GATED, int MT, int TW, int KW>
hipError_t launch_tile(const LinearCall& c, const LinearPlan& p, hipStream_t stream) {
  const int64_t tiles = (int64_t)p.grid.tiles_m * p.grid.groups;
  const unsigned blocks = (unsigned)((tiles * p.grid.splits + 7) / 8 * 8), joins = (unsigned)((tiles + 7) / 8 * 8);
  if constexpr (GATED && TW == 1 && (FMT == kFmtBlock || FMT == kFmtBlockBf16)) {
    if (p.border)
      k_linear_tile<FMT, GATED, MT, TW, KW, true><<<blocks, 256 * KW, 0, stream>>>(c, p.grid);
    else
      k_linear_tile<FMT, GATED, MT, TW, KW, false><<<blocks, 256 * KW, 0, stream>>>(c, p.grid);
  } else {
    k_linear_tile<FMT, GATED, MT, TW, KW, false><<<blocks, 256 * KW, 0, stream>>>(c, p.grid);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.grid.splits == 1) return e;
  k_linear_join<FMT, GATED, MT, TW><<<joins, 256, 0, stream>>>(c, p.grid);
  return hipGetLastError();
}

template <int FMT, bool GATED>
hipError_t launch_plan(const LinearCall& c, const LinearPlan& p, hipStream_t stream) {
  if (p.kind == LinearPlan::kStream) return launch_stream<FMT, GATED>(c, p, stream);
  if (p.mt == 4) return launch_tile<FMT, GATED, 4, 2, 1>(c, p, stream);
  if (p.mt == 2) return p.kw == 2 ? launch_tile<FMT, GATED, 2, 1, 2>(c, p, stream) : launch_tile<FMT, GATED, 2, 1, 1>(c, p, stream);
  if (p.kw == 4) return launch_tile<FMT, GATED, 1, 1, 4>(c, p, stream);
  return p.kw == 2 ? launch_tile<FMT, GATED, 1, 1, 2>(c, p, stream) : launch_tile<FMT, GATED, 1, 1, 1>(c, p, stream);
}

template <int FMT>
hipError_t launch_gate(const LinearCall& c, const LinearPlan& p, hipStream_t stream) {
  return is_gated(c.act) ? launch_plan<FMT, true>(c, p, stream) : launch_plan<FMT, false>(c, p, stream);
}

}  // namespace

int64_t linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int format, int act) {
  const LinearPlan p = linear_plan(m, n, k, format, act);
  if (p.grid.splits == 1) return 0;
  if (p.kind == LinearPlan::kStream)   // rows of sums, padded to four
    return m * p.grid.splits * 4 * (is_gated(act) ? 2 * ((n / 2 + 3) & ~(int64_t)3) : (n + 3) & ~(int64_t)3);
  return (int64_t)p.grid.tiles_m * p.grid.groups * p.grid.splits * p.slice;
}

int64_t linear_blocks(int64_t m, int64_t n, int64_t k, int format, int act) {
  const LinearPlan p = linear_plan(m, n, k, format, act);
  return ((int64_t)p.grid.tiles_m * p.grid.groups * p.grid.splits + 7) / 8 * 8;
}

hipError_t launch_linear(const LinearCall& c, hipStream_t stream) {
  const LinearPlan p = linear_plan(c.m, c.n, c.k, c.format, c.act);
  if (p.kind == LinearPlan::kSimple) {
    const unsigned blocks = (unsigned)((int64_t)p.grid.tiles_m * p.grid.groups);
    if (is_gated(c.act))
      k_linear_simple<true><<<blocks, 256, 0, stream>>>(c, p.grid.groups);
    else
      k_linear_simple<false><<<blocks, 256, 0, stream>>>(c, p.grid.groups);
    return hipGetLastError();
  }
  switch (c.format) {
    case kFmtBlock: return launch_gate<kFmtBlock>(c, p, stream);
    case kFmtMx: return launch_gate<kFmtMx>(c, p, stream);
    case kFmtBlockBf16: return launch_gate<kFmtBlockBf16>(c, p, stream);
    case kFmtRow: return launch_gate<kFmtRow>(c, p, stream);
    default: return launch_gate<kFmtTensor>(c, p, stream);
  }
}

}  // namespace fp8w
