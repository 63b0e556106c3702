// experts.hip -- matrix products grouped by expert on fp8 weights.
//
//   y[i][j] = sum_k x[rows[i]][k] * deq(W_e)[j][k],
//   offsets[e] <= i < offsets[e + 1],
// bf16 x and y, fp32 accumulation, or with W_e's halves g (rows 0..n/2) and
// u (rows n/2..n)
//   y[i][j] = silu(g) * u,  silu(g) = g / (1 + exp(-g)).
// Sizes of the groups are read on the device (a router's answer, no host
// synchronization): every workgroup finds its expert in the offsets.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.hpp"
#include "internal.hpp"

namespace fp8w {
namespace {

// A workgroup's tile: a run of at most `height` slots of one expert, and
// `group` of the n_groups along n.
struct TileAt {
  int expert;   // -1: no tile is left for this workgroup
  int slot0, count, group;
};

// Inclusive sums over the wave: sums along each row of 16 lanes by lane
// shifts, then the rows' totals by lane reads.
__device__ __forceinline__ int wave_prefix(int v) {
#define FP8W_ROW_SHR_ADD(n) v += __builtin_amdgcn_update_dpp(0, v, 0x110 + (n), 0xF, 0xF, false)
  FP8W_ROW_SHR_ADD(1);
  FP8W_ROW_SHR_ADD(2);
  FP8W_ROW_SHR_ADD(4);
  FP8W_ROW_SHR_ADD(8);
#undef FP8W_ROW_SHR_ADD
  const int a = __builtin_amdgcn_readlane(v, 15), b = __builtin_amdgcn_readlane(v, 31), c = __builtin_amdgcn_readlane(v, 47);
  const int row = (threadIdx.x & (kWave - 1)) >> 4;
  return v + (row > 0 ? a : 0) + (row > 1 ? b : 0) + (row > 2 ? c : 0);
}

// The runs of all experts, in expert order, each in n_groups tiles, held by a
// wave (the answers are the same in every lane).  The offsets are kept inside
// [0, slots], so that what a wrong offset names is still in bounds.
//
// Workgroups go round the 8 XCDs in turn, and each XCD has its own L2: it
// gets one contiguous eighth of the tiles, so that an expert's weights and
// rows are read by one XCD, or two.  That takes the number of tiles, so all
// offsets are read: 256 experts a pass, every load of a pass at once.
constexpr int kRunsFew = 256;   // experts of one pass
template <bool FEW>
struct Runs {
  static constexpr int kPass = kRunsFew / kWave;
  const int32_t* offsets;
  int experts, slots, height, n_groups, total;
  int from[kPass], last[kPass], upto[kPass];   // of experts e0 + 64 r + lane

  __device__ __forceinline__ int pass(int e0, int before) {   // returns the runs up to the pass's end
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int r = 0; r < kPass; ++r) {
      const int e = e0 + r * kWave + lane;
      from[r] = ld_global<int32_t>(offsets, (size_t)min(e, experts) * 4);
      last[r] = ld_global<int32_t>(offsets, (size_t)min(e + 1, experts) * 4);
    }
#pragma unroll
    for (int r = 0; r < kPass; ++r) {
      if (e0 + r * kWave >= experts) {
        from[r] = last[r] = 0;
        upto[r] = before;
        continue;
      }
      from[r] = min(max(from[r], 0), slots);
      last[r] = min(max(last[r], 0), slots);
      upto[r] = wave_prefix(tiles(r)) + before;
      before = __builtin_amdgcn_readlane(upto[r], kWave - 1);
    }
    return before;
  }
  __device__ __forceinline__ int tiles(int r) const {
    return last[r] > from[r] ? (last[r] - from[r] + height - 1) / height : 0;
  }
  __device__ __forceinline__ Runs(const int32_t* o, int e, int s, int h, int g)
      : offsets(o), experts(e), slots(s), height(h), n_groups(g), total(0) {
    if constexpr (FEW) {
      total = pass(0, 0);
    } else {
      for (int e0 = 0; e0 < experts; e0 += kPass * kWave) total = pass(e0, total);
    }
  }
  // Tile `place` of this workgroup's XCD.
  __device__ __forceinline__ TileAt at(int64_t place) {
    const int64_t share = ((int64_t)total * n_groups + 7) / 8;
    const int64_t id = (blockIdx.x & 7) * share + place;
    if (place >= share || id >= (int64_t)total * n_groups) return TileAt{-1, 0, 1, 0};
    const int run = (int)((uint32_t)id / (uint32_t)n_groups);
    TileAt t{-1, 0, 1, (int)((uint32_t)id - (uint32_t)run * (uint32_t)n_groups)};
    int before = 0;
    for (int e0 = 0; e0 < (FEW ? 1 : experts) && t.expert < 0; e0 += kPass * kWave) {
      if constexpr (!FEW) before = pass(e0, before);
#pragma unroll
      for (int r = 0; r < kPass; ++r) {
        if (e0 + r * kWave >= experts) break;
        const int first = upto[r] - tiles(r);
        const uint64_t mine = __ballot(run >= first && run < upto[r]);
        if (mine) {
          const int l = __builtin_ctzll(mine);
          const int slot0 = from[r] + (run - first) * height;
          t.expert = e0 + r * kWave + l;
          t.slot0 = __builtin_amdgcn_readlane(slot0, l);
          t.count = __builtin_amdgcn_readlane(min(height, last[r] - slot0), l);
        }
      }
    }
    return t;
  }
};

// The only tile of a workgroup.
__device__ __forceinline__ TileAt tile_at(const int32_t* offsets, int experts, int slots, int height, int n_groups) {
  if (experts <= kRunsFew) return Runs<true>(offsets, experts, slots, height, n_groups).at(blockIdx.x >> 3);
  return Runs<false>(offsets, experts, slots, height, n_groups).at(blockIdx.x >> 3);
}

// silu(g) * u within a few units of the last place of fp32: exp(-g) as 2^t
// times a first-order correction for what rounding t = -g log2 e lost, and
// the hardware reciprocal (an IEEE division of every output cost as many
// instructions as a third of the products at k = 2048).
__device__ __forceinline__ float silu_times(float g, float u) {
  constexpr float kLog2E = 0x1.715476p+0f, kLog2ELow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  // Beyond 200 either way 2^t is infinite and the result zero, or it is zero
  // and silu(g) is g, up to infinity.
  const float a = -__builtin_amdgcn_fmed3f(g, -200.0f, 200.0f);
  const float t = a * kLog2E;
  const float lost = __builtin_fmaf(a, kLog2ELow, __builtin_fmaf(a, kLog2E, -t));
  const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(lost, kLn2, 1.0f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// The simple kernel: one wave takes 16 weight rows (with SWIGLU 16 of each
// half) against 16 slots, operands straight from memory.  It takes what the
// others do not (experts_plan): block scales of two halves that a row quad
// would cross, and rows of at most three MX exponents; row and tensor scales
// never come here.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void k_experts_simple(ExpertsCall c, int n_groups) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const TileAt tile = tile_at(c.offsets, c.experts, c.slots, 16, n_groups);
  if (tile.expert < 0) return;
  const int n_out = SWIGLU ? c.n / 2 : c.n;
  const int n0 = (tile.group * 4 + wave) * 16;
  if (n0 >= n_out) return;
  const int i = lane & 15, g = lane >> 4;
  const int slot = tile.slot0 + min(i, tile.count - 1);
  int row = c.rows ? ld_global<int32_t>(c.rows, (size_t)slot * 4) : slot;
  const bool live = row >= 0 && row < c.x_rows;
  if (!live) row = 0;
  const uint8_t* w0 = c.codes + (size_t)tile.expert * c.n * c.k;
  const char* sc = static_cast<const char*>(c.scales) + (size_t)tile.expert * c.scale_bytes;
  f32x4 acc[2] = {};
  const int nkb = (c.k + 127) / 128, ng = (c.k + 31) / 32;
  for (int kb = 0; kb < nkb; ++kb) {
    f32x4 part[2] = {};
    for (int h = 0; h < 2; ++h) {
      const int col = kb * 128 + h * 64 + 16 * g;
      const bool in = col < c.k;
      uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
      if (in && live) {
        b0 = ld_global_u4(c.x, ((size_t)row * c.k + col) * 2);
        b1 = ld_global_u4(c.x, ((size_t)row * c.k + col) * 2 + 16);
      }
#pragma unroll
      for (int q = 0; q < (SWIGLU ? 2 : 1); ++q) {
        const int n = min(n0 + i, n_out - 1) + q * n_out;
        uint4 w = make_uint4(0, 0, 0, 0);
        float s = 1.0f;
        if (in) {
          w = ld_global_u4(w0, (size_t)n * c.k + col);
          if (c.format == kFmtMx) s = mx_scale(ld_global<uint8_t>(sc, (size_t)n * ng + col / 32));
        }
        bf16x8 a0, a1;
        a_operands<true>(w, s, a0, a1);
        part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, b0), part[q], 0, 0, 0);
        part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, b1), part[q], 0, 0, 0);
      }
    }
#pragma unroll
    for (int q = 0; q < (SWIGLU ? 2 : 1); ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = min(n0 + 4 * g + v, n_out - 1) + q * n_out;
        float s = 1.0f;
        if (c.format == kFmtBlock) s = ld_global<float>(sc, ((size_t)(n / 128) * nkb + kb) * 4);
        if (c.format == kFmtBlockBf16) s = bf16_lo(ld_global<uint16_t>(sc, ((size_t)(n / 128) * nkb + kb) * 2));
        acc[q][v] = __builtin_fmaf(s, part[q][v], acc[q][v]);
      }
  }
  if (i >= tile.count) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int n = n0 + 4 * g + v;
    if (n >= n_out) continue;
    const float r = SWIGLU ? silu_times(acc[0][v], acc[1][v]) : acc[0][v];
    st_global<uint16_t>(c.y, ((size_t)slot * n_out + n) * 2, (uint16_t)f32_to_bf16_rne(r));
  }
}

// 16 bytes a lane from memory to LDS at `to` + 16 * lane (`to` uniform).
__device__ __forceinline__ void stage16(const void* from, unsigned char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
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

// The wide kernel: 128 * TW weight rows against 32 * MT slots of one expert
// on the 32x32x16 MFMA, four waves of 32 * TW rows (SWIGLU: half of them of
// each half), two (TW = 2) or four workgroups a CU.
//
// Everything reaches LDS by loads that write it directly, in whole 128-byte
// lines (in the MFMA A layout a load instruction would touch 64 bytes of 16
// rows or 32 of 32, which took as long as the products themselves).
//   * Weights: a wave's rows of a 128-column block are its own 4 * TW KB.  At
//     the start of a block it takes them into registers in the A layout and
//     asks for the next block at once: a block's time to arrive.
//   * x: 64 columns of the slots for all four waves, three buffers, asked
//     for two steps ahead; one barrier a step.
// The waits name how many younger loads may still be on their way; a wait
// for everything would put the memory's latency into every step.
//
// A CU takes about 58 bytes a clock of such loads, and a wave that issues one
// while the queue is full stands still.  With TW = 2 they are therefore spread
// over the products of a step (12 and 4 of them between 32 products), instead
// of all at its start: 4096 tokens, 8 of 64 experts, gate and up 2048 x 2048,
// block scales 317 -> 298 us, down 2048 x 1024, row scales 156 -> 145 us.  (Of
// 534 us at k = 4096, row scales, 192 went when nothing was loaded, 7 when
// nothing was converted, 46 when all came out of L2.)
//
// A lane's 16 bytes of codes are two MFMA steps of 8 columns each, so step
// (p, s) takes columns 32p + 16(l/32) + 8s of the step, for weights and x
// alike.  LDS rows are 128 bytes, their 16-byte units XOR-swizzled by row / 2,
// so that any 16 consecutive rows fall into 16 different bank groups.
//
// A block scale multiplies its sums every 64 columns (a full block's sums
// would need as many registers as the accumulators, and with TW = 2 some 16
// registers a lane are spilled as it is); MX scales multiply the codes as
// they become bf16 (exact); row and tensor scales the results.  The same
// prefill, gate and up, by format: block 312 us, bf16 block 309, MX 275, row
// 270, tensor 268.
template <int FMT, bool SWIGLU, int MT, int TW>
__device__ __forceinline__ void experts_run(const ExpertsCall& c, const TileAt& at, unsigned char* ws, unsigned char* xs0,
                                            unsigned char* xs1, unsigned char* xs2) {
  constexpr bool kBlock = FMT == kFmtBlock || FMT == kFmtBlockBf16;
  constexpr bool kMx = FMT == kFmtMx;
  constexpr int kRows = 32 * TW;       // weight rows of a wave
  constexpr int kCols = SWIGLU ? kRows / 2 : kRows;   // outputs of a slot and wave
  constexpr int kXLoads = MT;          // x loads of a wave and step (1 KB each)
  constexpr int kWLoads = 4 * TW;      // weight loads of a wave and block
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane & 31, hh = lane >> 5;
  const int n_out = SWIGLU ? c.n / 2 : c.n;
  const int k = c.k, nkb = (k + 127) / 128, ng = (k + 31) / 32;

  const int n0 = (at.group * 4 + wave) * kCols;
  const uint8_t* codes = c.codes + (size_t)at.expert * c.n * k;
  const char* scales = static_cast<const char*>(c.scales) + (size_t)at.expert * c.scale_bytes;
  // Row r of the wave's (r may be uniform or a lane's): output out_row(r),
  // weight row half(r) further on.
  const auto out_row = [&](int r) { return n0 + r % kCols; };
  const auto half = [&](int r) { return r >= kCols ? n_out : 0; };
  unsigned char* wl = ws + wave * kRows * 128;

  // Load j of a wave's weights brings rows 8j + l/8; LDS place l%8 of a row
  // holds its unit (l%8) ^ (row / 2 % 8), so j odd the unit of j even ^ 4.
  // Rows past the end are the last one, columns past it the first ones (zeroed
  // by take_w; x has zeros there, so that no infinity of a column that is read
  // in their place meets them).  No branches: a load that
  // two paths share is one the compiler takes to write any of the arrays.
  // Offsets pass through an empty asm statement where they are used: the
  // addresses of all loads would otherwise be kept in registers throughout.
  const int wu = (lane & 7) ^ (lane >> 4);
  uint32_t wrow = (uint32_t)(lane >> 3) * (uint32_t)k;
  int wcol = 16 * wu;
  const auto load_w = [&](int kb, int j) __attribute__((always_inline)) {
    asm volatile("" : "+v"(wrow), "+v"(wcol)::"memory");
    const int c0 = kb * 128 + (wcol ^ (j & 1) * 64);
    const int row = min(out_row(8 * j), n_out - 1);
    const uint32_t within = (uint32_t)min(n_out - 1 - row, 7) * (uint32_t)k;
    stage16(codes + (size_t)(row + half(8 * j)) * k + (min(wrow, within) + (uint32_t)(c0 < k ? c0 : 0)), wl + j * 1024);
    asm volatile("" ::: "memory");
  };
  const auto request_w = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) load_w(kb, j);
  };
  // x rows a wave stages: 8 (MT * wave + j) + l/8, the same places (row / 2 % 8
  // = 4 (row / 8 % 2) + l/16)
  uint32_t xrow[kXLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int slot = at.slot0 + min(8 * (kXLoads * wave + j) + (lane >> 3), at.count - 1);
    const int row = c.rows ? ld_global<int32_t>(c.rows, (size_t)slot * 4) : slot;
    xrow[j] = row >= 0 && row < c.x_rows ? row : 0;
  }
  int xcol = 8 * (wu ^ (kXLoads * wave & 1) * 4);
  const auto load_x = [&](int step, int j, unsigned char* to) __attribute__((always_inline)) {
    asm volatile("" : "+v"(xcol), "+v"(xrow[j])::"memory");
    const int c0 = step * 64 + (xcol ^ (j & 1) * 32);
    // An offset from x either way: chosen between two addresses the MX tile
    // spilled (prefill 278 -> 282 us).
    const uint64_t x = reinterpret_cast<uint64_t>(c.x), none = reinterpret_cast<uint64_t>(&kNoColumns) - x;
    const uint64_t from = (uint64_t)xrow[j] * (uint32_t)(2 * k) + (uint32_t)(2 * c0);
    stage16(reinterpret_cast<const void*>(x + (c0 < k ? from : none)), to + (kXLoads * wave + j) * 1024);
    asm volatile("" ::: "memory");
  };
  const auto request_x = [&](int step, unsigned char* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) load_x(step, j, to);
  };
  // whether the slots a lane will store, 32q + i, have a row of x
  uint32_t live = 0;
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int slot = at.slot0 + min(32 * q + i, at.count - 1);
    const int row = c.rows ? ld_global<int32_t>(c.rows, (size_t)slot * 4) : slot;
    live |= row >= 0 && row < c.x_rows ? 1u << q : 0u;
  }

  // scales of the next block: a float a run of rows that lie in one scale
  // block (a half's, or a 32-row tile; scalar loads), or the four MX exponents
  // of the lane's row in each tile
  constexpr int kScales = kMx ? TW : SWIGLU ? 2 : TW;
  const auto scale_of = [](int t, int v) { return SWIGLU && TW == 1 ? v >> 3 : t; };   // of sum v of tile t
  const char* sp[kScales];
  float sc[kScales];
  uint32_t ex[kScales];
#pragma unroll
  for (int t = 0; t < kScales; ++t) {
    const int first = t * (kRows / kScales);
    if (kBlock) sp[t] = scales + (size_t)((min(out_row(first), n_out - 1) + half(first)) / 128) * nkb * (FMT == kFmtBlock ? 4 : 2);
    if (kMx) sp[t] = scales + (size_t)(min(out_row(32 * t + i), n_out - 1) + half(32 * t + i)) * ng;
  }
  const auto request_s = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kScales; ++t) {
      if (FMT == kFmtBlock) sc[t] = reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(sp[t]))[kb];
      if (FMT == kFmtBlockBf16)
        sc[t] = bf16_lo(reinterpret_cast<const __attribute__((address_space(4))) uint16_t*>(reinterpret_cast<uintptr_t>(sp[t]))[kb]);
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
  float s[kScales];
  uint32_t e[TW];
  const auto take_w = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        wr[t][p] = *reinterpret_cast<const uint4*>(&wl[(32 * t + i) * 128 + 16 * ((2 * p + hh) ^ (i >> 1 & 7))]);
    if (kb * 128 + 128 > k) {
      const int from = kb * 128 + 16 * (lane_fresh() >> 5);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int t = 0; t < TW; ++t)
          if (from + 32 * p >= k) wr[t][p] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < kScales; ++t) {
      if (kBlock) s[t] = sc[t];
      if (kMx) e[t] = ex[t] >> 8 * (4 * kb - min(4 * kb, ng - 4));
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): the codes are in registers
    request_s(kb + 1 < nkb ? kb + 1 : 0);         // the last block asks for one nobody takes
    __builtin_amdgcn_sched_barrier(0);
  };
  // 64 columns.  Scaled sums are settled after every 32 slots: left alone
  // the compiler starts all products first, each with sums of its own, and
  // spills.
  const auto step = [&](int h, const unsigned char* xb, const auto& load) __attribute__((always_inline)) {
    const auto read_b = [&](int q, int u) __attribute__((always_inline)) {
      return *reinterpret_cast<const bf16x8*>(&xb[(32 * q + i) * 128 + 16 * ((4 * (u >> 1) + 2 * hh + (u & 1)) ^ (i >> 1 & 7))]);
    };
    bf16x8 a[TW][4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) b[u] = read_b(0, u);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int t = 0; t < TW; ++t)
        a_operands<kMx>(wr[t][2 * h + p], kMx ? mx_scale((uint8_t)(e[t] >> 8 * (2 * h + p))) : 1.0f, a[t][2 * p], a[t][2 * p + 1]);
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      // No slots left, in the last run of an expert.  (With block scales the
      // branches cost registers that are not there; the wide tile's loads
      // stand between its products.)
      if (!kBlock && TW == 1 && q > 0 && 32 * q >= at.count) break;
      f32x16 part[TW];
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        if constexpr (kBlock) {
#pragma unroll
          for (int v = 0; v < 16; ++v) part[t][v] = 0.0f;
        } else {
          part[t] = acc[t][q];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int t = 0; t < TW; ++t) part[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[t][u], b[u], part[t], 0, 0, 0);
        // the operand's register is free: the next 32 slots' into it, three
        // products ahead of their use
        if (q + 1 < MT) b[u] = read_b(q + 1, u);
        if (TW == 2) load(4 * q + u);
        if (q + 1 < MT || u < 3) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        if constexpr (kBlock) {
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[t][q][v] = __builtin_fmaf(s[scale_of(t, v)], part[t][v], acc[t][q][v]);
          settle(acc[t][q]);
        } else {
          acc[t][q] = part[t];
        }
      }
    }
  };
  // A block of 128 columns: x steps 2kb and 2kb + 1 are in x0 and x1, and
  // the two after them go to x2 and x0.
  const auto block = [&](int kb, unsigned char* x0, unsigned char* x1, unsigned char* x2) __attribute__((always_inline)) {
    take_w(kb);
    const int next = kb + 1 < nkb ? kb + 1 : 0;
    const auto first = [&](int n) __attribute__((always_inline)) {   // 4 MT places for 8 + MT loads
      const int to = (n + 1) * (kWLoads + kXLoads) / (4 * MT);
#pragma unroll
      for (int j = n * (kWLoads + kXLoads) / (4 * MT); j < to; ++j) {
        if (j < kWLoads)
          load_w(next, j);
        else
          load_x(2 * next, j - kWLoads, x2);
      }
    };
    const auto second = [&](int n) __attribute__((always_inline)) {
      if (n % 4 == 0) load_x(2 * next + 1, n / 4, x0);
    };
    if (TW == 1) {
      request_w(next);
      request_x(2 * next, x2);
      __builtin_amdgcn_sched_barrier(0);
    }
    step(0, x0, first);
    land_and_meet<kWLoads + kXLoads>();           // younger than x1's: weights and x2's
    if (TW == 1) request_x(2 * next + 1, x0);
    step(1, x1, second);
    land_and_meet<kXLoads>();                     // the weights and x2's have landed
  };

  request_s(0);
  request_w(0);
  request_x(0, xs0);
  request_x(1, xs1);
  land_and_meet<kXLoads>();
  int kb = 0;
#pragma unroll 1
  for (; kb + 2 < nkb; kb += 3) {
    block(kb, xs0, xs1, xs2);
    block(kb + 1, xs2, xs0, xs1);
    block(kb + 2, xs1, xs2, xs0);
  }
  if (kb < nkb) block(kb, xs0, xs1, xs2);
  if (kb + 1 < nkb) block(kb + 1, xs2, xs0, xs1);
  vm_wait_all();   // nothing may land in LDS that is no longer ours

  // A lane holds slot 32q + l%32 and, for each v4, rows 8 v4 + 4 (l / 32) .. + 3
  // of each tile.  32 slots at a time go through the wave's own LDS (rows of
  // kCols outputs, units swizzled as above), so that they reach memory as
  // whole lines: 8-byte stores from here took 50 us on 134 MB.
  constexpr int kUnits = kCols / 8;
  float os[TW][16];
  if (FMT == kFmtRow || FMT == kFmtTensor) {
#pragma unroll
    for (int t = 0; t < TW; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = 32 * t + 8 * (v >> 2) + 4 * hh + (v & 3);
        os[t][v] = ld_global<float>(scales, FMT == kFmtRow ? (size_t)(min(out_row(r), n_out - 1) + half(r)) * 4 : 0);
      }
  }
  const bool vec = n_out % 8 == 0 && reinterpret_cast<uintptr_t>(c.y) % 16 == 0;
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    if (32 * q >= at.count) break;
    unsigned char* out = wl + (q & 1) * 64 * kCols;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {   // outputs 8u + 4 (l / 32) .. + 3 of the wave's
      const auto sum = [&](int r, int v) {   // of row r + 4 (l / 32) + v
        const int t = r / 32, w = r % 32 / 2 + v;
        return FMT == kFmtRow || FMT == kFmtTensor ? acc[t][q][w] * os[t][w] : acc[t][q][w];
      };
      float r[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float o = SWIGLU ? silu_times(sum(8 * u, v), sum(8 * u + kCols, v)) : sum(8 * u, v);
        r[v] = live >> q & 1 ? o : 0.0f;   // else the products of zeros
      }
      *reinterpret_cast<u32x2*>(out + i * 2 * kCols + 16 * (u ^ (i >> 1 & (kUnits - 1))) + 8 * hh) =
          u32x2{bf16_pair(r[0], r[1]), bf16_pair(r[2], r[3])};
    }
#pragma unroll
    for (int j = 0; j < kUnits / 2; ++j) {
      const int r = j * (kWave / kUnits) + lane / kUnits, u = lane % kUnits, n = n0 + 8 * u;
      const u32x4 v = *reinterpret_cast<const u32x4*>(out + r * 2 * kCols + 16 * (u ^ (r >> 1 & (kUnits - 1))));
      if (32 * q + r >= at.count || n >= n_out) continue;
      const size_t to = ((size_t)(at.slot0 + 32 * q + r) * n_out + n) * 2;
      if (vec) {
        st_global<u32x4>(c.y, to, v);
      } else {
#pragma unroll
        for (int w = 0; w < 8; ++w)
          if (n + w < n_out) st_global<uint16_t>(c.y, to + 2 * w, (uint16_t)(v[w >> 1] >> 16 * (w & 1)));
      }
    }
  }
}

template <int FMT, bool SWIGLU, int MT, int TW>
__global__ __launch_bounds__(256, TW == 2 ? 2 : 4) void k_experts_wide(ExpertsCall c, int n_groups) {
  // separate arrays: the compiler then knows that reads of one need not wait
  // for what is on its way into another
  __shared__ __attribute__((aligned(16))) unsigned char ws[4 * 32 * TW * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs0[32 * MT * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs1[32 * MT * 128];
  __shared__ __attribute__((aligned(16))) unsigned char xs2[32 * MT * 128];
  const TileAt at = tile_at(c.offsets, c.experts, c.slots, 32 * MT, n_groups);
  if (at.expert < 0) return;
  // These steps do not skip empty slots: an expert's last run as one of half
  // the height, where that holds it (32768 slots over 64 experts, gate and up
  // 2048 x 2048, block scales: 332 us without, 320 with; for the narrow tiles
  // the difference is within the noise).
  if constexpr (TW == 2) {
    if (at.count <= 16 * MT) {
      experts_run<FMT, SWIGLU, MT / 2, TW>(c, at, ws, xs0, xs1, xs2);
      return;
    }
  }
  experts_run<FMT, SWIGLU, MT, TW>(c, at, ws, xs0, xs1, xs2);
}

// The streaming kernel, for experts of a few slots: 16 * NT weight rows
// (SWIGLU: half of them of each half) against 16 slots, bound by the weights'
// way from HBM.
//
// The four waves share k: wave w takes the 128-column blocks w, w + 4, ...,
// one at a time: its weights (2 KB a 16-row tile, in whole lines, to the
// wave's own LDS) and operands of x are asked for together and waited for
// once.  Nothing is shared between waves until their sums meet in LDS at the
// end.  What keeps the memory busy is the number of workgroups a CU holds,
// eight of 16 KB, each at another point of its way from look-up to sums:
// four blocks at a time and two workgroups a CU took 65 us for 281 MB (32
// tokens on 128 experts), two and four 54 us, one and eight 52 us; a ring of
// two blocks in flight a wave 54 us.  NT = 4: 52 us, but 10.5 us for one
// token against 8.5 us.
template <int FMT, bool SWIGLU, int NT>
__global__ __launch_bounds__(256, 16 / NT) void k_experts_stream(ExpertsCall c, int n_groups) {
  constexpr bool kBlock = FMT == kFmtBlock || FMT == kFmtBlockBf16;
  constexpr bool kMx = FMT == kFmtMx;
  constexpr int kOut = SWIGLU ? NT / 2 : NT;       // 16-row tiles of outputs
  __shared__ __attribute__((aligned(16))) unsigned char ws[4][NT * 2048];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane & 15, g = lane >> 4;
  const TileAt at = tile_at(c.offsets, c.experts, c.slots, 16, n_groups);
  if (at.expert < 0) return;
  const int n_out = SWIGLU ? c.n / 2 : c.n;
  const int k = c.k, nkb = (k + 127) / 128, ng = (k + 31) / 32;
  const int n0 = at.group * 16 * kOut;
  const uint8_t* codes = c.codes + (size_t)at.expert * c.n * k;
  const char* scales = static_cast<const char*>(c.scales) + (size_t)at.expert * c.scale_bytes;
  const auto out_row = [&](int t) { return n0 + 16 * (t % kOut); };
  const auto half = [&](int t) { return t >= kOut ? n_out : 0; };
  unsigned char* wl = ws[wave];

  // Load j of a block brings rows 8j + l/8 (tile j / 2); LDS place l%8 of a
  // row holds its unit (l%8) ^ (row / 2 % 8).  Rows past the end are the
  // last one, columns past it the first ones, taken as zeros.
  const uint8_t* wp[2 * NT];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j)
    wp[j] = codes + (size_t)(min(out_row(j >> 1) + 8 * (j & 1) + (lane >> 3), n_out - 1) + half(j >> 1)) * k;
  const int wunit = (lane & 7) ^ (lane >> 4);   // j odd: ^ 4
  const auto request_w = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int col = kb * 128 + 16 * (wunit ^ (j & 1) * 4);
      stage16(wp[j] + (col < k ? col : 0), wl + j * 1024);
    }
  };
  // the first weights before anything that takes a second look-up
  if (wave < nkb) request_w(wave);

  const int slot = at.slot0 + min(i, at.count - 1);
  const int row = c.rows ? ld_global<int32_t>(c.rows, (size_t)slot * 4) : slot;
  const bool live = row >= 0 && row < c.x_rows;
  const uint16_t* xp = c.x + (size_t)(live ? row : 0) * k;
  const char* sp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // a lane's four sums are rows 4g .. of the tile: one scale block (the
    // halves start on a multiple of 4)
    if (kBlock) sp[t] = scales + (size_t)((min(out_row(t) + 4 * g, n_out - 1) + half(t)) / 128) * nkb * (FMT == kFmtBlock ? 4 : 2);
    if (kMx) sp[t] = scales + (size_t)(min(out_row(t) + i, n_out - 1) + half(t)) * ng;
  }

  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int kb = wave; kb < nkb; kb += 4) {
    uint4 x[4];
    float sc[NT];
    uint32_t ex[NT];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = kb * 128 + 64 * (u >> 1) + 16 * g + 8 * (u & 1);
      x[u] = ld_global_u4(xp, (size_t)(col < k ? col : 0) * 2);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (FMT == kFmtBlock) sc[t] = ld_global<float>(sp[t], (size_t)kb * 4);
      if (FMT == kFmtBlockBf16) sc[t] = bf16_lo(ld_global<uint16_t>(sp[t], (size_t)kb * 2));
      // four bytes that end with the row's last, where the block has fewer
      if (kMx) ex[t] = ld_global<u32_unaligned>(sp[t], (size_t)min(4 * kb, ng - 4)) >> 8 * (4 * kb - min(4 * kb, ng - 4));
    }
    vm_wait_all();
    asm volatile("" ::: "memory");
    if (kb * 128 + 128 > k) {   // zeros past k, where a column's infinity would meet the zero weights
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (kb * 128 + 64 * (u >> 1) + 16 * g >= k) x[u] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 part = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w = *reinterpret_cast<const uint4*>(wl + (16 * t + i) * 128 + 16 * ((4 * h + g) ^ (i >> 1)));
        if (kb * 128 + 64 * h + 16 * g >= k) w = make_uint4(0, 0, 0, 0);
        bf16x8 a0, a1;
        a_operands<kMx>(w, kMx ? mx_scale((uint8_t)(ex[t] >> 8 * (2 * h + (g >> 1)))) : 1.0f, a0, a1);
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, x[2 * h]), part, 0, 0, 0);
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, x[2 * h + 1]), part, 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(kBlock ? sc[t] : 1.0f, part[v], acc[t][v]);
    }
    if (kb + 4 < nkb) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the codes have been read
      request_w(kb + 4);
    }
  }

  // the waves' sums meet, each in its own part of LDS; wave t finishes the
  // outputs of tiles t, t + 4, ...
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(wl + (t * kWave + lane) * 16) = acc[t];
  __syncthreads();
  const auto total = [&](int t) {
    f32x4 v = *reinterpret_cast<const f32x4*>(ws[0] + (t * kWave + lane) * 16);
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(ws[w] + (t * kWave + lane) * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += o[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = min(out_row(t) + 4 * g + j, n_out - 1) + half(t);
      if (FMT == kFmtRow) v[j] *= ld_global<float>(scales, (size_t)r * 4);
      if (FMT == kFmtTensor) v[j] *= ld_global<float>(scales, 0);
    }
    return v;
  };
  if (i >= at.count) return;
  for (int t = wave; t < kOut; t += 4) {
    f32x4 v = total(t);
    if (SWIGLU) {
      const f32x4 u = total(t + kOut);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = silu_times(v[j], u[j]);
    }
    if (!live) v = f32x4{};   // the products of zeros
    const int n = out_row(t) + 4 * g;
    const size_t to = ((size_t)slot * n_out + n) * 2;
    if (n_out % 4 == 0) {
      if (n < n_out) st_global<u32x2>(c.y, to, u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < n_out) st_global<uint16_t>(c.y, to + 2 * j, (uint16_t)bf16_pair(v[j], 0.0f));
    }
  }
}

// Runs of `height` slots that any split of the slots over the experts can
// have: each expert ends with at most one run that is not full.
int64_t max_tiles(int64_t slots, int64_t experts, int64_t height) {
  const int64_t e = experts < slots ? experts : slots;
  return (slots + e * (height - 1)) / height;
}

}  // namespace

namespace {

constexpr int kStreamTiles = 2;   // 16-row weight tiles of a streaming workgroup

// The kernel of a call, by its sizes.
struct ExpertsPlan {
  enum Kind { kSimple, kStream, kNarrow, kWide } kind;
  int height;   // slots of a run
  int width;    // outputs of a group
};

// By the slots an expert has on average, from sweeps on MI355X (us).
//   E = 64, 4 choices, gate and up 2048 x 2048, block scales, at 2 / 4 / 8 / 12
//   slots an expert; the same at 24 / 48 / 64 / 96 / 128 / 160 / 256; down
//   2048 x 2048, row scales, at those:
//   streaming        36 44 54 65
//   128 x 64 tiles   43 51 55 55     62 73 85 103 122 143 198    62 69 81 97 114 134 186
//   256 x 128 tiles   .  .  . 53     65 84 91 106 116 131 178    59 73 85 92 101 116 156
// With 8 experts of 4096 x 2048 the narrow tiles' lead lasts (24 / 48 / 96 /
// 160 / 256 slots: 18 / 21 / 23 / 34 / 51 us against 21 / 27 / 28 / 31 / 48).
//
// Halves that do not start on a multiple of 32 rows would put a tile's rows
// in two scale blocks (the streaming kernel asks for 4), and rows of fewer
// than four MX exponents cannot be read four at a time.  What that costs where
// experts have many slots: 4096 tokens, 8 of 64 experts, k = 2048, block
// scales, halves of 192 / 352 / 992 / 1024 rows 100 / 134 / 312 / 312 us, of
// 176 / 360 / 1000 rows (streaming) 210 / 439 / 1194 us, of 1001 rows (simple)
// 1965 us; 32 tokens, halves of 352 and 1024 rows 16.3 and 45.0 us, of 360,
// 1000 and 1001 rows 16.7, 44.7 and 71.5 us.
ExpertsPlan experts_plan(int64_t experts, int64_t slots, int64_t n, int64_t k, bool swiglu, int format) {
  const bool block = format == kFmtBlock || format == kFmtBlockBf16;
  const int64_t average = slots / (experts < slots ? experts : slots);
  const int64_t split = swiglu && block ? n / 2 : 0;
  const int outputs = swiglu ? 1 : 2;   // of two weight rows
  if (split % 4 != 0 || (format == kFmtMx && k <= 96)) return {ExpertsPlan::kSimple, 16, 64};
  if (average <= 8 || split % 32 != 0) return {ExpertsPlan::kStream, 16, 8 * kStreamTiles * outputs};
  if (average <= 112) return {ExpertsPlan::kNarrow, 64, 64 * outputs};
  return {ExpertsPlan::kWide, 128, 128 * outputs};
}

int64_t experts_groups(const ExpertsPlan& p, int64_t n, bool swiglu) {
  return ((swiglu ? n / 2 : n) + p.width - 1) / p.width;
}

template <int FMT, bool SWIGLU>
void launch_plan(const ExpertsCall& c, const ExpertsPlan& p, unsigned blocks, int groups, hipStream_t stream) {
  switch (p.kind) {
    case ExpertsPlan::kStream: k_experts_stream<FMT, SWIGLU, kStreamTiles><<<blocks, 256, 0, stream>>>(c, groups); break;
    case ExpertsPlan::kNarrow: k_experts_wide<FMT, SWIGLU, 2, 1><<<blocks, 256, 0, stream>>>(c, groups); break;
    default: k_experts_wide<FMT, SWIGLU, 4, 2><<<blocks, 256, 0, stream>>>(c, groups); break;
  }
}

template <int FMT>
void launch_act(const ExpertsCall& c, const ExpertsPlan& p, unsigned blocks, int groups, hipStream_t stream) {
  if (c.swiglu)
    launch_plan<FMT, true>(c, p, blocks, groups, stream);
  else
    launch_plan<FMT, false>(c, p, blocks, groups, stream);
}

// Workgroups of one launch, a multiple of 8 (a share for every XCD).
int64_t plan_blocks(const ExpertsPlan& p, int64_t experts, int64_t slots, int64_t n, bool swiglu) {
  return (max_tiles(slots, experts, p.height) * experts_groups(p, n, swiglu) + 7) / 8 * 8;
}

}  // namespace

int64_t experts_blocks(int64_t experts, int64_t slots, int64_t n, int64_t k, bool swiglu, int format) {
  return plan_blocks(experts_plan(experts, slots, n, k, swiglu, format), experts, slots, n, swiglu);
}

hipError_t launch_gemm_experts(const ExpertsCall& c, hipStream_t stream) {
  const ExpertsPlan p = experts_plan(c.experts, c.slots, c.n, c.k, c.swiglu, c.format);
  const int groups = (int)experts_groups(p, c.n, c.swiglu);
  const unsigned blocks = (unsigned)plan_blocks(p, c.experts, c.slots, c.n, c.swiglu);
  if (p.kind == ExpertsPlan::kSimple) {
    if (c.swiglu)
      k_experts_simple<true><<<blocks, 256, 0, stream>>>(c, groups);
    else
      k_experts_simple<false><<<blocks, 256, 0, stream>>>(c, groups);
    return hipGetLastError();
  }
  switch (c.format) {
    case kFmtBlock: launch_act<kFmtBlock>(c, p, blocks, groups, stream); break;
    case kFmtMx: launch_act<kFmtMx>(c, p, blocks, groups, stream); break;
    case kFmtBlockBf16: launch_act<kFmtBlockBf16>(c, p, blocks, groups, stream); break;
    case kFmtRow: launch_act<kFmtRow>(c, p, blocks, groups, stream); break;
    default: launch_act<kFmtTensor>(c, p, blocks, groups, stream); break;
  }
  return hipGetLastError();
}

}  // namespace fp8w
