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

#include "device.hpp"
#include "internal.hpp"

namespace fp8w {
namespace {

// A run of at most `height` slots of one expert.
struct ExpertTile {
  int expert;   // -1: past the last tile
  int slot0, count;
};

// Tile `index` of all experts' runs of `height` slots, in expert order.  The
// offsets are kept inside [0, slots], so what a wrong offset names is still
// in bounds.  By a whole wave; the answer is the same in every lane.
__device__ __forceinline__ ExpertTile expert_tile(const int32_t* offsets, int experts, int slots, int height, int index) {
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;
  for (int e0 = 0; e0 < experts; e0 += kWave) {
    const int e = e0 + lane;
    int from = 0, to = 0;
    if (e < experts) {
      from = min(max(ld_global<int32_t>(offsets, (size_t)e * 4), 0), slots);
      to = min(max(ld_global<int32_t>(offsets, (size_t)e * 4 + 4), 0), slots);
    }
    const int tiles = to > from ? (to - from + height - 1) / height : 0;
    int upto = tiles;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int up = __shfl_up(upto, off);
      if (lane >= off) upto += up;
    }
    const int first = before + upto - tiles;
    const uint64_t mine = __ballot(index >= first && index < first + tiles);
    if (mine) {
      const int l = __builtin_ctzll(mine);
      const int slot0 = from + (index - first) * height;
      ExpertTile t;
      t.expert = e0 + l;
      t.slot0 = __builtin_amdgcn_readlane(slot0, l);
      t.count = __builtin_amdgcn_readlane(min(height, to - slot0), l);
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return ExpertTile{-1, 0, 0};
}

// A workgroup's tile: `group` of n_groups along n, a run of slots of one
// expert.  Workgroups go round the 8 XCDs in turn, and each XCD has its own
// L2: it gets one contiguous eighth of the tiles, in which a run's groups
// follow one another, so that an expert's weights and rows are read by one
// XCD, or two.
struct TileAt {
  int expert, slot0, count, group;
};
__device__ __forceinline__ int count_tiles(const int32_t* offsets, int experts, int slots, int height) {
  const int lane = threadIdx.x & (kWave - 1);
  int mine = 0;
  for (int e = lane; e < experts; e += kWave) {
    const int from = min(max(ld_global<int32_t>(offsets, (size_t)e * 4), 0), slots);
    const int to = min(max(ld_global<int32_t>(offsets, (size_t)e * 4 + 4), 0), slots);
    mine += to > from ? (to - from + height - 1) / height : 0;
  }
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) mine += __shfl_xor(mine, off);
  return __builtin_amdgcn_readfirstlane(mine);
}
__device__ __forceinline__ TileAt tile_at(const int32_t* offsets, int experts, int slots, int height, int n_groups) {
  const int64_t tiles = (int64_t)count_tiles(offsets, experts, slots, height) * n_groups;
  const int64_t share = (tiles + 7) / 8;
  const int64_t place = blockIdx.x >> 3, id = (blockIdx.x & 7) * share + place;
  if (place >= share || id >= tiles) return TileAt{-1, 0, 0, 0};
  const int run = (int)(id / n_groups);
  const ExpertTile t = expert_tile(offsets, experts, slots, height, run);
  return TileAt{t.expert, t.slot0, t.count, (int)(id - (int64_t)run * n_groups)};
}

__device__ __forceinline__ float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// The simple kernel: one wave takes 16 weight rows (with SWIGLU 16 of each
// half) against 16 slots, operands straight from memory.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void k_experts_simple(ExpertsCall c, int n_groups) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int group = blockIdx.x % n_groups;
  const ExpertTile tile = expert_tile(c.offsets, c.experts, c.slots, 16, blockIdx.x / n_groups);
  if (tile.expert < 0) return;
  const int n_out = SWIGLU ? c.n / 2 : c.n;
  const int n0 = (group * 4 + wave) * 16;
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
    float out[2] = {acc[0][v], acc[1][v]};
#pragma unroll
    for (int q = 0; q < (SWIGLU ? 2 : 1); ++q) {
      if (c.format == kFmtRow) out[q] *= ld_global<float>(sc, (size_t)(n + q * n_out) * 4);
      if (c.format == kFmtTensor) out[q] *= ld_global<float>(sc, 0);
    }
    const float r = SWIGLU ? silu_times(out[0], out[1]) : out[0];
    st_global<uint16_t>(c.y, ((size_t)slot * n_out + n) * 2, (uint16_t)f32_to_bf16_rne(r));
  }
}

// The tiled kernel: 256 weight rows against 16 * MT slots of one expert.
//
// Four waves take 64 weight rows each (SWIGLU: 32 of each half) against all
// the slots, so a wave's weights belong to it alone: they go from memory to
// its registers in the MFMA A layout (a lane holds row l%16, bytes 16(l/16)
// of each 64) one 128-column block ahead, and become bf16 there once for all
// slot tiles.  x is staged in LDS, two buffers, in 16-byte units XOR-swizzled
// by row % 16, so that both the writes and the B operand reads spread over
// the banks; one barrier a block.  Block scales multiply the fp32 sums of
// each 128-column block, MX scales the codes as they become bf16 (exact).
template <int FMT, bool SWIGLU, int MT>
__global__ __launch_bounds__(256, MT > 4 ? 1 : 2) void k_experts_tile(ExpertsCall c, int n_groups) {
  constexpr bool kBlock = FMT == kFmtBlock || FMT == kFmtBlockBf16;
  constexpr bool kMx = FMT == kFmtMx;
  constexpr int kSlots = 16 * MT;
  __shared__ __attribute__((aligned(16))) unsigned char xs[2][kSlots * 256];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int i = lane & 15, g = lane >> 4;
  const TileAt at = tile_at(c.offsets, c.experts, c.slots, kSlots, n_groups);
  if (at.expert < 0) return;
  const int n_out = SWIGLU ? c.n / 2 : c.n;
  const int k = c.k, nkb = (k + 127) / 128, ng = (k + 31) / 32;

  // weight row of 16-row tile t that lane i loads, cut to the last row
  const int n0 = at.group * (SWIGLU ? 128 : 256) + wave * (SWIGLU ? 32 : 64);
  const uint8_t* codes = c.codes + (size_t)at.expert * c.n * k;
  const char* scales = static_cast<const char*>(c.scales) + (size_t)at.expert * c.scale_bytes;
  const auto out_row = [&](int t) { return n0 + 16 * (SWIGLU ? t & 1 : t); };
  const auto half = [&](int t) { return SWIGLU && t >= 2 ? n_out : 0; };
  const uint8_t* wp[4];
  const char* sp[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int row = min(out_row(t) + i, n_out - 1) + half(t);
    wp[t] = codes + (size_t)row * k + 16 * g;
    if (kMx) sp[t] = scales + (size_t)row * ng;
    // a lane's four sums are rows 4g.. of the tile: one scale block (the
    // halves start on a multiple of 4)
    if (kBlock) sp[t] = scales + (size_t)((min(out_row(t) + 4 * g, n_out - 1) + half(t)) / 128) * nkb * (FMT == kFmtBlock ? 4 : 2);
  }
  // x rows this thread stages: slot 16q + tid/16, unit tid%16
  const uint16_t* xp[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int slot = at.slot0 + min(16 * q + tid / 16, at.count - 1);
    const int row = c.rows ? ld_global<int32_t>(c.rows, (size_t)slot * 4) : slot;
    xp[q] = c.x + (size_t)(row >= 0 && row < c.x_rows ? row : 0) * k + 8 * (tid & 15);
  }

  uint4 wr[4][2], xr[MT];
  float sc[4];
  uint8_t ex[4][2];
  const auto request = [&](int kb) {
    const bool whole = kb * 128 + 128 <= k;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (whole || kb * 128 + 64 * h + 16 * g < k)
          wr[t][h] = ld_global_u4(wp[t], (size_t)kb * 128 + 64 * h);
        else
          wr[t][h] = make_uint4(0, 0, 0, 0);
        if (kMx) ex[t][h] = ld_global<uint8_t>(sp[t], (size_t)min(4 * kb + 2 * h + (g >> 1), ng - 1));
      }
      if (FMT == kFmtBlock) sc[t] = ld_global<float>(sp[t], (size_t)kb * 4);
      if (FMT == kFmtBlockBf16) sc[t] = bf16_lo(ld_global<uint16_t>(sp[t], (size_t)kb * 2));
    }
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      if (whole || kb * 128 + 8 * (tid & 15) < k)
        xr[q] = ld_global_u4(xp[q], (size_t)kb * 256);
      else
        xr[q] = make_uint4(0, 0, 0, 0);
    }
  };
  const auto stage = [&](int buf) {
#pragma unroll
    for (int q = 0; q < MT; ++q)
      *reinterpret_cast<uint4*>(&xs[buf][(16 * q + tid / 16) * 256 + 16 * ((tid & 15) ^ (tid / 16))]) = xr[q];
  };

  f32x4 acc[4][MT];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int q = 0; q < MT; ++q) acc[t][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  request(0);
  stage(0);
  __syncthreads();
#pragma unroll 1
  for (int kb = 0; kb < nkb; ++kb) {
    bf16x8 a[4][4];
    float s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[t] = kBlock ? sc[t] : 1.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        a_operands<kMx>(wr[t][h], kMx ? mx_scale(ex[t][h]) : 1.0f, a[t][2 * h], a[t][2 * h + 1]);
    }
    if (kb + 1 < nkb) request(kb + 1);
    const unsigned char* xb = xs[kb & 1];
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      bf16x8 b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        b[u] = *reinterpret_cast<const bf16x8*>(&xb[(16 * q + i) * 256 + 16 * ((8 * (u >> 1) + 2 * g + (u & 1)) ^ i)]);
      f32x4 part[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) part[t] = kBlock ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[t][q];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][u], b[u], part[t], 0, 0, 0);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (kBlock) {
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[t][q][v] = __builtin_fmaf(s[t], part[t][v], acc[t][q][v]);
        } else {
          acc[t][q] = part[t];
        }
      }
    }
    if (kb + 1 < nkb) {
      stage((kb + 1) & 1);
      __syncthreads();
    }
  }

  // rows 4g .. 4g + 3 of each tile, for slot 16q + l%16
  float os[4][4];
  if (FMT == kFmtRow) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        os[t][v] = ld_global<float>(scales, (size_t)(min(out_row(t) + 4 * g + v, n_out - 1) + half(t)) * 4);
  }
  const float whole_scale = FMT == kFmtTensor ? ld_global<float>(scales, 0) : 1.0f;
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    if (16 * q + i >= at.count) continue;
    const int slot = at.slot0 + 16 * q + i;
    bool live = true;
    if (c.rows) {
      const int row = ld_global<int32_t>(c.rows, (size_t)slot * 4);
      live = row >= 0 && row < c.x_rows;   // else the products of zeros
    }
#pragma unroll
    for (int t = 0; t < (SWIGLU ? 2 : 4); ++t) {
      const int n = out_row(t) + 4 * g;
      uint32_t r[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float o = acc[t][q][v];
        if (FMT == kFmtRow) o *= os[t][v];
        if (FMT == kFmtTensor) o *= whole_scale;
        if (SWIGLU) {
          float u = acc[(t + 2) & 3][q][v];
          if (FMT == kFmtRow) u *= os[(t + 2) & 3][v];
          if (FMT == kFmtTensor) u *= whole_scale;
          o = silu_times(o, u);
        }
        r[v] = live ? f32_to_bf16_rne(o) : 0;
      }
      const size_t to = ((size_t)slot * n_out + n) * 2;
      if (n_out % 4 == 0) {
        if (n < n_out) st_global<u32x2>(c.y, to, u32x2{r[0] | (r[1] << 16), r[2] | (r[3] << 16)});
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n + v < n_out) st_global<uint16_t>(c.y, to + 2 * v, (uint16_t)r[v]);
      }
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

// The kernel of a call, by its sizes.  Slot tiles of 16 * mt, or 0 for the
// simple kernel: halves that do not start on a multiple of 4 rows would put
// a lane's four sums in two scale blocks.
int experts_mt(int64_t experts, int64_t slots, int64_t n, bool swiglu, int format) {
  const bool block = format == kFmtBlock || format == kFmtBlockBf16;
  if (swiglu && block && (n / 2) % 4 != 0) return 0;
  const int64_t average = slots / (experts < slots ? experts : slots);
  return average >= 96 ? 8 : average >= 40 ? 4 : average >= 12 ? 2 : 1;
}

int64_t experts_groups(int mt, int64_t n, bool swiglu) {
  const int64_t n_out = swiglu ? n / 2 : n, width = mt == 0 ? 64 : swiglu ? 128 : 256;
  return (n_out + width - 1) / width;
}

template <int FMT, bool SWIGLU>
void launch_tile(const ExpertsCall& c, int mt, unsigned blocks, int groups, hipStream_t stream) {
  switch (mt) {
    case 8: k_experts_tile<FMT, SWIGLU, 8><<<blocks, 256, 0, stream>>>(c, groups); break;
    case 4: k_experts_tile<FMT, SWIGLU, 4><<<blocks, 256, 0, stream>>>(c, groups); break;
    case 2: k_experts_tile<FMT, SWIGLU, 2><<<blocks, 256, 0, stream>>>(c, groups); break;
    default: k_experts_tile<FMT, SWIGLU, 1><<<blocks, 256, 0, stream>>>(c, groups); break;
  }
}

template <int FMT>
void launch_act(const ExpertsCall& c, int mt, unsigned blocks, int groups, hipStream_t stream) {
  if (c.swiglu)
    launch_tile<FMT, true>(c, mt, blocks, groups, stream);
  else
    launch_tile<FMT, false>(c, mt, blocks, groups, stream);
}

}  // namespace

// Workgroups of one launch, a multiple of 8 (a share for every XCD).
int64_t experts_blocks(int64_t experts, int64_t slots, int64_t n, bool swiglu, int format) {
  const int mt = experts_mt(experts, slots, n, swiglu, format);
  const int64_t tiles = max_tiles(slots, experts, mt == 0 ? 16 : 16 * mt) * experts_groups(mt, n, swiglu);
  return (tiles + 7) / 8 * 8;
}

hipError_t launch_gemm_experts(const ExpertsCall& c, hipStream_t stream) {
  const int mt = experts_mt(c.experts, c.slots, c.n, c.swiglu, c.format);
  const int groups = (int)experts_groups(mt, c.n, c.swiglu);
  const unsigned blocks = (unsigned)experts_blocks(c.experts, c.slots, c.n, c.swiglu, c.format);
  if (mt == 0) {
    if (c.swiglu)
      k_experts_simple<true><<<blocks, 256, 0, stream>>>(c, groups);
    else
      k_experts_simple<false><<<blocks, 256, 0, stream>>>(c, groups);
    return hipGetLastError();
  }
  switch (c.format) {
    case kFmtBlock: launch_act<kFmtBlock>(c, mt, blocks, groups, stream); break;
    case kFmtMx: launch_act<kFmtMx>(c, mt, blocks, groups, stream); break;
    case kFmtBlockBf16: launch_act<kFmtBlockBf16>(c, mt, blocks, groups, stream); break;
    case kFmtRow: launch_act<kFmtRow>(c, mt, blocks, groups, stream); break;
    default: launch_act<kFmtTensor>(c, mt, blocks, groups, stream); break;
  }
  return hipGetLastError();
}

}  // namespace fp8w
