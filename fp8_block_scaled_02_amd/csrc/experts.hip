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

// Runs of `height` slots that any split of the slots over the experts can
// have: each expert ends with at most one run that is not full.
int64_t max_tiles(int64_t slots, int64_t experts, int64_t height) {
  const int64_t e = experts < slots ? experts : slots;
  return (slots + e * (height - 1)) / height;
}

}  // namespace

int64_t experts_blocks(int64_t experts, int64_t slots, int64_t n, bool swiglu) {
  return max_tiles(slots, experts, 16) * (((swiglu ? n / 2 : n) + 63) / 64);
}

hipError_t launch_gemm_experts(const ExpertsCall& c, hipStream_t stream) {
  const int n_out = c.swiglu ? c.n / 2 : c.n;
  const int n_groups = (n_out + 63) / 64;
  const unsigned blocks = (unsigned)experts_blocks(c.experts, c.slots, c.n, c.swiglu);
  if (c.swiglu)
    k_experts_simple<true><<<blocks, 256, 0, stream>>>(c, n_groups);
  else
    k_experts_simple<false><<<blocks, 256, 0, stream>>>(c, n_groups);
  return hipGetLastError();
}

}  // namespace fp8w
