// linear.hip -- a dense layer's product on fp8 weights with its epilogue:
//
//   y = act(x . deq(W)^T + bias) + residual
//
// for any number of rows of x; bf16 x, fp32 sums, one rounding at the end.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// The simple kernel: one wave takes 16 weight rows (gated: 16 of each half)
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
  const int nkb = (c.k + 127) / 128, ng = (c.k + 31) / 32;
  for (int kb = 0; kb < nkb; ++kb) {
    f32x4 part[2] = {};
    for (int h = 0; h < 2; ++h) {
      const int col = kb * 128 + h * 64 + 16 * g;
      const bool in = col < c.k;
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
          if (c.format == kFmtMx) s = mx_scale(ld_global<uint8_t>(c.scales, (size_t)n * ng + col / 32));
        }
        bf16x8 a0, a1;
        a_operands<true>(w, s, a0, a1);
        part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, b0), part[q], 0, 0, 0);
        part[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, b1), part[q], 0, 0, 0);
      }
    }
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = min(n0 + 4 * g + v, n_out - 1) + q * n_out;
        float s = 1.0f;
        if (c.format == kFmtBlock) s = ld_global<float>(c.scales, ((size_t)(n / 128) * nkb + kb) * 4);
        if (c.format == kFmtBlockBf16) s = bf16_lo(ld_global<uint16_t>(c.scales, ((size_t)(n / 128) * nkb + kb) * 2));
        acc[q][v] = __builtin_fmaf(s, part[q][v], acc[q][v]);
      }
  }
  if (m0 + i >= c.m) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int n = n0 + 4 * g + v;
    if (n >= n_out) continue;
    float r[2];
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      const int nq = n + q * n_out;
      float s = 1.0f;
      if (c.format == kFmtRow) s = ld_global<float>(c.scales, (size_t)nq * 4);
      if (c.format == kFmtTensor) s = ld_global<float>(c.scales, 0);
      r[q] = __builtin_fmaf(s, acc[q][v], bias_of(c, nq));
    }
    store_one(c, m0 + i, n, GATED ? gated(c.act, r[0], r[1]) : activated(c.act, r[0]));
  }
}

bool is_gated(int act) { return act == kActSwiglu || act == kActGeglu; }

}  // namespace

int64_t linear_workspace_bytes(int64_t, int64_t, int64_t, int, int) { return 0; }

int64_t linear_blocks(int64_t m, int64_t n, int64_t, int, int act) {
  const int64_t n_out = is_gated(act) ? n / 2 : n;
  return (m + 15) / 16 * ((n_out + 63) / 64);
}

hipError_t launch_linear(const LinearCall& c, hipStream_t stream) {
  const bool gated = is_gated(c.act);
  const int groups = ((gated ? c.n / 2 : c.n) + 63) / 64;
  const unsigned blocks = (unsigned)linear_blocks(c.m, c.n, c.k, c.format, c.act);
  if (gated)
    k_linear_simple<true><<<blocks, 256, 0, stream>>>(c, groups);
  else
    k_linear_simple<false><<<blocks, 256, 0, stream>>>(c, groups);
  return hipGetLastError();
}

}  // namespace fp8w
