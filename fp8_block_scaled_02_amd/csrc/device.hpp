// device.hpp -- device helpers shared by the libfp8w kernels (gfx950 only).
//
// bf16 <-> fp32 bit helpers, the e4m3fn encoder, the e8m0 exponent rule and
// wavefront reductions.  Nothing here is shared with the CPU oracle.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8w {

constexpr int kWave = 64;       // CDNA wavefront width
constexpr int kTile = 128;      // block-scale tile edge, both axes
constexpr int kGroup = 32;      // elements per e8m0 scale, along K
constexpr uint32_t kF32Bits448 = 0x43E00000u;   // 448.0f
constexpr uint32_t kF32BitsMinNormalE4M3 = 0x3C800000u;   // 2^-6

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Loads and stores through the global address space.  Pointers read from a
// job table are generic; generic (flat) accesses also count against the LDS
// counter, so a wait for an LDS write would wait for the weight stream too.
// Scalar types only (the global address space does not bind to class types).
template <typename T>
__device__ __forceinline__ T ld_global(const void* p, size_t byte_offset = 0) {
  return *(const __attribute__((address_space(1))) T*)((const char*)p + byte_offset);
}
template <typename T>
__device__ __forceinline__ void st_global(void* p, size_t byte_offset, T v) {
  *(__attribute__((address_space(1))) T*)((char*)p + byte_offset) = v;
}
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 ld_global_u4(const void* p, size_t byte_offset) {
  const u32x4 v = ld_global<u32x4>(p, byte_offset);
  return make_uint4(v.x, v.y, v.z, v.w);
}
// Non-temporal 16-byte load, for data read exactly once (the weight stream):
// on MI355X it lifts a pure streaming read from about 6.3 to 6.8 TB/s.
__device__ __forceinline__ uint4 ld_stream_u4(const void* p, size_t byte_offset) {
  const u32x4 v = __builtin_nontemporal_load(
      (const __attribute__((address_space(1))) u32x4*)((const char*)p + byte_offset));
  return make_uint4(v.x, v.y, v.z, v.w);
}

// Non-temporal 8-byte store, for outputs written once (quantized codes).
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void st_stream_u2(void* p, size_t byte_offset, uint2 v) {
  __builtin_nontemporal_store(u32x2{v.x, v.y},
                              (__attribute__((address_space(1))) u32x2*)((char*)p + byte_offset));
}

// The same for 16 bytes.
__device__ __forceinline__ void st_stream_u4(void* p, size_t byte_offset, u32x4 v) {
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) u32x4*)((char*)p + byte_offset));
}

// s_waitcnt vmcnt(0), leaving the LDS/scalar and export counters alone
// (gfx9 encoding: vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8).
__device__ __forceinline__ void vm_wait_all() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// bf16 halves of a packed dword, widened exactly to fp32.
__device__ __forceinline__ float bf16_lo(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); }

// fp32 -> bf16 bits, round to nearest even (finite inputs; NaN stays NaN).
__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Two fp32 -> two bf16, a in the low half, by the hardware conversion (round
// to nearest even, NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// e4m3fn codes by the hardware conversion (v_cvt_pk_fp8_f32: round to
// nearest even, OCP e4m3fn on gfx950, sign kept, -0 -> 0x80) after clamping
// to [-448, 448], which is the saturation.  Measured on MI355X over every
// non-NaN fp32 bit pattern, in both byte positions of the packed result: the
// byte equals an integer RNE encoder of the bit pattern (top three mantissa
// bits kept, 20 dropped bits rounded to nearest even, exponent rebiased; the
// uniform 2^-9 grid below 2^-6) in every case.  Inputs must not be NaN.
__device__ __forceinline__ float clamp448(float q) { return __builtin_fminf(__builtin_fmaxf(q, -448.0f), 448.0f); }

// Four codes packed little-endian: a in bits 0-7, ..., d in bits 24-31.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(a), clamp448(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(c), clamp448(d), lo, true);
}

__device__ __forceinline__ uint32_t e4m3_code(float q) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(q), 0.0f, 0, false) & 0xFFu;
}

// MX exponent of a group from its amax (the fp32 bit pattern of a
// non-negative value): the smallest e with amax <= 448 * 2^e, clamped to
// [-127, 127].  With amax = 2^x * 1.f and 448 = 2^8 * 1.75, e = x - 8 when
// 1.f <= 1.75 and x - 7 otherwise.  fp32 subnormals and zero land below
// -127 and clamp there; no finite amax reaches 127.
__device__ __forceinline__ int e8m0_exponent(uint32_t amax_bits) {
  const int field = (int)(amax_bits >> 23);
  if (field == 0) return -127;
  const int e = field - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// Sum over aligned groups of `width` consecutive lanes (width a power of two
// <= 64).  Every lane of the group ends with the group's sum.
template <int width>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = width / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, width);
  return v;
}

template <int width>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
#pragma unroll
  for (int off = width / 2; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off, width);
    v = o > v ? o : v;
  }
  return v;
}

// The lane index, recomputed at every call (an opaque v_mbcnt pair): kernels
// at the register limit otherwise keep lane-derived row indices live from the
// start, and spill them.
__device__ __forceinline__ int lane_fresh() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// 2^(e - 127) as an exact fp32: a normal number for e >= 1, the subnormal
// 2^-127 for e == 0.
__device__ __forceinline__ float mx_scale(uint8_t e) {
  return __uint_as_float(e ? (uint32_t)e << 23 : 0x00400000u);
}

// Two e4m3 codes (bytes 0,1 or 2,3 of d) -> two bf16 (exact).
__device__ __forceinline__ bf16x2 cvt_lo(uint32_t d) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false);
}
__device__ __forceinline__ bf16x2 cvt_hi(uint32_t d) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true);
}

// Two e4m3 codes times the MX scale s = 2^(E-127), rounded to bf16, in one
// instruction.  Measured on MI355X over every code and every e8m0 byte
// 0..254: bit-identical to rounding fp32(code) * s (exact in fp32) to bf16;
// byte 255, E8M0's NaN, gives NaN where that product would be infinite (a
// non-finite weight, outside the contract either way).
template <bool HI>
__device__ __forceinline__ bf16x2 cvt_scaled(uint32_t d, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, s, HI);
}

// 16 e4m3 codes -> the two bf16x8 A operands of one 64-column chunk (first
// and last 8 K positions of each lane's 16), scaled by s for MX.
template <bool MX>
__device__ __forceinline__ void a_operands(uint4 d, float s, bf16x8& A0, bf16x8& A1) {
  bf16x2 a0, a1, a2, a3, b0, b1, b2, b3;
  if (MX) {
    a0 = cvt_scaled<false>(d.x, s), a1 = cvt_scaled<true>(d.x, s);
    a2 = cvt_scaled<false>(d.y, s), a3 = cvt_scaled<true>(d.y, s);
    b0 = cvt_scaled<false>(d.z, s), b1 = cvt_scaled<true>(d.z, s);
    b2 = cvt_scaled<false>(d.w, s), b3 = cvt_scaled<true>(d.w, s);
  } else {
    a0 = cvt_lo(d.x), a1 = cvt_hi(d.x), a2 = cvt_lo(d.y), a3 = cvt_hi(d.y);
    b0 = cvt_lo(d.z), b1 = cvt_hi(d.z), b2 = cvt_lo(d.w), b3 = cvt_hi(d.w);
  }
  A0 = bf16x8{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
  A1 = bf16x8{b0[0], b0[1], b1[0], b1[1], b2[0], b2[1], b3[0], b3[1]};
}

}  // namespace fp8w
