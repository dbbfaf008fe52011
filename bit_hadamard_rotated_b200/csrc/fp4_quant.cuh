// fp4_quant.cuh -- the quantiser's arithmetic on 16 values in registers,
// shared by hq_fp4_quantize and the expert layer's first product.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "hq_internal.h"

namespace hq {
namespace fp4 {

// The block scale of amax: the scale byte and its value times the tensor
// scale.  In IEEE single precision, as the header defines it.
template <int FMT>
__device__ __forceinline__ void block_scale(float amax, float ts, uint32_t& byte, float& eff) {
  if constexpr (FMT == HQ_FP4_NV) {
    byte = __nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(6.f, ts)), __NV_SATFINITE, __NV_E4M3);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    eff = __fmul_rn(__half2float(__half(h)), ts);
  } else {
    // floor(log2 amax) - 2, at least -127: the exponent field of a normal
    // amax less 2 (a subnormal amax gives the smallest scale either way)
    const int f = static_cast<int>(__float_as_uint(amax) >> 23) - 2;
    byte = static_cast<uint32_t>(max(f, 0));
    eff = byte == 0 ? __uint_as_float(1u << 22) : __uint_as_float(byte << 23);
  }
}

// Two fp32 values in one 64-bit register pair, for the packed fp32 pipe.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void un2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// x / eff for 16 values.  An E8M0 scale is a power of two and so is its
// reciprocal (2^-125 to 2^127): one exact product.  Otherwise, where 1 / eff is
// far from under- and overflow, by Markstein's quotient correction (IBM J. Res.
// Dev. 34, 1990): with y the correctly rounded 1 / eff, q = x y is within an
// ulp and q + (x - q eff) y, both steps fused, rounds to the correctly rounded
// quotient; so ties between codes are met exactly, at 3 packed operations for
// two values instead of two divisions.
template <int FMT>
__device__ __forceinline__ void quotients(float (&v)[16], float eff) {
  if (FMT == HQ_FP4_MX || (eff >= 0x1p-100f && eff <= 0x1p100f)) {
    const float yf = FMT == HQ_FP4_MX ? __uint_as_float(static_cast<uint32_t>(
                                            254 - max(static_cast<int>(__float_as_uint(eff) >> 23), 0)) << 23)
                                      : __frcp_rn(eff);
    const uint64_t y = f2(yf, yf), n = f2(-eff, -eff);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t x = f2(v[2 * i], v[2 * i + 1]);
      uint64_t q = mul2(x, y);
      if constexpr (FMT == HQ_FP4_NV) q = fma2(fma2(q, n, x), y, q);
      un2(q, v[2 * i], v[2 * i + 1]);
    }
  } else if (eff > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], eff);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = copysignf(0.f, v[i]);
  }
}

// Two values to two E2M1 codes (low nibble first), round to nearest even,
// saturating.  One conversion per statement: four with their bytes packed by a
// vector mov in one statement were compiled to zeros in one of the kernels
// (CUDA 12.9; its test is the equality of the fused and the two-step product).
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
  return to_e2m1x2(v[0], v[1]) | to_e2m1x2(v[2], v[3]) << 8 | to_e2m1x2(v[4], v[5]) << 16 |
         to_e2m1x2(v[6], v[7]) << 24;
}

__device__ __forceinline__ float2 from_e2m1x2(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct Packed16 {
  uint2 codes;    // 16 codes, low nibble first
  uint32_t byte;  // the block's scale
  float eff;      // its value times the tensor scale
};

// 16 values of a block to codes and scale.  E8M0 blocks are two threads' 16
// values, lanes `mate` apart (all lanes of the warp take part).
template <int FMT>
__device__ __forceinline__ Packed16 pack16(float (&v)[16], float ts, int mate) {
  // The largest magnitude as a bit pattern: magnitudes order as their
  // patterns, infinity and NaN lie above all finite ones.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  if constexpr (FMT == HQ_FP4_MX) top = max(top, __shfl_xor_sync(~0u, top, mate));
  Packed16 p;
  block_scale<FMT>(__uint_as_float(top), ts, p.byte, p.eff);
  if (top >= 0x7F800000u) {  // the format's NaN as the scale, over codes of zero
    p.byte = FMT == HQ_FP4_NV ? 0x7Fu : 0xFFu;
    p.eff = __uint_as_float(0x7FC00000u);
    p.codes = make_uint2(0, 0);
    return p;
  }
  quotients<FMT>(v, p.eff);
  p.codes.x = to_e2m1x8(v);
  p.codes.y = to_e2m1x8(v + 8);
  return p;
}

}  // namespace fp4
}  // namespace hq
