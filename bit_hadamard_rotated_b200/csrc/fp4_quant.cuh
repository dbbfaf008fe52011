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

// x / eff for 16 values.  Where 1 / eff is far from under- and overflow, by
// Markstein's quotient correction (IBM J. Res. Dev. 34, 1990): with y the
// correctly rounded 1 / eff, q = x y is within an ulp and q + (x - q eff) y,
// both steps fused, rounds to the correctly rounded quotient; so ties between
// codes are met exactly, at 3 operations a value instead of a division.
__device__ __forceinline__ void quotients(float (&v)[16], float eff) {
  if (eff >= 0x1p-100f && eff <= 0x1p100f) {
    const float y = __frcp_rn(eff);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = __fmul_rn(v[i], y);
      v[i] = __fmaf_rn(__fmaf_rn(-q, eff, v[i]), y, q);
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
// saturating.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
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
  float amax = 0.f;
  bool fine = true;  // every value finite
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(v[i]);
    amax = fmaxf(amax, m);
    fine = fine && m < INFINITY;
  }
  if constexpr (FMT == HQ_FP4_MX) {
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, mate));
    fine = __shfl_xor_sync(~0u, static_cast<int>(fine), mate) && fine;
  }
  Packed16 p;
  block_scale<FMT>(amax, ts, p.byte, p.eff);
  if (!fine) {  // the format's NaN as the scale, over codes of zero
    p.byte = FMT == HQ_FP4_NV ? 0x7Fu : 0xFFu;
    p.eff = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  } else {
    quotients(v, p.eff);
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = to_e2m1x2(v[2 * i], v[2 * i + 1]);
  p.codes.x = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24;
  p.codes.y = w[4] | w[5] << 8 | w[6] << 16 | w[7] << 24;
  return p;
}

}  // namespace fp4
}  // namespace hq
