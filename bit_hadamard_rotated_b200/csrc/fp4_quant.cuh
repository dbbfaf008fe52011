// fp4_quant.cuh -- the quantiser's arithmetic on 16 values in registers,
// shared by hq_fp4_quantize and the expert layer's first product.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "hq_internal.h"
#include "hq_io.cuh"

namespace hq {
namespace fp4 {

// Whether 1 / b stays far from under- and overflow.
__device__ __forceinline__ bool mid_range(float b) { return b >= 0x1p-100f && b <= 0x1p100f; }

// x / b, correctly rounded up to 2^100 and above that at least 2^100 (every
// scale saturates long before), for x = 0 or of middling size like b > 0 and
// y = 1 / b correctly rounded: Markstein's quotient correction (IBM J. Res.
// Dev. 34, 1990).  q = x y is within an ulp, and q + (x - q b) y, both steps
// fused, rounds to the correctly rounded quotient.  The bound on q keeps
// x - q b from inf - inf where x y overflows.
__device__ __forceinline__ float quotient(float x, float b, float y) {
  const float q = fminf(__fmul_rn(x, y), 0x1p100f);
  return __fmaf_rn(__fmaf_rn(-q, b, x), y, q);
}

// 6 times the tensor scale and its reciprocal (NV).
struct SixTs {
  float ts, six, y;
  bool mid;
  __device__ __forceinline__ explicit SixTs(const float* p) {
    if (p == nullptr) {
      ts = 1.f, six = 6.f, y = 1.f / 6.f, mid = true;
    } else {
      ts = __ldg(p);
      six = __fmul_rn(6.f, ts);
      mid = mid_range(six);
      y = mid ? __frcp_rn(six) : 0.f;
    }
  }
};

// The block scale of amax: the scale byte and its value times the tensor
// scale.  In IEEE single precision, as the header defines it.
template <int FMT>
__device__ __forceinline__ void block_scale(float amax, const SixTs& t, uint32_t& byte, float& eff) {
  if constexpr (FMT == HQ_FP4_NV) {
    const float v = t.mid && (amax == 0.f || mid_range(amax)) ? quotient(amax, t.six, t.y) : __fdiv_rn(amax, t.six);
    byte = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    eff = __fmul_rn(__half2float(__half(h)), t.ts);
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
// reciprocal (2^-125 to 2^127): one exact product.  Otherwise as quotient()
// above, two values at a time, so that ties between codes are met exactly at 3
// packed operations instead of two divisions; where the block's largest
// magnitude, amax, is far beyond its (saturated) scale, quotients could
// overflow and are divided out.
//
// The corrected quotient is computed negated, -q = x (-y), then -q + (x - q b)
// (-y), and the codes' signs are flipped back: for x = -0 the negated sum is
// +0 - 0 = +0, so -0 again, where q + (x - q b) y would be -0 + 0 = +0.
// Returns what the codes have to be xored with: their signs, or 0.
template <int FMT>
__device__ __forceinline__ uint32_t quotients(float (&v)[16], float amax, float eff) {
  if (FMT == HQ_FP4_MX || (mid_range(eff) && amax <= __fmul_rn(eff, 0x1p20f))) {
    const float yf = FMT == HQ_FP4_MX ? __uint_as_float(static_cast<uint32_t>(
                                            254 - max(static_cast<int>(__float_as_uint(eff) >> 23), 0)) << 23)
                                      : -__frcp_rn(eff);
    const uint64_t y = f2(yf, yf), b = f2(eff, eff);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t x = f2(v[2 * i], v[2 * i + 1]);
      uint64_t q = mul2(x, y);
      if constexpr (FMT == HQ_FP4_NV) q = fma2(fma2(q, b, x), y, q);
      un2(q, v[2 * i], v[2 * i + 1]);
    }
    return FMT == HQ_FP4_NV ? 0x88888888u : 0u;
  }
  if (eff > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], eff);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = copysignf(0.f, v[i]);
  }
  return 0;
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

// The largest magnitude of 16 values, as its bit pattern: magnitudes order as
// their patterns, infinity and NaN lie above all finite ones.
__device__ __forceinline__ uint32_t top_of(const float (&v)[16]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return top;
}

// 16 values of a block, largest magnitude `top`, to codes and scale.  E8M0
// blocks are two threads' 16 values, lanes `mate` apart (all lanes of the warp
// take part).
template <int FMT>
__device__ __forceinline__ Packed16 pack16(float (&v)[16], uint32_t top, const SixTs& ts, int mate) {
  if constexpr (FMT == HQ_FP4_MX) top = max(top, __shfl_xor_sync(~0u, top, mate));
  Packed16 p;
  block_scale<FMT>(__uint_as_float(top), ts, p.byte, p.eff);
  if (top >= 0x7F800000u) {  // the format's NaN as the scale, over codes of zero
    p.byte = FMT == HQ_FP4_NV ? 0x7Fu : 0xFFu;
    p.eff = __uint_as_float(0x7FC00000u);
    p.codes = make_uint2(0, 0);
    return p;
  }
  const uint32_t signs = quotients<FMT>(v, __uint_as_float(top), p.eff);
  p.codes.x = to_e2m1x8(v) ^ signs;
  p.codes.y = to_e2m1x8(v + 8) ^ signs;
  return p;
}

// 16 consecutive values of a row as loaded.
template <typename T>
struct Raw16 {
  static constexpr int N = sizeof(T);  // 16-byte vectors
  uint4 u[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack(float (&v)[16]) const {
    const T* t = reinterpret_cast<const T*>(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = to_f32<T>(t[i]);
  }
  // top_of, for 16-bit types two values at a time on their own patterns.
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      float v[16];
      unpack(v);
      return top_of(v);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
      uint32_t m = w[0] & 0x7FFF7FFFu;
      m = __vmaxu2(m, w[1] & 0x7FFF7FFFu);
#pragma unroll
      for (int i = 2; i < 8; i += 2) m = __vimax3_u16x2(m, w[i] & 0x7FFF7FFFu, w[i + 1] & 0x7FFF7FFFu);
      const uint32_t h = max(m & 0xFFFFu, m >> 16);
      const unsigned short s = static_cast<unsigned short>(h);
      return __float_as_uint(to_f32<T>(*reinterpret_cast<const T*>(&s)));
    }
  }
};

}  // namespace fp4
}  // namespace hq
