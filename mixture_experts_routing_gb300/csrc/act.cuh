// The experts' gated activation and its derivative, and the MX (E8M0 + E4M3)
// conversions, shared by the kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// Gated activation act(gate) of the FFN and its derivative ("Permute-Free
// Grouped GEMM for MoE (bf16, gfx950)", section 3 act(gate)*up; section 8:
// silu and gelu): 0 = silu(v) = v sigma(v); 1 = gelu(v) = v Phi(v) (the erf
// form); act_grad: sigma(v)(1 + v(1 - sigma(v))), Phi(v) + v phi(v).
template <int act>
__device__ __forceinline__ float act_fwd(float v) {
  if (act == 1) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  return __fdividef(v, 1.0f + __expf(-v));
}

// The factor both share: act(v) = v c(v) with c = sigma (silu) or Phi (gelu),
// and act'(v) from c: c (1 + v (1 - c)) for silu, c + v phi(v) for gelu. The
// backward evaluates c once per element and derives both from it.
template <int act>
__device__ __forceinline__ float act_core(float v) {
  if (act == 1) return 0.5f * (1.0f + erff(v * 0.70710678118654752f));
  return __fdividef(1.0f, 1.0f + __expf(-v));
}

template <int act>
__device__ __forceinline__ float act_grad_core(float v, float c) {
  if (act == 1) return c + v * (__expf(-0.5f * v * v) * 0.39894228040143268f);
  return c * (1.0f + v * (1.0f - c));
}

// 2^-s for s in [-127, 127], from its bits (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ float pow2_neg(int s) {
  const int e = 127 - s;
  return e > 0 ? __int_as_float(e << 23) : __int_as_float(0x00400000);
}

// floor(log2(a)) - 8 clamped to [-127, 127] for a finite a >= 0; -127 for a = 0.
__device__ __forceinline__ int mx_block_exponent(float a) {
  const uint32_t b = __float_as_uint(a);
  if (b == 0u) return -127;
  const int ef = (int)(b >> 23);
  const int fl = ef > 0 ? ef - 127 : (31 - __clz((int)(b & 0x7FFFFFu))) - 149;
  return min(127, max(-127, fl - 8));
}

// 2^(byte - 127) for an E8M0 byte; 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  if (byte == 255u) return __int_as_float(0x7FC00000);
  return byte ? __int_as_float((int)(byte << 23)) : __int_as_float(0x00400000);
}

// Two E4M3 codes of (lo, hi), lo in the low byte: nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The values of two E4M3 codes (exact in half precision).
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

}  // namespace moe
