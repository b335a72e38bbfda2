// The router's fp32 exp and the live token count, shared by the kernels that route.
#pragma once
#include <stdint.h>

namespace moe {

// fp32 exp: Cody-Waite reduction v = n ln2 + r (ln 2 split into an fp32 head
// and an fp32 tail), degree-7 Taylor polynomial of e^r in Horner form with
// fma, scale by 2^n through the exponent field. Domain v <= 0 (softmax);
// v < -87 gives +0. Every operation is an explicitly rounded IEEE op.
__device__ __forceinline__ float route_exp(float v) {
  if (v < -87.0f) return 0.0f;
  const float log2e = __uint_as_float(0x3FB8AA3Bu);
  const float ln2_hi = __uint_as_float(0x3F317218u);
  const float ln2_lo = __uint_as_float(0xB102E308u);
  const float n = rintf(__fmul_rn(v, log2e));
  float r = __fmaf_rn(-n, ln2_hi, v);
  r = __fmaf_rn(-n, ln2_lo, r);
  float p = __uint_as_float(0x39500D01u);         // 1/7!
  p = __fmaf_rn(p, r, __uint_as_float(0x3AB60B61u));  // 1/6!
  p = __fmaf_rn(p, r, __uint_as_float(0x3C088889u));  // 1/5!
  p = __fmaf_rn(p, r, __uint_as_float(0x3D2AAAABu));  // 1/4!
  p = __fmaf_rn(p, r, __uint_as_float(0x3E2AAAABu));  // 1/3!
  p = __fmaf_rn(p, r, 0.5f);
  p = __fmaf_rn(p, r, 1.0f);
  p = __fmaf_rn(p, r, 1.0f);
  const float scale = __uint_as_float((uint32_t)((int)n + 127) << 23);
  return __fmul_rn(p, scale);
}

// Live token count: *n_dev clamped to [0, Nmax], or Nmax without a device
// count. Buffers and grids are sized for Nmax (the static bound a captured
// graph was built for); tokens at or past the live count are absent.
__device__ __forceinline__ int live_tokens(const int32_t* n_dev, int Nmax) {
  if (!n_dev) return Nmax;
  const int v = *n_dev;
  return v < 0 ? 0 : (v > Nmax ? Nmax : v);
}

}  // namespace moe
