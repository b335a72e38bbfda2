// AdamW over many tensors in one launch, with states in 32 or in 8 bits.
//
//   g = scale * grad; m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2
//   p -= lr (m / (1-b1^t) / (sqrt(v / (1-b2^t)) + eps) + decay p)
//
// The tensors' table is a kernel argument. The work is cut into blocks of 256 values
// of one tensor (those that share a scale in 8 bits); a warp takes a block, a lane eight
// values of it.
//
// 32 bits: bound by memory, 44 million bf16 weights with f32 masters and bf16 gradients in
// 192 us, 6.4 TB/s of the 6.8 that a copy reaches. 8 bits: 277 million with f32 gradients
// in 837 us, 6.0 TB/s; a value takes some 90 instructions of a lane, 72 % of the issue slots are
// used. At 824 us, before roots had a smallest code (+4) and decay was added to the update first
// (+9), it took 799 without the exact root or without the hash, and 955 with the next block
// loaded ahead of this one's work, which cost the fourth block an SM. A launch carries its whole
// table, 21 KB: of a call's 5.6 us of host time for a few tensors 0.9.
#include "act.cuh"
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"

#include <math.h>

namespace moe {
namespace {

struct Table {
  int n;                               // tensors
  int last;                            // this launch ends the step
  float b1, b2, o1, o2;                // the betas, and 1 - beta
  float log_b1, log_b2;                // ln of the betas
  AdamwArgs a;
  int64_t end[kAdamwTensors];          // blocks of the tensors up to and with this one
  AdamwTensor t[kAdamwTensors];
};
static_assert(sizeof(Table) < 32000, "a kernel's arguments are at most 32764 bytes");

// Two rounds of xor-shift and odd multiplication: 32 bits of which each depends on all of v.
// Shifts and multipliers are published ones, of the least bias found for this form (C. Wellons,
// "Prospecting for Hash Functions", 2018). The factors of the index and of the step are the
// prime next to 2^32 over the golden ratio (Knuth's multiplicative hashing) and, for the index's
// upper half, a prime that Y. Collet's 32-bit hash uses: any odd ones would do.
__device__ __host__ __forceinline__ uint32_t mix32(uint32_t v) {
  v = (v ^ (v >> 16)) * 0x7FEB352Du;
  v = (v ^ (v >> 15)) * 0x846CA68Bu;
  return v ^ (v >> 16);
}

// Scale of a block whose largest magnitude has these bits, and what brings it to 448 times
// 2^-120 (see codes4): products with constants and one reciprocal, each rounded.
__device__ __forceinline__ float scale_of(uint32_t top, float* inv) {
  const float t = __uint_as_float(top);
  const bool some = t >= 0x1p-100f && top < 0x7F800000u;
  *inv = some ? __fmul_rn(__frcp_rn(t), 448.0f) : 0.0f;
  return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : some ? __fmul_rn(t, 1.0f / 448.0f) : 0.0f;
}

// Four E4M3 codes of v * inv, magnitudes at most 448, in a word. Scaled by 2^-120, a float's
// exponent field is the code's, and its subnormals are the code's too: the code is the upper
// bits, and the lower 20 are what is rounded. The dither, 16 bits of d from bit SHIFT on and
// a half of the last of them, carries into the code with their probability. It does not
// reach over 448: 2^20 - 8 at most, and a value is at most two units above its code.
// scaled: 2^-120 is already in inv (exact for inv of 2^-6 or more). least: the smallest code.
template <int SHIFT, bool SIGN>
__device__ __forceinline__ uint32_t codes4(const float* v, float inv, bool scaled, const uint32_t* d, uint32_t least) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f = __fmul_rn(fabsf(v[i]), inv);
    if (!scaled) f = __fmul_rn(f, 0x1p-120f);
    const uint32_t dither = SHIFT ? (d[i] >> 12) & 0xFFFF0u : (d[i] << 4) & 0xFFFF0u;
    x[i] = __float_as_uint(f) + dither + 8u;
    if (!SIGN) x[i] = max(x[i], least << 20);
    x[i] <<= 4;  // the code in bits 24-30
    if (SIGN) x[i] = (x[i] & 0x7FFFFFFFu) | (__float_as_uint(v[i]) & 0x80000000u);
  }
  return __byte_perm(__byte_perm(x[0], x[1], 0x0073), __byte_perm(x[2], x[3], 0x0073), 0x5410);
}

// The larger, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight values of a lane: four at 4 lane and four at 128 + 4 lane of the block, so that every
// vector access of a warp is one run. full: the block lies in the tensor; else values past
// the end read as zeros and are not written.
__device__ __forceinline__ void load4(const float* p, float (&v)[8], int at) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[at] = q.x; v[at + 1] = q.y; v[at + 2] = q.z; v[at + 3] = q.w;
}
__device__ __forceinline__ void load8(const float* p, int lane, bool full, int left, float (&v)[8]) {
  if (full) {
    load4(p + 4 * lane, v, 0);
    load4(p + 128 + 4 * lane, v, 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = 4 * lane + (i & 3) + (i >> 2) * 128;
    v[i] = k < left ? p[k] : 0.0f;
  }
}
__device__ __forceinline__ void store8(float* p, int lane, bool full, int left, const float (&v)[8]) {
  if (full) {
    *reinterpret_cast<float4*>(p + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 128 + 4 * lane) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = 4 * lane + (i & 3) + (i >> 2) * 128;
    if (k < left) p[k] = v[i];
  }
}
__device__ __forceinline__ void load8_bf16(const uint16_t* p, int lane, bool full, int left, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (full) {
      const uint2 q = *reinterpret_cast<const uint2*>(p + h * 128 + 4 * lane);
      v[4 * h] = __uint_as_float(q.x << 16);
      v[4 * h + 1] = __uint_as_float(q.x & 0xFFFF0000u);
      v[4 * h + 2] = __uint_as_float(q.y << 16);
      v[4 * h + 3] = __uint_as_float(q.y & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = h * 128 + 4 * lane + i;
        v[4 * h + i] = k < left ? __uint_as_float((uint32_t)p[k] << 16) : 0.0f;
      }
    }
  }
}
__device__ __forceinline__ void store8_bf16(uint16_t* p, int lane, bool full, int left, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * h], v[4 * h + 1]), hi = __floats2bfloat162_rn(v[4 * h + 2], v[4 * h + 3]);
    const uint32_t a = *reinterpret_cast<const uint32_t*>(&lo), b = *reinterpret_cast<const uint32_t*>(&hi);
    if (full) {
      *reinterpret_cast<uint2*>(p + h * 128 + 4 * lane) = make_uint2(a, b);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = h * 128 + 4 * lane + i;
        if (k < left) p[k] = (uint16_t)((i < 2 ? a : b) >> (16 * (i & 1)));
      }
    }
  }
}
// Codes, four bytes a word.
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int lane, int h, bool full, int left) {
  if (full) return *reinterpret_cast<const uint32_t*>(p + h * 128 + 4 * lane);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = h * 128 + 4 * lane + i;
    if (k < left) c |= (uint32_t)p[k] << (8 * i);
  }
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int lane, int h, bool full, int left, uint32_t c) {
  if (full) {
    *reinterpret_cast<uint32_t*>(p + h * 128 + 4 * lane) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = h * 128 + 4 * lane + i;
    if (k < left) p[k] = (uint8_t)(c >> (8 * i));
  }
}
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float (&v)[8], int at) {
  const float2 a = e4m3x2_value(codes & 0xFFFFu), b = e4m3x2_value(codes >> 16);
  v[at] = __fmul_rn(a.x, scale);
  v[at + 1] = __fmul_rn(a.y, scale);
  v[at + 2] = __fmul_rn(b.x, scale);
  v[at + 3] = __fmul_rn(b.y, scale);
}

__device__ __forceinline__ float rcp_approx(float v) {  // within 2^-23 of 1/v; v is eps at least, not subnormal
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float sqrt_approx(float v) {  // within 2^-22 of the root, subnormal v included
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// m, v and the root that is stored are rounded operation by operation, so that a step can be
// repeated elsewhere bit for bit. The update itself takes the fast root and reciprocal:
// 2^-21 of an update is far below the weight's own rounding.
template <int BITS>
__global__ void __launch_bounds__(256, 4) adamw_kernel(const __grid_constant__ Table tab) {
  griddep_wait();
  griddep_launch_dependents();
  const AdamwArgs& a = tab.a;
  const int lane = threadIdx.x & 31;
  const int t = a.steps[0] + 1;
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  const bool skip = !isfinite(scale);
  if (!skip) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    const float c1 = -expm1f((float)t * tab.log_b1), c2 = -expm1f((float)t * tab.log_b2);
    const float lr1 = lr / c1, rc2 = sqrtf(1.0f / c2);
    const uint32_t key = mix32((uint32_t)t * 0x9E3779B1u + a.seed);
    const float b1 = tab.b1, b2 = tab.b2, o1 = tab.o1, o2 = tab.o2, eps = a.eps;
    const int64_t all = tab.n ? tab.end[tab.n - 1] : 0;
    const int64_t step = (int64_t)gridDim.x * 8;
    int64_t blk = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int cur = 0, hi = tab.n - 1;  // this warp's first tensor; the later ones are near
    while (cur < hi) {
      const int mid = (cur + hi) >> 1;
      if (blk < tab.end[mid]) hi = mid; else cur = mid + 1;
    }
    for (; blk < all; blk += step) {
      while (blk >= tab.end[cur]) ++cur;
      const AdamwTensor& w = tab.t[cur];
      const int64_t own = blk - (cur ? tab.end[cur - 1] : 0);
      const int64_t at = own * kAdamwBlock;
      const int left = (int)min((int64_t)kAdamwBlock, w.n - at);
      const bool full = left == kAdamwBlock;
      float* pp = (w.master ? w.master : static_cast<float*>(w.param)) + at;
      float g[8], p[8], m[8], v[8];
      uint32_t cm[2], cv[2];
      float ms = 0.0f, vs = 0.0f;
      if (w.grad_bf16) load8_bf16(static_cast<const uint16_t*>(w.grad) + at, lane, full, left, g);
      else load8(static_cast<const float*>(w.grad) + at, lane, full, left, g);
      load8(pp, lane, full, left, p);
      if (BITS == 8) {
        ms = w.m_scale[own];
        vs = w.v_scale[own];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cm[h] = load_codes(static_cast<const uint8_t*>(w.m) + at, lane, h, full, left);
          cv[h] = load_codes(static_cast<const uint8_t*>(w.v) + at, lane, h, full, left);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          decode4(cm[h], ms, m, 4 * h);
          decode4(cv[h], vs, v, 4 * h);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
      } else {
        load8(static_cast<const float*>(w.m) + at, lane, full, left, m);
        load8(static_cast<const float*>(w.v) + at, lane, full, left, v);
      }
      const float decay = lr * w.decay;
      float ma = 0.0f, va = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gi = __fmul_rn(g[i], scale);
        m[i] = __fadd_rn(__fmul_rn(m[i], b1), __fmul_rn(gi, o1));
        v[i] = __fadd_rn(__fmul_rn(v[i], b2), __fmul_rn(__fmul_rn(gi, gi), o2));
        float root;
        if (BITS == 8) {
          root = v[i] = __fsqrt_rn(v[i]);
          ma = max_nan(ma, fabsf(m[i]));
          va = max_nan(va, root);
        } else {
          root = sqrt_approx(v[i]);
        }
        // both small terms first, then one rounding of the weight: 1 - decay as a factor would be a
        // multiple of 2^-24, so that a decay of 1e-7 became 1.2e-7 and one of 2.5e-8 nothing
        p[i] -= fmaf(lr1 * m[i], rcp_approx(fmaf(root, rc2, eps)), p[i] * decay);
      }
      store8(pp, lane, full, left, p);
      if (w.master) store8_bf16(static_cast<uint16_t*>(w.param) + at, lane, full, left, p);
      if (BITS == 8) {
        float im, iv;
        const uint32_t mt = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(ma) & 0x7FFFFFFFu);
        const uint32_t vt = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(va) & 0x7FFFFFFFu);
        ms = scale_of(mt, &im);
        vs = scale_of(vt, &iv);
        if (lane == 0) {
          w.m_scale[own] = ms;
          w.v_scale[own] = vs;
        }
        // `first` is a multiple of 256, so the index's upper half is the block's
        const uint64_t idx = (uint64_t)(w.first + at);
        const uint32_t base = ((uint32_t)idx + 4u * lane) * 0x9E3779B1u + (uint32_t)(idx >> 32) * 0x85EBCA77u + key;
        const bool scaled = fminf(im, iv) >= 0x1p-6f;  // else a state passes 28672 (or a block is of zeros)
        // A root of code 0 would leave the next step an m that may have been rounded up to a code
        // of its own over (1-b2) g^2 alone: updates of hundreds of lr where a block's values are
        // 10^4 apart (two of lr with code 1, which reads high what lies below 2^-9 / 448 of the
        // largest: such a weight moves less than it would). Blocks of zeros stay at 0.
        const uint32_t least = iv > 0.0f;
        if (scaled) {
          im *= 0x1p-120f;
          iv *= 0x1p-120f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t d[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = mix32(base + (uint32_t)(h * 128 + i) * 0x9E3779B1u);
          const uint32_t qm = scaled ? codes4<0, true>(m + 4 * h, im, true, d, 0u) : codes4<0, true>(m + 4 * h, im, false, d, 0u);
          const uint32_t qv = scaled ? codes4<16, false>(v + 4 * h, iv, true, d, least) : codes4<16, false>(v + 4 * h, iv, false, d, least);
          store_codes(static_cast<uint8_t*>(w.m) + at, lane, h, full, left, qm);
          store_codes(static_cast<uint8_t*>(w.v) + at, lane, h, full, left, qv);
        }
      } else {
        store8(static_cast<float*>(w.m) + at, lane, full, left, m);
        store8(static_cast<float*>(w.v) + at, lane, full, left, v);
      }
    }
  }
  // the last block to finish advances the step: every block has read it by then
  if (!tab.last || skip) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&a.steps[1], 1) == (int)gridDim.x - 1) {
      a.steps[1] = 0;
      a.steps[0] = t;
    }
  }
}

}  // namespace

int launch_adamw(const AdamwArgs& a, const AdamwTensor* t, int n, int last, cudaStream_t s) {
  static DeviceOnce once;
  int sms = 0;
  cudaError_t e = once_per_device(once, &sms, [](int dev, int* v) {
    return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
  if (e != cudaSuccess) return -(int)e;
  Table tab;
  tab.n = n;
  tab.last = last;
  tab.a = a;
  tab.b1 = (float)a.beta1;
  tab.b2 = (float)a.beta2;
  tab.o1 = (float)(1.0 - a.beta1);
  tab.o2 = (float)(1.0 - a.beta2);
  tab.log_b1 = (float)log(a.beta1);
  tab.log_b2 = (float)log(a.beta2);
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    blocks += (t[i].n + kAdamwBlock - 1) / kAdamwBlock;
    tab.end[i] = blocks;
    tab.t[i] = t[i];
  }
  int64_t grid = (blocks + 7) / 8;
  const int per_sm = 4;
  if (grid > per_sm * sms) grid = per_sm * sms;
  if (grid < 1) grid = 1;
  e = launch_pdl(a.bits == 8 ? adamw_kernel<8> : adamw_kernel<32>, dim3((unsigned)grid), dim3(256), 0, s, tab);
  return e != cudaSuccess ? -(int)e : 1;
}

}  // namespace moe
