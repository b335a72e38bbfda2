// AdamW over many tensors in one launch, with states in 32 or in 8 bits.
//
//   g = scale * grad; m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2
//   p -= lr (m / (1-b1^t) / (sqrt(v / (1-b2^t)) + eps) + decay p)
//
// The tensors' table is a kernel argument. The work is cut into blocks of 256 values
// of one tensor (those that share a scale in 8 bits); a warp takes a block, a lane
// eight consecutive values of it.
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
__device__ __host__ __forceinline__ uint32_t mix32(uint32_t v) {
  v = (v ^ (v >> 16)) * 0x7FEB352Du;
  v = (v ^ (v >> 15)) * 0x846CA68Bu;
  return v ^ (v >> 16);
}

__device__ __forceinline__ uint32_t top_of(float v, uint32_t top) {
  return max(top, __float_as_uint(v) & 0x7FFFFFFFu);
}

__device__ __forceinline__ uint32_t warp_top(uint32_t top) { return __reduce_max_sync(0xFFFFFFFFu, top); }

// Scale of a block whose largest magnitude has these bits, and what brings it to 448.
__device__ __forceinline__ float scale_of(uint32_t top, float* inv) {
  *inv = 0.0f;
  if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float t = __uint_as_float(top);
  if (t < 0x1p-100f) return 0.0f;
  *inv = __fdiv_rn(448.0f, t);
  return __fdiv_rn(t, 448.0f);
}

// E4M3 code of v * inv (magnitude at most 448): scaled by 2^-120, a float's exponent
// field is the code's (its subnormals too), so the code is the upper bits and the lower
// 20 are what is rounded; dither (16 bits) carries into the code with their probability.
__device__ __forceinline__ uint32_t code_of(float v, float inv, uint32_t dither) {
  const uint32_t b = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(v), inv), 0x1p-120f));
  return min((b + dither * 16u + 8u) >> 20, 126u) | (v < 0.0f ? 128u : 0u);
}

template <int BITS>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ Table tab) {
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
    const float ic1 = 1.0f / c1, ic2 = 1.0f / c2;
    const uint32_t key = mix32((uint32_t)t * 0x9E3779B1u + a.seed);
    const float b1 = tab.b1, b2 = tab.b2, o1 = tab.o1, o2 = tab.o2;
    const int64_t all = tab.n ? tab.end[tab.n - 1] : 0;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t blk = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); blk < all; blk += step) {
      int lo = 0, hi = tab.n - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (blk < tab.end[mid]) hi = mid; else lo = mid + 1;
      }
      const AdamwTensor& w = tab.t[lo];
      const int64_t own = blk - (lo ? tab.end[lo - 1] : 0);
      const int64_t at = own * kAdamwBlock + lane * 8;
      float ms = 0.0f, vs = 0.0f;
      if (BITS == 8) {
        ms = w.m_scale[own];
        vs = w.v_scale[own];
      }
      float m[8], v[8];
      uint32_t mt = 0, vt = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t k = at + i;
        m[i] = v[i] = 0.0f;
        if (k < w.n) {
          float g = w.grad_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(w.grad)[k] << 16)
                                : static_cast<const float*>(w.grad)[k];
          g = __fmul_rn(g, scale);
          float mo, vo;
          if (BITS == 8) {
            mo = __fmul_rn(e4m3x2_value(static_cast<const uint8_t*>(w.m)[k]).x, ms);
            vo = __fmul_rn(e4m3x2_value(static_cast<const uint8_t*>(w.v)[k]).x, vs);
            vo = __fmul_rn(vo, vo);
          } else {
            mo = static_cast<const float*>(w.m)[k];
            vo = static_cast<const float*>(w.v)[k];
          }
          m[i] = __fadd_rn(__fmul_rn(mo, b1), __fmul_rn(g, o1));
          v[i] = __fadd_rn(__fmul_rn(vo, b2), __fmul_rn(__fmul_rn(g, g), o2));
          const float up = m[i] * ic1 / (sqrtf(v[i] * ic2) + a.eps);
          float* pp = w.master ? w.master + k : static_cast<float*>(w.param) + k;
          const float p = *pp - lr * (up + w.decay * *pp);
          *pp = p;
          if (w.master) static_cast<__nv_bfloat16*>(w.param)[k] = __float2bfloat16_rn(p);
          if (BITS == 8) {
            v[i] = __fsqrt_rn(v[i]);
            mt = top_of(m[i], mt);
            vt = top_of(v[i], vt);
          } else {
            static_cast<float*>(w.m)[k] = m[i];
            static_cast<float*>(w.v)[k] = v[i];
          }
        }
      }
      if (BITS == 8) {
        float im, iv;
        mt = warp_top(mt);
        vt = warp_top(vt);
        ms = scale_of(mt, &im);
        vs = scale_of(vt, &iv);
        if (lane == 0) {
          w.m_scale[own] = ms;
          w.v_scale[own] = vs;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t k = at + i;
          if (k >= w.n) continue;
          const uint64_t idx = (uint64_t)(w.first + k);
          const uint32_t d = mix32((uint32_t)idx * 0x9E3779B1u + (uint32_t)(idx >> 32) * 0x85EBCA77u + key);
          static_cast<uint8_t*>(w.m)[k] = mt < 0x7F800000u ? (uint8_t)code_of(m[i], im, d & 0xFFFFu) : 0x7F;
          static_cast<uint8_t*>(w.v)[k] = vt < 0x7F800000u ? (uint8_t)code_of(v[i], iv, d >> 16) : 0x7F;
        }
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
  if (grid > 8 * sms) grid = 8 * sms;
  if (grid < 1) grid = 1;
  e = launch_pdl(a.bits == 8 ? adamw_kernel<8> : adamw_kernel<32>, dim3((unsigned)grid), dim3(256), 0, s, tab);
  return e != cudaSuccess ? -(int)e : 1;
}

}  // namespace moe
