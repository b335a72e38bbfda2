// Layer norm (and its RMS form) of bf16 rows, forward and backward.
//
//   forward   s = bf16(x + add); mean, var over the row; y = (s - mean) r w + b
//   backward  z = (s - mean) r, g = dy w;
//             dx = r (g - z mean(g z) - mean(g)) + dx_add
//             dweight = sum over rows of dy z, dbias = sum of dy
//
// A block takes whole rows, a thread the same columns of every row, 8 at a time.
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kVec = 2;        // groups of 8 columns a thread holds
constexpr int kMaxParts = 304;

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  v[0] = __uint_as_float(q.x << 16);
  v[1] = __uint_as_float(q.x & 0xFFFF0000u);
  v[2] = __uint_as_float(q.y << 16);
  v[3] = __uint_as_float(q.y & 0xFFFF0000u);
  v[4] = __uint_as_float(q.z << 16);
  v[5] = __uint_as_float(q.z & 0xFFFF0000u);
  v[6] = __uint_as_float(q.w << 16);
  v[7] = __uint_as_float(q.w & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The sum of v over the block, the same in every thread; `slot` (32 floats) is not
// written again before every thread has passed a later block_sum of another slot.
__device__ __forceinline__ float block_sum(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < warps; ++w) t += slot[w];
  return t;
}

template <bool RMS>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float slots[2][2][32];
  const int H = a.H;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x, turn ^= 1) {
    float v[kVec][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * 8;
      if (c < H) {
        unpack8(*reinterpret_cast<const uint4*>(a.x + row * H + c), v[j]);
        if (a.add) {
          float r[8];
          unpack8(*reinterpret_cast<const uint4*>(a.add + row * H + c), r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] += r[i];
          const uint4 q = pack8(v[j]);
          *reinterpret_cast<uint4*>(a.sum + row * H + c) = q;
          unpack8(q, v[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[j][i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      }
    }
    float mean = 0.0f;
    if (!RMS) mean = block_sum(sum, slots[turn][0]) / (float)H;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * 8;
      if (c < H) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][i] -= mean;
          sq += v[j][i] * v[j][i];
        }
      }
    }
    const float r = 1.0f / sqrtf(block_sum(sq, slots[turn][1]) / (float)H + a.eps);
    if (threadIdx.x == 0) {
      if (!RMS && a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * 8;
      if (c >= H) continue;
      float w[8], o[8];
      load8(a.w + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = v[j][i] * r * w[i];
      if (a.b) {
        load8(a.b + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += w[i];
      }
      *reinterpret_cast<uint4*>(a.y + row * H + c) = pack8(o);
    }
  }
}

template <bool RMS>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float slots[2][2][32];
  const int H = a.H;
  float dw[kVec][8] = {}, db[kVec][8] = {};
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x, turn ^= 1) {
    const float mean = RMS ? 0.0f : a.mean[row], r = a.rstd[row];
    float z[kVec][8], g[kVec][8];
    float sg = 0.0f, sgz = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * 8;
      if (c < H) {
        float w[8];
        unpack8(*reinterpret_cast<const uint4*>(a.x + row * H + c), z[j]);
        unpack8(*reinterpret_cast<const uint4*>(a.dy + row * H + c), g[j]);
        load8(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[j][i] = (z[j][i] - mean) * r;
          dw[j][i] += g[j][i] * z[j][i];
          db[j][i] += g[j][i];
          g[j][i] *= w[i];
          sg += g[j][i];
          sgz += g[j][i] * z[j][i];
        }
      }
    }
    const float mz = block_sum(sgz, slots[turn][0]) / (float)H;
    const float mg = RMS ? 0.0f : block_sum(sg, slots[turn][1]) / (float)H;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * 8;
      if (c >= H) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = r * (g[j][i] - z[j][i] * mz - mg);
      if (a.add) {
        float t[8];
        unpack8(*reinterpret_cast<const uint4*>(a.add + row * H + c), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += t[i];
      }
      *reinterpret_cast<uint4*>(a.dx + row * H + c) = pack8(o);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * 8;
    if (c >= H) continue;
    float* p = a.part + (int64_t)blockIdx.x * 2 * H + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = dw[j][i];
      p[H + i] = db[j][i];
    }
  }
}

// dw and db from the blocks' partial sums, in block order.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* part, int parts, int H, float* dw,
                                                         float* db) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= 2 * H) return;
  float* out = c < H ? dw : db;
  if (!out) return;
  float t = 0.0f;
  for (int p = 0; p < parts; ++p) t += part[(int64_t)p * 2 * H + c];
  out[c < H ? c : c - H] = t;
}

int threads_of(int H) { return ((H + 8 * kVec - 1) / (8 * kVec) + 31) / 32 * 32; }

int parts_of(int64_t N) { return (int)(N < kMaxParts ? N : kMaxParts); }

}  // namespace

int launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(a.N < 2432 ? a.N : 2432);
  const cudaError_t e = launch_pdl(a.rms ? norm_forward_kernel<true> : norm_forward_kernel<false>, dim3(grid),
                                   dim3(threads_of(a.H)), 0, s, a);
  return e != cudaSuccess ? -(int)e : 1;
}

int64_t norm_backward_workspace_bytes(int64_t N, int H) { return (int64_t)parts_of(N) * 2 * H * 4; }

int launch_norm_backward(const NormArgs& a, cudaStream_t s) {
  const int parts = parts_of(a.N);
  cudaError_t e = launch_pdl(a.rms ? norm_backward_kernel<true> : norm_backward_kernel<false>, dim3(parts),
                             dim3(threads_of(a.H)), 0, s, a);
  if (e != cudaSuccess) return -(int)e;
  e = launch_pdl(norm_parts_kernel, dim3((2 * a.H + 255) / 256), dim3(256), 0, s, (const float*)a.part, parts, a.H,
                 a.dw, a.db);
  return e != cudaSuccess ? -(int)e : 2;
}

}  // namespace moe
