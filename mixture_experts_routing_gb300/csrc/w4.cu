// Products with 4-bit weights and group scales, for the few tokens of a decode
// step: w[r,c] = scale[r, c/group] * (nibble[r,c] - 8).
//
//   matvec    y[t,:] = w x[t,:]
//   experts   h[t,k,:] = act(W13g[e] x_t) * (W13u[e] x_t), e = topk_ids[t,k]
//             y[t,:] = add[t,:] + sum_k p[t,k] W2[e] h[t,k,:]
//
// One warp per output value; each lane takes eight columns (one 32-bit word of
// codes) a step and multiplies their sum by the group's scale.
#include "act.cuh"
#include "moe_internal.h"
#include "shared_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// One row times one vector, the whole warp's sum in every lane.
__device__ __forceinline__ float dot_row(const uint8_t* q, const uint16_t* scale,
                                         const uint16_t* x, int cols, int group, int lane) {
  float sum = 0.0f;
  for (int c = lane * 8; c < cols; c += 256) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q + c / 2);
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      part = fmaf((float)((int)((w >> (4 * j)) & 15u) - 8), bf(x[c + j]), part);
    sum = fmaf(part, bf(scale[c / group]), sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum;
}

__global__ void __launch_bounds__(kWarps * 32) w4_matvec_kernel(const uint16_t* x, const uint8_t* q,
                                                                const uint16_t* scale, int rows,
                                                                int cols, int group, uint16_t* y) {
  const int lane = threadIdx.x & 31, r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  const float v = dot_row(q + (size_t)r * (cols / 2), scale + (size_t)r * (cols / group),
                          x + (size_t)blockIdx.y * cols, cols, group, lane);
  if (lane == 0) y[(size_t)blockIdx.y * rows + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__global__ void __launch_bounds__(kWarps * 32) w4_fc1_kernel(const W4Args a) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int r = blockIdx.y, t = r / a.K, e = a.topk_ids[r];
  if (i >= a.I || e < 0 || e >= a.E) return;
  const size_t row = (size_t)e * 2 * a.I + i, up = row + a.I;
  const uint16_t* x = a.x + (size_t)t * a.H;
  const int ng = a.H / a.group;
  const float g = dot_row(a.w13 + row * (a.H / 2), a.w13_scale + row * ng, x, a.H, a.group, lane);
  const float u = dot_row(a.w13 + up * (a.H / 2), a.w13_scale + up * ng, x, a.H, a.group, lane);
  const float h = (a.activation ? act_fwd<1>(g) : act_fwd<0>(g)) * u;
  if (lane == 0) a.h[(size_t)r * a.I + i] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
}

__global__ void __launch_bounds__(kWarps * 32) w4_fc2_kernel(const W4Args a) {
  const int lane = threadIdx.x & 31, c = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = blockIdx.y;
  if (c >= a.H) return;
  float y = a.add ? bf(a.add[(size_t)t * a.H + c]) : 0.0f;
  for (int k = 0; k < a.K; ++k) {
    const int r = t * a.K + k, e = a.topk_ids[r];
    if (e < 0 || e >= a.E) continue;
    const size_t row = (size_t)e * a.H + c;
    y = fmaf(a.topk_p[r], dot_row(a.w2 + row * (a.I / 2), a.w2_scale + row * (a.I / a.group),
                                  a.h + (size_t)r * a.I, a.I, a.group, lane), y);
  }
  if (lane == 0) a.y[(size_t)t * a.H + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

// One warp per group of a row: scale = bf16(max|w| / 7) (1 for a group of
// zeros), code = round(w / scale) to even, within -8..7, stored plus 8.
__global__ void __launch_bounds__(kWarps * 32) w4_quantize_kernel(const uint16_t* m, int64_t groups,
                                                                  int group, uint8_t* q,
                                                                  uint16_t* scale) {
  const int lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (g >= groups) return;
  // group / 32 values a lane, at most four: two to a byte, so lanes hold pairs
  float v[4];
  float top = 0.0f;
  const int pairs = group / 2;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = lane + 32 * j;
    const uint32_t w = at < pairs ? *reinterpret_cast<const uint32_t*>(m + g * group + 2 * at) : 0u;
    v[2 * j] = __uint_as_float(w << 16);
    v[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
    top = fmaxf(top, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(top, 7.0f));
  const float s = __bfloat162float(sb) > 0.0f ? __bfloat162float(sb) : 1.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = lane + 32 * j;
    if (at >= pairs) break;
    const int lo = max(-8, min(7, __float2int_rn(__fdiv_rn(v[2 * j], s))));
    const int hi = max(-8, min(7, __float2int_rn(__fdiv_rn(v[2 * j + 1], s))));
    q[g * pairs + at] = (uint8_t)((lo + 8) | ((hi + 8) << 4));
  }
  if (lane == 0) scale[g] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

}  // namespace

int launch_w4_matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                     int cols, int group, uint16_t* y, cudaStream_t s) {
  w4_matvec_kernel<<<dim3((rows + kWarps - 1) / kWarps, N), kWarps * 32, 0, s>>>(x, q, scale, rows,
                                                                                cols, group, y);
  const cudaError_t err = cudaGetLastError();
  return err != cudaSuccess ? -(int)err : 1;
}

int launch_w4_ffn(const W4Args& a, cudaStream_t s) {
  w4_fc1_kernel<<<dim3((a.I + kWarps - 1) / kWarps, a.N * a.K), kWarps * 32, 0, s>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return -(int)err;
  w4_fc2_kernel<<<dim3((a.H + kWarps - 1) / kWarps, a.N), kWarps * 32, 0, s>>>(a);
  err = cudaGetLastError();
  return err != cudaSuccess ? -(int)err : 2;
}

int launch_w4_quantize(const uint16_t* m, int64_t rows, int cols, int group, uint8_t* q,
                       uint16_t* scale, cudaStream_t s) {
  const int64_t groups = rows * (cols / group);
  const int64_t blocks = (groups + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return -(int)cudaErrorInvalidValue;
  w4_quantize_kernel<<<(unsigned)blocks, kWarps * 32, 0, s>>>(m, groups, group, q, scale);
  const cudaError_t err = cudaGetLastError();
  return err != cudaSuccess ? -(int)err : 1;
}

}  // namespace moe
