// The whole layer for a few tokens in bf16.
#include "act.cuh"
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"
#include "route_math.cuh"

namespace moe {
namespace {

struct FewWs {
  size_t logits, ids, p, h, total;
};

FewWs layout(int N, int H, int E, int K, int I) {
  FewWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  w.logits = take((size_t)N * E * 4);
  w.ids = take((size_t)N * K * 4);
  w.p = take((size_t)N * K * 4);
  w.h = take((size_t)N * K * I * 2);
  w.total = off;
  return w;
}

__global__ void __launch_bounds__(256) few_logits_kernel(const FewArgs a, float* logits) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[8][32];
  const int t = blockIdx.y, c = threadIdx.x & 31, s = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
  if (t >= live_tokens(a.n_dev, a.N)) return;
  float sum = 0.0f;
  if (e < a.E)
    for (int h = s; h < a.H; h += 8)
      sum = fmaf(__uint_as_float((uint32_t)a.x[(size_t)t * a.H + h] << 16), a.wr[(size_t)h * a.E + e], sum);
  part[s][c] = sum;
  __syncthreads();
  if (s || e >= a.E) return;
  for (int i = 1; i < 8; ++i) sum += part[i][c];
  logits[(size_t)t * a.E + e] = sum + (a.bias ? a.bias[e] : 0.0f);
}

__global__ void __launch_bounds__(32) few_select_kernel(const FewArgs a, const float* logits, int* ids, float* ps) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, lane = threadIdx.x;
  if (t >= live_tokens(a.n_dev, a.N)) return;
  float v[8], top = -INFINITY;
  for (int j = 0; j < 8; ++j) {
    const int e = lane + 32 * j;
    v[j] = e < a.E ? logits[(size_t)t * a.E + e] : -INFINITY;
    top = fmaxf(top, v[j]);
  }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.0f;
  for (int j = 0; j < 8; ++j) {
    if (lane + 32 * j < a.E) sum += v[j] = route_exp(v[j] - top);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  uint32_t taken = 0;
  float d = 0.0f, my_p = 0.0f;
  int my_id = 0;
  for (int j = 0; j < 8; ++j) v[j] = v[j] / sum;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0, mine = 0xFFFFFFFFu;
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < a.E && !((taken >> j) & 1u)) best = max(best, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    for (int j = 7; j >= 0; --j)
      if (lane + 32 * j < a.E && !((taken >> j) & 1u) && (__float_as_uint(v[j]) & 0x7FFFFFFFu) == best) mine = lane + 32 * j;
    const int e = (int)__reduce_min_sync(0xFFFFFFFFu, mine);
    if ((e & 31) == lane) taken |= 1u << (e >> 5);
    const float p = __uint_as_float(best);
    d += p;
    if (lane == k) { my_id = e; my_p = p; }
  }
  if (lane < a.K) {
    const float p = a.renorm ? my_p / d : my_p;
    const size_t at = (size_t)t * a.K + lane;
    ids[at] = my_id;
    ps[at] = p;
    if (a.topk_ids) a.topk_ids[at] = my_id;
    if (a.topk_p) a.topk_p[at] = p;
  }
}

// sum of n products of two bf16 rows over a warp's lanes (n a multiple of 8)
__device__ __forceinline__ float dot_row(const uint16_t* x, const uint16_t* w, int n, int lane) {
  float s = 0.0f;
  for (int k = lane * 8; k < n; k += 256) {
    const uint4 p = *reinterpret_cast<const uint4*>(x + k), q = *reinterpret_cast<const uint4*>(w + k);
    const uint32_t* pp = &p.x;
    const uint32_t* qq = &q.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(pp[i] << 16), __uint_as_float(qq[i] << 16), s);
      s = fmaf(__uint_as_float(pp[i] & 0xFFFF0000u), __uint_as_float(qq[i] & 0xFFFF0000u), s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

template <int ACT>
__global__ void __launch_bounds__(256) few_fc1_kernel(const FewArgs a, const int* ids, uint16_t* h) {
  griddep_wait();
  griddep_launch_dependents();
  const int route = blockIdx.y, t = route / a.K, lane = threadIdx.x & 31, f = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= live_tokens(a.n_dev, a.N) || f >= a.I) return;
  const uint16_t* w = a.w13 + (size_t)ids[route] * 2 * a.I * a.H;
  const float g = dot_row(a.x + (size_t)t * a.H, w + (size_t)f * a.H, a.H, lane);
  const float u = dot_row(a.x + (size_t)t * a.H, w + ((size_t)a.I + f) * a.H, a.H, lane);
  if (lane == 0) reinterpret_cast<__nv_bfloat16*>(h)[(size_t)route * a.I + f] = __float2bfloat16_rn(act_fwd<ACT>(g) * u);
}

__global__ void __launch_bounds__(256) few_fc2_kernel(const FewArgs a, const int* ids, const float* ps, const uint16_t* h) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.y, lane = threadIdx.x & 31, c = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= live_tokens(a.n_dev, a.N) || c >= a.H) return;
  float y = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    const int route = t * a.K + k;
    const float p = ps[route];
    if (p != 0.0f)
      y += p * dot_row(h + (size_t)route * a.I, a.w2 + ((size_t)ids[route] * a.H + c) * a.I, a.I, lane);
  }
  if (lane == 0) {
    if (a.add) y += __uint_as_float((uint32_t)a.add[(size_t)t * a.H + c] << 16);
    reinterpret_cast<__nv_bfloat16*>(a.y)[(size_t)t * a.H + c] = __float2bfloat16_rn(y);
  }
}

}  // namespace

int64_t few_workspace_bytes(int N, int H, int E, int K, int I) { return (int64_t)layout(N, H, E, K, I).total; }

int launch_few(const FewArgs& a, cudaStream_t s) {
  const FewWs w = layout(a.N, a.H, a.E, a.K, a.I);
  float* logits = reinterpret_cast<float*>(a.ws + w.logits);
  int* ids = reinterpret_cast<int*>(a.ws + w.ids);
  float* ps = reinterpret_cast<float*>(a.ws + w.p);
  uint16_t* h = reinterpret_cast<uint16_t*>(a.ws + w.h);
  cudaError_t e = launch_pdl(few_logits_kernel, dim3((a.E + 31) / 32, a.N), dim3(256), 0, s, a, logits);
  if (e == cudaSuccess)
    e = launch_pdl(few_select_kernel, dim3(a.N), dim3(32), 0, s, a, (const float*)logits, ids, ps);
  if (e == cudaSuccess)
    e = launch_pdl(a.activation ? few_fc1_kernel<1> : few_fc1_kernel<0>, dim3((a.I + 7) / 8, a.N * a.K), dim3(256), 0,
                   s, a, (const int*)ids, h);
  if (e == cudaSuccess)
    e = launch_pdl(few_fc2_kernel, dim3((a.H + 7) / 8, a.N), dim3(256), 0, s, a, (const int*)ids, (const float*)ps,
                   (const uint16_t*)h);
  return e != cudaSuccess ? -(int)e : 4;
}

}  // namespace moe
