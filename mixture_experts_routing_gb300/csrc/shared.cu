// The shared expert: a gated feed-forward block that every token passes, its
// 8-bit activation checkpoint and its backward.
//
//   forward   g = x Wg, u = x Wu, h = act(g) u, y = h Wd (+ add)
//   kept      [g | u] as MX blocks: E4M3 codes, one E8M0 byte per 32 values
//   backward  from the kept values: a = act(g) u, da = dy Wd^T,
//             dg = da u act'(g), du = da act(g),
//             dx = dg Wg^T + du Wu^T (+ add), dW13 = [dg du]^T x, dW2 = dy^T a
//
// Each contraction is one launch of a tiled kernel with its own epilogue.
#include "act.cuh"
#include "moe_internal.h"
#include "shared_internal.h"

namespace moe {
namespace {

constexpr int kT = 64;   // output tile edge
constexpr int kTK = 16;  // contraction per step

enum Epi { kEpiGated = 0, kEpiOut = 1, kEpiGatedBwd = 2 };

struct SimpleParams {
  const uint16_t* a;      // element (m, k) at a[m * a_m + k * a_k]
  const uint16_t* b;      // element (n, k) at b[n * b_n + k * b_k]
  const uint16_t* b2;     // kEpiGated: the up rows
  int64_t a_m, a_k, b_n, b_k;
  int M, N, K;
  const uint16_t* add;    // kEpiOut: [M,N] or null
  void* out;              // kEpiOut: [M,N] (bf16, or f32 with out_f32); else h [M,N] bf16
  int out_f32;
  uint16_t* dpre;         // kEpiGatedBwd: [M,2N]
  uint8_t* ck;            // [M,2N] codes
  uint8_t* ck_sf;         // [M,2N/32]
  int activation;
};

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Stores four consecutive values of a row as MX codes; the eight threads of a
// 32-value block find its largest magnitude together. A block that holds an
// infinity or a NaN gets the scale byte 255, which reads as NaN.
__device__ __forceinline__ void keep4(const float (&v)[4], bool in, uint8_t* ck, uint8_t* sf,
                                      bool first) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (!in) return;
  const bool finite = top < 0x7F800000u;
  const int s = finite ? mx_block_exponent(__uint_as_float(top)) : 0;
  const float f = pow2_neg(s);
  const uint32_t c = e4m3x2(v[0] * f, v[1] * f) | (e4m3x2(v[2] * f, v[3] * f) << 16);
  *reinterpret_cast<uint32_t*>(ck) = c;
  if (first) *sf = finite ? (uint8_t)(s + 127) : (uint8_t)255;
}

template <int EPI>
__global__ void __launch_bounds__(256) shared_gemm_kernel(const SimpleParams p) {
  __shared__ float as[kTK][kT + 1], bs[kTK][kT + 1], cs[EPI == kEpiGated ? kTK : 1][kT + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int m0 = blockIdx.y * kT, n0 = blockIdx.x * kT;
  float acc[4][4] = {}, acc2[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kTK) {
#pragma unroll
    for (int j = 0; j < kT * kTK / 256; ++j) {
      const int e = threadIdx.x + 256 * j;
      // the contiguous dimension of each operand goes with the thread index
      const int ak = p.a_k == 1 ? e % kTK : e / kT, am = p.a_k == 1 ? e / kTK : e % kT;
      const int bk = p.b_k == 1 ? e % kTK : e / kT, bn = p.b_k == 1 ? e / kTK : e % kT;
      as[ak][am] = (m0 + am < p.M && k0 + ak < p.K)
                       ? bf(p.a[(m0 + am) * p.a_m + (k0 + ak) * p.a_k]) : 0.0f;
      const bool in = n0 + bn < p.N && k0 + bk < p.K;
      bs[bk][bn] = in ? bf(p.b[(n0 + bn) * p.b_n + (k0 + bk) * p.b_k]) : 0.0f;
      if (EPI == kEpiGated) cs[bk][bn] = in ? bf(p.b2[(n0 + bn) * p.b_n + (k0 + bk) * p.b_k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTK; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
          if (EPI == kEpiGated) acc2[i][j] = fmaf(as[k][ty * 4 + i], cs[k][tx * 4 + j], acc2[i][j]);
        }
    }
    __syncthreads();
  }
  const int n = n0 + tx * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    const bool in = m < p.M && n < p.N;  // N is a multiple of 8: all four or none
    const size_t row = (size_t)m * p.N;
    if (EPI == kEpiGated) {
      if (p.ck) {
        const size_t at = 2 * row + n, sa = (size_t)m * (p.N / 16) + n / 32;
        keep4(acc[i], in, p.ck + at, p.ck_sf + sa, (tx & 7) == 0);
        keep4(acc2[i], in, p.ck + at + p.N, p.ck_sf + sa + p.N / 32, (tx & 7) == 0);
      }
      if (in)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = p.activation ? act_fwd<1>(acc[i][j]) : act_fwd<0>(acc[i][j]);
          static_cast<uint16_t*>(p.out)[row + n + j] = to_bf(a * acc2[i][j]);
        }
    } else if (EPI == kEpiGatedBwd) {
      if (in) {
        const size_t sa = (size_t)m * (p.N / 16) + n / 32;
        const float fg = e8m0_value(p.ck_sf[sa]), fu = e8m0_value(p.ck_sf[sa + p.N / 32]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float g = e4m3x2_value(p.ck[2 * row + n + j]).x * fg;
          const float u = e4m3x2_value(p.ck[2 * row + p.N + n + j]).x * fu;
          const float c = p.activation ? act_core<1>(g) : act_core<0>(g);
          const float d = p.activation ? act_grad_core<1>(g, c) : act_grad_core<0>(g, c);
          p.dpre[2 * row + n + j] = to_bf(acc[i][j] * u * d);
          p.dpre[2 * row + p.N + n + j] = to_bf(acc[i][j] * g * c);
          static_cast<uint16_t*>(p.out)[row + n + j] = to_bf(g * c * u);
        }
      }
    } else if (in) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = acc[i][j] + (p.add ? bf(p.add[row + n + j]) : 0.0f);
        if (p.out_f32) static_cast<float*>(p.out)[row + n + j] = v;
        else static_cast<uint16_t*>(p.out)[row + n + j] = to_bf(v);
      }
    }
  }
}

template <int EPI>
cudaError_t launch_simple(const SimpleParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.N + kT - 1) / kT), (unsigned)((p.M + kT - 1) / kT));
  shared_gemm_kernel<EPI><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

int launch_shared_forward(const SharedArgs& a, cudaStream_t s) {
  SimpleParams p{};
  p.a = a.x; p.a_m = a.H; p.a_k = 1;
  p.b = a.w13; p.b2 = a.w13 + (size_t)a.I * a.H; p.b_n = a.H; p.b_k = 1;
  p.M = a.N; p.N = a.I; p.K = a.H;
  p.out = a.h; p.ck = a.ck; p.ck_sf = a.ck_sf; p.activation = a.activation;
  cudaError_t err = launch_simple<kEpiGated>(p, s);
  if (err != cudaSuccess) return -(int)err;
  p = SimpleParams{};
  p.a = a.h; p.a_m = a.I; p.a_k = 1;
  p.b = a.w2; p.b_n = a.I; p.b_k = 1;
  p.M = a.N; p.N = a.H; p.K = a.I;
  p.add = a.add; p.out = a.y;
  err = launch_simple<kEpiOut>(p, s);
  return err != cudaSuccess ? -(int)err : 2;
}

int launch_shared_backward(const SharedArgs& a, cudaStream_t s) {
  SimpleParams p{};  // da = dy Wd^T: w2 [H,I] read along its rows
  p.a = a.dy; p.a_m = a.H; p.a_k = 1;
  p.b = a.w2; p.b_n = 1; p.b_k = a.I;
  p.M = a.N; p.N = a.I; p.K = a.H;
  p.out = a.h; p.dpre = a.dpre; p.ck = a.ck; p.ck_sf = a.ck_sf; p.activation = a.activation;
  cudaError_t err = launch_simple<kEpiGatedBwd>(p, s);
  if (err != cudaSuccess) return -(int)err;
  p = SimpleParams{};  // dx = [dg du] W13
  p.a = a.dpre; p.a_m = 2 * a.I; p.a_k = 1;
  p.b = a.w13; p.b_n = 1; p.b_k = a.H;
  p.M = a.N; p.N = a.H; p.K = 2 * a.I;
  p.add = a.add; p.out = a.dx;
  err = launch_simple<kEpiOut>(p, s);
  if (err != cudaSuccess) return -(int)err;
  p = SimpleParams{};  // dW13 = [dg du]^T x
  p.a = a.dpre; p.a_m = 1; p.a_k = 2 * a.I;
  p.b = a.x; p.b_n = 1; p.b_k = a.H;
  p.M = 2 * a.I; p.N = a.H; p.K = a.N;
  p.out = a.dw13; p.out_f32 = a.grad_f32;
  err = launch_simple<kEpiOut>(p, s);
  if (err != cudaSuccess) return -(int)err;
  p = SimpleParams{};  // dW2 = dy^T h
  p.a = a.dy; p.a_m = 1; p.a_k = a.H;
  p.b = a.h; p.b_n = 1; p.b_k = a.I;
  p.M = a.H; p.N = a.I; p.K = a.N;
  p.out = a.dw2; p.out_f32 = a.grad_f32;
  err = launch_simple<kEpiOut>(p, s);
  return err != cudaSuccess ? -(int)err : 4;
}

}  // namespace moe
