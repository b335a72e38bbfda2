// Launch interface of the layer for a few tokens (few.cu), of layer norm (norm.cu)
// and of AdamW (adamw.cu) for moe_abi.cu. Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFewMaxTokens = 64;

struct FewArgs {
  int N, H, E, K, I, renorm, activation;
  const uint16_t* x;       // [N,H]
  const float* wr;         // [H,E]
  const float* bias;       // [E] or null
  const uint16_t* w13;     // [E,2I,H]
  const uint16_t* w2;      // [E,H,I]
  const uint16_t* add;     // [N,H] or null
  const int32_t* n_dev;    // live tokens, or null
  uint16_t* y;             // [N,H]
  int32_t* topk_ids;       // [N,K] or null
  float* topk_p;           // [N,K] or null
  uint8_t* ws;             // few_workspace_bytes
  uint32_t* err;           // device error word (bounded waits)
};

int64_t few_workspace_bytes(int N, int H, int E, int K, int I);
// Each returns the number of kernels launched (>= 0) or a negative cudaError_t.
int launch_few(const FewArgs& a, cudaStream_t s);

struct NormArgs {
  int64_t N;
  int H, rms;
  float eps;
  const uint16_t* x;
  const uint16_t* add;     // forward: added to x; backward: added to dx; or null
  const float* w;
  const float* b;          // or null
  uint16_t* sum;           // forward, or null
  uint16_t* y;             // forward
  float* mean;             // forward output (or null), backward input; null for rms
  float* rstd;
  const uint16_t* dy;
  uint16_t* dx;
  float* dw;
  float* db;               // or null
  float* part;             // backward workspace
  uint32_t* err;           // device error word (bounded waits)
};

constexpr int kNormMaxParts = 256;  // blocks of the backward: partial sums of dw and db

int launch_norm_forward(const NormArgs& a, cudaStream_t s);
int64_t norm_backward_workspace_bytes(int64_t N, int H);
int launch_norm_backward(const NormArgs& a, cudaStream_t s);

constexpr int kAdamwTensors = 240;  // of one launch: their table is a kernel argument
constexpr int kAdamwBlock = 256;    // values that share the scale of an 8-bit state

struct AdamwTensor {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  int64_t first;
  float decay;
  int grad_bf16;
};

struct AdamwArgs {
  double beta1, beta2;
  float lr, eps;
  int bits;
  uint32_t seed;
  const float* lr_dev;
  const float* grad_scale;
  int32_t* steps;
};

int launch_adamw(const AdamwArgs& a, const AdamwTensor* t, int n, int last, cudaStream_t s);

}  // namespace moe
