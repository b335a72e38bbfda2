// Launch interface of the shared expert (shared.cu) and of the 4-bit products
// (w4.cu) for moe_abi.cu. Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct SharedArgs {
  int N, H, I, activation;
  const uint16_t* x;     // [N,H]
  const uint16_t* w13;   // [2I,H]: gate rows, then up rows
  const uint16_t* w2;    // [H,I]
  const uint16_t* add;   // forward: [N,H] added to y, or null; backward: added to dx, or null
  uint16_t* h;           // [N,I] act(g) u (backward: of the checkpointed g, u)
  uint16_t* y;           // [N,H]
  uint8_t* ck;           // [N,2I] E4M3 codes of [g | u], or null (forward without a checkpoint)
  uint8_t* ck_sf;        // [N,2I/32] E8M0 bytes
  const uint16_t* dy;    // [N,H]
  uint16_t* dpre;        // [N,2I] [dg | du]
  uint16_t* dx;          // [N,H]
  void* dw13;            // [2I,H]
  void* dw2;             // [H,I]
  int grad_f32;          // dw13, dw2 are f32 (else bf16)
  uint32_t* err;         // device error word (bounded waits)
};

// Each returns the number of kernels launched (>= 0) or a negative cudaError_t.
int launch_shared_forward(const SharedArgs& a, cudaStream_t s);
int launch_shared_forward_few(const SharedArgs& a, cudaStream_t s);  // shared_few.cu
int launch_shared_backward(const SharedArgs& a, cudaStream_t s);

constexpr int kW4MaxRoutes = 1024;  // routes of a decode batch, rows of a product

struct W4Args {
  int N, H, E, K, I, group, activation;
  const int32_t* topk_ids;  // [N,K], -1: no route
  const float* topk_p;      // [N,K]
  const uint16_t* x;        // [N,H]
  const uint8_t* w13;       // [E,2I,H/2]
  const uint16_t* w13_scale;  // [E,2I,H/group] bf16
  const uint8_t* w2;        // [E,H,I/2]
  const uint16_t* w2_scale;  // [E,H,I/group] bf16
  const uint16_t* add;      // [N,H] or null
  uint8_t* ws;              // w4_workspace_bytes
  uint16_t* h;              // [N*K,I] in the workspace (set by launch_w4_ffn)
  uint16_t* y;              // [N,H]
};

int64_t w4_workspace_bytes(int N, int K, int H, int I);

int launch_w4_ffn(const W4Args& a, cudaStream_t s);
int launch_w4_matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                     int cols, int group, uint16_t* y, cudaStream_t s);
int launch_w4_quantize(const uint16_t* m, int64_t rows, int cols, int group, uint8_t* q,
                       uint16_t* scale, cudaStream_t s);

}  // namespace moe
