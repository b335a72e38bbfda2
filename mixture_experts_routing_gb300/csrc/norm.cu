// Layer norm (and its RMS form) of bf16 rows, forward and backward.
//
//   forward   s = bf16(x + add); mean, var over the row; y = (s - mean) r w + b
//   backward  z = (s - mean) r, g = dy w;
//             dx = r (g - z mean(g z) - mean(g)) + dx_add
//             dweight = sum over rows of dy z, dbias = sum of dy
//
// Bound by memory: every row is read and written once. One block an SM walks over its
// share of the rows; a thread keeps the same 8 (or 16) columns of every row, so weight,
// bias and the sums over rows stay in its registers. Rows arrive through a ring of bulk
// copies: about 100 KB are under way while a row is summed, which loads into registers
// could not reach next to those sums.
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr uint32_t kRingBytes = 200u << 10;
constexpr int kMaxStages = 8;
constexpr uint32_t kErrWaitRows = 1u << 5;  // rows never arrived

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

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// How a block takes its rows: `lanes` threads a row (a power of two up to 32, else whole
// warps), `rows` rows at a time.
struct Plan {
  int lanes, rows, threads;
  int64_t steps;     // row groups
  int stages;
  uint32_t stage;    // bytes: `tensors` x rows x H x 2
};

// Sums of v over a row's threads, the same in all of them. slot: a float per warp and value;
// it is written again two calls later at the earliest, behind another barrier.
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], const Plan& p, float (*slot)[NV]) {
  const int width = p.lanes < 32 ? p.lanes : 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (p.lanes <= 32) return;
  const int warp = threadIdx.x >> 5, per = p.lanes >> 5, first = warp / per * per;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) slot[warp][i] = v[i];
  __syncthreads();
  const int l = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = l < per ? slot[first + l][i] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

// The block's ring of row groups: TENSORS arrays, each `rows` rows of it, a bulk copy each.
template <int TENSORS>
struct Rows {
  uint64_t* full;
  uint32_t base;
  int64_t N;
  int H;
  Plan p;
  const uint16_t* from[TENSORS];

  __device__ __forceinline__ uint32_t at(int stage, int tensor) const {
    return base + (uint32_t)stage * p.stage + (uint32_t)tensor * (p.stage / TENSORS);
  }
  __device__ __forceinline__ void load(int64_t step, int stage) const {  // one thread
    const int64_t row = step * p.rows;
    const uint32_t bytes = (uint32_t)(min((int64_t)p.rows, N - row) * H * 2), bar = smem_u32(&full[stage]);
    mbar_arrive_expect_tx(bar, bytes * TENSORS);
#pragma unroll
    for (int i = 0; i < TENSORS; ++i) bulk_load(at(stage, i), from[i] + row * H, bytes, bar);
  }
};

// KV: groups of 8 columns a thread holds.
template <bool RMS, bool ADD, int KV>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_forward_kernel(const NormArgs a, const Plan p) {
  constexpr int kTensors = ADD ? 2 : 1;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ float slots[4][kMaxThreads / 32][1];
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  Rows<kTensors> rows{full, (smem_u32(smem) + 127u) & ~127u, a.N, a.H, p, {}};
  rows.from[0] = a.x;
  if (ADD) rows.from[kTensors - 1] = a.add;
  if (threadIdx.x == 0)
    for (int i = 0; i < p.stages; ++i) {
      const int64_t step = blockIdx.x + (int64_t)i * gridDim.x;
      if (step < p.steps) rows.load(step, i);
    }
  const int H = a.H, mine = threadIdx.x / p.lanes, lane = threadIdx.x - mine * p.lanes;
  const float inv_h = 1.0f / (float)H;
  float w[KV][8], b[KV][8];
#pragma unroll
  for (int j = 0; j < KV; ++j) {
    const int c = (j * p.lanes + lane) * 8;
    if (c < H) {
      load8(a.w + c, w[j]);
      if (a.b) load8(a.b + c, b[j]);
    }
    if (c >= H || !a.b) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[j][i] = 0.0f;
    }
  }
  int stage = 0, turn = 0;
  uint32_t par = 0;
  bool ok = true;  // after a wait that ran out: no more copies and waits, but every barrier
  for (int64_t step = blockIdx.x; step < p.steps; step += gridDim.x) {
    ok = ok && mbar_wait(smem_u32(&full[stage]), par, a.err, kErrWaitRows);
    const int64_t row = step * p.rows + mine;
    const bool live = row < a.N;  // the last group may have fewer rows
    float v[KV][8], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      const int c = (j * p.lanes + lane) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (c < H && live) {
        unpack8(lds16(rows.at(stage, 0) + (uint32_t)(mine * H + c) * 2), v[j]);
        if (ADD) {
          float r[8];
          unpack8(lds16(rows.at(stage, 1) + (uint32_t)(mine * H + c) * 2), r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] += r[i];
          const uint4 q = pack8(v[j]);
          *reinterpret_cast<uint4*>(a.sum + row * H + c) = q;
          unpack8(q, v[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += v[j][i];
      }
    }
    float mean = 0.0f;
    if (!RMS) {
      row_sum(sum, p, slots[turn]);
      mean = sum[0] * inv_h;
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if ((j * p.lanes + lane) * 8 < H) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][i] -= mean;
          sq[0] += v[j][i] * v[j][i];
        }
      }
    }
    row_sum(sq, p, slots[turn + 1]);
    turn ^= 2;
    // every thread has the stage's rows in registers behind this barrier (row_sum has one of
    // its own where a row takes several warps)
    if (p.lanes <= 32) __syncthreads();
    if (threadIdx.x == 0) {
      const int64_t next = step + (int64_t)p.stages * gridDim.x;
      if (ok && next < p.steps) rows.load(next, stage);
    }
    if (++stage == p.stages) { stage = 0; par ^= 1u; }
    if (!live) continue;
    const float r = 1.0f / sqrtf(sq[0] * inv_h + a.eps);
    if (lane == 0) {
      if (!RMS && a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      const int c = (j * p.lanes + lane) * 8;
      if (c >= H) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(v[j][i] * r, w[j][i], b[j][i]);
      *reinterpret_cast<uint4*>(a.y + row * H + c) = pack8(o);
    }
  }
}

template <bool RMS, bool ADD, int KV>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_kernel(const NormArgs a, const Plan p) {
  constexpr int kTensors = ADD ? 3 : 2;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ float slots[2][kMaxThreads / 32][2];
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // the weight (not of the widest rows, which need the room), then the ring: with w in
  // registers too the sums would spill, and the ring leaves the first-level cache no room
  const uint32_t base = ((smem_u32(smem) + 127u) & ~127u) + (KV == 1 ? ((uint32_t)a.H * 4 + 127u) & ~127u : 0u);
  float* ws = reinterpret_cast<float*>(smem + (base - smem_u32(smem))) - a.H;
  Rows<kTensors> rows{full, base, a.N, a.H, p, {}};
  rows.from[0] = a.x;
  rows.from[1] = a.dy;
  if (ADD) rows.from[kTensors - 1] = a.add;
  if (threadIdx.x == 0)
    for (int i = 0; i < p.stages; ++i) {
      const int64_t step = blockIdx.x + (int64_t)i * gridDim.x;
      if (step < p.steps) rows.load(step, i);
    }
  const int H = a.H, mine = threadIdx.x / p.lanes, lane = threadIdx.x - mine * p.lanes;
  const float inv_h = 1.0f / (float)H;
  if (KV == 1)
    for (int c = threadIdx.x * 4; c < H; c += p.threads * 4)
      *reinterpret_cast<float4*>(ws + c) = *reinterpret_cast<const float4*>(a.w + c);
  __syncthreads();
  float dw[KV][8] = {}, db[KV][8] = {};
  int stage = 0, turn = 0;
  uint32_t par = 0;
  bool ok = true;  // after a wait that ran out: no more copies and waits, but every barrier
  for (int64_t step = blockIdx.x; step < p.steps; step += gridDim.x, turn ^= 1) {
    const int64_t row = step * p.rows + mine;
    const bool live = row < a.N;
    float mean = 0.0f, r = 0.0f;
    if (live) {
      if (!RMS) mean = a.mean[row];
      r = a.rstd[row];
    }
    ok = ok && mbar_wait(smem_u32(&full[stage]), par, a.err, kErrWaitRows);
    float z[KV][8], g[KV][8], s[2] = {0.0f, 0.0f};
    uint4 add[KV];
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      const int c = (j * p.lanes + lane) * 8;
      if (c < H && live) {
        const uint32_t off = (uint32_t)(mine * H + c) * 2;
        float w[8];
        unpack8(lds16(rows.at(stage, 0) + off), z[j]);
        unpack8(lds16(rows.at(stage, 1) + off), g[j]);
        if (ADD) add[j] = lds16(rows.at(stage, kTensors - 1) + off);
        load8(KV == 1 ? ws + c : a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[j][i] = (z[j][i] - mean) * r;
          dw[j][i] = fmaf(g[j][i], z[j][i], dw[j][i]);
          db[j][i] += g[j][i];
          g[j][i] *= w[i];
          s[0] = fmaf(g[j][i], z[j][i], s[0]);
          if (!RMS) s[1] += g[j][i];
        }
      }
    }
    row_sum(s, p, slots[turn]);
    if (p.lanes <= 32) __syncthreads();
    if (threadIdx.x == 0) {
      const int64_t next = step + (int64_t)p.stages * gridDim.x;
      if (ok && next < p.steps) rows.load(next, stage);
    }
    if (++stage == p.stages) { stage = 0; par ^= 1u; }
    if (!live) continue;
    const float mz = s[0] * inv_h, mg = RMS ? 0.0f : s[1] * inv_h;
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      const int c = (j * p.lanes + lane) * 8;
      if (c >= H) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = r * (g[j][i] - z[j][i] * mz - mg);
      if (ADD) {
        float t[8];
        unpack8(add[j], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += t[i];
      }
      *reinterpret_cast<uint4*>(a.dx + row * H + c) = pack8(o);
    }
  }
  // the block's sums: its rows' groups are added in order through shared memory
  float* part = a.part + (int64_t)blockIdx.x * 2 * H;
  float* sums = reinterpret_cast<float*>(smem + (base - smem_u32(smem)));  // [2][H]: every copy has landed and was read
  __syncthreads();
  for (int turn2 = 0; turn2 < p.rows; ++turn2) {
    if (mine == turn2) {
#pragma unroll
      for (int j = 0; j < KV; ++j) {
        const int c = (j * p.lanes + lane) * 8;
        if (c >= H) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = turn2 ? sums[c + i] + dw[j][i] : dw[j][i], y = turn2 ? sums[H + c + i] + db[j][i] : db[j][i];
          if (turn2 == p.rows - 1) {
            part[c + i] = x;
            part[H + c + i] = y;
          } else {
            sums[c + i] = x;
            sums[H + c + i] = y;
          }
        }
      }
    }
    __syncthreads();
  }
}

// dw and db from the blocks' partial sums: 32 columns a block, eight runs of the parts, added
// in order.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* part, int parts, int H, float* dw, float* db) {
  __shared__ float sums[8][32];
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < 2 * H) {
    const int p0 = q * parts / 8, p1 = (q + 1) * parts / 8;
#pragma unroll 8
    for (int p = p0; p < p1; ++p) t += part[(int64_t)p * 2 * H + c];
  }
  sums[q][threadIdx.x & 31] = t;
  __syncthreads();
  if (q || c >= 2 * H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += sums[i][threadIdx.x];
  if (c < H) dw[c] = t;
  else if (db) db[c - H] = t;
}

constexpr int kWide = 8192;  // columns from which a thread takes 16 of a row instead of 8

uint32_t weight_bytes(int H) { return H > kWide ? 0u : ((uint32_t)H * 4 + 127u) & ~127u; }

Plan plan_of(int64_t N, int H, int tensors, uint32_t ring) {
  Plan p{};
  const int groups = (H / 8 + (H > kWide)) / (H > kWide ? 2 : 1);
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < groups) p.lanes *= 2;
  if (groups > 32) p.lanes = (groups + 31) / 32 * 32;
  p.rows = kMaxThreads / p.lanes;
  p.threads = (p.rows * p.lanes + 31) / 32 * 32;
  const uint32_t row = (uint32_t)H * 2 * tensors;
  while (p.rows > 1 && (uint64_t)p.rows * row > ring / 3) p.rows /= 2;
  p.threads = p.rows * p.lanes;
  p.steps = (N + p.rows - 1) / p.rows;
  p.stage = (uint32_t)p.rows * row;
  p.stages = (int)(ring / p.stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  return p;
}

template <typename K>
cudaError_t ring_smem(K* kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 128);
}

template <bool RMS, bool ADD>
cudaError_t opt_in() {
  cudaError_t e = ring_smem(norm_forward_kernel<RMS, ADD, 1>);
  if (e == cudaSuccess) e = ring_smem(norm_forward_kernel<RMS, ADD, 2>);
  if (e == cudaSuccess) e = ring_smem(norm_backward_kernel<RMS, ADD, 1>);
  if (e == cudaSuccess) e = ring_smem(norm_backward_kernel<RMS, ADD, 2>);
  return e;
}

int sm_count(cudaError_t* err) {
  static DeviceOnce once;
  int sms = 0;
  *err = once_per_device(once, &sms, [](int dev, int* v) {
    cudaError_t e = opt_in<false, false>();
    if (e == cudaSuccess) e = opt_in<false, true>();
    if (e == cudaSuccess) e = opt_in<true, false>();
    if (e == cudaSuccess) e = opt_in<true, true>();
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
  return sms;
}

unsigned grid_of(const Plan& p, int sms) { return (unsigned)(p.steps < sms ? p.steps : sms); }

template <int KV>
cudaError_t forward(const NormArgs& a, const Plan& p, unsigned grid, cudaStream_t s) {
  auto k = a.rms ? (a.add ? norm_forward_kernel<true, true, KV> : norm_forward_kernel<true, false, KV>)
                 : (a.add ? norm_forward_kernel<false, true, KV> : norm_forward_kernel<false, false, KV>);
  return launch_pdl(k, dim3(grid), dim3(p.threads), p.stages * p.stage + 128, s, a, p);
}

template <int KV>
cudaError_t backward(const NormArgs& a, const Plan& p, unsigned grid, cudaStream_t s) {
  auto k = a.rms ? (a.add ? norm_backward_kernel<true, true, KV> : norm_backward_kernel<true, false, KV>)
                 : (a.add ? norm_backward_kernel<false, true, KV> : norm_backward_kernel<false, false, KV>);
  const uint32_t ring = p.stages * p.stage, sums = 8u * (uint32_t)a.H;  // the block's sums take the ring's place
  return launch_pdl(k, dim3(grid), dim3(p.threads), weight_bytes(a.H) + (ring > sums ? ring : sums) + 128, s, a, p);
}

}  // namespace

int launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int sms = sm_count(&e);
  if (e != cudaSuccess) return -(int)e;
  const Plan p = plan_of(a.N, a.H, a.add ? 2 : 1, kRingBytes);
  e = a.H > kWide ? forward<2>(a, p, grid_of(p, sms), s) : forward<1>(a, p, grid_of(p, sms), s);
  return e != cudaSuccess ? -(int)e : 1;
}

int64_t norm_backward_workspace_bytes(int64_t N, int H) {
  return (N < kNormMaxParts ? N : kNormMaxParts) * 2 * H * 4;
}

int launch_norm_backward(const NormArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  int sms = sm_count(&e);
  if (e != cudaSuccess) return -(int)e;
  if (sms > kNormMaxParts) sms = kNormMaxParts;
  const Plan p = plan_of(a.N, a.H, a.add ? 3 : 2, kRingBytes - weight_bytes(a.H));
  const unsigned grid = grid_of(p, sms);
  e = a.H > kWide ? backward<2>(a, p, grid, s) : backward<1>(a, p, grid, s);
  if (e != cudaSuccess) return -(int)e;
  e = launch_pdl(norm_parts_kernel, dim3((2 * a.H + 31) / 32), dim3(256), 0, s, (const float*)a.part, (int)grid, a.H,
                 a.dw, a.db);
  return e != cudaSuccess ? -(int)e : 2;
}

}  // namespace moe
