// Layer norm (and its RMS form) of bf16 rows, forward and backward.
//
//   forward   s = bf16(x + add); mean, var over the row; y = (s - mean) r w + b
//   backward  z = (s - mean) r, g = dy w;
//             dx = r (g - z mean(g z) - mean(g)) + dx_add
//             dweight = sum over rows of dy z, dbias = sum of dy
//
// Bound by memory: every row is read and written once. One block an SM (forward: two up to
// 8192 columns) walks over its share of the rows; a thread keeps the same 8 (or 16) columns of every row, so weight,
// bias and the sums over rows stay in its registers. Rows arrive through a ring of bulk
// copies: some 100 KB are under way while a row is summed, which loads into registers
// could not reach next to those sums. Measured at 4096 rows of 7168 with the residual: the
// forward 42 us, 5.6 TB/s, the backward 46.5 us, 5.1 TB/s, both of 6.8 that a copy reaches;
// the backward's loads, stores and barriers alone, without its sums, take 43.6. RMS with the
// residual 42 and 45. 2048 rows of 16384: forward 48.5, backward 108, whose threads spill.
// Narrow rows: a backward block adds its row groups one after another at the end, so 16384 rows
// take 16, 18, 24 us at 256, 128, 64 columns, one row of 64 takes 22 and one of 8 146.
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr uint32_t kRingBytes = 200u << 10;
// Three groups of rows under way, 130 KB of the backward's 7168 columns, measured best (4096
// rows of them: 48.7 us with two, 46.5 with three, 47.7 with as many as fit).
constexpr int kMaxStages = 3;
constexpr uint32_t kNone = 0xFFFFFFFFu;  // no step

// Two fp32 values in one register pair, worked on by one instruction: the kernels are short of
// issue slots before they are short of memory (the backward of 7168 columns took 350
// instructions a thread and row, and 57 us, without them).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ F2 unpack2(uint32_t q) { return f2(__uint_as_float(q << 16), __uint_as_float(q & 0xFFFF0000u)); }
__device__ __forceinline__ void unpack8(const uint4& q, F2 (&v)[4]) {
  v[0] = unpack2(q.x);
  v[1] = unpack2(q.y);
  v[2] = unpack2(q.z);
  v[3] = unpack2(q.w);
}
__device__ __forceinline__ uint32_t pack2(F2 a) {
  const float2 f = split(a);
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
}
__device__ __forceinline__ void load8(const float* p, F2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = f2(a.x, a.y);
  v[1] = f2(a.z, a.w);
  v[2] = f2(b.x, b.y);
  v[3] = f2(b.z, b.w);
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
  uint32_t steps;    // row groups
  int stages;
  uint32_t stage;    // bytes: `tensors` x rows x H x 2
};

// Sums over a row's threads, the same in all of them. WIDE: a row takes several warps, which
// meet in slot (a value a warp; written again two calls later at the earliest, behind another
// barrier); else it takes `lanes` lanes of one warp.
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, int lanes, int first_warp, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (WIDE || o < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (!WIDE) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (lanes >> 5) ? slot[first_warp + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// The sums of a and of b. (Half a warp for each of them would halve the shuffles, but the
// selections that it takes cost as much: 4096 rows of 7168, backward, 47.6 us so, 48.6 that way.)
template <bool WIDE>
__device__ __forceinline__ float2 row_sums(float a, float b, int lanes, int first_warp, float2* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (WIDE || o < lanes) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
  if (!WIDE) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 v = make_float2(0.0f, 0.0f);
  if (lane < (lanes >> 5)) v = slot[first_warp + lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  return v;
}

// The block's ring of row groups: TENSORS arrays, each `rows` rows of it, a bulk copy each.
template <int TENSORS>
struct Rows {
  uint64_t* full;
  uint32_t base, N;
  int H;
  Plan p;
  const uint16_t* from[TENSORS];

  // By the first threads of the first warps, a copy each (a block has eight warps at least);
  // the copies may land before the bytes are announced.
  __device__ __forceinline__ bool loads() const { return threadIdx.x < 32 * TENSORS && (threadIdx.x & 31) == 0; }
  __device__ __forceinline__ void load(uint32_t step, int stage) const {
    const int warp = threadIdx.x >> 5;
    const uint32_t row = step * p.rows, part = p.stage / TENSORS;
    const uint32_t bytes = min((uint32_t)p.rows, N - row) * H * 2, bar = smem_u32(&full[stage]);
    if (warp == 0) mbar_arrive_expect_tx(bar, bytes * TENSORS);
#pragma unroll
    for (int i = 0; i < TENSORS; ++i)
      if (i == warp) bulk_load(base + stage * p.stage + i * part, from[i] + (size_t)row * H, bytes, bar);
  }

  // After a wait that ran out at step `failed`: this thread's copies for it and for the steps
  // behind it are waited for, with the same limit each, so that none is under way when the
  // block leaves.
  __device__ __forceinline__ void drain(uint32_t failed, uint32_t* err) const {
    const uint32_t turn = (failed - blockIdx.x) / gridDim.x;
    for (uint32_t i = 0; i < (uint32_t)p.stages && failed + i * gridDim.x < p.steps; ++i)
      mbar_wait(smem_u32(&full[(turn + i) % p.stages]), (turn + i) / p.stages & 1u, err, kErrWaitRows);
  }
};

// KV: groups of 8 columns a thread holds. T: threads of a block at most, 1024 / T blocks an SM.
template <bool RMS, bool ADD, int KV, bool WIDE, int T>
__global__ void __launch_bounds__(T, kMaxThreads / T) norm_forward_kernel(const NormArgs a, const Plan p) {
  constexpr int kTensors = ADD ? 2 : 1;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ float slots[2][2][T / 32];
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  Rows<kTensors> rows{full, (smem_u32(smem) + 127u) & ~127u, (uint32_t)a.N, a.H, p, {}};
  rows.from[0] = a.x;
  if (ADD) rows.from[kTensors - 1] = a.add;
  const bool loads = rows.loads();
  if (loads)
    for (int i = 0; i < p.stages; ++i)
      if (blockIdx.x + i * gridDim.x < p.steps) rows.load(blockIdx.x + i * gridDim.x, i);
  const int H = a.H, mine = threadIdx.x / p.lanes, lane = threadIdx.x - mine * p.lanes;
  const int first_warp = WIDE ? mine * (p.lanes >> 5) : 0, column2 = p.lanes * 8;
  const float inv_h = 1.0f / (float)H;
  bool in[KV];
  F2 w[KV][4], b[KV][4];
#pragma unroll
  for (int j = 0; j < KV; ++j) {
    const int c = lane * 8 + j * column2;
    in[j] = c < H;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = b[j][i] = f2(0.0f);
    if (in[j]) {
      load8(a.w + c, w[j]);
      if (a.b) load8(a.b + c, b[j]);
    }
  }
  const uint32_t N = (uint32_t)a.N, rows_on = gridDim.x * p.rows, tensor = p.stage / kTensors;
  const uint32_t mine_at = rows.base + (uint32_t)(mine * H + lane * 8) * 2;
  uint32_t row = blockIdx.x * p.rows + mine, from = mine_at, par = 0;
  int stage = 0, turn = 0;
  uint32_t failed = kNone;  // the step of a wait that ran out: no more copies and waits after it, but every barrier
  for (uint32_t step = blockIdx.x; step < p.steps; step += gridDim.x, row += rows_on, turn ^= 1) {
    if (failed == kNone && !mbar_wait(smem_u32(&full[stage]), par, a.err, kErrWaitRows)) failed = step;
    const bool live = row < N;  // the last group may have fewer rows
    const size_t at = (size_t)row * H + lane * 8;
    F2 v[KV][4], sum = f2(0.0f);
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      uint4 q = make_uint4(0, 0, 0, 0);
      const bool here = in[j] && live;
      if (here) q = lds16(from + j * column2 * 2);
      unpack8(q, v[j]);
      if (ADD && here) {
        F2 r[4];
        unpack8(lds16(from + tensor + j * column2 * 2), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], r[i]);
        q = pack8(v[j]);
        *reinterpret_cast<uint4*>(a.sum + at + j * column2) = q;
        unpack8(q, v[j]);
      }
      if (!RMS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = add2(sum, v[j][i]);
      }
    }
    float mean = 0.0f;
    if (!RMS) {
      const float2 s = split(sum);
      mean = row_sum<WIDE>(s.x + s.y, p.lanes, first_warp, slots[turn][0]) * inv_h;
    }
    F2 sq = f2(0.0f);
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if (RMS || in[j]) {  // columns past the row are zeros, not minus the mean
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!RMS) v[j][i] = add2(v[j][i], f2(-mean));
          sq = fma2(v[j][i], v[j][i], sq);
        }
      }
    }
    const float2 s = split(sq);
    float mine_sq = s.x + s.y;
    // A row that holds an infinity is NaN throughout. The mean makes it so; without one 1 / inf
    // would bring the others to 0. (Finite values whose squares are infinite stay finite.)
    if (RMS && isinf(mine_sq)) {
#pragma unroll
      for (int j = 0; j < KV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = split(v[j][i]);
          if (isinf(u.x) || isinf(u.y)) mine_sq = __uint_as_float(0x7FC00000u);
        }
    }
    const float var = row_sum<WIDE>(mine_sq, p.lanes, first_warp, slots[turn][1]) * inv_h;
    // every thread has the stage's rows in registers behind this barrier (row_sum has one of
    // its own where a row takes several warps)
    if (!WIDE) __syncthreads();
    if (loads && failed == kNone && step + p.stages * gridDim.x < p.steps) rows.load(step + p.stages * gridDim.x, stage);
    from += p.stage;
    if (++stage == p.stages) { stage = 0; from = mine_at; par ^= 1u; }
    if (!live) continue;
    const float r = 1.0f / sqrtf(var + a.eps);
    if (lane == 0) {
      if (!RMS && a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if (!in[j]) continue;
      F2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fma2(mul2(v[j][i], f2(r)), w[j][i], b[j][i]);
      *reinterpret_cast<uint4*>(a.y + at + j * column2) = pack8(o);
    }
  }
  if (loads && failed != kNone) rows.drain(failed, a.err);
}

template <bool RMS, bool ADD, int KV, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_kernel(const NormArgs a, const Plan p) {
  constexpr int kTensors = ADD ? 3 : 2;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ float2 slots[2][kMaxThreads / 32];
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
  Rows<kTensors> rows{full, base, (uint32_t)a.N, a.H, p, {}};
  rows.from[0] = a.x;
  rows.from[1] = a.dy;
  if (ADD) rows.from[kTensors - 1] = a.add;
  const bool loads = rows.loads();
  if (loads)
    for (int i = 0; i < p.stages; ++i)
      if (blockIdx.x + i * gridDim.x < p.steps) rows.load(blockIdx.x + i * gridDim.x, i);
  const int H = a.H, mine = threadIdx.x / p.lanes, lane = threadIdx.x - mine * p.lanes;
  const int first_warp = WIDE ? mine * (p.lanes >> 5) : 0, column2 = p.lanes * 8;
  const float inv_h = 1.0f / (float)H;
  if (KV == 1)
    for (int c = threadIdx.x * 4; c < H; c += p.threads * 4)
      *reinterpret_cast<float4*>(ws + c) = *reinterpret_cast<const float4*>(a.w + c);
  __syncthreads();
  F2 dw[KV][4], db[KV][4];
#pragma unroll
  for (int j = 0; j < KV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = f2(0.0f);
  const uint32_t N = (uint32_t)a.N, rows_on = gridDim.x * p.rows, tensor = p.stage / kTensors;
  const uint32_t mine_at = base + (uint32_t)(mine * H + lane * 8) * 2;
  uint32_t row = blockIdx.x * p.rows + mine, from = mine_at, par = 0;
  int stage = 0, turn = 0;
  uint32_t failed = kNone;  // the step of a wait that ran out: no more copies and waits after it, but every barrier
  float next_mean = 0.0f, next_r = 0.0f;  // a step ahead: their way from memory is longer than a step
  auto stats = [&](uint32_t row) {
    if (row < N) {
      if (!RMS) next_mean = a.mean[row];
      next_r = a.rstd[row];
    }
  };
  stats(row);
  for (uint32_t step = blockIdx.x; step < p.steps; step += gridDim.x, row += rows_on, turn ^= 1) {
    const bool live = row < N;
    const float mean = next_mean, r = next_r;
    stats(row + rows_on);
    if (failed == kNone && !mbar_wait(smem_u32(&full[stage]), par, a.err, kErrWaitRows)) failed = step;
    F2 z[KV][4], g[KV][4], sg = f2(0.0f), sgz = f2(0.0f);
    uint4 res[KV];
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      const int c = lane * 8 + j * column2;
      if (c < H && live) {
        const uint32_t off = from + j * column2 * 2;
        F2 w[4];
        unpack8(lds16(off), z[j]);
        unpack8(lds16(off + tensor), g[j]);
        if (ADD) res[j] = lds16(off + 2 * tensor);
        load8(KV == 1 ? ws + c : a.w + c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!RMS) z[j][i] = add2(z[j][i], f2(-mean));
          z[j][i] = mul2(z[j][i], f2(r));
          dw[j][i] = fma2(g[j][i], z[j][i], dw[j][i]);
          db[j][i] = add2(db[j][i], g[j][i]);
          g[j][i] = mul2(g[j][i], w[i]);
          sgz = fma2(g[j][i], z[j][i], sgz);
          if (!RMS) sg = add2(sg, g[j][i]);
        }
      }
    }
    const float2 u = split(sgz), t = split(sg);
    float2 s;
    if (RMS) s = make_float2(row_sum<WIDE>(u.x + u.y, p.lanes, first_warp, reinterpret_cast<float*>(slots[turn])), 0.0f);
    else s = row_sums<WIDE>(u.x + u.y, t.x + t.y, p.lanes, first_warp, slots[turn]);
    if (!WIDE) __syncthreads();
    if (loads && failed == kNone && step + p.stages * gridDim.x < p.steps) rows.load(step + p.stages * gridDim.x, stage);
    from += p.stage;
    if (++stage == p.stages) { stage = 0; from = mine_at; par ^= 1u; }
    if (!live) continue;
    const size_t at = (size_t)row * H + lane * 8;
    const F2 mz = f2(-s.x * inv_h), mg = f2(-s.y * inv_h);
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if (lane * 8 + j * column2 >= H) continue;
      F2 o[4], t[4];
      if (ADD) unpack8(res[j], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = fma2(z[j][i], mz, g[j][i]);
        if (!RMS) o[i] = add2(o[i], mg);
        o[i] = ADD ? fma2(o[i], f2(r), t[i]) : mul2(o[i], f2(r));
      }
      *reinterpret_cast<uint4*>(a.dx + at + j * column2) = pack8(o);
    }
  }
  if (loads && failed != kNone) rows.drain(failed, a.err);
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
        for (int i = 0; i < 8; i += 4) {
          const float2 x0 = split(dw[j][i / 2]), x1 = split(dw[j][i / 2 + 1]), y0 = split(db[j][i / 2]), y1 = split(db[j][i / 2 + 1]);
          float4 x = make_float4(x0.x, x0.y, x1.x, x1.y), y = make_float4(y0.x, y0.y, y1.x, y1.y);
          float4* xs = reinterpret_cast<float4*>(sums + c + i);
          float4* ys = reinterpret_cast<float4*>(sums + H + c + i);
          if (turn2) {
            const float4 u = *xs, v = *ys;
            x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
            y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
          }
          if (turn2 == p.rows - 1) {
            xs = reinterpret_cast<float4*>(part + c + i);
            ys = reinterpret_cast<float4*>(part + H + c + i);
          }
          *xs = x;
          *ys = y;
        }
      }
    }
    __syncthreads();
  }
}

// dw and db from the blocks' partial sums: 8 groups of 4 columns a block, the parts in 32 runs
// (five parts each, under way at once: with 8 runs of 19 the kernel took 9 us for 2048 columns),
// added in order.
constexpr int kRuns = 32, kGroups = 8;
__global__ void __launch_bounds__(kRuns * kGroups) norm_parts_kernel(const float* part, int parts, int H, float* dw, float* db) {
  __shared__ float4 sums[kRuns][kGroups];
  griddep_wait();
  griddep_launch_dependents();
  const int g = threadIdx.x % kGroups, q = threadIdx.x / kGroups, c = (blockIdx.x * kGroups + g) * 4;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool wanted = c < (db ? 2 * H : H);
  if (wanted) {
    const int p0 = q * parts / kRuns, p1 = (q + 1) * parts / kRuns;
#pragma unroll 8
    for (int p = p0; p < p1; ++p) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)p * 2 * H + c);
      t = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
    }
  }
  sums[q][g] = t;
  __syncthreads();
  if (q || !wanted) return;
#pragma unroll
  for (int i = 1; i < kRuns; ++i) {
    const float4 v = sums[i][g];
    t = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
  }
  *reinterpret_cast<float4*>(c < H ? dw + c : db + (c - H)) = t;
}

constexpr int kWide = 8192;  // columns from which a thread takes 16 of a row instead of 8

uint32_t weight_bytes(int H) { return H > kWide ? 0u : ((uint32_t)H * 4 + 127u) & ~127u; }

Plan plan_of(int64_t N, int H, int tensors, uint32_t ring, int kv, int threads) {
  Plan p{};
  const int groups = (H / 8 + kv - 1) / kv;
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < groups) p.lanes *= 2;
  if (groups > 32) p.lanes = (groups + 31) / 32 * 32;
  p.rows = threads / p.lanes;  // several of them fill a third of the ring at most, one of 16384 columns half of it
  const uint32_t row = (uint32_t)H * 2 * tensors;
  p.threads = p.rows * p.lanes;
  p.steps = (uint32_t)((N + p.rows - 1) / p.rows);
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
  cudaError_t e = ring_smem(norm_forward_kernel<RMS, ADD, 2, false, 512>);
  if (e == cudaSuccess) e = ring_smem(norm_forward_kernel<RMS, ADD, 2, true, 512>);
  if (e == cudaSuccess) e = ring_smem(norm_forward_kernel<RMS, ADD, 2, true, 1024>);
  if (e == cudaSuccess) e = ring_smem(norm_backward_kernel<RMS, ADD, 1, false>);
  if (e == cudaSuccess) e = ring_smem(norm_backward_kernel<RMS, ADD, 1, true>);
  if (e == cudaSuccess) e = ring_smem(norm_backward_kernel<RMS, ADD, 2, true>);
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

unsigned grid_of(const Plan& p, int blocks) { return p.steps < (unsigned)blocks ? p.steps : (unsigned)blocks; }

template <bool RMS, bool ADD>
cudaError_t forward(const NormArgs& a, int sms, cudaStream_t s) {
  const int threads = a.H > kWide ? 1024 : 512, blocks = kMaxThreads / threads;
  const Plan p = plan_of(a.N, a.H, ADD ? 2 : 1, kRingBytes / blocks, 2, threads);
  auto k = a.H > kWide     ? norm_forward_kernel<RMS, ADD, 2, true, 1024>
           : p.lanes > 32 ? norm_forward_kernel<RMS, ADD, 2, true, 512>
                          : norm_forward_kernel<RMS, ADD, 2, false, 512>;
  return launch_pdl(k, dim3(grid_of(p, sms * blocks)), dim3(p.threads), p.stages * p.stage + 128, s, a, p);
}

template <bool RMS, bool ADD>
cudaError_t backward(const NormArgs& a, int sms, unsigned* grid, cudaStream_t s) {
  const Plan p = plan_of(a.N, a.H, ADD ? 3 : 2, kRingBytes - weight_bytes(a.H), a.H > kWide ? 2 : 1, kMaxThreads);
  *grid = grid_of(p, sms);
  auto k = a.H > kWide     ? norm_backward_kernel<RMS, ADD, 2, true>
           : p.lanes > 32 ? norm_backward_kernel<RMS, ADD, 1, true>
                          : norm_backward_kernel<RMS, ADD, 1, false>;
  const uint32_t ring = p.stages * p.stage, sums = 8u * (uint32_t)a.H;  // the block's sums take the ring's place
  return launch_pdl(k, dim3(*grid), dim3(p.threads), weight_bytes(a.H) + (ring > sums ? ring : sums) + 128, s, a, p);
}

}  // namespace

int launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int sms = sm_count(&e);
  if (e != cudaSuccess) return -(int)e;
  e = a.rms ? (a.add ? forward<true, true>(a, sms, s) : forward<true, false>(a, sms, s))
            : (a.add ? forward<false, true>(a, sms, s) : forward<false, false>(a, sms, s));
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
  unsigned grid = 0;
  e = a.rms ? (a.add ? backward<true, true>(a, sms, &grid, s) : backward<true, false>(a, sms, &grid, s))
            : (a.add ? backward<false, true>(a, sms, &grid, s) : backward<false, false>(a, sms, &grid, s));
  if (e != cudaSuccess) return -(int)e;
  e = launch_pdl(norm_parts_kernel, dim3((2 * a.H + 4 * kGroups - 1) / (4 * kGroups)), dim3(kRuns * kGroups), 0, s,
                 (const float*)a.part, (int)grid, a.H,
                 a.dw, a.db);
  return e != cudaSuccess ? -(int)e : 2;
}

}  // namespace moe
