// Products with 4-bit weights and group scales, for the few tokens of a decode
// step: w[r,c] = scale[r, c/group] * (nibble[r,c] - 8).
//
//   matvec    y[t,:] = w x[t,:]
//   experts   h[t,k,:] = act(W13g[e] x_t) * (W13u[e] x_t), e = topk_ids[t,k]
//             y[t,:] = add[t,:] + sum_k p[t,k] W2[e] h[t,k,:]
//
// The time is that of reading the codes once, so the kernels are built around
// that stream: a warp takes 16 rows and walks 128-column blocks of them, each
// lane loading 16 bytes (32 codes) of its two rows straight into registers,
// kAhead blocks ahead. The codes become the A operand of mma.sync m16n8k16 (the
// products need 8 columns for 1 to 8 tokens, and the operands are already in
// registers, which tcgen05.mma cannot read B or A from without a trip through
// shared or tensor memory): a mask and an OR put four bits into the mantissa of
// bf16 128 + code, one subtraction makes it code - 8, exactly. The order of the
// columns within a block is free as long as x follows it, so no weight is
// shuffled. The sums of one group are scaled in fp32 and added up in fp32. The
// warps of a block split the columns and add their parts in a fixed order.
#include "act.cuh"
#include "moe_internal.h"
#include "ptx.cuh"
#include "shared_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 128;       // columns a warp takes at a time
constexpr int kMaxRoutes = 1024;  // N*K, at most

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Within a block, lane t of a quad holds four words of eight codes; word j
// covers columns word_col(t, j) .. + 7, so that the 16 columns of one MMA (two
// MMAs a word) lie in one group.
template <int GROUP>
__device__ __forceinline__ int word_col(int t, int j) {
  if (GROUP == 128) return 32 * t + 8 * j;
  if (GROUP == 64) return 64 * (j >> 1) + 16 * t + 8 * (j & 1);
  return 32 * j + 8 * t;
}

// The four words of block kb of a row; words past the last column stay 0 (their
// x is 0).
template <int GROUP>
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int kb, int t, int cols) {
  const uint8_t* at = row + kb * (kBlock / 2);
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (GROUP == 128) {
    w = __ldg(reinterpret_cast<const uint4*>(at) + t);
  } else if constexpr (GROUP == 64) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(at) + t);
    w.x = a.x;
    w.y = a.y;
    if (kb * kBlock + 64 < cols) {
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(at) + 4 + t);
      w.z = b.x;
      w.w = b.y;
    }
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(at) + t;
    const int left = cols - kb * kBlock;
    w.x = __ldg(p);
    if (left > 32) w.y = __ldg(p + 4);
    if (left > 64) w.z = __ldg(p + 8);
    if (left > 96) w.w = __ldg(p + 12);
  }
  return w;
}

// Eight codes as four pairs of bf16 code - 8: columns (0,4), (1,5), (2,6), (3,7).
__device__ __forceinline__ void open_codes(uint32_t w, uint32_t (&d)[4]) {
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;  // 128 + code
    const __nv_bfloat162 b = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
    d[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes and scales of one block of MT tiles of 16 rows (this lane's rows g and
// g + 8 of each).
template <int MT, int GROUP>
struct Block {
  uint4 w[MT][2];
  uint16_t s[MT][2][kBlock / GROUP];

  // q[m][i], sc[m][i]: this lane's rows; cols columns
  __device__ __forceinline__ void load(const uint8_t* const (&q)[MT][2],
                                       const uint16_t* const (&sc)[MT][2], int kb, int t,
                                       int cols) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[m][i] = load_codes<GROUP>(q[m][i], kb, t, cols);
#pragma unroll
        for (int j = 0; j < kBlock / GROUP; ++j)
          s[m][i][j] = (kb * kBlock + j * GROUP < cols)
                           ? __ldg(sc[m][i] + kb * (kBlock / GROUP) + j) : (uint16_t)0;
      }
  }

  // acc[m][n] += (rows of tile m) x (tokens of tile n); x[n]: this lane's token
  // (column g of tile n) or null; tiles not in `live` (the same for all lanes)
  // are left out. P: weights of the two token columns this lane holds of each tile.
  template <int NT, bool P>
  __device__ __forceinline__ void multiply(const uint16_t* const (&x)[NT], uint32_t live, int kb,
                                           int t, int cols, const float (&p)[NT][2],
                                           float (&acc)[MT][NT][4]) const {
    constexpr int kGroups = kBlock / GROUP, kWords = 4 / kGroups;
#pragma unroll
    for (int grp = 0; grp < kGroups; ++grp) {
      if (kb * kBlock + grp * GROUP >= cols) break;
      float part[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[m][n][i] = 0.0f;
#pragma unroll
      for (int jj = 0; jj < kWords; ++jj) {
        const int j = grp * kWords + jj;
        uint4 v[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          v[n] = make_uint4(0u, 0u, 0u, 0u);
          if (x[n])
            v[n] = *reinterpret_cast<const uint4*>(x[n] + kb * kBlock + word_col<GROUP>(t, j));
        }
        uint32_t a[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4& q = w[m][i];
            open_codes(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w, a[m][i]);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (NT > 1 && !((live >> n) & 1u)) continue;
          const uint32_t b0 = __byte_perm(v[n].x, v[n].z, 0x5410), b1 = __byte_perm(v[n].x, v[n].z, 0x7632);
          const uint32_t b2 = __byte_perm(v[n].y, v[n].w, 0x5410), b3 = __byte_perm(v[n].y, v[n].w, 0x7632);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma16816(part[m][n], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b0, b1);
            mma16816(part[m][n], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b2, b3);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float s0 = bf(s[m][0][grp]), s1 = bf(s[m][1][grp]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (NT > 1 && !((live >> n) & 1u)) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            acc[m][n][i] = fmaf(P ? s0 * p[n][i] : s0, part[m][n][i], acc[m][n][i]);
            acc[m][n][2 + i] = fmaf(P ? s1 * p[n][i] : s1, part[m][n][2 + i], acc[m][n][2 + i]);
          }
        }
      }
    }
  }
};

// Every kWarps-th block of a row tile from this warp's own on, kAhead loads ahead.
template <int MT, int NT, int GROUP, int kAhead>
__device__ __forceinline__ void stream_rows(const uint8_t* const (&q)[MT][2],
                                            const uint16_t* const (&sc)[MT][2],
                                            const uint16_t* const (&x)[NT], uint32_t live, int warp,
                                            int t, int cols, float (&acc)[MT][NT][4]) {
  const int blocks = (cols + kBlock - 1) / kBlock;
  const float none[NT][2] = {};
  Block<MT, GROUP> ring[kAhead];
#pragma unroll
  for (int d = 0; d < kAhead; ++d)
    if (warp + d * kWarps < blocks) ring[d].load(q, sc, warp + d * kWarps, t, cols);
  for (int kb = warp; kb < blocks; kb += kAhead * kWarps) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int at = kb + d * kWarps;
      if (at < blocks) {
        ring[d].template multiply<NT, false>(x, live, at, t, cols, none, acc);
        if (at + kAhead * kWarps < blocks) ring[d].load(q, sc, at + kAhead * kWarps, t, cols);
      }
    }
  }
}

// The warps' sums of MT x 16 rows x NT x 8 tokens side by side in shared memory:
// part[((warp * MT + m) * 16 + row) * 8 NT + token].
template <int MT, int NT>
__device__ __forceinline__ void leave_parts(float* part, int warp, int g, int t,
                                            const float (&acc)[MT][NT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* at = part + ((warp * MT + m) * 16 + g) * 8 * NT + 8 * n + 2 * t;
      *reinterpret_cast<float2*>(at) = make_float2(acc[m][n][0], acc[m][n][1]);
      *reinterpret_cast<float2*>(at + 8 * 8 * NT) = make_float2(acc[m][n][2], acc[m][n][3]);
    }
}

template <int NT, int GROUP>
__global__ void __launch_bounds__(kThreads) w4_matvec_kernel(const uint16_t* x, const uint8_t* q,
                                                             const uint16_t* scale, int N, int rows,
                                                             int cols, uint16_t* y) {
  __shared__ float part[kWarps * 16 * 8 * NT];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * NT;
  const uint8_t* qr[1][2];
  const uint16_t* sr[1][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // a row past the last one reads the last one
    const size_t r = (size_t)min(r0 + g + 8 * i, rows - 1);
    qr[0][i] = q + r * (cols / 2);
    sr[0][i] = scale + r * (cols / GROUP);
  }
  const uint16_t* xt[NT];
  uint32_t live = 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = t0 + 8 * n + g;
    xt[n] = tok < N ? x + (size_t)tok * cols : nullptr;
    live |= (t0 + 8 * n < N) ? 1u << n : 0u;
  }
  float acc[1][NT][4] = {};
  stream_rows<1, NT, GROUP, NT == 1 ? 4 : 2>(qr, sr, xt, live, warp, t, cols, acc);
  leave_parts<1, NT>(part, warp, g, t, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += kThreads) {
    const int tok = t0 + (i >> 4), r = r0 + (i & 15);
    if (tok >= N || r >= rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[(w * 16 + (i & 15)) * 8 * NT + (i >> 4)];
    y[(size_t)tok * rows + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

// First product: block (16 features, route r). The first route of an expert does
// the work of all its routes, in passes of 8 NT; the others leave.
template <int NT, int GROUP>
__global__ void __launch_bounds__(kThreads) w4_fc1_kernel(const W4Args a) {
  __shared__ float part[kWarps * 2 * 16 * 8 * NT];
  __shared__ int16_t routes[kMaxRoutes];
  __shared__ int count;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r = blockIdx.y, R = a.N * a.K;
  const int e = a.topk_ids[r];
  if (e < 0 || e >= a.E) return;
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < R; i0 += 32) {
      const int i = i0 + lane;
      const bool same = i < R && a.topk_ids[i] == e;
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, same);
      if (same) routes[n + __popc(b & ((1u << lane) - 1u))] = (int16_t)i;
      n += __popc(b);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  if (routes[0] != r) return;
  const int n_routes = count, i0 = blockIdx.x * 16;
  const uint8_t* qr[2][2];
  const uint16_t* sr[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t row = (size_t)e * 2 * a.I + (size_t)m * a.I + i0 + g + 8 * i;
      qr[m][i] = a.w13 + row * (a.H / 2);
      sr[m][i] = a.w13_scale + row * (a.H / GROUP);
    }
  for (int c0 = 0; c0 < n_routes; c0 += 8 * NT) {
    const uint16_t* xt[NT];
    uint32_t live = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int at = c0 + 8 * n + g;
      xt[n] = at < n_routes ? a.x + (size_t)(routes[at] / a.K) * a.H : nullptr;
      live |= (c0 + 8 * n < n_routes) ? 1u << n : 0u;
    }
    float acc[2][NT][4] = {};
    stream_rows<2, NT, GROUP, 2>(qr, sr, xt, live, warp, t, a.H, acc);
    leave_parts<2, NT>(part, warp, g, t, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kThreads) {
      const int at = c0 + (i >> 4);
      if (at >= n_routes) continue;
      float gv = 0.0f, uv = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gv += part[((w * 2) * 16 + (i & 15)) * 8 * NT + (i >> 4)];
        uv += part[((w * 2 + 1) * 16 + (i & 15)) * 8 * NT + (i >> 4)];
      }
      const float h = (a.activation ? act_fwd<1>(gv) : act_fwd<0>(gv)) * uv;
      a.h[(size_t)routes[at] * a.I + i0 + (i & 15)] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
    }
    __syncthreads();
  }
}

// Second product and the sum over a token's routes: block (16 output columns,
// 8 NT tokens) goes through the experts that its tokens chose, in ascending
// order, the (expert, block of columns) pairs dealt out to the warps; a column
// of the products is a token, weighted by its probability for the expert.
// Dynamic shared memory: prob [items][8 NT] f32, slot [items][8 NT] i8; at the
// end the warps' sums.
template <int NT, int GROUP>
__global__ void __launch_bounds__(kThreads) w4_fc2_kernel(const W4Args a) {
  constexpr int kTok = 8 * NT;
  extern __shared__ float prob[];
  float* part = prob;
  __shared__ int16_t item_of[kMaxExperts], expert_of[kMaxExperts];
  __shared__ int warp_items[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16, t0 = blockIdx.y * kTok;
  const int tokens = min(kTok, a.N - t0), R = tokens * a.K;
  const int32_t* ids = a.topk_ids + (size_t)t0 * a.K;
  const float* ps = a.topk_p + (size_t)t0 * a.K;
  // The first product's kernel let this one start after every earlier kernel had
  // finished, and writes neither the routes nor the weights: only h has to wait.
  for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) item_of[e] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < R; i += kThreads) {
    const int e = __ldcg(ids + i);
    if (e >= 0 && e < a.E) item_of[e] = 0;
  }
  __syncthreads();
  static_assert(kThreads == kMaxExperts, "one thread per expert");
  const bool used = item_of[threadIdx.x] == 0;
  const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, used);
  if (lane == 0) warp_items[warp] = __popc(ballot);
  __syncthreads();
  int before = 0, items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? warp_items[w] : 0;
    items += warp_items[w];
  }
  if (used) {
    const int at = before + __popc(ballot & ((1u << lane) - 1u));
    item_of[threadIdx.x] = (int16_t)at;
    expert_of[at] = (int16_t)threadIdx.x;
  }
  int8_t* slot = reinterpret_cast<int8_t*>(prob + items * kTok);
  for (int i = threadIdx.x; i < items * kTok; i += kThreads) {
    prob[i] = 0.0f;
    slot[i] = -1;
  }
  __syncthreads();
  if ((int)threadIdx.x < tokens) {
    // a token that names an expert twice gets both probabilities
    for (int k = 0; k < a.K; ++k) {
      const int e = __ldcg(ids + threadIdx.x * a.K + k);
      if (e < 0 || e >= a.E) continue;
      const int at = item_of[e] * kTok + threadIdx.x;
      prob[at] += __ldcg(ps + threadIdx.x * a.K + k);
      if (slot[at] < 0) slot[at] = (int8_t)k;
    }
  }
  __syncthreads();

  const int blocks = (a.I + kBlock - 1) / kBlock;
  constexpr int kAhead = NT == 1 ? 4 : 2;
  Block<1, GROUP> ring[kAhead];
  int item_l = 0, kb_l = warp;  // what is loaded next
  auto load_next = [&](Block<1, GROUP>& b) {
    while (kb_l >= blocks) {
      kb_l -= blocks;
      ++item_l;
    }
    if (item_l < items) {
      const uint8_t* q[1][2];
      const uint16_t* sc[1][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t row = (size_t)expert_of[item_l] * a.H + r0 + g + 8 * i;
        q[0][i] = a.w2 + row * (a.I / 2);
        sc[0][i] = a.w2_scale + row * (a.I / GROUP);
      }
      b.load(q, sc, kb_l, t, a.I);
    }
    kb_l += kWarps;
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load_next(ring[d]);
  griddep_wait();
  griddep_launch_dependents();

  float acc[1][NT][4] = {};
  const uint16_t* ht[NT];
  float p[NT][2];
  uint32_t live = 0;
  int item = 0, kb = warp, have = -1;
  bool more = true;
  while (more) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      while (kb >= blocks) {
        kb -= blocks;
        ++item;
      }
      if (item >= items) {
        more = false;
        break;
      }
      if (item != have) {
        have = item;
        live = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int k = slot[item * kTok + 8 * n + g];
          ht[n] = k >= 0 ? a.h + ((size_t)(t0 + 8 * n + g) * a.K + k) * a.I : nullptr;
          p[n][0] = prob[item * kTok + 8 * n + 2 * t];
          p[n][1] = prob[item * kTok + 8 * n + 2 * t + 1];
          live |= __any_sync(0xFFFFFFFFu, k >= 0) ? 1u << n : 0u;
        }
      }
      ring[d].template multiply<NT, true>(ht, live, kb, t, a.I, p, acc);
      load_next(ring[d]);
      kb += kWarps;
    }
  }
  __syncthreads();  // every warp is done with prob and slot
  leave_parts<1, NT>(part, warp, g, t, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kTok; i += kThreads) {
    const int tok = t0 + (i >> 4), c = r0 + (i & 15);
    if (tok >= a.N) continue;
    const size_t at = (size_t)tok * a.H + c;
    float v = a.add ? bf(a.add[at]) : 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[(w * 16 + (i & 15)) * kTok + (i >> 4)];
    a.y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
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

namespace {

template <int NT>
cudaError_t matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                   int cols, int group, uint16_t* y, cudaStream_t s) {
  const dim3 grid((rows + 15) / 16, (N + 8 * NT - 1) / (8 * NT));
  auto* k = group == 128 ? w4_matvec_kernel<NT, 128>
                         : group == 64 ? w4_matvec_kernel<NT, 64> : w4_matvec_kernel<NT, 32>;
  return launch_pdl(k, grid, dim3(kThreads), 0, s, x, q, scale, N, rows, cols, y);
}

template <int NT>
cudaError_t fc1(const W4Args& a, cudaStream_t s) {
  const dim3 grid(a.I / 16, a.N * a.K);
  auto* k = a.group == 128 ? w4_fc1_kernel<NT, 128>
                           : a.group == 64 ? w4_fc1_kernel<NT, 64> : w4_fc1_kernel<NT, 32>;
  return launch_pdl(k, grid, dim3(kThreads), 0, s, a);
}

template <int NT>
cudaError_t fc2(const W4Args& a, cudaStream_t s) {
  const int tokens = a.N < 8 * NT ? a.N : 8 * NT;
  const int items = a.E < tokens * a.K ? a.E : tokens * a.K;
  const dim3 grid(a.H / 16, (a.N + 8 * NT - 1) / (8 * NT));
  // at most 256 x 32 x 5 bytes: within the 48 KB a kernel has without asking
  size_t smem = (size_t)items * 8 * NT * 5;
  if (smem < (size_t)kWarps * 16 * 8 * NT * 4) smem = (size_t)kWarps * 16 * 8 * NT * 4;
  auto* k = a.group == 128 ? w4_fc2_kernel<NT, 128>
                           : a.group == 64 ? w4_fc2_kernel<NT, 64> : w4_fc2_kernel<NT, 32>;
  return launch_pdl(k, grid, dim3(kThreads), smem, s, a);
}

}  // namespace

int launch_w4_matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                     int cols, int group, uint16_t* y, cudaStream_t s) {
  const cudaError_t err = N <= 8 ? matvec<1>(x, q, scale, N, rows, cols, group, y, s)
                                 : N <= 16 ? matvec<2>(x, q, scale, N, rows, cols, group, y, s)
                                           : matvec<4>(x, q, scale, N, rows, cols, group, y, s);
  return err != cudaSuccess ? -(int)err : 1;
}

int launch_w4_ffn(const W4Args& a, cudaStream_t s) {
  // tokens an expert serves at once: by the mean number of its routes
  cudaError_t err = a.N <= 8 || a.N * a.K <= 4 * a.E ? fc1<1>(a, s)
                                                     : a.N * a.K <= 12 * a.E ? fc1<2>(a, s) : fc1<4>(a, s);
  if (err != cudaSuccess) return -(int)err;
  err = a.N <= 8 ? fc2<1>(a, s) : a.N <= 16 ? fc2<2>(a, s) : fc2<4>(a, s);
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
