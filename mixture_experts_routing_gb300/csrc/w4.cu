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

  // q, sc: this lane's row g of the first tile; row g + 8 is `eight` rows on (8,
  // unless the matrix ends before it), the next tile `tile` rows
  __device__ __forceinline__ void load(const uint8_t* q, const uint16_t* sc, int eight, int tile,
                                       int kb, int t, int cols) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t rows = (size_t)(m * tile + i * eight);
        w[m][i] = load_codes<GROUP>(q + rows * (cols / 2), kb, t, cols);
#pragma unroll
        for (int j = 0; j < kBlock / GROUP; ++j)
          s[m][i][j] = (kb * kBlock + j * GROUP < cols)
                           ? __ldg(sc + rows * (cols / GROUP) + kb * (kBlock / GROUP) + j)
                           : (uint16_t)0;
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
template <int NT, int GROUP, int kAhead>
__device__ __forceinline__ void stream_rows(const uint8_t* q, const uint16_t* sc, int eight,
                                            const uint16_t* const (&x)[NT], uint32_t live, int warp,
                                            int t, int cols, float (&acc)[1][NT][4]) {
  const int blocks = (cols + kBlock - 1) / kBlock;
  const float none[NT][2] = {};
  Block<1, GROUP> ring[kAhead];
#pragma unroll
  for (int d = 0; d < kAhead; ++d)
    if (warp + d * kWarps < blocks) ring[d].load(q, sc, eight, 0, warp + d * kWarps, t, cols);
  for (int kb = warp; kb < blocks; kb += kAhead * kWarps) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int at = kb + d * kWarps;
      if (at < blocks) {
        ring[d].template multiply<NT, false>(x, live, at, t, cols, none, acc);
        if (at + kAhead * kWarps < blocks)
          ring[d].load(q, sc, eight, 0, at + kAhead * kWarps, t, cols);
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
  __shared__ __align__(16) float part[kWarps * 16 * 8 * NT];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * NT;
  const int row = min(r0 + g, rows - 1);  // a row past the last one reads the last one
  const uint16_t* xt[NT];
  uint32_t live = 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = t0 + 8 * n + g;
    xt[n] = tok < N ? x + (size_t)tok * cols : nullptr;
    live |= (t0 + 8 * n < N) ? 1u << n : 0u;
  }
  float acc[1][NT][4] = {};
  stream_rows<NT, GROUP, NT == 1 ? 4 : 2>(q + (size_t)row * (cols / 2), scale + (size_t)row * (cols / GROUP),
                                          min(8, rows - 1 - row), xt, live, warp, t, cols, acc);
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

// Routes grouped by expert, in shared memory, by the whole block: pieces of at
// most `most` routes of one expert, experts ascending, routes in their order.
struct Groups {
  int16_t order[kMaxRoutes];                          // routes, sorted by expert
  int16_t expert[kMaxExperts + kMaxRoutes / 8];       // of each piece
  int16_t first[kMaxExperts + kMaxRoutes / 8];        // its first place in `order`
  int16_t count[kMaxExperts + kMaxRoutes / 8];
  int16_t rank[kMaxRoutes];                           // of a route among its expert's
  int16_t routes[kMaxExperts];                        // of each expert
  int scan[2][kWarps];
  int pieces;
};

__device__ __forceinline__ void group_routes(Groups& G, const int32_t* ids, int R, int E,
                                             int most) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kThreads == kMaxExperts, "one thread per expert");
  G.routes[threadIdx.x] = 0;
  __syncthreads();
  if (warp == 0) {  // 32 routes at a time, in order: each gets its rank within its expert
    for (int i0 = 0; i0 < R; i0 += 32) {
      const int i = i0 + lane;
      const int id = i < R ? ids[i] : -1;
      const int e = id >= 0 && id < E ? id : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int base = e >= 0 ? G.routes[e] : 0;
      __syncwarp();
      if (e >= 0 && before == 0) G.routes[e] = (int16_t)(base + __popc(same));
      if (i < R) G.rank[i] = (int16_t)(base + before);
      __syncwarp();
    }
  }
  __syncthreads();
  // exclusive sums over the experts of their routes and of their pieces
  const int n = G.routes[threadIdx.x], np = (n + most - 1) / most;
  int sn = n, sp = np;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int vn = __shfl_up_sync(0xFFFFFFFFu, sn, o), vp = __shfl_up_sync(0xFFFFFFFFu, sp, o);
    if (lane >= o) {
      sn += vn;
      sp += vp;
    }
  }
  if (lane == 31) {
    G.scan[0][warp] = sn;
    G.scan[1][warp] = sp;
  }
  __syncthreads();
  int on = sn - n, op = sp - np;
  for (int w = 0; w < warp; ++w) {
    on += G.scan[0][w];
    op += G.scan[1][w];
  }
  G.routes[threadIdx.x] = (int16_t)on;  // now: where the expert's routes begin
  for (int j = 0; j < np; ++j) {
    G.expert[op + j] = (int16_t)threadIdx.x;
    G.first[op + j] = (int16_t)(on + j * most);
    G.count[op + j] = (int16_t)min(most, n - j * most);
  }
  if (threadIdx.x == kThreads - 1) G.pieces = op + np;
  __syncthreads();
  for (int i = threadIdx.x; i < R; i += kThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E) G.order[G.routes[e] + G.rank[i]] = (int16_t)i;
  }
  __syncthreads();
}

// First product. A unit is 16 features (their gate and up rows) of one expert's
// piece of at most 8 NT routes; a team of S warps, which split the columns,
// takes every teams-th unit, its loads running on from unit to unit. Teams of
// a block take neighbouring features of the same expert.
template <int NT, int GROUP>
__global__ void __launch_bounds__(kThreads, 2) w4_fc1_kernel(const W4Args a, const int S) {
  constexpr int kAhead = 2, kPart = 2 * 16 * 8 * NT;
  __shared__ Groups G;
  __shared__ __align__(16) float part[kWarps * kPart];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  group_routes(G, a.topk_ids, a.N * a.K, a.E, 8 * NT);
  const int team = (blockIdx.x * kWarps + warp) / S, teams = gridDim.x * kWarps / S;
  const int member = warp % S, i_tiles = a.I / 16, units = G.pieces * i_tiles;
  const int blocks = (a.H + kBlock - 1) / kBlock;

  Block<2, GROUP> ring[kAhead];
  int unit_l = team, kb_l = member;  // what is loaded next
  const uint8_t* q_l = nullptr;
  const uint16_t* s_l = nullptr;
  int have_l = -1;
  auto load_next = [&](Block<2, GROUP>& b) {
    while (kb_l >= blocks && unit_l < units) {
      kb_l = member;
      unit_l += teams;
    }
    if (unit_l >= units) return;
    if (unit_l != have_l) {
      have_l = unit_l;
      const int piece = unit_l / i_tiles, i0 = (unit_l - piece * i_tiles) * 16;
      const size_t row = (size_t)G.expert[piece] * 2 * a.I + i0 + g;
      q_l = a.w13 + row * (a.H / 2);
      s_l = a.w13_scale + row * (a.H / GROUP);
    }
    b.load(q_l, s_l, 8, a.I, kb_l, t, a.H);
    kb_l += S;
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load_next(ring[d]);

  const float none[NT][2] = {};
  float acc[2][NT][4] = {};
  const uint16_t* xt[NT];
  uint32_t live = 0;
  int unit = team, kb = member;
  auto begin = [&]() {  // the tokens of the unit's piece
    const int piece = unit / i_tiles, first = G.first[piece], n = G.count[piece];
    live = 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = 8 * j + g;
      xt[j] = at < n ? a.x + (size_t)(G.order[first + at] / a.K) * a.H : nullptr;
      live |= 8 * j < n ? 1u << j : 0u;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  };
  auto end = [&]() {  // h of the unit
    const int piece = unit / i_tiles, i0 = (unit - piece * i_tiles) * 16;
    const int first = G.first[piece], n = G.count[piece];
    if (S > 1) {
      float* mine = part + warp * kPart;
      leave_parts<2, NT>(mine, 0, g, t, acc);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / S), "r"(32 * S) : "memory");
      const float* all = part + (warp - member) * kPart;
      for (int i = member * 32 + lane; i < 16 * 8 * NT; i += 32 * S) {
        if ((i >> 4) >= n) break;
        float gv = 0.0f, uv = 0.0f;
        for (int w = 0; w < S; ++w) {
          gv += all[w * kPart + (i & 15) * 8 * NT + (i >> 4)];
          uv += all[w * kPart + (16 + (i & 15)) * 8 * NT + (i >> 4)];
        }
        const float h = (a.activation ? act_fwd<1>(gv) : act_fwd<0>(gv)) * uv;
        a.h[(size_t)G.order[first + (i >> 4)] * a.I + i0 + (i & 15)] =
            __bfloat16_as_ushort(__float2bfloat16_rn(h));
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / S), "r"(32 * S) : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 8 * j + 2 * t + (i & 1);
          if (at >= n) continue;
          const float gv = acc[0][j][i];
          const float h = (a.activation ? act_fwd<1>(gv) : act_fwd<0>(gv)) * acc[1][j][i];
          a.h[(size_t)G.order[first + at] * a.I + i0 + g + 8 * (i >> 1)] =
              __bfloat16_as_ushort(__float2bfloat16_rn(h));
        }
    }
  };
  if (unit < units) begin();
  while (unit < units) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      while (kb >= blocks && unit < units) {
        end();
        kb = member;
        unit += teams;
        if (unit < units) begin();
      }
      if (unit >= units) break;
      ring[d].template multiply<NT, false>(xt, live, kb, t, a.H, none, acc);
      load_next(ring[d]);
      kb += S;
    }
  }
}

// Second product and the sum over a token's routes: block (16 output columns,
// 8 NT tokens) goes through the experts that its tokens chose, in ascending
// order; a team of S warps, which split the columns, takes every teams-th
// expert. A column of the products is a token, weighted by its probability for
// the expert. Dynamic shared memory: prob [items][8 NT] f32, slot [items][8 NT]
// i8; at the end the warps' sums.
template <int NT, int GROUP, int W>
__global__ void __launch_bounds__(W * 32, W == 16 ? 1 : 2) w4_fc2_kernel(const W4Args a, const int S) {
  constexpr int kTok = 8 * NT;
  extern __shared__ __align__(16) float prob[];
  float* part = prob;
  __shared__ int16_t item_of[kMaxExperts], expert_of[kMaxExperts];
  __shared__ int warp_items[kMaxExperts / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16, t0 = blockIdx.y * kTok;
  const int tokens = min(kTok, a.N - t0), R = tokens * a.K;
  const int32_t* ids = a.topk_ids + (size_t)t0 * a.K;
  const float* ps = a.topk_p + (size_t)t0 * a.K;
  // The first product's kernel let this one start after every earlier kernel had
  // finished, and writes neither the routes nor the weights: only h has to wait.
  static_assert(W * 32 >= kMaxExperts, "a thread for each expert");
  const int e_mine = threadIdx.x;
  if (e_mine < kMaxExperts) item_of[e_mine] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < R; i += W * 32) {
    const int e = __ldcg(ids + i);
    if (e >= 0 && e < a.E) item_of[e] = 0;
  }
  __syncthreads();
  const bool used = e_mine < kMaxExperts && item_of[e_mine] == 0;
  const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, used);
  if (lane == 0 && e_mine < kMaxExperts) warp_items[warp] = __popc(ballot);
  __syncthreads();
  int before = 0, items = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    before += w < warp ? warp_items[w] : 0;
    items += warp_items[w];
  }
  if (used) {
    const int at = before + __popc(ballot & ((1u << lane) - 1u));
    item_of[e_mine] = (int16_t)at;
    expert_of[at] = (int16_t)e_mine;
  }
  int8_t* slot = reinterpret_cast<int8_t*>(prob + items * kTok);
  for (int i = threadIdx.x; i < items * kTok; i += W * 32) {
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

  constexpr int kAhead = NT == 4 ? 2 : 4;
  const int teams = W / S;
  const int blocks = (a.I + kBlock - 1) / kBlock, member = warp % S;
  Block<1, GROUP> ring[kAhead];
  int item_l = warp / S, kb_l = member, have_l = -1;  // what is loaded next
  const uint8_t* q_l = nullptr;
  const uint16_t* s_l = nullptr;
  auto load_next = [&](Block<1, GROUP>& b) {
    while (kb_l >= blocks && item_l < items) {
      kb_l = member;
      item_l += teams;
    }
    if (item_l >= items) return;
    if (item_l != have_l) {
      have_l = item_l;
      const size_t row = (size_t)expert_of[item_l] * a.H + r0 + g;
      q_l = a.w2 + row * (a.I / 2);
      s_l = a.w2_scale + row * (a.I / GROUP);
    }
    b.load(q_l, s_l, 8, 0, kb_l, t, a.I);
    kb_l += S;
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load_next(ring[d]);
  griddep_wait();
  griddep_launch_dependents();

  float acc[1][NT][4] = {};
  const uint16_t* ht[NT];
  float p[NT][2];
  uint32_t live = 0;
  int item = warp / S, kb = member, have = -1;
  while (item < items) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      while (kb >= blocks && item < items) {
        kb = member;
        item += teams;
      }
      if (item >= items) break;
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
      kb += S;
    }
  }
  __syncthreads();  // every warp is done with prob and slot
  leave_parts<1, NT>(part, warp, g, t, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kTok; i += W * 32) {
    const int tok = t0 + (i >> 4), c = r0 + (i & 15);
    if (tok >= a.N) continue;
    const size_t at = (size_t)tok * a.H + c;
    float v = a.add ? bf(a.add[at]) : 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[(w * 16 + (i & 15)) * kTok + (i >> 4)];
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

template <int NT, int GROUP>
cudaError_t fc1(const W4Args& a, cudaStream_t s) {
  static DeviceOnce once;
  int sms = 0;
  const cudaError_t err = once_per_device(once, &sms, [](int dev, int* v) {
    return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
  if (err != cudaSuccess) return err;
  // units there may be, and the warps of two blocks an SM
  const int64_t routes = (int64_t)a.N * a.K, warps = 2 * sms * kWarps;
  const int64_t units = (routes < a.E ? routes : a.E) * (a.I / 16);
  const int S = units * 8 <= warps ? 8 : units * 4 <= warps ? 4 : units * 2 <= warps ? 2 : 1;
  return launch_pdl(w4_fc1_kernel<NT, GROUP>, dim3(2 * sms), dim3(kThreads), 0, s, a, S);
}

template <int NT>
cudaError_t fc1(const W4Args& a, cudaStream_t s) {
  return a.group == 128 ? fc1<NT, 128>(a, s) : a.group == 64 ? fc1<NT, 64>(a, s) : fc1<NT, 32>(a, s);
}

template <int NT, int GROUP, int W>
cudaError_t fc2(const W4Args& a, cudaStream_t s) {
  const int tokens = a.N < 8 * NT ? a.N : 8 * NT;
  const int items = a.E < tokens * a.K ? a.E : tokens * a.K;
  const dim3 grid(a.H / 16, (a.N + 8 * NT - 1) / (8 * NT));
  // at most 256 x 32 x 5 bytes: within the 48 KB a kernel has without asking
  size_t smem = (size_t)items * 8 * NT * 5;
  if (smem < (size_t)W * 16 * 8 * NT * 4) smem = (size_t)W * 16 * 8 * NT * 4;
  const int S = items * 8 <= W ? 8 : items * 4 <= W ? 4 : items * 2 <= W ? 2 : 1;
  return launch_pdl(w4_fc2_kernel<NT, GROUP, W>, grid, dim3(W * 32), smem, s, a, S);
}

template <int NT, int GROUP>
cudaError_t fc2(const W4Args& a, cudaStream_t s) {
  // narrow outputs have fewer blocks than SMs to fill: more warps each
  return (int64_t)(a.H / 16) * ((a.N + 8 * NT - 1) / (8 * NT)) <= 256 ? fc2<NT, GROUP, 16>(a, s)
                                                                      : fc2<NT, GROUP, 8>(a, s);
}

template <int NT>
cudaError_t fc2(const W4Args& a, cudaStream_t s) {
  return a.group == 128 ? fc2<NT, 128>(a, s) : a.group == 64 ? fc2<NT, 64>(a, s) : fc2<NT, 32>(a, s);
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
  cudaError_t err = a.N <= 8 || a.N * a.K <= 4 * a.E ? fc1<1>(a, s) : fc1<2>(a, s);
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
