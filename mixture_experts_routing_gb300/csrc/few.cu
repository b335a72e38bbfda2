// The whole layer for a few tokens in bf16: two kernels.
//
//   logits   l[t,e] = x_t . W_r[:,e] + b[e]. A cluster of eight blocks shares the
//            contraction of 16 experts and adds its parts through distributed shared
//            memory; on the way it clears the work counters of the second kernel.
//   experts  every block picks the experts of all tokens for itself (a warp a token),
//            then the blocks stream the chosen experts' weights, tile by tile:
//              FC1   8 gate and 8 up rows of an expert times its tokens; h = act(g) u
//              FC2   16 rows of W_down times the same tokens' h, to o [route][column]
//            The last block to finish a column tile adds up its tokens' routes.
//
// The time is that of reading the weights, so a tile is a run of 16 weight rows that
// passes through a ring in shared memory (a TMA copy of 16 rows x 1024 or 512 columns a
// stage) into mma.sync, once for each unit of the expert's tokens (8, 16 or 32: see
// build_units), weights as the 16 rows, tokens as the 8 columns: four warps split the
// columns of a stage, so a tile needs no split between blocks, and there are enough tiles
// to keep all SMs busy from one token on (128-row tiles of the 5th-generation tensor
// cores would leave 8 experts x 2048 features with fewer tiles than there are turns to
// share out). A block draws its tiles from one counter, FC1's before FC2's, so a block
// that waits for an expert's h waits only for tiles that running blocks already hold: the
// kernel needs no co-residency, and the ring fills with W_down while it waits.
//
// Measured, called in a row with changing inputs: 1 token, 8 of 256 experts of 7168 x 2048,
// 113 us (705 MB: 6.3 TB/s over the whole call, 7 once the weights flow, of 6.8 that a copy
// reaches); 33 tokens, 8 of 128 of 2048 x 768, 163 to 176 us by the experts hit; 64 tokens,
// 2 of 8 of 512 x 1024, 32 us: some 18 are the chain of its waits, the rest eight tiles an SM
// of 16 to 32 KB, each of which pays a tile's set-up and a copy of its unit's tokens. The logits
// take 2 us of one token's call (2048 columns) to 5 us of 33 tokens'.
#include "act.cuh"
#include "layer_internal.h"
#include "moe_internal.h"
#include "ptx.cuh"
#include "route_math.cuh"
#include "tmap.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- workspace
struct FewWs {
  size_t logits, count, h, o, total;
};

constexpr int kMaxUnits = kMaxExperts + kFewMaxTokens * kMaxTopK / 8;  // an expert's tokens, 8 or more at a time

// [0] next tile, [1 + u] tiles of unit u's h that are written, then of every 16 columns the
// units whose products are in o
__host__ __device__ inline int count_words(int H) { return 1 + kMaxUnits + H / 16; }

FewWs layout(int N, int H, int E, int K, int I) {
  FewWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  w.logits = take((size_t)N * E * 4);
  w.count = take((size_t)count_words(H) * 4);
  w.h = take((size_t)N * K * I * 2);
  w.o = take((size_t)N * K * H * 4);
  w.total = off;
  return w;
}

// ---------------------------------------------------------------- logits
constexpr int kLogitThreads = 256;
constexpr int kLogitSplit = 8;   // blocks of a cluster: parts of the contraction
constexpr int kLogitCols = 16;   // experts of a cluster
constexpr int kLogitTok = 8;     // tokens at a time

// A thread takes four experts and every 64th pair of rows of the block's part; a row pair
// of x is one 32-bit load. Four pairs' weights are under way at once: with one, a decode
// step's 14 rows a thread waited for memory seven times. Chain of a logit: H / 1024
// pairs, 3 lanes, 8 warps, 8 blocks. blockIdx.y: eight tokens.
__global__ void __cluster_dims__(kLogitSplit, 1, 1) __launch_bounds__(kLogitThreads)
    few_logits_kernel(const FewArgs a, float* logits, int32_t* count) {
  __shared__ float warp_part[8][kLogitTok][kLogitCols];
  __shared__ __align__(16) float part[kLogitTok][kLogitCols];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * kLogitThreads + threadIdx.x; i < count_words(a.H); i += gridDim.x * kLogitThreads)
      count[i] = 0;
  const int t0 = blockIdx.y * kLogitTok, n = min(kLogitTok, live_tokens(a.n_dev, a.N) - t0);
  if (n <= 0) return;  // the whole cluster
  const int rank = blockIdx.x % kLogitSplit, e0 = blockIdx.x / kLogitSplit * kLogitCols;
  const int q = threadIdx.x & 3, r = threadIdx.x >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.H / 2, p0 = (int)((int64_t)rank * pairs / kLogitSplit), p1 = (int)((int64_t)(rank + 1) * pairs / kLogitSplit);
  const int e = e0 + 4 * q;
  const bool vec = (a.E & 3) == 0 && (reinterpret_cast<uintptr_t>(a.wr) & 15) == 0;
  constexpr int kStep = kLogitThreads / 4, kAhead = 4;
  float acc[kLogitTok][4] = {};
  for (int p = p0 + r; p < p1; p += kAhead * kStep) {
    float w[kAhead][2][4];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* row = a.wr + (size_t)(2 * (p + s * kStep) + i) * a.E + e;
        const bool in = p + s * kStep < p1;
        if (vec) {
          const float4 v = in && e < a.E ? *reinterpret_cast<const float4*>(row) : make_float4(0.f, 0.f, 0.f, 0.f);
          w[s][i][0] = v.x; w[s][i][1] = v.y; w[s][i][2] = v.z; w[s][i][3] = v.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[s][i][j] = in && e + j < a.E ? row[j] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kLogitTok; ++t) {
      if (t < n) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          if (p + s * kStep < p1) {
            const uint32_t x = reinterpret_cast<const uint32_t*>(a.x + (size_t)(t0 + t) * a.H)[p + s * kStep];
            const float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xFFFF0000u);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(x1, w[s][1][j], fmaf(x0, w[s][0][j], acc[t][j]));
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kLogitTok; ++t) {
    if (t < n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) acc[t][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[t][j], o);
        if (lane < 4) warp_part[warp][t][4 * q + j] = acc[t][j];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < n * kLogitCols) {
    const int t = threadIdx.x / kLogitCols, c = threadIdx.x % kLogitCols;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += warp_part[w][t][c];
    part[t][c] = s;
  }
  cluster_sync_all();
  const int c = threadIdx.x;
  if (rank < n && c < kLogitCols && e0 + c < a.E) {  // block `rank` adds up token t0 + rank
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kLogitSplit; ++k) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&part[rank][c]), (uint32_t)k)));
      s += v;
    }
    logits[(size_t)(t0 + rank) * a.E + e0 + c] = s + (a.bias ? a.bias[e0 + c] : 0.0f);
  }
  cluster_sync_all();  // no block leaves while another reads its part
}
static_assert(kLogitTok <= kLogitSplit, "one token of the chunk per block of the cluster");

// ---------------------------------------------------------------- experts
constexpr int kMmaWarps = 4, kEpiWarps = 4, kFinishWarps = 2;
constexpr int kFewThreads = (kMmaWarps + 2 + kEpiWarps + kFinishWarps) * 32;
constexpr int kPosts = 8;        // column tiles posted to the finishing warps
constexpr int kRows = 16;        // weight rows of a tile
constexpr int kDrawn = 3;        // tiles drawn ahead
constexpr int kMaxStages = 8;
constexpr uint32_t kRingBytes = 209u << 10;  // with the buffers of the sums

struct FewShared {
  uint64_t wfull[kMaxStages], afull[kMaxStages], empty[kMaxStages], named[kMaxStages], rfull[kEpiWarps], rempty[kEpiWarps];
  int tile[kMaxStages];            // of the stage, -1: no more
  int red_tile[kEpiWarps];
  uint64_t pfull[kPosts], pempty[kPosts];
  int post_row[kPosts], post_first[kPosts], posts;
  int ids[kFewMaxTokens * kMaxTopK];
  float p[kFewMaxTokens * kMaxTopK];
  uint16_t list[kFewMaxTokens * kMaxTopK];  // routes by expert, tokens ascending
  uint32_t mask[kMaxExperts][2];   // tokens of an expert
  uint16_t base[kMaxExperts];      // an expert's first route in list
  uint16_t unit_e[kMaxUnits], unit_at[kMaxUnits], unit_n[kMaxUnits];
  uint8_t unit_done[kMaxUnits];    // seen complete by the activations' warp
  int warp_sum[kMaxExperts / 32][3];
  int units, groups;               // units; groups of 8 tokens in one at most
  uint32_t by_per, by_run;         // 2^32 / (FC1 tiles of a unit) and / (16 units), rounded up
};

// A logit as a key that orders like it, a NaN above all and 0 for none; and back.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 and 0 are equal
  return isnan(l) ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t k) {
  return __uint_as_float(k == 0xFFFFFFFFu ? 0x7FC00000u : (k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Pick k of token t.
__device__ __forceinline__ void keep_pick(const FewArgs& a, FewShared& s, int t, int k, int id, float p, bool out) {
  const int at = t * a.K + k;
  s.ids[at] = id;
  s.p[at] = p;
  if (p != 0.0f) atomicOr(&s.mask[id][t >> 5], 1u << (t & 31));  // p = 0 is not read; a NaN is not 0
  if (out && a.topk_ids) a.topk_ids[at] = id;
  if (out && a.topk_p) a.topk_p[at] = p;
}

// The K experts of a token by a warp. The picks go by the logits (ties to the lower id):
// probabilities are needed of the K picked alone, and their sum over all experts only where
// it is not divided out again. Lane l holds experts l, l+32, ..., PER of them. One token at a
// time: two in turns filled each other's waits, but the larger code came from memory at
// every launch (1 token, 7168 x 2048: 115.0 us with both forms, 113.7 with this one).
template <int PER>
__device__ __forceinline__ void pick(const FewArgs& a, const float* logits, int t, FewShared& s, bool out) {
  const int lane = threadIdx.x & 31;
  uint32_t key[PER], first[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    first[j] = e < a.E ? __float_as_uint(__ldcg(logits + (size_t)t * a.E + e)) : 0u;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = first[j] = lane + 32 * j < a.E ? key_of(__uint_as_float(first[j])) : 0u;
  float top = 0.0f, my_l = 0.0f;
  int my_id = 0;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) best = max(best, key[j]);
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t mine = 0xFFFFFFFFu;
#pragma unroll
    for (int j = PER - 1; j >= 0; --j)
      if (key[j] == best) mine = lane + 32 * j;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, mine);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (e == (uint32_t)(lane + 32 * j)) key[j] = 0;
    if (k == 0) top = logit_of(best);
    if (lane == k) { my_id = (int)e; my_l = logit_of(best); }
  }
  my_l = lane < a.K ? route_exp(__fsub_rn(my_l, top)) : 0.0f;
  float all = my_l;
  if (!a.renorm) {
    all = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (lane + 32 * j < a.E) all += route_exp(__fsub_rn(logit_of(first[j]), top));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (lane < a.K) keep_pick(a, s, t, lane, my_id, __fdiv_rn(my_l, all), out);
}

// The same with at most eight experts: four tokens t0 .. t0+3 a warp, eight lanes each (64
// tokens, top-2 of 8: a turn of all warps instead of six).
__device__ __forceinline__ void pick_eighths(const FewArgs& a, const float* logits, int t0, int n, FewShared& s, bool out) {
  const int lane = threadIdx.x & 31, e = lane & 7, t = t0 + (lane >> 3);
  const bool in = t < n && e < a.E;
  const uint32_t first = in ? key_of(__ldcg(logits + (size_t)t * a.E + e)) : 0u;
  uint32_t key = first;
  float top = 0.0f, my_l = 0.0f;
  int my_id = 0;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = key, id = 0;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    id = key == best ? e : 8;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) id = min(id, __shfl_xor_sync(0xFFFFFFFFu, id, o));
    if (id == (uint32_t)e) key = 0;
    if (k == 0) top = logit_of(best);
    if (e == k) { my_id = (int)id; my_l = logit_of(best); }
  }
  my_l = e < a.K ? route_exp(__fsub_rn(my_l, top)) : 0.0f;
  float all = my_l;
  if (!a.renorm) all = in ? route_exp(__fsub_rn(logit_of(first), top)) : 0.0f;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (e < a.K && t < n) keep_pick(a, s, t, e, my_id, __fdiv_rn(my_l, all), out);
}

// The units (an expert's tokens, at most 8, 16 or 32 at a time) from the masks; all threads.
// The blocks build the same lists, each for itself.
__device__ __forceinline__ void build_units(const FewArgs& a, int n, FewShared& s) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int c = 0;
  if (e < kMaxExperts) {
    c = __popc(s.mask[e][0]) + __popc(s.mask[e][1]);
    const int u8 = __reduce_add_sync(0xFFFFFFFFu, (c + 7) / 8), u16 = __reduce_add_sync(0xFFFFFFFFu, (c + 15) / 16);
    const int u32 = __reduce_add_sync(0xFFFFFFFFu, (c + 31) / 32);
    if (lane == 0) s.warp_sum[warp][0] = u8, s.warp_sum[warp][1] = u16, s.warp_sum[warp][2] = u32;
  }
  __syncthreads();
  int u8 = 0, u16 = 0, u32 = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    u8 += s.warp_sum[w][0];
    u16 += s.warp_sum[w][1];
    u32 += s.warp_sum[w][2];
  }
  // Units of 16 and of 32 tokens take 1.3 and 1.55 times one of 8 (their stages are shorter);
  // an expert's second unit finds weights of the first in the second-level cache, at the sizes
  // measured. 64 tokens, 6 of 64 experts (6 tokens each, some over 8), with 8, 16, 32: 4096 x
  // 1408 380, 457, 552 us, 7168 x 2048 895, 1086, 1304; 4 of 32 of 7168 x 2048 (8 each) 546,
  // 587, 687 (at the rule's border: it takes 16); 2 of 8 (16 each) 258, 263, 243, of 512 x 1024
  // 42, 37, 35.
  const int per = 10 * u8 <= 13 * u16 && 20 * u8 <= 31 * u32 ? 8 : 26 * u16 <= 31 * u32 ? 16 : 32;
  __syncthreads();  // the sums are written again below
  const int u = (c + per - 1) / per;
  int cs = c, us = u;  // inclusive sums over the warp's experts
  if (e < kMaxExperts) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, cs, o), y = __shfl_up_sync(0xFFFFFFFFu, us, o);
      if (lane >= o) { cs += x; us += y; }
    }
    if (lane == 31) { s.warp_sum[warp][0] = cs; s.warp_sum[warp][1] = us; }
  }
  __syncthreads();
  if (e < kMaxExperts) {
    int c0 = cs - c, u0 = us - u, all = 0;
#pragma unroll
    for (int w = 0; w < kMaxExperts / 32; ++w) {
      if (w < warp) { c0 += s.warp_sum[w][0]; u0 += s.warp_sum[w][1]; }
      all += s.warp_sum[w][1];
    }
    s.base[e] = (uint16_t)c0;
    for (int i = 0; i < u; ++i) {
      s.unit_e[u0 + i] = (uint16_t)e;
      s.unit_at[u0 + i] = (uint16_t)(c0 + i * per);
      s.unit_n[u0 + i] = (uint16_t)min(per, c - i * per);
      s.unit_done[u0 + i] = 0;
    }
    if (e == 0) {
      s.units = all;
      s.groups = per / 8;
      // exact quotients: dividend x divisor stays below 2^32 (at most 384 units of 2048 tiles
      // by 2048, and 384 x 1024 by 16 x 384)
      s.by_per = 0xFFFFFFFFu / (uint32_t)(a.I / 8) + 1u;
      s.by_run = 0xFFFFFFFFu / (uint32_t)max(16, 16 * all) + 1u;
    }
  }
  __syncthreads();
  for (int r = threadIdx.x; r < n * a.K; r += kFewThreads) {
    const int t = r / a.K, id = s.ids[r];
    const uint32_t m0 = s.mask[id][0], m1 = s.mask[id][1], bit = 1u << (t & 31);
    if (((t < 32 ? m0 : m1) & bit) == 0 || s.p[r] == 0.0f) continue;
    const int rank = t < 32 ? __popc(m0 & (bit - 1u)) : __popc(m0) + __popc(m1 & (bit - 1u));
    s.list[s.base[id] + rank] = (uint16_t)r;
  }
  __syncthreads();
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int ld_relaxed(const int32_t* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(int32_t* p) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}

// Columns of a stage, by the groups of 8 tokens of a unit. A stage's 16 rows are one copy,
// [64 columns][row], each row of 64 columns swizzled over its 128 bytes: copies of 4 KB kept
// the copying warp busy for longer than memory took (1 token, 7168 x 2048: 128 us, with one
// of 16 KB 116; 33 tokens, 2048 x 768: 195 us with two of 16 KB, 188 with one of 32).
__host__ __device__ constexpr int stage_cols(int groups) { return groups == 1 ? 1024 : 512; }

// Sizes by the groups of 8 tokens of a unit.
template <int G>
struct Ring {
  // Columns of a stage: long ones leave the warps of the products fewer waits (1 token, 7168 x
  // 2048: 140 us with 512, 124 with 1024), where the tokens leave room for four (16 tokens of
  // 512 x 1024: 48 us with five stages of 512, 52 with two of 1024).
  static constexpr int kCols = stage_cols(G);
  static constexpr uint32_t kPitch = kCols * 2 + 16;  // of the activations' rows: 16 bytes apart in banks
  static constexpr uint32_t kWeights = kCols * 2 * kRows;
  static constexpr uint32_t kStage = (kWeights + kPitch * 8 * G + 1023u) & ~1023u;
  static constexpr uint32_t kRed = kMmaWarps * G * 512u;  // of one buffer of the sums
  static constexpr uint32_t kFit = (kRingBytes - 1024u - kEpiWarps * kRed) / kStage;
  static constexpr uint32_t kStages = kFit < kMaxStages ? kFit : kMaxStages;
};

// A place in the ring: stage, and the parity of its turn.
template <int G>
struct Turn {
  uint32_t st = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++st == Ring<G>::kStages) {
      st = 0;
      par ^= 1u;
    }
  }
};

struct TileOf {
  int fc2, unit, row;  // row: first feature, or first column
  int cols;            // contraction
};

// FC1 tiles: unit by unit, so that the first ones are complete early. FC2 tiles: 16 column
// tiles of every unit at a time: outputs are finished all along and not at the end alone, and
// neighbouring blocks read neighbouring rows.
__device__ __forceinline__ TileOf tile_of(const FewArgs& a, const FewShared& s, int tile) {
  TileOf t;
  const int per = a.I / 8, tiles1 = s.units * per;
  t.fc2 = tile >= tiles1;
  if (!t.fc2) {
    t.unit = (int)__umulhi((uint32_t)tile, s.by_per);
    t.row = (tile - t.unit * per) * 8;
    t.cols = a.H;
  } else {
    const int i = tile - tiles1, run = 16 * s.units, c16 = (int)__umulhi((uint32_t)i, s.by_run), r = i - c16 * run;
    const int wide = min(16, a.H / kRows - 16 * c16);
    t.unit = wide == 16 ? r >> 4 : r / wide;
    t.row = (16 * c16 + r - t.unit * wide) * kRows;
    t.cols = a.I;
  }
  return t;
}

// ---------------------------------------------------------------- roles
template <int G>
__device__ __forceinline__ void weights_role(const CUtensorMap& tm1, const CUtensorMap& tm2, const FewArgs& a, FewShared& s,
                                             int32_t* count, int (&drawn)[kDrawn], uint32_t ring) {
  using R = Ring<G>;
  const int lane = threadIdx.x & 31;
  const int tiles = s.units * (a.I / 8 + a.H / kRows);
  const uint64_t policy = policy_evict_first();
  uint32_t it = 0;
  Turn<G> at;
  bool ok = true;
  auto load = [&](int tile) {
    const TileOf t = tile_of(a, s, tile);
    const int e = s.unit_e[t.unit];
    for (int k = 0; k < t.cols; k += R::kCols, ++it, at.next()) {
      if (it >= R::kStages && !mbar_wait_warp(smem_u32(&s.empty[at.st]), at.par ^ 1u, a.err, kErrWaitEmpty)) return false;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&s.wfull[at.st]), dst = ring + at.st * R::kStage;
        s.tile[at.st] = tile;
        mbar_arrive(smem_u32(&s.named[at.st]));
        mbar_arrive_expect_tx(bar, R::kWeights);  // columns past the end count as zeros
        if (t.fc2)
          tma_load_3d(dst, &tm2, 0, e * a.H + t.row, k / 64, bar, policy);
        else
          tma_load_4d(dst, &tm1, 0, t.row, 2 * e, k / 64, bar, policy);
      }
      __syncwarp();
    }
    return true;
  };
  // Three numbers are under way, each in a register of its own: a short tile's copies are
  // issued in half the time that the counter takes to answer.
  bool more = true;
  while (more) {
#pragma unroll
    for (int i = 0; i < kDrawn; ++i) {
      const int tile = __shfl_sync(0xFFFFFFFFu, drawn[i], 0);
      more = tile < tiles;
      if (!more) break;
      if (lane == 0) drawn[i] = atomicAdd(count, 1);
      more = ok = load(tile);
      if (!more) break;
    }
  }
  // the end, told through one more stage; and no copy of this warp is under way when it leaves
  ok = ok && (it < R::kStages || mbar_wait_warp(smem_u32(&s.empty[at.st]), at.par ^ 1u, a.err, kErrWaitEmpty));
  if (ok && lane == 0) {
    s.tile[at.st] = -1;
    mbar_arrive(smem_u32(&s.named[at.st]));
    mbar_arrive(smem_u32(&s.wfull[at.st]));
  }
  __syncwarp();
  // the copy before the end's stage has been used; its barrier is a phase further
  for (uint32_t j = it >= R::kStages ? it - R::kStages + (ok ? 1 : 0) : 0; j < it; ++j)
    if (!mbar_wait_warp(smem_u32(&s.wfull[j % R::kStages]), (j / R::kStages) & 1u, a.err, kErrWaitFull)) break;
}

template <int G>
__device__ __forceinline__ void activations_role(const FewArgs& a, FewShared& s, const int32_t* count, const uint16_t* h, uint32_t ring) {
  using R = Ring<G>;
  const int lane = threadIdx.x & 31;
  int tile = -2, k = 0, rows = 0;
  TileOf t{};
  uint64_t from = 0;  // lane i: the row of the unit's token i
  for (Turn<G> at;; at.next()) {
    if (!mbar_wait_warp(smem_u32(&s.named[at.st]), at.par, a.err, kErrWaitEmpty)) break;
    const int now = s.tile[at.st];
    if (now < 0) {
      mbar_arrive(smem_u32(&s.afull[at.st]));
      break;
    }
    if (now != tile) {
      tile = now;
      k = 0;
      t = tile_of(a, s, tile);
      if (t.fc2 && !s.unit_done[t.unit]) {
        // h is complete when all tiles of its features have said so. An answer takes a
        // microsecond under load, so all units are asked at once.
        const int want = a.I / 8;
        const uint64_t t0 = globaltimer_ns();
        bool ok = true;
        for (uint32_t i = 1;; ++i) {
          bool have = false;
          for (int u0 = lane; u0 < s.units; u0 += 128) {
            int v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = ld_relaxed(count + 1 + min(u0 + 32 * q, kMaxUnits - 1));
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (u0 + 32 * q < s.units && v[q] >= want) {
                s.unit_done[u0 + 32 * q] = 1;
                have |= u0 + 32 * q == t.unit;
              }
          }
          if (__any_sync(0xFFFFFFFFu, have)) break;
          if ((i & 255u) == 0u && __any_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > 2000000000ull)) {
            if (lane == 0) atomicOr(a.err, kErrWaitUnit);
            ok = false;
            break;
          }
        }
        if (!ok) break;
        __threadfence();
        __syncwarp();
      }
      rows = s.unit_n[t.unit];
      if (lane < rows) {
        const int r = s.list[s.unit_at[t.unit] + lane];
        from = reinterpret_cast<uint64_t>(t.fc2 ? h + (size_t)r * a.I : a.x + (size_t)(r / a.K) * a.H);
      }
    } else {
      k += R::kCols;
    }
    const int pieces = min(R::kCols, t.cols - k) / 8;
    const uint32_t dst = ring + at.st * R::kStage + R::kWeights + lane * 16;
#pragma unroll 4
    for (int i = 0; i < rows; ++i) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, from, i)) + k + lane * 8;
#pragma unroll
      for (int j = 0; j < R::kCols / 8; j += 32)
        if (lane + j < pieces) cp_async_16(dst + i * R::kPitch + j * 16, src + j * 8, 16);
    }
    cp_async_mbar_arrive_noinc(smem_u32(&s.afull[at.st]));
  }
  cp_async_wait_all();
}

// A warp takes a quarter of a stage's columns, 64 (one swizzled piece of a box) at a time.
template <int G>
__device__ __forceinline__ void products_role(const FewArgs& a, FewShared& s, uint32_t ring, uint32_t red) {
  using R = Ring<G>;
  constexpr int kPieces = R::kCols / 64 / kMmaWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // weights: 16-byte part c of row r at (c ^ r) of its 128 bytes
  uint32_t woff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    woff[j] = ring + (lane & 15) * 128 + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4);
  // activations: two steps of 16 columns at a time
  const uint32_t boff = ring + R::kWeights + (lane & 7) * R::kPitch + (lane >> 3) * 16;
  constexpr int kChains = G == 1 ? kPieces : 1;  // sums that do not wait for one another
  float acc[kChains][G][4];
  int tile = -2, left = 0, done = 0;
  for (Turn<G> at;; at.next()) {
    if (!mbar_wait_warp(smem_u32(&s.wfull[at.st]), at.par, a.err, kErrWaitFull) ||
        !mbar_wait_warp(smem_u32(&s.afull[at.st]), at.par, a.err, kErrWaitFull))
      break;
    const int now = s.tile[at.st];
    if (now < 0) {  // the end, for every warp of the outputs
      for (int i = 0; i < kEpiWarps; ++i, ++done) {
        const int b = done % kEpiWarps;
        if (done >= kEpiWarps && !mbar_wait_warp(smem_u32(&s.rempty[b]), (done / kEpiWarps - 1) & 1u, a.err, kErrWaitAccum)) break;
        if (warp == 0 && lane == 0) s.red_tile[b] = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.rfull[b]));
      }
      break;
    }
    if (now != tile) {
      tile = now;
      left = tile < s.units * (a.I / 8) ? a.H : a.I;
#pragma unroll
      for (int c = 0; c < kChains; ++c)
#pragma unroll
        for (int g = 0; g < G; ++g) acc[c][g][0] = acc[c][g][1] = acc[c][g][2] = acc[c][g][3] = 0.0f;
    }
    const uint32_t base = at.st * R::kStage;
    uint32_t wf[kPieces][4][4], xf[kPieces][G][2][4];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int piece = warp + p * kMmaWarps;
      if (piece * 64 < left) {
        const uint32_t wat = base + piece * 2048, xat = boff + base + piece * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) ldmatrix4(wf[p][j], woff[j] + wat);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) ldmatrix4(xf[p][g][j], xat + g * 8 * R::kPitch + j * 64);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        if ((warp + p * kMmaWarps) * 64 < left) {
#pragma unroll
          for (int g = 0; g < G; ++g)
            mma16816(acc[p % kChains][g], wf[p][j], xf[p][g][j / 2][j % 2 * 2], xf[p][g][j / 2][j % 2 * 2 + 1]);
        }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.empty[at.st]));
    left -= R::kCols;
    if (left > 0) continue;
    // the warps' sums of the tile, [warp][group][row][token]
    const int b = done % kEpiWarps;
    if (done >= kEpiWarps && !mbar_wait_warp(smem_u32(&s.rempty[b]), (done / kEpiWarps - 1) & 1u, a.err, kErrWaitAccum)) break;
    if (warp == 0 && lane == 0) s.red_tile[b] = tile;
#pragma unroll
    for (int c = 1; c < kChains; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][0][i] += acc[c][0][i];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t to = red + b * R::kRed + (uint32_t)(warp * G + g) * 512u + (lane >> 2) * 32 + (lane & 3) * 8;
      asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to), "f"(acc[0][g][0]), "f"(acc[0][g][1]) : "memory");
      asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to + 256), "f"(acc[0][g][2]), "f"(acc[0][g][3]) : "memory");
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.rfull[b]));
    ++done;
  }
}

// Column tiles whose products are all in o, from the warps of the outputs to the finishing
// ones. A post is 16 columns and every `parts`-th group of 16 tokens; post i goes to
// finishing warp i % kFinishWarps. By one thread.
__device__ __forceinline__ void post(const FewArgs& a, FewShared& s, int row, int parts) {
  const int first = atomicAdd(&s.posts, parts);
  for (int i = 0; i < parts; ++i) {
    const uint32_t at = (uint32_t)(first + i), slot = at % kPosts, turn = at / kPosts;
    if (turn > 0 && !mbar_wait(smem_u32(&s.pempty[slot]), (turn - 1) & 1u, a.err, kErrWaitAccum)) return;
    s.post_row[slot] = row;
    s.post_first[slot] = i | (parts << 16);
    mbar_arrive(smem_u32(&s.pfull[slot]));
  }
}

// y of the posted columns: four lanes a token, two tokens a lane under way at once. Warps of
// their own: the reads of a tile's routes take microseconds, and while a warp of the outputs
// spent them its buffer stood still (33 tokens of 2048 x 768: 199 us with two tokens under
// way there, 212 with one).
__device__ __forceinline__ void finish_role(const FewArgs& a, FewShared& s, int n, const float* o) {
  const int lane = threadIdx.x & 31;
  for (uint32_t at = (threadIdx.x >> 5) - (kMmaWarps + 2 + kEpiWarps);; at += kFinishWarps) {
    const uint32_t slot = at % kPosts;
    if (!mbar_wait_warp(smem_u32(&s.pfull[slot]), (at / kPosts) & 1u, a.err, kErrWaitAccum)) break;
    const int row = s.post_row[slot], part = s.post_first[slot] & 0xFFFF, parts = s.post_first[slot] >> 16;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.pempty[slot]));
    if (row < 0) break;
    const int c = row + 4 * (lane & 3);
    constexpr int kTwo = 2;
    for (int t0 = 16 * part + (lane >> 2); t0 < n; t0 += 16 * parts) {
      float4 y[kTwo] = {};
      for (int k0 = 0; k0 < a.K; k0 += 8) {
        float4 v[kTwo][8];
        float p[kTwo][8];
#pragma unroll
        for (int i = 0; i < kTwo; ++i) {
          const int t = t0 + 8 * i;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            p[i][k] = t < n && k0 + k < a.K ? s.p[t * a.K + k0 + k] : 0.0f;
            // a route of probability 0 has no product
            v[i][k] = p[i][k] != 0.0f ? __ldcg(reinterpret_cast<const float4*>(o + ((size_t)t * a.K + k0 + k) * a.H + c))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
#pragma unroll
        for (int i = 0; i < kTwo; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[i].x = fmaf(p[i][k], v[i][k].x, y[i].x);
            y[i].y = fmaf(p[i][k], v[i][k].y, y[i].y);
            y[i].z = fmaf(p[i][k], v[i][k].z, y[i].z);
            y[i].w = fmaf(p[i][k], v[i][k].w, y[i].w);
          }
      }
#pragma unroll
      for (int i = 0; i < kTwo; ++i) {
        if (t0 + 8 * i >= n) break;
        const size_t to = (size_t)(t0 + 8 * i) * a.H + c;
        if (a.add) {
          const uint2 q = *reinterpret_cast<const uint2*>(a.add + to);
          y[i].x += __uint_as_float(q.x << 16);
          y[i].y += __uint_as_float(q.x & 0xFFFF0000u);
          y[i].z += __uint_as_float(q.y << 16);
          y[i].w += __uint_as_float(q.y & 0xFFFF0000u);
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y[i].x, y[i].y), hi = __floats2bfloat162_rn(y[i].z, y[i].w);
        *reinterpret_cast<uint2*>(a.y + to) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
}

// A warp takes every fourth tile, from a buffer of its own: making a tile's values visible
// to the other blocks costs it about a microsecond, which three other tiles hide.
template <int ACT, int G>
__device__ __forceinline__ void outputs_role(const FewArgs& a, FewShared& s, int32_t* count, uint16_t* h, float* o,
                                             const float* red) {
  using R = Ring<G>;
  const int w = (threadIdx.x >> 5) - kMmaWarps - 2, lane = threadIdx.x & 31;
  int32_t* col_count = count + 1 + kMaxUnits;
  const float* r = red + w * (R::kRed / 4);
  // An FC2 tile's products are counted when the warp gets its next tile: by then they have
  // reached memory and the fence finds little to wait for; the count is read after that tile.
  int last_row = -1, counted = -1, arrived = 0;
  auto count_last = [&]() {
    counted = last_row;
    if (last_row >= 0 && lane == 0) {
      __threadfence();
      arrived = atomicAdd(col_count + last_row / kRows, 1);
    }
  };
  auto complete = [&]() { return counted >= 0 && __shfl_sync(0xFFFFFFFFu, arrived, 0) == s.units - 1; };
  for (uint32_t par = 0;; par ^= 1u) {
    // also after a wait that ran out, every warp comes to the barrier
    const bool ok = mbar_wait_warp(smem_u32(&s.rfull[w]), par, a.err, kErrWaitAccum);
    const int tile = ok ? s.red_tile[w] : -1;
    if (tile < 0) {
      // the last columns are what the launch ends with: all finishing warps share their tokens
      if (ok) {
        count_last();
        if (complete() && lane == 0) {
          __threadfence();
          post(a, s, counted, kFinishWarps);
        }
      }
      __syncwarp();
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
      if (w == 0 && lane == 0) post(a, s, -1, kFinishWarps);
      break;
    }
    const TileOf t = tile_of(a, s, tile);
    const int tok = s.unit_n[t.unit], at = s.unit_at[t.unit];
    if (!t.fc2) {
      for (int i = lane; i < 8 * tok; i += 32) {
        const int f = i & 7, c = i >> 3;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int m = 0; m < kMmaWarps; ++m) {
          const float* q = r + (m * G + (c >> 3)) * 128 + f * 8 + (c & 7);
          g += q[0];
          u += q[64];
        }
        // bf16, as the tensor cores take it and the ordinary layer has it: without an addend y is off
        // by 1.4 times what h in 32 bits gives (7 tokens, 4096 x 1408: 0.0024 against 0.0017)
        reinterpret_cast<__nv_bfloat16*>(h)[(size_t)s.list[at + c] * a.I + t.row + f] = __float2bfloat16_rn(act_fwd<ACT>(g) * u);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&s.rempty[w]));
        red_release(count + 1 + t.unit);
      }
    } else {
      count_last();
      for (int i = lane; i < 16 * tok; i += 32) {
        const int f = i & 15, c = i >> 4;
        float v = 0.0f;
#pragma unroll
        for (int m = 0; m < kMmaWarps; ++m) v += r[(m * G + (c >> 3)) * 128 + f * 8 + (c & 7)];
        o[(size_t)s.list[at + c] * a.H + t.row + f] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.rempty[w]));
      if (complete() && lane == 0) {
        __threadfence();
        post(a, s, counted, 1);
      }
      last_row = t.row;
    }
    __syncwarp();
  }
}

template <int ACT, int G>
__device__ __forceinline__ void roles(const CUtensorMap& tm1, const CUtensorMap& tm2, const FewArgs& a, FewShared& s,
                                      int32_t* count, int (&drawn)[kDrawn], uint16_t* h, float* o, uint8_t* smem) {
  const uint32_t ring = (smem_u32(smem) + 1023u) & ~1023u, red = ring + Ring<G>::kStages * Ring<G>::kStage;
  const int warp = threadIdx.x >> 5;
  if (warp == kMmaWarps)
    weights_role<G>(tm1, tm2, a, s, count, drawn, ring);
  else if (warp == kMmaWarps + 1)
    activations_role<G>(a, s, count, h, ring);
  else if (warp < kMmaWarps)
    products_role<G>(a, s, ring, red);
  else if (warp < kMmaWarps + 2 + kEpiWarps)
    outputs_role<ACT, G>(a, s, count, h, o, reinterpret_cast<const float*>(smem + (red - smem_u32(smem))));
}

struct Maps {
  CUtensorMap w13[2], w2[2];  // boxes as wide as the stages of one group, and of more
};

template <int ACT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_experts_kernel(const __grid_constant__ Maps tm, const FewArgs a,
                       const float* logits, int32_t* count, uint16_t* h, float* o) {
  extern __shared__ uint8_t smem[];
  __shared__ FewShared s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&s.wfull[i]), 1);
      mbar_init(smem_u32(&s.afull[i]), 32);
      mbar_init(smem_u32(&s.named[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), kMmaWarps);
    }
    for (int i = 0; i < kEpiWarps; ++i) {
      mbar_init(smem_u32(&s.rfull[i]), kMmaWarps);
      mbar_init(smem_u32(&s.rempty[i]), 1);
    }
    for (int i = 0; i < kPosts; ++i) {
      mbar_init(smem_u32(&s.pfull[i]), 1);
      mbar_init(smem_u32(&s.pempty[i]), 1);
    }
    s.posts = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm.w13[0]);
    tma_prefetch_desc(&tm.w2[0]);
  }
  for (int i = threadIdx.x; i < 2 * kMaxExperts; i += kFewThreads) (&s.mask[0][0])[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  int drawn[kDrawn] = {};  // this block's first tiles, under way while the experts are picked
  if (warp == kMmaWarps && lane == 0) {
#pragma unroll
    for (int i = 0; i < kDrawn; ++i) drawn[i] = atomicAdd(count, 1);
  }
  const int n = live_tokens(a.n_dev, a.N);
  __syncthreads();
  const bool out = blockIdx.x == 0;
  if (a.E <= 8)
    for (int t = 4 * warp; t < n; t += 4 * (kFewThreads / 32)) pick_eighths(a, logits, t, n, s, out);
  else
    for (int t = warp; t < n; t += kFewThreads / 32) {
      if (a.E <= 32) pick<1>(a, logits, t, s, out);
      else if (a.E <= 64) pick<2>(a, logits, t, s, out);
      else if (a.E <= 128) pick<4>(a, logits, t, s, out);
      else pick<8>(a, logits, t, s, out);
    }
  __syncthreads();
  build_units(a, n, s);
  if (s.units == 0) return;
  if (warp >= kMmaWarps + 2 + kEpiWarps)
    finish_role(a, s, n, o);
  else if (s.groups == 1)
    roles<ACT, 1>(tm.w13[0], tm.w2[0], a, s, count, drawn, h, o, smem);
  else if (s.groups == 2)
    roles<ACT, 2>(tm.w13[1], tm.w2[1], a, s, count, drawn, h, o, smem);
  else
    roles<ACT, 4>(tm.w13[1], tm.w2[1], a, s, count, drawn, h, o, smem);
}

}  // namespace

int64_t few_workspace_bytes(int N, int H, int E, int K, int I) { return (int64_t)layout(N, H, E, K, I).total; }

int launch_few(const FewArgs& a, cudaStream_t s) {
  static DeviceOnce once;
  int sms = 0;
  cudaError_t e = once_per_device(once, &sms, [](int dev, int* v) {
    cudaError_t err = cudaFuncSetAttribute(few_experts_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(few_experts_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    return err != cudaSuccess ? err : cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
  if (e != cudaSuccess) return -(int)e;
  Maps tm;
  for (int i = 0; i < 2; ++i)
    if (!make_map_halves(&tm.w13[i], a.w13, (uint64_t)a.H, (uint64_t)a.I, 2ull * a.E, 8, 2, stage_cols(1 + i) / 64) ||
        !make_map_mn3d(&tm.w2[i], a.w2, (uint64_t)a.I, (uint64_t)a.E * a.H, kRows, stage_cols(1 + i) / 64))
      return -(int)cudaErrorInvalidValue;
  const FewWs w = layout(a.N, a.H, a.E, a.K, a.I);
  float* logits = reinterpret_cast<float*>(a.ws + w.logits);
  int32_t* count = reinterpret_cast<int32_t*>(a.ws + w.count);
  e = launch_pdl(few_logits_kernel, dim3((a.E + kLogitCols - 1) / kLogitCols * kLogitSplit, (a.N + kLogitTok - 1) / kLogitTok), dim3(kLogitThreads), 0, s, a,
                 logits, count);
  if (e == cudaSuccess)
    e = launch_pdl(a.activation ? few_experts_kernel<1> : few_experts_kernel<0>, dim3(sms), dim3(kFewThreads), kRingBytes, s,
                   tm, a, (const float*)logits, count, reinterpret_cast<uint16_t*>(a.ws + w.h),
                   reinterpret_cast<float*>(a.ws + w.o));
  return e != cudaSuccess ? -(int)e : 2;
}

}  // namespace moe
