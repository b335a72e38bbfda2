// The shared expert's contractions on the 5th-generation tensor cores.
//
// D[m, n] = sum_k A[m, k] B[n, k]; the launches:
//   gated      D = x W13^T      epilogue h = act(g) u, 8-bit checkpoint of g, u
//   out        D = h W2^T       epilogue (+ add)
//   gated bwd  D = dy W2        epilogue dg, du and h from the checkpoint
//   gradients  D = [dg du] W13 (+ add), [dg du]^T x and dy^T h in one launch: they
//              need nothing of one another, and one list of their tiles leaves one
//              partly filled turn of the SMs instead of three
// Where the backward's tiles are too few for the SMs, the pairs of a cluster share a
// tile's contraction (SHARED).
// A and B are read as they lie in memory: K-major, or MN-major where the
// contraction index is the row of the matrix (no transposed copy is written).
//
// A tile is 256 x 256, computed by a pair of CTAs (cluster of two,
// tcgen05 cta_group::2): each CTA stages its 128 rows of A and its 128 rows of
// B and holds its 128 accumulator rows (256 TMEM columns) in its own TMEM, so a
// stage of 64 contraction values is 32 KB per SM for 256 x 128 x 64
// multiply-adds, half of what a tile of the same size costs one CTA alone. Two
// accumulators fit TMEM: the epilogue of a tile runs under the next tile's
// MMAs. For the gated forward the even CTA stages the gate rows of 128
// features and the odd CTA the up rows of the same features, so a thread of
// the epilogue finds both pre-activations in its own TMEM lane.
//
// Persistent: pair p takes tiles p, p + pairs, ... Both CTAs' TMA copies
// signal the even CTA's stage barrier; its commits release the stage in both.
// Warps: 0 = TMA producer, 1 = TMEM allocator and (even CTA) MMA issuer, 2-9 =
// epilogue (two warps per TMEM lane quarter, half the columns each). Outputs
// leave through the warp's 4 KB of shared memory and a TMA store, which clips
// the ragged edges.
#include "act.cuh"
#include "moe_internal.h"
#include "ptx.cuh"
#include "shared_internal.h"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kBM = 128;              // rows of A per CTA, rows of B per CTA
constexpr int kBK = 64;               // contraction values per stage
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kOpBytes = kBM * kBK * 2;      // 16 KB: one operand's stage
constexpr uint32_t kStageBytes = 2 * kOpBytes;
constexpr uint32_t kEpiBytes = 4096;              // per epilogue warp
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kEpiWarps * kEpiBytes + 1024;
constexpr int kBand = 8;              // M tiles walked together before the next N tile

enum Epi { kGated = 0, kOut = 1, kGatedBwd = 2, kGrads = 3 };

constexpr int kMaxProblems = 3;

// One contraction of a launch.
struct Problem {
  int M, N;              // output rows and columns (gated: columns of h)
  int k_tiles;
  int w;                 // rows of B that a CTA stages: a tile has 2w columns (gated: w features)
  int m_tiles, n_tiles;
  int begin;             // of its tiles in the launch's list
  int amn;               // kGrads: A read MN-major
  int has_add;           // kOut, kGrads
  int f32;               // kGrads: f32 output
};

struct MmaParams {
  Problem pr[kMaxProblems];
  int problems, tiles;
  int split;             // pairs of a cluster, which share a tile's contraction (below)
  int up;                // kGated: rows of B from a feature's gate row to its up row
  const uint8_t* ck_in;  // kGatedBwd: [M,2N] codes, [M,2N/32] bytes
  const uint8_t* sf_in;
  uint8_t* ck;           // kGated: the same as outputs, or null
  uint8_t* sf;
  uint32_t* err;
};

// Of each problem: A, B, the output, what is added (kOut); kGatedBwd (one problem):
// the outputs dg, du and h in o[0], x[0] and o[1].
struct Maps {
  CUtensorMap a[kMaxProblems], b[kMaxProblems], o[kMaxProblems], x[kMaxProblems];
  CUtensorMap o16;  // kGated: the output in boxes of 16 columns
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Where 16-byte piece c of row r lies in a staged box of 64-byte rows (32 bf16
// columns, 64-byte swizzle).
__device__ __forceinline__ uint32_t at64(int r, int c) {
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// This lane's row of 32 bf16 values, as pairs or to be rounded, into a staged box.
__device__ __forceinline__ void stage_pairs(uint32_t buf, int lane, const uint32_t (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(buf + at64(lane, c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void stage_row(uint32_t buf, int lane, const float (&v)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
  stage_pairs(buf, lane, w);
}

__device__ __forceinline__ void store_box(const CUtensorMap* m, uint32_t buf, int x, int y,
                                          int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(m, buf, x, y);
    bulk_commit();
  }
}

// 32 values of a row as one MX block: codes (two 16-byte stores) and the scale
// byte. A block that holds an infinity or a NaN gets the byte 255.
__device__ __forceinline__ void keep_block(const float (&v)[32], uint8_t* ck, uint8_t* sf) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  const bool finite = top < 0x7F800000u;
  const int s = finite ? mx_block_exponent(__uint_as_float(top)) : 0;
  const float f = pow2_neg(s);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = e4m3x2(v[4 * j] * f, v[4 * j + 1] * f) |
           (e4m3x2(v[4 * j + 2] * f, v[4 * j + 3] * f) << 16);
  reinterpret_cast<uint4*>(ck)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(ck)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  *sf = finite ? (uint8_t)(s + 127) : (uint8_t)255;
}

__device__ __forceinline__ void tmem_row32(uint32_t at, float (&v)[32]) {
  uint32_t a[16], b[16];
  tmem_ld16(at, a);
  tmem_ld16(at + 16, b);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[j] = __uint_as_float(a[j]);
    v[16 + j] = __uint_as_float(b[j]);
  }
}

// TMA load into this CTA's shared memory that signals `bar`, the shared::cluster
// address of a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, int x, int y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"((uint64_t)m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

struct Tile {
  int pr;    // problem
  int m, n;  // first row of the pair, first column (gated: first feature)
};

// Tile t of the list: the problems one after another, M tiles in bands of kBand,
// walked M first within a band.
template <int EPI>
__device__ __forceinline__ Tile tile_of(const MmaParams& p, int t) {
  Tile T;
  T.pr = 0;
#pragma unroll
  for (int i = 1; i < kMaxProblems; ++i)
    if (i < p.problems && t >= p.pr[i].begin) T.pr = i;
  const Problem& P = p.pr[T.pr];
  t -= P.begin;
  const int per = kBand * P.n_tiles;
  const int band = t / per, r = t - band * per;
  const int rows = min(kBand, P.m_tiles - band * kBand);
  const int n = r / rows;
  T.m = (band * kBand + (r - n * rows)) * 2 * kBM;
  T.n = n * (EPI == kGated ? P.w : 2 * P.w);
  return T;
}

// Which operands are read MN-major: the launch's kind tells, but for the gradients.
template <int EPI>
__device__ __forceinline__ bool kAMn(const Problem& P) { return EPI == kGrads && P.amn; }
template <int EPI>
__device__ __forceinline__ bool kBMn(const Problem& P) { return EPI == kGatedBwd || EPI == kGrads; }

// SHARED: the cluster's p.split pairs share the contraction of its only tile. A
// kernel of its own: with the split read at run time every launch took 0.5 us more.
template <int EPI, int ACT, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    shared_mma_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MmaParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t tmem_full_bar[2];
  __shared__ __align__(8) uint64_t tmem_empty_bar[2];
  __shared__ __align__(8) uint64_t add_bar[kEpiWarps][2];
  __shared__ uint32_t tmem_base_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SHARED ? p.split : 1;
  const uint32_t rank = cluster_ctarank(), crank = rank & 1u, even = SHARED ? rank & ~1u : 0u;
  const int part = SHARED ? (int)(rank >> 1) : 0;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tiles = p.tiles;
  const int pair = blockIdx.x / (2 * split), pairs = gridDim.x / (2 * split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tmem_full_bar[b]), 1);
      mbar_init(smem_u32(&tmem_empty_bar[b]), 2 * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w)
      for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&add_bar[w][b]), 1);
    mbar_fence_init();
  }
  if (warp == 0 && lane < p.problems) {
    tma_prefetch_desc(&maps.a[lane]);
    tma_prefetch_desc(&maps.b[lane]);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_base_s), 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are set up before the first remote signal
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    uint32_t g = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const Tile T = tile_of<EPI>(p, t);
      const Problem& P = p.pr[T.pr];
      // what the loop needs, in registers: a read of the parameters by problem in
      // every step made the launch 9 % slower
      const CUtensorMap *ma = &maps.a[T.pr], *mb = &maps.b[T.pr];
      const bool amn = kAMn<EPI>(P), bmn = kBMn<EPI>(P);
      const int k0 = P.k_tiles * part / split, k1 = P.k_tiles * (part + 1) / split, w = P.w;
      const uint32_t bar0 = mapa_shared(smem_u32(&full_bar[0]), even);
      const int am = T.m + (int)crank * kBM;
      // the odd CTA's rows of B: the second half of the tile's columns (gated: the up rows)
      const int bn = T.n + (int)crank * (EPI == kGated ? p.up : w);
      // of both CTAs: K-major boxes of w rows, MN-major ones of 64 columns
      const uint32_t bytes = 2 * (kOpBytes + (bmn ? (w > 64 ? kOpBytes : kOpBytes / 2) : (uint32_t)w * 128u));
      for (int kt = k0; kt < k1; ++kt, ++g) {
        const uint32_t s = g % kStages, u = g / kStages;
        if (u > 0 && !mbar_wait_cluster_warp(smem_u32(&empty_bar[s]), (u - 1u) & 1u, p.err,
                                             kErrWaitEmpty)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t bar = bar0 + 8u * s;
          if (crank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), bytes);
          const uint32_t a = sbase + s * kStageBytes, b = a + kOpBytes;
          const int k = kt * kBK;
          // K-major: one box of all rows; MN-major: boxes of 64 columns
          if (amn) {
            tma_load_2d_pair(a, ma, am, k, bar);
            tma_load_2d_pair(a + kOpBytes / 2, ma, am + 64, k, bar);
          } else {
            tma_load_2d_pair(a, ma, k, am, bar);
          }
          if (bmn) {
            tma_load_2d_pair(b, mb, bn, k, bar);
            if (w > 64) tma_load_2d_pair(b + kOpBytes / 2, mb, bn + 64, k, bar);
          } else {
            tma_load_2d_pair(b, mb, k, bn, bar);
          }
        }
        __syncwarp();
      }
    }
    // neither CTA leaves with a copy under way, after a wait that ran out too: both CTAs'
    // signal the even one's barriers
    if (crank == 0)
      for (uint32_t j = g > kStages ? g - kStages : 0; j < g; ++j)
        if (!mbar_wait_cluster_warp(smem_u32(&full_bar[j % kStages]), (j / kStages) & 1u, p.err, kErrWaitFull))
          break;
    __syncwarp();
    if (SHARED) cluster_sync_all();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (crank == 0) {
      uint32_t g = 0, tc = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++tc) {
        const Tile T = tile_of<EPI>(p, t);
        const Problem& P = p.pr[T.pr];
        const bool amn = kAMn<EPI>(P), bmn = kBMn<EPI>(P);
        const int k0 = P.k_tiles * part / split, k1 = P.k_tiles * (part + 1) / split;
        const uint32_t idesc = idesc_bf16_f32(2 * kBM, 2 * P.w) |
                               (amn ? kIdescAMnMajor : 0u) | (bmn ? kIdescBMnMajor : 0u);
        // 16 contraction values: 32 bytes along a K-major row, 16 rows of an MN-major
        // tile (descriptors count in 16 bytes)
        const uint64_t a_step = amn ? 128u : 2u, b_step = bmn ? 128u : 2u;
        const uint64_t a_base = amn ? sdesc_sw128_mn(sbase) : sdesc_sw128(sbase);
        const uint64_t b_base = bmn ? sdesc_sw128_mn(sbase + kOpBytes) : sdesc_sw128(sbase + kOpBytes);
        const uint32_t b = tc & 1u, bu = tc >> 1;
        if (bu > 0 && !mbar_wait_cluster_warp(smem_u32(&tmem_empty_bar[b]), (bu - 1u) & 1u, p.err,
                                              kErrWaitAccum))
          break;
        tc_fence_after();
        for (int kt = k0; kt < k1; ++kt, ++g) {
          const uint32_t s = g % kStages, u = g / kStages;
          if (!mbar_wait_cluster_warp(smem_u32(&full_bar[s]), u & 1u, p.err, kErrWaitFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint64_t at = (uint64_t)(s * (kStageBytes >> 4));
#pragma unroll
            for (uint32_t kk = 0; kk < kBK / 16; ++kk)
              umma_bf16_pair(tmem + b * 256u, a_base + at + kk * a_step, b_base + at + kk * b_step, idesc,
                             ((kt - k0) | (int)kk) != 0);
            umma_commit_pair(smem_u32(&empty_bar[s]), (uint16_t)(3u << even));
          }
          __syncwarp();
        }
        if (lane == 0) umma_commit_pair(smem_u32(&tmem_full_bar[b]), (uint16_t)(3u << even));  // also after an abort
        __syncwarp();
      }
    }
    __syncwarp();
    if (SHARED) cluster_sync_all();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    const uint32_t buf0 = sbase + kStages * kStageBytes + (uint32_t)ew * kEpiBytes;
    // adds: phases of this warp's add barriers so far; turn: which of its two boxes the
    // next chunk uses (they alternate from tile to tile too: a store may still read the
    // last one)
    uint32_t tc = 0, adds[2] = {0, 0}, turn = 0;
    // this warp's chunks of a tile: of a shared one, the pair's
    const int first = half + 2 * part, step = 2 * split;
    bool met = !SHARED;
    for (int t = pair; t < tiles; t += pairs, ++tc) {
      const Tile T = tile_of<EPI>(p, t);
      const Problem& P = p.pr[T.pr];
      const CUtensorMap *mo = &maps.o[T.pr], *mx = &maps.x[T.pr];
      const uint32_t b = tc & 1u, bu = tc >> 1;
      const int row0 = T.m + (int)crank * kBM + q * 32, row = row0 + lane;
      const uint32_t tl = tmem + b * 256u + ((uint32_t)(q * 32) << 16);
      const int M = P.M, N = P.N, w = P.w;
      // 32-column chunks of the tile that hold output values; this warp takes every second
      const int cols = min(EPI == kGated ? w : 2 * w, N - T.n);
      const int chunks = row0 < M ? (cols + 31) / 32 : 0;
      const bool add = (EPI == kOut || EPI == kGrads) && P.has_add;
      auto load_add = [&](int c, uint32_t i) {  // the tile's i-th chunk of this warp
        if (c < chunks && lane == 0) {
          const uint32_t box = (turn + i) & 1u, bar = smem_u32(&add_bar[ew][box]);
          mbar_arrive_expect_tx(bar, 2048);
          tma_load_2d_pair(buf0 + box * 2048u, mx, T.n + 32 * c, row0, bar);
        }
      };
      auto added = [&](uint32_t i) {  // waits for that load
        const uint32_t box = (turn + i) & 1u, use = adds[box]++;
        return mbar_wait_warp(smem_u32(&add_bar[ew][box]), use & 1u, p.err, kErrWaitAccum);
      };
      if (add && first < chunks) {  // under the tile's MMAs: the first two chunks of what is added
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        load_add(first, 0);
        load_add(first + step, 1);
      }
      // the checkpoint of a chunk is loaded a chunk ahead, the first under the tile's MMAs
      uint4 nx[4] = {};
      uint32_t nsf = 0;
      auto load_kept = [&](int c) {
        if (EPI == kGatedBwd && c < chunks && row < M) {
          const uint8_t* from = p.ck_in + (size_t)row * 2 * N + T.n + 32 * c;
          const uint8_t* sf = p.sf_in + (size_t)row * (N / 16) + T.n / 32 + c;
          nx[0] = reinterpret_cast<const uint4*>(from)[0];
          nx[1] = reinterpret_cast<const uint4*>(from)[1];
          nx[2] = reinterpret_cast<const uint4*>(from + N)[0];
          nx[3] = reinterpret_cast<const uint4*>(from + N)[1];
          nsf = (uint32_t)sf[0] | ((uint32_t)sf[N / 32] << 8);
        }
      };
      load_kept(first);
      if (!mbar_wait_cluster_warp(smem_u32(&tmem_full_bar[b]), bu & 1u, p.err, kErrWaitAccum)) {
        if (add && first < chunks) added(0);
        if (add && first + step < chunks) added(1);
        break;
      }
      tc_fence_after();
      if (SHARED) {
        // the other pairs' chunks to where they read them: the stages, whose last MMA is done
        for (int c = half; c < chunks; c += 2) {
          if ((c >> 1) % split == part) continue;
          float v[32];
          tmem_row32(tl + 32u * (uint32_t)c, v);
          const uint32_t at = sbase + (uint32_t)(c * kBM + q * 32 + lane) * 128u;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(at + (uint32_t)((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]),
                         __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                         __float_as_uint(v[4 * j + 3]));
        }
        __syncwarp();
        cluster_sync_all();
        met = true;
      }
      uint32_t nth = 0;
      for (int c = first; c < chunks; c += step, ++nth) {
        const int col = T.n + 32 * c;
        const uint32_t odd = (turn + nth) & 1u, buf = buf0 + odd * 2048u;
        float v[32];
        tmem_row32(tl + 32u * (uint32_t)c, v);
        if (SHARED) {  // the pairs' sums, in their order
          float sum[32] = {};
          const uint32_t at = sbase + (uint32_t)(c * kBM + q * 32 + lane) * 128u;
          for (int r = 0; r < split; ++r) {
            if (r == part) {
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[j] += v[j];
              continue;
            }
            const uint32_t from = mapa_shared(at, 2u * (uint32_t)r + crank);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 o = ld_cluster_v4(from + (uint32_t)((j ^ (lane & 7)) << 4));
              sum[4 * j] += o.x;
              sum[4 * j + 1] += o.y;
              sum[4 * j + 2] += o.z;
              sum[4 * j + 3] += o.w;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[j];
        }
        if (EPI == kGrads && P.f32) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 128-byte rows, 128-byte swizzle
            st_shared_v4(buf0 + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) << 4)),
                         __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                         __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
          store_box(mo, buf0, col, row0, lane);
        } else if constexpr (EPI == kOut || EPI == kGrads) {
          if (add) {
            if (!added(nth)) {
              if (c + step < chunks) added(nth + 1);
              t = tiles;  // the last tile of this warp
              break;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 w = ld_shared_v4(buf + at64(lane, j));
              const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[8 * j + 2 * i] += __uint_as_float(a[i] << 16);
                v[8 * j + 2 * i + 1] += __uint_as_float(a[i] & 0xFFFF0000u);
              }
            }
          } else {
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
          }
          stage_row(buf, lane, v);
          store_box(mo, buf, col, row0, lane);
          if (add && c + 2 * step < chunks) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            load_add(c + 2 * step, nth + 2);
          }
        } else if constexpr (EPI == kGated) {
          float u[32];
          tmem_row32(tl + (uint32_t)w + 32u * (uint32_t)c, u);
          if (p.ck && row < M) {
            const size_t at = (size_t)row * 2 * N + col, sa = (size_t)row * (N / 16) + col / 32;
            keep_block(v, p.ck + at, p.sf + sa);
            keep_block(u, p.ck + at + N, p.sf + sa + N / 32);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = act_fwd<ACT>(v[j]) * u[j];
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          if (32 * c + 32 <= w) {
            stage_row(buf, lane, v);
            store_box(mo, buf, col, row0, lane);
          } else {  // the tile ends after 16 columns
#pragma unroll
            for (int j = 0; j < 2; ++j)
              st_shared_v4(buf + (uint32_t)(lane * 32 + j * 16), pack_bf16(v[8 * j], v[8 * j + 1]),
                           pack_bf16(v[8 * j + 2], v[8 * j + 3]), pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                           pack_bf16(v[8 * j + 6], v[8 * j + 7]));
            store_box(&maps.o16, buf, col, row0, lane);
          }
        } else {  // kGatedBwd
          const uint32_t gw[8] = {nx[0].x, nx[0].y, nx[0].z, nx[0].w, nx[1].x, nx[1].y, nx[1].z, nx[1].w};
          const uint32_t uw[8] = {nx[2].x, nx[2].y, nx[2].z, nx[2].w, nx[3].x, nx[3].y, nx[3].z, nx[3].w};
          const float fg = e8m0_value(nsf & 255u), fu = e8m0_value(nsf >> 8);
          load_kept(c + step);
          uint32_t dg[16], du[16], h[16];  // pairs of bf16
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t sh = (j & 1) * 16;
            const float2 g2 = e4m3x2_value((gw[j >> 1] >> sh) & 0xFFFFu);
            const float2 u2 = e4m3x2_value((uw[j >> 1] >> sh) & 0xFFFFu);
            float a[2], d[2], e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float g = (i ? g2.y : g2.x) * fg, u = (i ? u2.y : u2.x) * fu;
              const float da = v[2 * j + i], k = act_core<ACT>(g), act = g * k;
              d[i] = da * u * act_grad_core<ACT>(g, k);
              e[i] = da * act;
              a[i] = act * u;
            }
            dg[j] = pack_bf16(d[0], d[1]);
            du[j] = pack_bf16(e[0], e[1]);
            h[j] = pack_bf16(a[0], a[1]);
          }
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          stage_pairs(buf0, lane, dg);
          store_box(mo, buf0, col, row0, lane);
          stage_pairs(buf0 + 2048u, lane, du);
          store_box(mx, buf0 + 2048u, col, row0, lane);
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          stage_pairs(buf0, lane, h);
          store_box(&maps.o[1], buf0, col, row0, lane);
        }
      }
      turn += nth;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (crank == 0)
          mbar_arrive(smem_u32(&tmem_empty_bar[b]));
        else
          mbar_arrive_remote_relaxed(mapa_shared(smem_u32(&tmem_empty_bar[b]), even));
        // the store of an f32 chunk reads both boxes, and a bf16 chunk of the next tile
        // waits for all stores but the newest only
        if (EPI == kGrads && P.f32) bulk_wait_read<0>();
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (!met) cluster_sync_all();  // after an abort
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// bf16 [rows, cols], row pitch `pitch` elements, boxes of box_cols x box_rows.
bool map2d(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch,
           uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw,
           CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, uint32_t bytes = 2) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand [rows, cols]: K-major boxes of 64 contraction values x `box_rows`
// rows, or (mn) MN-major boxes of 64 columns x 64 contraction values.
bool operand_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, bool mn,
                 uint32_t box_rows = kBM) {
  return map2d(m, base, cols, rows, cols, 64, mn ? 64 : box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool out_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch) {
  return map2d(m, base, cols, rows, pitch, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

constexpr int kMaxSplit = 4;

void set_cluster(cudaLaunchAttribute& a, int ctas) {
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)ctas;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
}

// Clusters of `split` pairs resident at once (0 where one does not fit), and the kernel's
// shared-memory opt-in, once per device.
template <int EPI, int ACT, bool SHARED>
int max_clusters(int split, cudaError_t* err) {
  static DeviceOnce once[kMaxSplit + 1];
  int n = 0;
  *err = count_per_device(once[split], &n, [&](int, int* v) {
    auto* k = shared_mma_kernel<EPI, ACT, SHARED>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    set_cluster(attr[0], 2 * split);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(v, k, &cfg);
  });
  return n;
}

Problem problem(int M, int N, int64_t K, bool amn = false) {
  Problem P{};
  P.M = M;
  P.N = N;
  P.k_tiles = (int)((K + kBK - 1) / kBK);
  P.amn = amn;
  return P;
}

// In k-tiles of the widest tile, as tile_cost below.
constexpr double kShareCost = 5;   // for each pair more that shares a tile
constexpr double kLaunchCost = 8;  // of a launch more (4 and 13: the same choices but for few)

// How long a tile of width w takes, in k-tiles of the widest: its MMAs, or its
// operands' way into shared memory (128 + w rows a CTA, MN-major B in boxes of 64; the
// widest tile's operands take 0.82 of its MMAs' time), and what a tile costs beside its
// contraction.
double tile_cost(int w, int k_tiles, bool mn) {
  const double mma = w / 128.0, operands = 0.82 * (128 + (mn ? (w > 64 ? 128 : 64) : w)) / 256.0;
  return k_tiles * (mma > operands ? mma : operands) + 1.5;
}

void set_width(Problem& P, int w, bool gated) {
  P.w = w;
  P.m_tiles = (P.M + 2 * kBM - 1) / (2 * kBM);
  const int wide = gated ? w : 2 * w;
  P.n_tiles = (P.N + wide - 1) / wide;
}

// The width of the launch's tiles (one for all its problems) whose longest pair ends
// first: pair p takes tiles p, p + pairs, ... of the list, so a last turn that few
// tiles fill costs as much as a full one. 8192 x 2048 x 768, the gated product: 128
// -> 96 features, 2.5 turns that cost 3 become 3.4 that cost 2.9.
double pick_width(Problem* pr, int n, int pairs, bool gated, bool mn, int step) {
  double least = 0;
  int best = 128;
  for (int w = 128; w >= 64; w -= step) {
    double cost[kMaxProblems];
    int64_t begin[kMaxProblems + 1] = {0};
    for (int i = 0; i < n; ++i) {
      set_width(pr[i], w, gated);
      cost[i] = tile_cost(w, pr[i].k_tiles, mn);
      begin[i + 1] = begin[i] + (int64_t)pr[i].m_tiles * pr[i].n_tiles;
    }
    // pair p has begin / pairs + (p < begin % pairs) tiles of those before `begin`, so
    // its load changes only at the p that are such remainders
    int64_t turns[kMaxProblems + 1];
    int rest[kMaxProblems + 1];
    for (int i = 0; i <= n; ++i) {
      turns[i] = begin[i] / pairs;
      rest[i] = (int)(begin[i] - turns[i] * pairs);
    }
    double longest = 0;
    for (int c = 0; c <= n; ++c) {
      const int p = rest[c];  // the first is 0
      double sum = 0;
      for (int i = 0; i < n; ++i)
        sum += cost[i] * (double)(turns[i + 1] + (p < rest[i + 1]) - turns[i] - (p < rest[i]));
      longest = sum > longest ? sum : longest;
    }
    if (w == 128 || longest < 0.97 * least) {
      least = longest;
      best = w;
    }
  }
  for (int i = 0; i < n; ++i) set_width(pr[i], best, gated);
  return least;
}

// Contractions whose tiles are too few for the SMs: the pairs of a cluster share a
// tile, each a part of the contraction, and each adds up some of its columns from all
// (a tile for each cluster then, not a list for each pair). Sets the width and returns
// the pairs of a cluster. Backward, 64 tokens: 7168 x 2048 96 us without, 65 with;
// 1024 x 352 18.7 and 17.9; 1000 tokens, 4096 x 1408 75 and 70; 4000 tokens, 256 x 128,
// whose weight gradients are a few long contractions, 32 and 25.
template <int EPI, int ACT>
int pick_split(Problem* pr, int n, int step, double* cost, cudaError_t* err) {
  const int pairs = max_clusters<EPI, ACT, false>(1, err);
  if (pairs <= 0) return 0;
  *cost = pick_width(pr, n, pairs, false, true, step);
  int best = 1, w = pr[0].w, shortest = pr[0].k_tiles;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    tiles += (int64_t)pr[i].m_tiles * pr[i].n_tiles;
    shortest = pr[i].k_tiles < shortest ? pr[i].k_tiles : shortest;
  }
  if (tiles < pairs)
    for (int split = 2; split <= kMaxSplit && split <= shortest; ++split) {
      const int clusters = max_clusters<EPI, ACT, true>(split, err);
      if (*err != cudaSuccess) return 0;
      for (int v = 128; v >= 64; v -= step) {
        double longest = 0;
        tiles = 0;
        for (int i = 0; i < n; ++i) {
          set_width(pr[i], v, false);
          tiles += (int64_t)pr[i].m_tiles * pr[i].n_tiles;
          const double c = tile_cost(v, (pr[i].k_tiles + split - 1) / split, true);
          longest = c > longest ? c : longest;
        }
        if (tiles > clusters) continue;
        const double c = longest + kShareCost * (split - 1);
        if (c < 0.97 * *cost) {
          *cost = c;
          best = split;
          w = v;
        }
      }
    }
  for (int i = 0; i < n; ++i) set_width(pr[i], w, false);
  return best;
}

// The problems come longest contraction first: the pairs take tiles in turn, so the
// short ones even the pairs out.
template <int EPI, int ACT>
cudaError_t launch(const Maps& maps, MmaParams p, int pairs, cudaStream_t s) {
  int64_t tiles = 0;
  for (int i = 0; i < p.problems; ++i) {
    p.pr[i].begin = (int)tiles;
    tiles += (int64_t)p.pr[i].m_tiles * p.pr[i].n_tiles;
    if (tiles > INT32_MAX / 4) return cudaErrorInvalidValue;
  }
  p.tiles = (int)tiles;
  if (p.split < 1) p.split = 1;
  const int n = p.split > 1 || p.tiles < pairs ? p.tiles : pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * p.split * n));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  set_cluster(attr[1], 2 * p.split);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if constexpr (EPI == kGatedBwd || EPI == kGrads)
    if (p.split > 1) return cudaLaunchKernelEx(&cfg, shared_mma_kernel<EPI, ACT, true>, maps, p);
  return cudaLaunchKernelEx(&cfg, shared_mma_kernel<EPI, ACT, false>, maps, p);
}

template <int ACT>
cudaError_t forward(const SharedArgs& a, cudaStream_t s) {
  cudaError_t err = cudaSuccess;
  int pairs = max_clusters<kGated, ACT, false>(1, &err);
  if (pairs <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  Maps m{};
  MmaParams p{};
  p.err = a.err;
  p.problems = 1;
  p.pr[0] = problem(a.N, a.I, a.H);
  // a checkpoint block of 32 features lies in one tile
  pick_width(p.pr, 1, pairs, true, false, a.ck ? 32 : 16);
  p.up = a.I;
  p.ck = a.ck;
  p.sf = a.ck_sf;
  if (!operand_map(&m.a[0], a.x, a.H, a.N, false) ||
      !operand_map(&m.b[0], a.w13, a.H, 2 * (int64_t)a.I, false, (uint32_t)p.pr[0].w) ||
      !out_map(&m.o[0], a.h, a.I, a.N, a.I) ||
      !map2d(&m.o16, a.h, a.I, a.N, a.I, 16, 32, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  err = launch<kGated, ACT>(m, p, pairs, s);
  if (err != cudaSuccess) return err;
  pairs = max_clusters<kOut, 0, false>(1, &err);
  if (pairs <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  p = MmaParams{};
  p.err = a.err;
  p.problems = 1;
  p.pr[0] = problem(a.N, a.H, a.I);
  p.pr[0].has_add = a.add != nullptr;
  pick_width(p.pr, 1, pairs, false, false, 16);
  if (!operand_map(&m.a[0], a.h, a.I, a.N, false) ||
      !operand_map(&m.b[0], a.w2, a.I, a.H, false, (uint32_t)p.pr[0].w) ||
      !out_map(&m.o[0], a.y, a.H, a.N, a.H) || (a.add && !out_map(&m.x[0], a.add, a.H, a.N, a.H)))
    return cudaErrorInvalidValue;
  return launch<kOut, 0>(m, p, pairs, s);
}

template <int ACT>
cudaError_t backward(const SharedArgs& a, cudaStream_t s, int* launches) {
  cudaError_t err = cudaSuccess;
  // da = dy W2; dg, du and h from the checkpoint
  Maps m{};
  MmaParams p{};
  p.err = a.err;
  p.problems = 1;
  p.pr[0] = problem(a.N, a.I, a.H);
  double cost;
  p.split = pick_split<kGatedBwd, ACT>(p.pr, 1, 16, &cost, &err);
  if (p.split <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  int pairs = max_clusters<kGatedBwd, ACT, false>(1, &err);
  p.ck_in = a.ck;
  p.sf_in = a.ck_sf;
  if (!operand_map(&m.a[0], a.dy, a.H, a.N, false) || !operand_map(&m.b[0], a.w2, a.I, a.H, true) ||
      !out_map(&m.o[0], a.dpre, a.I, a.N, 2 * (int64_t)a.I) ||
      !out_map(&m.x[0], a.dpre + a.I, a.I, a.N, 2 * (int64_t)a.I) || !out_map(&m.o[1], a.h, a.I, a.N, a.I))
    return cudaErrorInvalidValue;
  err = launch<kGatedBwd, ACT>(m, p, pairs, s);
  if (err != cudaSuccess) return err;
  // dx = [dg du] W13, dW13 = [dg du]^T x and dW2 = dy^T h in one launch
  pairs = max_clusters<kGrads, 0, false>(1, &err);
  if (pairs <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  m = Maps{};
  p = MmaParams{};
  p.err = a.err;
  Problem dx = problem(a.N, a.H, 2 * (int64_t)a.I);
  dx.has_add = a.add != nullptr;
  Problem dw[2] = {problem(2 * a.I, a.H, a.N, true), problem(a.H, a.I, a.N, true)};
  dw[0].f32 = dw[1].f32 = a.grad_f32;
  const bool dx_first = 2 * (int64_t)a.I >= a.N;
  int ix = dx_first ? 0 : 2, i13 = dx_first ? 1 : 0, i2 = dx_first ? 2 : 1;
  p.pr[ix] = dx;
  p.pr[i13] = dw[0];
  p.pr[i2] = dw[1];
  p.problems = 3;
  p.split = pick_split<kGrads, 0>(p.pr, 3, 32, &cost, &err);
  if (p.split <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  // few tokens: dx's few tiles of a long contraction would outlast all others, so they
  // are shared out in a launch of their own
  double alone = 0;
  const int split = pick_split<kGrads, 0>(&dx, 1, 16, &alone, &err);
  if (split <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  if (split > 1 && alone + kLaunchCost + pick_width(dw, 2, pairs, false, true, 32) < cost) {
    MmaParams o{};
    o.err = a.err;
    o.problems = 1;
    o.pr[0] = dx;
    o.split = split;
    if (!operand_map(&m.a[0], a.dpre, 2 * (int64_t)a.I, a.N, false) ||
        !operand_map(&m.b[0], a.w13, a.H, 2 * (int64_t)a.I, true) || !out_map(&m.o[0], a.dx, a.H, a.N, a.H) ||
        (a.add && !out_map(&m.x[0], a.add, a.H, a.N, a.H)))
      return cudaErrorInvalidValue;
    err = launch<kGrads, 0>(m, o, pairs, s);
    if (err != cudaSuccess) return err;
    ++*launches;
    m = Maps{};
    p.pr[0] = dw[0];
    p.pr[1] = dw[1];
    p.problems = 2;
    p.split = 1;
    ix = -1;
    i13 = 0;
    i2 = 1;
  }
  auto grad_map = [&](CUtensorMap* t, void* d, int64_t cols, int64_t rows) {
    return a.grad_f32 ? map2d(t, d, cols, rows, cols, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)
                      : out_map(t, d, cols, rows, cols);
  };
  if (ix >= 0 && (!operand_map(&m.a[ix], a.dpre, 2 * (int64_t)a.I, a.N, false) ||
                  !operand_map(&m.b[ix], a.w13, a.H, 2 * (int64_t)a.I, true) ||
                  !out_map(&m.o[ix], a.dx, a.H, a.N, a.H) || (a.add && !out_map(&m.x[ix], a.add, a.H, a.N, a.H))))
    return cudaErrorInvalidValue;
  if (!operand_map(&m.a[i13], a.dpre, 2 * (int64_t)a.I, a.N, true) ||
      !operand_map(&m.b[i13], a.x, a.H, a.N, true) || !grad_map(&m.o[i13], a.dw13, a.H, 2 * (int64_t)a.I) ||
      !operand_map(&m.a[i2], a.dy, a.H, a.N, true) || !operand_map(&m.b[i2], a.h, a.I, a.N, true) ||
      !grad_map(&m.o[i2], a.dw2, a.I, a.H))
    return cudaErrorInvalidValue;
  return launch<kGrads, 0>(m, p, pairs, s);
}

}  // namespace

int launch_shared_forward(const SharedArgs& a, cudaStream_t s) {
  // up to 512 tokens the pairs' tiles of 256 rows are too few to fill the SMs: 400
  // tokens, 7168 x 2048: 55 us against 60; 2048 x 768: 19 against 23; from 700 on
  // the pairs are faster on wide layers (71 against 97)
  if (a.N <= 512) return launch_shared_forward_few(a, s);
  const cudaError_t err = a.activation ? forward<1>(a, s) : forward<0>(a, s);
  return err != cudaSuccess ? -(int)err : 2;
}

int launch_shared_backward(const SharedArgs& a, cudaStream_t s) {
  int launches = 2;
  const cudaError_t err = a.activation ? backward<1>(a, s, &launches) : backward<0>(a, s, &launches);
  return err != cudaSuccess ? -(int)err : launches;
}

}  // namespace moe
