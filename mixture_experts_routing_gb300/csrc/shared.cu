// The shared expert's contractions on the 5th-generation tensor cores.
//
// D[m, n] = sum_k A[m, k] B[n, k], one launch per contraction:
//   gated      D = x W13^T      epilogue h = act(g) u, 8-bit checkpoint of g, u
//   out        D = h W2^T, or [dg du] W13   epilogue (+ add), bf16
//   gated bwd  D = dy W2        epilogue dg, du and h from the checkpoint
//   grad       D = [dg du]^T x, or dy^T h   bf16 or f32
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

enum Epi { kGated = 0, kOut = 1, kGatedBwd = 2, kGradF32 = 3 };

struct MmaParams {
  int M, N;              // output rows and columns (gated: columns of h)
  int k_tiles;
  int m_tiles, n_tiles;  // tiles of 256 rows; of 256 columns (gated: 128 features)
  int b_pair_off;        // rows of B between the CTAs' halves: 128, or I (gated)
  int has_add;           // kOut
  const uint8_t* ck_in;  // kGatedBwd: [M,2N] codes, [M,2N/32] bytes
  const uint8_t* sf_in;
  uint8_t* ck;           // kGated: the same as outputs, or null
  uint8_t* sf;
  uint32_t* err;
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

// Where 16-byte piece c of row r lies in a staged box of 64-byte rows (32 bf16
// columns, 64-byte swizzle).
__device__ __forceinline__ uint32_t at64(int r, int c) {
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// This lane's row of 32 bf16 values into a staged box.
__device__ __forceinline__ void stage_row(uint32_t buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(buf + at64(lane, c), pack_bf16(v[8 * c], v[8 * c + 1]),
                 pack_bf16(v[8 * c + 2], v[8 * c + 3]), pack_bf16(v[8 * c + 4], v[8 * c + 5]),
                 pack_bf16(v[8 * c + 6], v[8 * c + 7]));
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

// Tile t: M tiles in bands of kBand, walked M first within a band.
__device__ __forceinline__ void tile_of(const MmaParams& p, int t, int& m, int& n) {
  const int per = kBand * p.n_tiles;
  const int band = t / per, r = t - band * per;
  const int rows = min(kBand, p.m_tiles - band * kBand);
  n = r / rows;
  m = band * kBand + (r - n * rows);
}

template <int EPI, int ACT, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
    shared_mma_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ CUtensorMap tmO2,
                      const __grid_constant__ CUtensorMap tmO3, const MmaParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t tmem_full_bar[2];
  __shared__ __align__(8) uint64_t tmem_empty_bar[2];
  __shared__ __align__(8) uint64_t add_bar[kEpiWarps][2];
  __shared__ uint32_t tmem_base_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tiles = p.m_tiles * p.n_tiles;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

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
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
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
      int m, n;
      tile_of(p, t, m, n);
      const int am = m * 2 * kBM + (int)crank * kBM;
      const int bn = n * (EPI == kGated ? kBM : 2 * kBM) + (int)crank * p.b_pair_off;
      for (int kt = 0; kt < p.k_tiles; ++kt, ++g) {
        const uint32_t s = g % kStages, u = g / kStages;
        if (u > 0 && !mbar_wait_cluster_warp(smem_u32(&empty_bar[s]), (u - 1u) & 1u, p.err,
                                             kErrWaitEmpty)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t bar = mapa_shared(smem_u32(&full_bar[s]), 0);
          if (crank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), 2 * kStageBytes);
          const uint32_t a = sbase + s * kStageBytes, b = a + kOpBytes;
          const int k = kt * kBK;
          if (AMN) {
            tma_load_2d_pair(a, &tmA, am, k, bar);
            tma_load_2d_pair(a + kOpBytes / 2, &tmA, am + 64, k, bar);
          } else {
            tma_load_2d_pair(a, &tmA, k, am, bar);
          }
          if (BMN) {
            tma_load_2d_pair(b, &tmB, bn, k, bar);
            tma_load_2d_pair(b + kOpBytes / 2, &tmB, bn + 64, k, bar);
          } else {
            tma_load_2d_pair(b, &tmB, k, bn, bar);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (crank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(2 * kBM, 2 * kBM) | (AMN ? kIdescAMnMajor : 0u) |
                                 (BMN ? kIdescBMnMajor : 0u);
      // 16 contraction values: 32 bytes along a K-major row, 16 rows of an MN-major tile
      constexpr uint32_t a_step = AMN ? 2048u : 32u, b_step = BMN ? 2048u : 32u;
      uint32_t g = 0, tc = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++tc) {
        const uint32_t b = tc & 1u, bu = tc >> 1;
        if (bu > 0 && !mbar_wait_cluster_warp(smem_u32(&tmem_empty_bar[b]), (bu - 1u) & 1u, p.err,
                                              kErrWaitAccum))
          break;
        tc_fence_after();
        for (int kt = 0; kt < p.k_tiles; ++kt, ++g) {
          const uint32_t s = g % kStages, u = g / kStages;
          if (!mbar_wait_cluster_warp(smem_u32(&full_bar[s]), u & 1u, p.err, kErrWaitFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t a0 = sbase + s * kStageBytes, b0 = a0 + kOpBytes;
#pragma unroll
            for (uint32_t kk = 0; kk < kBK / 16; ++kk)
              umma_bf16_pair(tmem + b * 256u,
                             AMN ? sdesc_sw128_mn(a0 + kk * a_step) : sdesc_sw128(a0 + kk * a_step),
                             BMN ? sdesc_sw128_mn(b0 + kk * b_step) : sdesc_sw128(b0 + kk * b_step),
                             idesc, (kt | (int)kk) != 0);
            umma_commit_pair(smem_u32(&empty_bar[s]), 3);
          }
          __syncwarp();
        }
        if (lane == 0) umma_commit_pair(smem_u32(&tmem_full_bar[b]), 3);  // also after an abort
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    const uint32_t buf0 = sbase + kStages * kStageBytes + (uint32_t)ew * kEpiBytes;
    uint32_t tc = 0, adds[2] = {0, 0};  // adds: phases of this warp's add barriers so far
    for (int t = pair; t < tiles; t += pairs, ++tc) {
      int m, n;
      tile_of(p, t, m, n);
      const uint32_t b = tc & 1u, bu = tc >> 1;
      const int row0 = m * 2 * kBM + (int)crank * kBM + q * 32, row = row0 + lane;
      const int col0 = n * (EPI == kGated ? kBM : 2 * kBM) + half * (EPI == kGated ? kBM / 2 : kBM);
      const uint32_t tl = tmem + b * 256u + ((uint32_t)(q * 32) << 16) +
                          (uint32_t)(half * (EPI == kGated ? kBM / 2 : kBM));
      // 32-column chunks of this warp that hold output values
      const int nch = row0 < p.M ? max(0, min(EPI == kGated ? 2 : 4, (p.N - col0 + 31) / 32)) : 0;
      const bool add = EPI == kOut && p.has_add;
      auto load_add = [&](int c) {
        if (lane == 0) {
          const uint32_t bar = smem_u32(&add_bar[ew][c & 1]);
          mbar_arrive_expect_tx(bar, 2048);
          tma_load_2d_pair(buf0 + (uint32_t)(c & 1) * 2048u, &tmO2, col0 + 32 * c, row0, bar);
        }
      };
      if (add && nch > 0) {  // under the tile's MMAs: the first two chunks of what is added
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        load_add(0);
        if (nch > 1) load_add(1);
      }
      if (!mbar_wait_cluster_warp(smem_u32(&tmem_full_bar[b]), bu & 1u, p.err, kErrWaitAccum)) break;
      tc_fence_after();
#pragma unroll 2
      for (int c = 0; c < nch; ++c) {
        const int col = col0 + 32 * c;
        const uint32_t buf = buf0 + (uint32_t)(c & 1) * 2048u;
        float v[32];
        tmem_row32(tl + 32u * (uint32_t)c, v);
        if constexpr (EPI == kOut) {
          if (add) {
            const uint32_t use = adds[c & 1]++;
            if (!mbar_wait_warp(smem_u32(&add_bar[ew][c & 1]), use & 1u, p.err, kErrWaitAccum)) break;
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
          store_box(&tmO, buf, col, row0, lane);
          if (add && c + 2 < nch) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            load_add(c + 2);
          }
        } else if constexpr (EPI == kGradF32) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 128-byte rows, 128-byte swizzle
            st_shared_v4(buf0 + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) << 4)),
                         __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                         __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
          store_box(&tmO, buf0, col, row0, lane);
        } else if constexpr (EPI == kGated) {
          float u[32];
          tmem_row32(tl + (uint32_t)kBM + 32u * (uint32_t)c, u);
          if (p.ck && row < p.M) {
            const size_t at = (size_t)row * 2 * p.N + col, sa = (size_t)row * (p.N / 16) + col / 32;
            keep_block(v, p.ck + at, p.sf + sa);
            keep_block(u, p.ck + at + p.N, p.sf + sa + p.N / 32);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = act_fwd<ACT>(v[j]) * u[j];
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          stage_row(buf, lane, v);
          store_box(&tmO, buf, col, row0, lane);
        } else {  // kGatedBwd
          uint4 gc[2] = {}, uc[2] = {};
          float fg = 0.0f, fu = 0.0f;
          if (row < p.M) {
            const size_t at = (size_t)row * 2 * p.N + col, sa = (size_t)row * (p.N / 16) + col / 32;
            gc[0] = reinterpret_cast<const uint4*>(p.ck_in + at)[0];
            gc[1] = reinterpret_cast<const uint4*>(p.ck_in + at)[1];
            uc[0] = reinterpret_cast<const uint4*>(p.ck_in + at + p.N)[0];
            uc[1] = reinterpret_cast<const uint4*>(p.ck_in + at + p.N)[1];
            fg = e8m0_value(p.sf_in[sa]);
            fu = e8m0_value(p.sf_in[sa + p.N / 32]);
          }
          const uint32_t gw[8] = {gc[0].x, gc[0].y, gc[0].z, gc[0].w, gc[1].x, gc[1].y, gc[1].z, gc[1].w};
          const uint32_t uw[8] = {uc[0].x, uc[0].y, uc[0].z, uc[0].w, uc[1].x, uc[1].y, uc[1].z, uc[1].w};
          float du[32], h[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t sh = (j & 1) * 16;
            const float2 g2 = e4m3x2_value((gw[j >> 1] >> sh) & 0xFFFFu);
            const float2 u2 = e4m3x2_value((uw[j >> 1] >> sh) & 0xFFFFu);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float g = (i ? g2.y : g2.x) * fg, u = (i ? u2.y : u2.x) * fu;
              const float da = v[2 * j + i];
              const float k = act_core<ACT>(g);
              const float a = g * k;
              v[2 * j + i] = da * u * act_grad_core<ACT>(g, k);
              du[2 * j + i] = da * a;
              h[2 * j + i] = a * u;
            }
          }
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          stage_row(buf0, lane, v);
          store_box(&tmO, buf0, col, row0, lane);
          stage_row(buf0 + 2048u, lane, du);
          store_box(&tmO2, buf0 + 2048u, col, row0, lane);
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          stage_row(buf0, lane, h);
          store_box(&tmO3, buf0, col, row0, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (crank == 0)
          mbar_arrive(smem_u32(&tmem_empty_bar[b]));
        else
          mbar_arrive_remote_relaxed(mapa_shared(smem_u32(&tmem_empty_bar[b]), 0));
      }
    }
    if (lane == 0) bulk_wait_all();
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

// An operand [rows, cols]: K-major boxes of 64 k x 128 rows, or (mn) MN-major
// boxes of 64 columns x 64 k.
bool operand_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, bool mn) {
  return map2d(m, base, cols, rows, cols, 64, mn ? 64 : 128, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool out_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch) {
  return map2d(m, base, cols, rows, pitch, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// Pairs resident at once, and the kernel's shared-memory opt-in, once per device.
template <int EPI, int ACT, bool AMN, bool BMN>
int max_pairs(cudaError_t* err) {
  static DeviceOnce once;
  int n = 0;
  *err = once_per_device(once, &n, [](int, int* v) {
    auto* k = shared_mma_kernel<EPI, ACT, AMN, BMN>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(v, k, &cfg);
  });
  return *err == cudaSuccess ? n : 0;
}

template <int EPI, int ACT, bool AMN, bool BMN>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                   const CUtensorMap& o2, const CUtensorMap& o3, MmaParams p, int64_t K,
                   cudaStream_t s) {
  p.k_tiles = (int)((K + kBK - 1) / kBK);
  p.m_tiles = (p.M + 2 * kBM - 1) / (2 * kBM);
  const int bn = EPI == kGated ? kBM : 2 * kBM;
  p.n_tiles = (p.N + bn - 1) / bn;
  if ((int64_t)p.m_tiles * p.n_tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  cudaError_t err = cudaSuccess;
  const int pairs = max_pairs<EPI, ACT, AMN, BMN>(&err);
  if (pairs <= 0) return err != cudaSuccess ? err : cudaErrorUnknown;
  const int n = p.m_tiles * p.n_tiles < pairs ? p.m_tiles * p.n_tiles : pairs;
  return launch_pdl_pairs(shared_mma_kernel<EPI, ACT, AMN, BMN>, dim3(2 * n), dim3(kThreads),
                          kSmemBytes, s, a, b, o, o2, o3, p);
}

}  // namespace

int launch_shared_forward(const SharedArgs& a, cudaStream_t s) {
  if (a.N <= 256) return launch_shared_forward_few(a, s);
  CUtensorMap x, w13, w2, h_in, h_out, y, add{};
  if (!operand_map(&x, a.x, a.H, a.N, false) || !operand_map(&w13, a.w13, a.H, 2 * a.I, false) ||
      !operand_map(&h_in, a.h, a.I, a.N, false) || !operand_map(&w2, a.w2, a.I, a.H, false) ||
      !out_map(&h_out, a.h, a.I, a.N, a.I) || !out_map(&y, a.y, a.H, a.N, a.H) ||
      (a.add && !out_map(&add, a.add, a.H, a.N, a.H)))
    return -1;
  MmaParams p{};
  p.err = a.err;
  p.M = a.N;
  p.N = a.I;
  p.b_pair_off = a.I;
  p.ck = a.ck;
  p.sf = a.ck_sf;
  cudaError_t err = a.activation ? launch<kGated, 1, false, false>(x, w13, h_out, h_out, h_out, p, a.H, s)
                                 : launch<kGated, 0, false, false>(x, w13, h_out, h_out, h_out, p, a.H, s);
  if (err != cudaSuccess) return -(int)err;
  p = MmaParams{};
  p.err = a.err;
  p.M = a.N;
  p.N = a.H;
  p.b_pair_off = kBM;
  p.has_add = a.add != nullptr;
  err = launch<kOut, 0, false, false>(h_in, w2, y, a.add ? add : y, y, p, a.I, s);
  return err != cudaSuccess ? -(int)err : 2;
}

int launch_shared_backward(const SharedArgs& a, cudaStream_t s) {
  CUtensorMap dy, w2, dg, du, h, dpre, w13, dx, add{}, dpre_t, x_t, dy_t, h_t, dw13, dw2;
  const CUtensorMapDataType f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const bool f = a.grad_f32 != 0;
  if (!operand_map(&dy, a.dy, a.H, a.N, false) || !operand_map(&w2, a.w2, a.I, a.H, true) ||
      !out_map(&dg, a.dpre, a.I, a.N, 2 * a.I) || !out_map(&du, a.dpre + a.I, a.I, a.N, 2 * a.I) ||
      !out_map(&h, a.h, a.I, a.N, a.I) || !operand_map(&dpre, a.dpre, 2 * a.I, a.N, false) ||
      !operand_map(&w13, a.w13, a.H, 2 * a.I, true) || !out_map(&dx, a.dx, a.H, a.N, a.H) ||
      (a.add && !out_map(&add, a.add, a.H, a.N, a.H)) ||
      !operand_map(&dpre_t, a.dpre, 2 * a.I, a.N, true) || !operand_map(&x_t, a.x, a.H, a.N, true) ||
      !operand_map(&dy_t, a.dy, a.H, a.N, true) || !operand_map(&h_t, a.h, a.I, a.N, true) ||
      !(f ? map2d(&dw13, a.dw13, a.H, 2 * a.I, a.H, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B, f32, 4)
          : out_map(&dw13, a.dw13, a.H, 2 * a.I, a.H)) ||
      !(f ? map2d(&dw2, a.dw2, a.I, a.H, a.I, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B, f32, 4)
          : out_map(&dw2, a.dw2, a.I, a.H, a.I)))
    return -1;
  MmaParams p{};  // da = dy W2; dg, du and h from the checkpoint
  p.err = a.err;
  p.M = a.N;
  p.N = a.I;
  p.b_pair_off = kBM;
  p.ck_in = a.ck;
  p.sf_in = a.ck_sf;
  cudaError_t err = a.activation ? launch<kGatedBwd, 1, false, true>(dy, w2, dg, du, h, p, a.H, s)
                                 : launch<kGatedBwd, 0, false, true>(dy, w2, dg, du, h, p, a.H, s);
  if (err != cudaSuccess) return -(int)err;
  p.ck_in = p.sf_in = nullptr;
  p.N = a.H;  // dx = [dg du] W13
  p.has_add = a.add != nullptr;
  err = launch<kOut, 0, false, true>(dpre, w13, dx, a.add ? add : dx, dx, p, 2 * (int64_t)a.I, s);
  if (err != cudaSuccess) return -(int)err;
  p.has_add = 0;
  p.M = 2 * a.I;  // dW13 = [dg du]^T x
  err = f ? launch<kGradF32, 0, true, true>(dpre_t, x_t, dw13, dw13, dw13, p, a.N, s)
          : launch<kOut, 0, true, true>(dpre_t, x_t, dw13, dw13, dw13, p, a.N, s);
  if (err != cudaSuccess) return -(int)err;
  p.M = a.H;  // dW2 = dy^T h
  p.N = a.I;
  err = f ? launch<kGradF32, 0, true, true>(dy_t, h_t, dw2, dw2, dw2, p, a.N, s)
          : launch<kOut, 0, true, true>(dy_t, h_t, dw2, dw2, dw2, p, a.N, s);
  return err != cudaSuccess ? -(int)err : 4;
}

}  // namespace moe
