// The shared expert's forward for few tokens on the 5th-generation tensor cores.
//
// With few tokens the time is that of streaming the weights, so the weights are
// the MMA's 128 rows and the tokens its columns (N = 16 .. 128): a tile costs no
// more MMA or shared memory than its tokens need. The few tiles there are would
// leave most SMs idle, so S CTAs of a cluster split a tile's contraction; each
// leaves its sums [token][row] in its shared memory, and after a cluster barrier
// the CTAs share out the tokens' outputs, adding the S parts in rank order
// through distributed shared memory (no atomics, no workspace, no second launch).
//
//   gated   rows 0-63 of a tile are gate rows of 64 features, rows 64-127 their up
//           rows; h = act(g) u, and the 8-bit checkpoint of g, u if asked for
//   out     y = h W2^T (+ add)
//
// Warps: 0 = TMA producer, 1 = TMEM allocator and MMA issuer, 2-5 = TMEM reads;
// all of them share the outputs. The second product's weights do not depend on
// the first one, so its ring is filled before it waits for the first kernel.
#include "act.cuh"
#include "moe_internal.h"
#include "ptx.cuh"
#include "shared_internal.h"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 192;
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr int kMaxTok = 128;  // of a tile
// A ring of about 100 KB leaves room for a second block on the SM, of this kernel or of
// the next, which fills its own while this one runs.
constexpr uint32_t kRing = 104u << 10;
constexpr int kMaxStages = kRing / (kABytes + 16 * kBK * 2);  // of the fewest tokens
// the sums of a tile take the place of its stages
static_assert(kRing - (kABytes + kMaxTok * kBK * 2) >= kMaxTok * kBM * 4, "the ring holds the sums");

struct FewParams {
  int N, M;          // tokens; output columns (gated: features)
  int n_tok;         // tokens of a tile (a multiple of 16, at most kMaxTok)
  int m_tiles;
  int second;        // rows from a tile's first 64 weight rows to its second 64
  int k_tiles;
  int stages;
  uint32_t tmem_cols;
  int early;         // the weights may be read before the previous kernel has finished
  const uint16_t* add;  // out: [N,M] or null
  uint16_t* out;     // [N,M]
  uint8_t* ck;       // gated: [N,2M] codes and [N,2M/32] bytes, or null
  uint8_t* sf;
  uint32_t* err;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// The sum, in rank order, of the four values at this shared-memory address in the S
// CTAs of the cluster; all the reads are under way before the first is needed.
template <int S>
__device__ __forceinline__ float4 sum_ranks(uint32_t at) {
  float4 a[S];
#pragma unroll
  for (int s = 0; s < S; ++s) a[s] = ld_cluster_f4(mapa_shared(at, (uint32_t)s));
#pragma unroll
  for (int s = 1; s < S; ++s) {
    a[0].x += a[s].x;
    a[0].y += a[s].y;
    a[0].z += a[s].z;
    a[0].w += a[s].w;
  }
  return a[0];
}
__device__ __forceinline__ float4 sum_ranks(uint32_t at, uint32_t S) {
  switch (S) {
    case 8: return sum_ranks<8>(at);
    case 7: return sum_ranks<7>(at);
    case 6: return sum_ranks<6>(at);
    case 5: return sum_ranks<5>(at);
    case 4: return sum_ranks<4>(at);
    case 3: return sum_ranks<3>(at);
    case 2: return sum_ranks<2>(at);
    default: return sum_ranks<1>(at);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four consecutive values of a row as MX codes; the eight lanes of a 32-value
// block find its largest magnitude together. A block that holds an infinity or a
// NaN gets the scale byte 255, which reads as NaN.
__device__ __forceinline__ void keep4(const float4& v, bool in, uint8_t* ck, uint8_t* sf, bool first) {
  uint32_t top = max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                     max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (!in) return;
  const bool finite = top < 0x7F800000u;
  const int s = finite ? mx_block_exponent(__uint_as_float(top)) : 0;
  const float f = pow2_neg(s);
  *reinterpret_cast<uint32_t*>(ck) = e4m3x2(v.x * f, v.y * f) | (e4m3x2(v.z * f, v.w * f) << 16);
  if (first) *sf = finite ? (uint8_t)(s + 127) : (uint8_t)255;
}

template <bool GATED, int ACT>
__global__ void __launch_bounds__(kThreads)
    shared_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t tmem_base_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_ctarank();
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = kABytes + (uint32_t)p.n_tok * 128u;
  const int tile = blockIdx.x / S, mt = tile % p.m_tiles, nt = tile / p.m_tiles;
  const int row0 = mt * (GATED ? 64 : kBM), tok0 = nt * p.n_tok;
  const int k0 = (int)((int64_t)rank * p.k_tiles / S), k1 = (int)((int64_t)(rank + 1) * p.k_tiles / S);
  const int kt = k1 - k0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(&done_bar), 1);
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_base_s), p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
    auto load_w = [&](int i) {
      if (lane == 0) {
        const uint32_t s = (uint32_t)(i % p.stages), bar = smem_u32(&full_bar[s]);
        const uint32_t a = sbase + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_load_2d(a, &tmW, (k0 + i) * kBK, row0, bar, stream);
        tma_load_2d(a + kABytes / 2, &tmW, (k0 + i) * kBK, row0 + p.second, bar, stream);
      }
    };
    auto load_x = [&](int i) {
      if (lane == 0) {
        const uint32_t s = (uint32_t)(i % p.stages);
        tma_load_2d(sbase + s * stage_bytes + kABytes, &tmX, (k0 + i) * kBK, tok0,
                    smem_u32(&full_bar[s]), keep);
      }
    };
    const int ahead = min(p.stages, kt);
    if (p.early)
      for (int i = 0; i < ahead; ++i) load_w(i);
    griddep_wait();
    griddep_launch_dependents();
    for (int i = 0; i < ahead; ++i) {
      if (!p.early) load_w(i);
      load_x(i);
    }
    int i = ahead;
    for (; i < kt; ++i) {
      if (!mbar_wait_warp(smem_u32(&empty_bar[i % p.stages]), (uint32_t)(i / p.stages - 1) & 1u, p.err,
                          kErrWaitEmpty))
        break;
      load_w(i);
      load_x(i);
      __syncwarp();
    }
    // the block leaves with no copy under way, after a wait that ran out too
    for (int j = max(0, i - p.stages); j < i; ++j)
      if (!mbar_wait_warp(smem_u32(&full_bar[j % p.stages]), (uint32_t)(j / p.stages) & 1u, p.err, kErrWaitFull))
        break;
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16_f32(kBM, p.n_tok);
    for (int i = 0; i < kt; ++i) {
      const uint32_t s = (uint32_t)(i % p.stages);
      if (!mbar_wait_warp(smem_u32(&full_bar[s]), (uint32_t)(i / p.stages) & 1u, p.err, kErrWaitFull)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t a0 = sbase + s * stage_bytes, b0 = a0 + kABytes;
#pragma unroll
        for (uint32_t kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, sdesc_sw128(a0 + kk * 32u), sdesc_sw128(b0 + kk * 32u), idesc, (i | (int)kk) != 0);
        umma_commit(smem_u32(&empty_bar[s]));
      }
      __syncwarp();
    }
    // also after an abort: the outputs are then of no use, and the error word says so
    if (lane == 0) umma_commit(smem_u32(&done_bar));
    __syncwarp();
    griddep_wait();
  } else {
    // ------------------------------------------------------------ sums to shared memory
    griddep_wait();
    const int q = warp & 3, row = q * 32 + lane;
    const bool ok = mbar_wait_warp(smem_u32(&done_bar), 0, p.err, kErrWaitAccum);
    if (ok) {
      tc_fence_after();
      const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
      const int live = min(p.n_tok, p.N - tok0);
      for (int c = 0; c < live; c += 16) {
        uint32_t v[16];
        tmem_ld16(tl + (uint32_t)c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)  // the ring is free: every MMA has read its stage
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(sbase + (uint32_t)(((c + j) * kBM + row) * 4)), "r"(v[j])
                       : "memory");
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (S > 1) cluster_sync_all();
  // ------------------------------------------------------------ outputs
  // item: four rows of one token's sums (gated: the gate rows, and the same up rows)
  constexpr int kPer = GATED ? 16 : 32;
  const int items = min(p.n_tok, p.N - tok0) * kPer;
  for (int base = (int)rank * kThreads; base < items; base += (int)S * kThreads) {
    const int i = base + (int)threadIdx.x, tok = i / kPer, r4 = (i % kPer) * 4;
    const bool in = i < items && row0 + r4 < p.M;
    float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
    if (in) {
      const uint32_t at = sbase + (uint32_t)((tok * kBM + r4) * 4);
      g = sum_ranks(at, S);
      if (GATED) u = sum_ranks(at + 64u * 4u, S);
    }
    const size_t row = (size_t)(tok0 + tok), out = row * p.M + row0 + r4;
    if (GATED) {
      if (p.ck) {  // kPer divides 32 twice: eight lanes hold one block
        uint8_t* sf = p.sf + row * (p.M / 16) + (row0 + r4) / 32;
        keep4(g, in, p.ck + 2 * row * p.M + row0 + r4, sf, (lane & 7) == 0);
        keep4(u, in, p.ck + (2 * row + 1) * p.M + row0 + r4, sf + p.M / 32, (lane & 7) == 0);
      }
      if (in)
        *reinterpret_cast<uint2*>(p.out + out) =
            make_uint2(pack_bf16(act_fwd<ACT>(g.x) * u.x, act_fwd<ACT>(g.y) * u.y),
                       pack_bf16(act_fwd<ACT>(g.z) * u.z, act_fwd<ACT>(g.w) * u.w));
    } else if (in) {
      if (p.add) {
        const uint2 a = *reinterpret_cast<const uint2*>(p.add + out);
        g.x += __uint_as_float(a.x << 16);
        g.y += __uint_as_float(a.x & 0xFFFF0000u);
        g.z += __uint_as_float(a.y << 16);
        g.w += __uint_as_float(a.y & 0xFFFF0000u);
      }
      *reinterpret_cast<uint2*>(p.out + out) = make_uint2(pack_bf16(g.x, g.y), pack_bf16(g.z, g.w));
    }
  }
  if (S > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// Clusters of S CTAs of this kernel that run at once (0 where one does not fit), once per
// device: two CTAs an SM (the query counts one, since the kernel allocates tensor memory).
template <bool GATED, int ACT>
int max_clusters(int S, cudaError_t* err) {
  static DeviceOnce once[9];
  int n = 0;
  *err = count_per_device(once[S], &n, [&](int, int* v) {
    auto* k = shared_few_kernel<GATED, ACT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing + 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(v, k, &cfg);
  });
  return 2 * n;
}

template <bool GATED, int ACT>
cudaError_t launch(const void* w, int64_t w_rows, const void* x, int K, FewParams p, cudaStream_t s) {
  p.m_tiles = (p.M + (GATED ? 63 : 127)) / (GATED ? 64 : 128);
  p.k_tiles = (K + kBK - 1) / kBK;
  // Tokens of a tile: 64 while the tiles are few enough that clusters still split each:
  // their sums pass through shared memory in half the time (128 tokens, 2048 x 768: 17.4
  // -> 14.9 us); else each further tile reads the weights again (200 tokens, 7168 x 2048:
  // 45.5 us in tiles of 64, 35.3 in tiles of 128). Short contractions, which are not
  // split: fewer tokens instead (100 tokens, 304 x 256: 11.6 us in tiles of 64, 8.6 of 16;
  // 64 tokens, 2048 x 768: 11.3 and 13.0).
  const int parts = p.k_tiles < 6 ? 1 : p.k_tiles < 15 ? p.k_tiles / 3 : 5;
  int tok = parts == 1 ? 16 : parts < 4 ? 32 : 64;
  while (tok < kMaxTok && p.m_tiles * ((p.N + tok - 1) / tok) > 300 / parts) tok *= 2;
  const int n_tiles = (p.N + tok - 1) / tok;
  p.n_tok = ((p.N + n_tiles - 1) / n_tiles + 15) / 16 * 16;
  p.tmem_cols = 32;
  while ((int)p.tmem_cols < p.n_tok) p.tmem_cols *= 2;
  const int tiles = p.m_tiles * n_tiles;
  // CTAs a tile: the most whose clusters all run at once, with three stages each at
  // least (500 tokens, 4096 x 1408, gated: two 39 us, three 37, four 46: a second turn)
  int S = p.k_tiles / 3 < 8 ? p.k_tiles / 3 : 8;
  if (S < 1) S = 1;
  for (;; --S) {  // the query also asks for the shared memory
    cudaError_t err = cudaSuccess;
    const int most = max_clusters<GATED, ACT>(S, &err);
    if (err != cudaSuccess) return err;
    if (S == 1 || tiles <= most) break;
  }
  const uint32_t stage = kABytes + (uint32_t)p.n_tok * 128u;
  p.stages = (int)(kRing / stage);
  CUtensorMap tw, tx;
  if (!make_map(&tw, w, (uint64_t)K, (uint64_t)w_rows, 64, 64) ||
      !make_map(&tx, x, (uint64_t)K, (uint64_t)p.N, 64, (uint32_t)p.n_tok))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (uint32_t)p.stages * stage + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, shared_few_kernel<GATED, ACT>, tw, tx, p);
}

}  // namespace

int launch_shared_forward_few(const SharedArgs& a, cudaStream_t s) {
  FewParams p{};
  p.err = a.err;
  p.N = a.N;
  p.M = a.I;
  p.second = a.I;
  p.out = a.h;
  p.ck = a.ck;
  p.sf = a.ck_sf;
  cudaError_t err = a.activation ? launch<true, 1>(a.w13, 2 * (int64_t)a.I, a.x, a.H, p, s)
                                 : launch<true, 0>(a.w13, 2 * (int64_t)a.I, a.x, a.H, p, s);
  if (err != cudaSuccess) return -(int)err;
  p = FewParams{};
  p.err = a.err;
  p.N = a.N;
  p.M = a.H;
  p.second = 64;
  p.early = 1;
  p.add = a.add;
  p.out = a.y;
  err = launch<false, 0>(a.w2, a.H, a.h, a.I, p, s);
  return err != cudaSuccess ? -(int)err : 2;
}

}  // namespace moe
