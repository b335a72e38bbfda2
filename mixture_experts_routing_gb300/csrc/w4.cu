// Products with 4-bit weights and group scales, for the few tokens of a decode
// step: w[r,c] = scale[r, c/group] * (nibble[r,c] - 8).
//
//   matvec    y[t,:] = w x[t,:]
//   experts   h[t,k,:] = act(W13g[e] x_t) * (W13u[e] x_t), e = topk_ids[t,k]
//             y[t,:] = add[t,:] + sum_k p[t,k] W2[e] h[t,k,:]
//
// The time is that of reading the codes once, so the kernels are built around
// that stream. A warp takes 16 rows. The codes become the A operand of mma.sync
// m16n8k16: the products need 8 columns for 1 to 8 tokens, and the opened codes are
// in registers, where tcgen05.mma takes no operand from. A mask and an OR put four
// bits into the mantissa of bf16 128 + code, one subtraction makes it code - 8,
// exactly. The order of the columns within a group is free as long as x follows
// it, so no weight is moved between lanes. The sums of one group are scaled in
// fp32 and added up in fp32. Warps that share a row tile split its columns and add
// their parts in a fixed order.
//
// Experts, and one token's matvec (Rows): a lane loads 16 bytes of its two rows
// straight into registers, four blocks of 128 columns ahead; x is laid out in shared
// memory once per block of threads. Several tokens that share experts: one small kernel groups the
// routes by expert, the blocks of the products share out the rows of the experts and
// multiply each by all its routes, or 2 to 8 of them at a time (an expert's weights
// come from HBM once), and a last kernel adds up each token's routes.
// Several tokens' matvec (Stream): codes, scales and x come through each warp's own
// ring of shared-memory stages.
#include "act.cuh"
#include "moe_internal.h"
#include "ptx.cuh"
#include "shared_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kShare = 128;       // columns are dealt out to warps in multiples of these
constexpr int kMaxRoutes = kW4MaxRoutes;  // N*K, at most: the grouping kernel's shared arrays

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Where value i of h goes: each eight in the order 0 4 1 5 2 6 3 7, as the pairs
// of open_codes lie.
__device__ __forceinline__ int permuted(int i) { return (i & ~7) | ((i & 3) << 1) | ((i >> 2) & 1); }

// Eight codes as four pairs of bf16 code - 8: columns (0,4), (1,5), (2,6), (3,7).
// The mask and the OR are one instruction (the compiler makes two of them: 27 %
// more ALU work, a 7168 x 7168 product 9.1 us instead of 7.7).
__device__ __forceinline__ void open_codes(uint32_t w, uint32_t (&d)[4]) {
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v;  // 128 + code
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(v)
        : "r"(w >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
    const __nv_bfloat162 b = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
    d[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// c = a b, or c += a b
template <bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Member m of S takes columns [share(m), share(m + 1)).
__device__ __forceinline__ int share(int m, int S, int cols) {
  return min(cols, (int)((int64_t)m * ((cols + kShare - 1) / kShare) / S) * kShare);
}

// A warp's stream of blocks: 16 rows (g and g + 8 of lane 4g + t, the second
// anywhere in the matrix) by kCols columns, and the same columns of up to TOK
// tokens. A stage holds
//  - the codes, 16-byte piece c of row r at place c ^ swizzle(r), so that reads of
//    4, 8 or 16 bytes a lane spread over the banks;
//  - each row's scales, as the 4-byte words they lie in (a row of scales starts at
//    any even address);
//  - x, token by token, 8 columns (16 bytes) a place (x_place): eight lanes that read
//    together find different banks, and four lanes that copy 64 bytes leave them
//    together. 13 tokens, 4104 x 4096, group 64 or 128: 7.5 and 6.9 us; 8.4 with only
//    32 bytes together, 15 with 16.
// Lane 4g + t takes words of eight codes: word j < GROUP/32 of a group covers its
// columns (GROUP/4) t + 8j .. + 7, so that the 16 columns of an MMA (two MMAs a
// word) lie in one group.
template <int GROUP, int TOK>
struct Stream {
  static constexpr int kCols = 128;
  static constexpr int kAhead = TOK == 8 ? 3 : 2;    // stages
  static constexpr int kNT = TOK / 8;                // tiles of 8 tokens
  static constexpr int kG = kCols / GROUP;           // scales of a row in a block
  static constexpr int kWords = GROUP / 32;          // words of a lane in a group
  static constexpr int kScaleBytes = kG == 1 ? 4 : 2 * kG + 4;  // the words a row's scales touch
  static constexpr int kCodes = 16 * kCols / 2;
  static constexpr int kX = kCodes + 16 * kScaleBytes;
  static constexpr int kStage = (kX + TOK * kCols * 2 + 127) / 128 * 128;
  static constexpr int kBytes = kAhead * kStage;     // of a warp
  static constexpr int kCopies = TOK / 2;            // x copies of a lane in a block

  uint32_t base;           // the warp's ring
  int fill = 0, take = 0;  // offsets of the stage filled and taken next
  int lane, g, t;
  const uint8_t* q;        // row g, at piece t of the block copied next
  int64_t q8;              // bytes from there to the second row
  const uint16_t* scales;  // of the whole matrix
  int64_t si, s_end;       // this lane's scale (lanes 0-15: row lane), number of scales
  int rs;                  // scales of a row
  int left;                // columns of the share from the block copied next on
  const uint16_t* x[kCopies];  // this lane's 8 columns of its tokens in that block
  int tokens;

  static __device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 3; }
  // The 16-byte place within a token's columns of word j of lane t of group grp.
  static __device__ __forceinline__ int x_place(int grp, int t, int j, int odd) {
    return kWords == 1 ? (4 * grp + t) ^ (odd << 2)
                       : 2 * (kWords == 2 ? 4 * grp + t : (2 * t + (j >> 1)) ^ (t >> 1)) + ((j & 1) ^ odd);
  }

  __device__ __forceinline__ void init(uint8_t* ring, int warp, int lane_, int64_t second, int cols,
                                       const uint16_t* sc, int64_t rows) {
    base = smem_u32(ring) + (uint32_t)(warp * kBytes);
    lane = lane_;
    g = lane >> 2;
    t = lane & 3;
    q8 = second * (cols / 2);
    scales = sc;
    rs = cols / GROUP;
    s_end = rows * rs;
  }

  // The token whose columns this lane copies with its i-th copy.
  __device__ __forceinline__ int token(int i) const { return 2 * i + (lane >> 4); }
  __device__ __forceinline__ int x_col() const { return (lane & (kCols / 8 - 1)) * 8; }

  // Continues with columns [c0, c1) of the rows whose row g is `row` and whose row
  // lane % 16 is `srow`, and of n tokens; the caller sets x[] (column c0 + x_col()).
  __device__ __forceinline__ void seek(const uint8_t* codes, int64_t row, int64_t srow, int c0,
                                       int c1, int cols, int n) {
    q = codes + row * (cols / 2) + c0 / 2 + 16 * t;
    si = srow * rs + c0 / GROUP;
    left = c1 - c0;
    tokens = n;
  }

  __device__ __forceinline__ void copy() {
    const uint32_t st = base + (uint32_t)fill;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      cp_async_16(st + (uint32_t)((g + 8 * i) * (kCols / 2) + ((t ^ swizzle(g)) << 4)),
                  q + (i ? q8 : 0), GROUP == 128 || 32 * t < left ? 16u : 0u);
    if (lane < 16) {
      const int64_t w = si >> 1;
      const uint16_t* src = scales + 2 * w;
      const int n = (int)min(s_end - 2 * w, (int64_t)(kScaleBytes / 2));  // scales from there on
#pragma unroll
      for (int j = 0; j < kScaleBytes / 4; ++j)
        cp_async_4(st + (uint32_t)(kCodes + lane * kScaleBytes + j * 4), n > 2 * j ? src + 2 * j : scales,
                   n > 2 * j + 1 ? 4u : n > 2 * j ? 2u : 0u);
    }
    const int c = x_col() / 8, in = c % (GROUP / 8);
    const int place = x_place(c / (GROUP / 8), in / kWords, in % kWords, lane >> 4);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const bool there = token(i) < tokens && x_col() < left;
      cp_async_16(st + (uint32_t)(kX + token(i) * kCols * 2 + place * 16), there ? x[i] : scales,
                  there ? 16u : 0u);
      x[i] += kCols;
    }
    q += kCols / 2;
    si += kG;
    left -= kCols;
  }
  __device__ __forceinline__ void commit() {
    cp_async_commit();
    fill = fill + kStage == kBytes ? 0 : fill + kStage;
  }

  // acc[n] += rows x (tokens of tile n) for the block taken next, of which `valid`
  // columns and `n_tok` tokens count. PERMUTED: each eight values of x lie in the
  // order 0 4 1 5 2 6 3 7. `odd`: whether the block's scales of this lane's rows
  // start at an odd place of the matrix.
  template <bool PERMUTED>
  __device__ __forceinline__ void multiply(int odd, int valid, int n_tok, float (&acc)[kNT][4]) {
    cp_async_wait<kAhead - 1>();
    __syncwarp();
    const uint32_t at = base + (uint32_t)take;
    const uint32_t xt = at + (uint32_t)(kX + g * kCols * 2);
    const uint32_t sc = at + (uint32_t)(kCodes + g * kScaleBytes + odd * 2);
#pragma unroll
    for (int grp = 0; grp < kG; ++grp) {
      if (grp > 0 && valid <= grp * GROUP) break;
      uint32_t w[2][kWords];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t row = at + (uint32_t)((g + 8 * i) * (kCols / 2));
        if constexpr (GROUP == 128) {
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                       : "r"(row + (uint32_t)(((4 * grp + t) ^ swizzle(g)) << 4))
                       : "memory");
        } else if constexpr (GROUP == 64) {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                       : "=r"(w[i][0]), "=r"(w[i][1])
                       : "r"(row + (uint32_t)((((2 * grp + (t >> 1)) ^ swizzle(g)) << 4) + (t & 1) * 8))
                       : "memory");
        } else {
          asm volatile("ld.shared.u32 %0, [%1];"
                       : "=r"(w[i][0])
                       : "r"(row + (uint32_t)(((grp ^ swizzle(g)) << 4) + t * 4))
                       : "memory");
        }
      }
      float s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(v)
                     : "r"(sc + (uint32_t)(8 * i * kScaleBytes + 2 * grp))
                     : "memory");
        s[i] = bf(v);
      }
      float part[kNT][4];
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        uint32_t a[2][4];
        open_codes(w[0][j], a[0]);
        open_codes(w[1][j], a[1]);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          if (n > 0 && 8 * n >= n_tok) break;
          uint4 u;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                       : "r"(xt + (uint32_t)(n * 8 * kCols * 2 + (x_place(grp, t, j, g & 1) << 4)))
                       : "memory");
          const uint32_t b0 = PERMUTED ? u.x : __byte_perm(u.x, u.z, 0x5410);
          const uint32_t b1 = PERMUTED ? u.y : __byte_perm(u.x, u.z, 0x7632);
          const uint32_t b2 = PERMUTED ? u.z : __byte_perm(u.y, u.w, 0x5410);
          const uint32_t b3 = PERMUTED ? u.w : __byte_perm(u.y, u.w, 0x7632);
          if (j == 0) mma16816<true>(part[n], a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
          else mma16816<false>(part[n], a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
          mma16816<false>(part[n], a[0][2], a[1][2], a[0][3], a[1][3], b2, b3);
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if (n > 0 && 8 * n >= n_tok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(s[i >> 1], part[n][i], acc[n][i]);
      }
    }
    __syncwarp();  // the stage may be filled again
    take = take + kStage == kBytes ? 0 : take + kStage;
  }
};

// A warp's sums of 16 rows x 8 NT tokens in shared memory: part[row * 8 NT + token].
template <int NT>
__device__ __forceinline__ void leave_part(float* part, int g, int t, const float (&acc)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* at = part + g * 8 * NT + 8 * n + 2 * t;
    *reinterpret_cast<float2*>(at) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(at + 8 * 8 * NT) = make_float2(acc[n][2], acc[n][3]);
  }
}

__device__ __forceinline__ uint8_t* ring_of(uint8_t* dynamic) {
  return dynamic + (-smem_u32(dynamic) & 127u);
}

template <int GROUP, int TOK>
__global__ void __launch_bounds__(kThreads, 2)
    w4_matvec_kernel(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                     int cols, uint16_t* y) {
  using St = Stream<GROUP, TOK>;
  constexpr int kTok = 8 * St::kNT;
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ __align__(16) float part[kWarps * 16 * kTok];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16, t0 = blockIdx.y * TOK, n = min(TOK, N - t0);
  const int row = min(r0 + g, rows - 1);  // a row past the last one reads the last one
  const int c0 = share(warp, kWarps, cols), c1 = share(warp + 1, kWarps, cols);
  const int blocks = (c1 - c0 + St::kCols - 1) / St::kCols;
  St st;
  st.init(ring_of(dynamic), warp, lane, min(8, rows - 1 - row), cols, scale, rows);
  st.seek(q, row, min(r0 + (lane & 15), rows - 1), c0, c1, cols, n);
#pragma unroll
  for (int i = 0; i < St::kCopies; ++i)
    st.x[i] = x + (size_t)(t0 + min(st.token(i), n - 1)) * cols + c0 + st.x_col();
#pragma unroll
  for (int d = 0; d < St::kAhead; ++d) {
    if (d < blocks) st.copy();
    st.commit();
  }
  const int odd = ((row & 1) * st.rs + c0 / GROUP) & 1;
  float acc[St::kNT][4] = {};
  for (int b = 0; b < blocks; ++b) {
    st.template multiply<false>((odd + b * St::kG) & 1, c1 - c0 - b * St::kCols, n, acc);
    if (b + St::kAhead < blocks) st.copy();
    st.commit();
  }
  leave_part<St::kNT>(part + warp * 16 * kTok, g, t, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * n; i += kThreads) {
    const int r = r0 + (i & 15);
    if (r >= rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[(w * 16 + (i & 15)) * kTok + (i >> 4)];
    y[(size_t)(t0 + (i >> 4)) * rows + r] = to_bf(v);
  }
}

// ------------------------------------------------------------------ rows in registers
// Lane 4g + t takes 16 bytes (32 columns) of its two rows of every block of 128
// columns. A block may hold kG groups, whose sums must not mix: the MMA's columns
// tell them apart. Column c of B is token c / kG and takes x only at the columns of
// the block's group c % kG (zeros elsewhere), so one MMA gives the sums of kG groups
// for 8 / kG tokens side by side, and P of them those of P times as many.
constexpr int kRowsAhead = 4;  // six: 4 to 5 % slower
constexpr int kRowsBlock = 128;

__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int GROUP, int P>
struct Rows {
  static constexpr int kG = kRowsBlock / GROUP;
  static constexpr int kTok = 8 / kG;         // tokens of an MMA
  static constexpr int kHeld = kG > 1 ? 1 : 2;  // tokens whose sums a lane holds, an MMA
  const uint8_t* q;   // row g, this lane's place in the block fetched next
  const uint16_t* s;
  int64_t q8, s8;     // on to the second row
  int n, cols, t, g;  // blocks, columns
  uint4 w[kRowsAhead][2];
  uint32_t sc[kRowsAhead][2];  // the scales of this lane's one or two groups
  bool pairs;  // rows of scales start at even places: two make an aligned word
  float sum[P][2][kHeld];

  // Row g at `row`, the second `second` rows on, columns [c0, c1), c0 a multiple of 128.
  __device__ __forceinline__ void begin(const uint8_t* codes, const uint16_t* scales, int64_t row,
                                        int64_t second, int row_cols, int c0, int c1, int lane) {
    t = lane & 3;
    g = lane >> 2;
    cols = c1 - c0;
    n = (cols + kRowsBlock - 1) / kRowsBlock;
    q = codes + row * (row_cols / 2) + c0 / 2 + 16 * t;
    s = scales + row * (row_cols / GROUP) + c0 / GROUP + first_group();
    q8 = second * (row_cols / 2);
    s8 = second * (row_cols / GROUP);
    pairs = row_cols / GROUP % 2 == 0;
    clear();
#pragma unroll
    for (int d = 0; d < kRowsAhead; ++d) fetch(d, q + d * (kRowsBlock / 2), s + d * kG, d);
  }
  // the first group of a block whose sums this lane holds
  __device__ __forceinline__ int first_group() const { return kG == 4 ? 2 * (t & 1) : 0; }
  // Block `at` of a tile, its codes and scales at qa and s0, into place d.
  __device__ __forceinline__ void fetch(int d, const uint8_t* qa, const uint16_t* s0, int at) {
    if (at >= n) return;
    const int left = cols - at * kRowsBlock;
    if (GROUP == 128 || 32 * t < left) {
      w[d][0] = ld_codes(qa);
      w[d][1] = ld_codes(qa + q8);
    }
    if (kG == 1) {
      sc[d][0] = __ldg(s0);
      sc[d][1] = __ldg(s0 + s8);
    } else if (first_group() * GROUP < left) {
      if (pairs) {
        sc[d][0] = __ldg(reinterpret_cast<const uint32_t*>(s0));
        sc[d][1] = __ldg(reinterpret_cast<const uint32_t*>(s0 + s8));
      } else {
        const bool both = (first_group() + 1) * GROUP < left;
        sc[d][0] = __ldg(s0) | (both ? (uint32_t)__ldg(s0 + 1) << 16 : 0u);
        sc[d][1] = __ldg(s0 + s8) | (both ? (uint32_t)__ldg(s0 + s8 + 1) << 16 : 0u);
      }
    } else {
      sc[d][0] = sc[d][1] = 0u;
    }
  }
  // x: the laid-out columns from c0 on of the first token, `stride` bytes on to the
  // next; `tokens` of them (columns without a token take another's, and their sums are
  // not used). STREAM: with `more`, another tile follows, `next` rows on: a place that
  // this tile is through with takes that one's block.
  template <bool STREAM = false>
  __device__ __forceinline__ void run(uint32_t x, uint32_t stride, int tokens, bool more = false, int next = 0,
                                      int row_cols = 0) {
    const bool mine = kG == 1 || t / (GROUP / 32) == g % kG;  // this lane's column takes x of its columns
    const int live = P == 1 ? 1 : (tokens + kTok - 1) / kTok;
    uint32_t xp[P];
#pragma unroll
    for (int i = 0; i < P; ++i) xp[i] = x + (uint32_t)min(g / kG + i * kTok, tokens - 1) * stride + (uint32_t)t * 16u;
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = make_uint4(0u, 0u, 0u, 0u);
    const uint8_t* qn = q + (int64_t)next * (row_cols / 2);
    const uint16_t* sn = s + (int64_t)next * (row_cols / GROUP);
    for (int b = 0; b < n; b += kRowsAhead) {
#pragma unroll
      for (int d = 0; d < kRowsAhead; ++d) {
        if (b + d >= n) break;
        float p[P][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0[4], a1[4];
          open_codes(j == 0 ? w[d][0].x : j == 1 ? w[d][0].y : j == 2 ? w[d][0].z : w[d][0].w, a0);
          open_codes(j == 0 ? w[d][1].x : j == 1 ? w[d][1].y : j == 2 ? w[d][1].z : w[d][1].w, a1);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (i > 0 && i >= live) break;
            // lanes whose column takes no x keep their zeros
            asm volatile(
                "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n"
                " @p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n}"
                : "+r"(u[j].x), "+r"(u[j].y), "+r"(u[j].z), "+r"(u[j].w)
                : "r"(xp[i] + (uint32_t)(d * 256 + j * 64)), "r"((int)mine)
                : "memory");
            if (j == 0) mma16816<true>(p[i], a0[0], a1[0], a0[1], a1[1], u[j].x, u[j].y);
            else mma16816<false>(p[i], a0[0], a1[0], a0[1], a1[1], u[j].x, u[j].y);
            mma16816<false>(p[i], a0[2], a1[2], a0[3], a1[3], u[j].z, u[j].w);
          }
        }
        // columns 2t and 2t + 1 are this lane's: two tokens, or two groups of one
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (i > 0 && i >= live) break;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              sum[i][r][kG == 1 ? j : 0] =
                  fmaf(__uint_as_float(kG == 1 || j == 0 ? sc[d][r] << 16 : sc[d][r] & 0xFFFF0000u), p[i][2 * r + j],
                       sum[i][r][kG == 1 ? j : 0]);
        }
        if constexpr (STREAM) {
          const bool here = b + d + kRowsAhead < n;
          fetch(d, (here ? q + kRowsAhead * (kRowsBlock / 2) : qn) + d * (kRowsBlock / 2),
                (here ? s + kRowsAhead * kG : sn) + d * kG, here ? b + d + kRowsAhead : more ? d : n);
        } else {
          fetch(d, q + (d + kRowsAhead) * (kRowsBlock / 2), s + (d + kRowsAhead) * kG, b + d + kRowsAhead);
        }
      }
      q += kRowsAhead * (kRowsBlock / 2);
      s += kRowsAhead * kG;
#pragma unroll
      for (int i = 0; i < P; ++i) xp[i] += kRowsAhead * 256;
    }
    if (STREAM) {
      q = qn;
      s = sn;
    }
    if (kG == 4)  // two lanes hold the four groups of a token
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) sum[i][r][0] += __shfl_xor_sync(0xFFFFFFFFu, sum[i][r][0], 1);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < kHeld; ++j) sum[i][0][j] = sum[i][1][j] = 0.0f;
  }
  // Where the sums go: to(row of the tile, token, value), for the tokens below n.
  template <class F>
  __device__ __forceinline__ void give(int tokens, F to) const {
    each(tokens, [&](int tok, float v0, float v1) {
      to(g, tok, v0);
      to(g + 8, tok, v1);
    });
  }
  // to(token, row g's, row g + 8's)
  template <class F>
  __device__ __forceinline__ void each(int tokens, F to) const {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int tok = i * kTok + (kG == 1 ? 2 * t + j : kG == 2 ? t : t >> 1);
        if (tok >= tokens || (kG == 4 && (t & 1))) continue;
        to(tok, sum[i][0][j], sum[i][1][j]);
      }
  }
};

// Columns [c0, c1) of x (c0 a multiple of 128), block by block in shared memory
// (256 bytes from c0 on): word j of lane t at place 4j + t, its eight values in the
// order of open_codes; zeros to the end of the last block. By one warp.
template <bool PERMUTED>
__device__ __forceinline__ void lay_out(uint32_t to, const uint16_t* x, int c0, int c1, int lane) {
  for (int c = c0 / 8 + lane; c < (c1 + kRowsBlock - 1) / kRowsBlock * (kRowsBlock / 8); c += 32) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (c * 8 < c1) v = __ldcg(reinterpret_cast<const uint4*>(x) + c);
    const uint32_t at = to + (uint32_t)(((c & ~15) + (c & 3) * 4 + ((c & 15) >> 2)) * 16 - c0 * 2);
    if (PERMUTED)
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    else
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(__byte_perm(v.x, v.z, 0x5410)),
                   "r"(__byte_perm(v.x, v.z, 0x7632)), "r"(__byte_perm(v.y, v.w, 0x5410)),
                   "r"(__byte_perm(v.y, v.w, 0x7632))
                   : "memory");
  }
  __syncwarp();
}

constexpr int kOneWarps = 4;

// Blocks an SM that the registers allow without spills: groups told apart by the
// MMA's columns take more. 7168 x 7168, group 64: 4 blocks 9.8 us, 6 12.9 us (some
// registers spilled); group 128: 9.2 and 8.1 us. One token's experts of 7168 x 2048,
// group 64: 48 us, 57.7 us.
constexpr int one_blocks(int group) { return group == 128 ? 6 : 4; }

template <int GROUP>
__global__ void __launch_bounds__(kOneWarps * 32, one_blocks(GROUP))
    w4_matvec_one_kernel(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int rows,
                         int cols, uint16_t* y) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float part[kOneWarps][16];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int r0 = blockIdx.x * 16, row = min(r0 + g, rows - 1);
  const int c0 = share(warp, kOneWarps, cols), c1 = share(warp + 1, kOneWarps, cols);
  Rows<GROUP, 1> o;
  o.begin(q, scale, row, min(8, rows - 1 - row), cols, c0, c1, lane);
  const uint32_t xs = smem_u32(dynamic) + (uint32_t)c0 * 2;
  lay_out<false>(xs, x, c0, c1, lane);
  o.run(xs, 0, 1);
  o.give(1, [&](int r, int, float v) { part[warp][r] = v; });
  __syncthreads();
  if (threadIdx.x < 16 && r0 + (int)threadIdx.x < rows) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kOneWarps; ++w) v += part[w][threadIdx.x];
    y[r0 + threadIdx.x] = to_bf(v);
  }
}

// The token's route of this lane (lane < K): its expert, -1 for none or one named
// before, and the token's whole probability of it.
__device__ __forceinline__ int one_route(const W4Args& a, int token, int lane, float* p) {
  int e = lane < a.K ? __ldcg(a.topk_ids + token * a.K + lane) : -1;
  if (e < 0 || e >= a.E) e = -1;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
  if (p) {
    const float mine = lane < a.K ? __ldcg(a.topk_p + token * a.K + lane) : 0.0f;
    *p = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      const float v = __shfl_sync(0xFFFFFFFFu, mine, k);
      if ((same >> k) & 1u) *p += v;
    }
  }
  return __ffs(same) - 1 == lane ? e : -1;
}

// Block (8 features, route): rows g of its tile are gate rows, rows g + 8 up rows.
template <int GROUP>
__global__ void __launch_bounds__(kOneWarps * 32, one_blocks(GROUP)) w4_fc1_one_kernel(const W4Args a) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float part[kOneWarps][16];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int token = blockIdx.z;
  const int e = __shfl_sync(0xFFFFFFFFu, one_route(a, token, lane, nullptr), blockIdx.y);
  if (e < 0) return;
  const int i0 = blockIdx.x * 8;
  const int c0 = share(warp, kOneWarps, a.H), c1 = share(warp + 1, kOneWarps, a.H);
  Rows<GROUP, 1> o;
  o.begin(a.w13, a.w13_scale, (int64_t)e * 2 * a.I + i0 + g, a.I, a.H, c0, c1, lane);
  const uint32_t xs = smem_u32(dynamic) + (uint32_t)c0 * 2;
  lay_out<false>(xs, a.x + (size_t)token * a.H, c0, c1, lane);
  o.run(xs, 0, 1);
  o.give(1, [&](int r, int, float v) { part[warp][r] = v; });
  __syncthreads();
  if (threadIdx.x < 8) {
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int w = 0; w < kOneWarps; ++w) {
      gate += part[w][threadIdx.x];
      up += part[w][8 + threadIdx.x];
    }
    const float h = (a.activation ? act_fwd<1>(gate) : act_fwd<0>(gate)) * up;
    a.h[(size_t)(token * a.K + blockIdx.y) * a.I + i0 + permuted(threadIdx.x)] = to_bf(h);
  }
}

// Block (16 output columns): the 128-column blocks of the token's experts, one
// expert after the other, are dealt out to the warps in runs.
template <int GROUP>
__global__ void __launch_bounds__(kThreads, one_blocks(GROUP) / 2) w4_fc2_one_kernel(const W4Args a) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float part[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // The first product's kernel let this one start after every earlier kernel had
  // finished, and writes neither the routes nor the weights: only h has to wait.
  float p_lane;
  const int token = blockIdx.y;
  const int e_lane = one_route(a, token, lane, &p_lane);
  uint32_t routes = __ballot_sync(0xFFFFFFFFu, e_lane >= 0);
  const int r0 = blockIdx.x * 16, per = (a.I + kRowsBlock - 1) / kRowsBlock;
  const int total = __popc(routes) * per;
  int at = warp * total / kWarps;
  const int end = (warp + 1) * total / kWarps;
  for (int skip = at / per; skip > 0; --skip) routes &= routes - 1;
  float lo = 0.0f, hi = 0.0f;
  bool waited = false;
  while (at < end) {  // the run's part of one expert
    const int r = __ffs(routes) - 1, b0 = at % per, b1 = min(per, b0 + end - at);
    const int e = __shfl_sync(0xFFFFFFFFu, e_lane, r);
    const float p = __shfl_sync(0xFFFFFFFFu, p_lane, r);
    const int c0 = b0 * kRowsBlock, c1 = min(a.I, b1 * kRowsBlock);
    Rows<GROUP, 1> o;
    o.begin(a.w2, a.w2_scale, (int64_t)e * a.H + r0 + g, 8, a.I, c0, c1, lane);
    if (!waited) griddep_wait();
    waited = true;
    const uint32_t hs = smem_u32(dynamic) + (uint32_t)(r * per + b0) * 256u;
    lay_out<true>(hs, a.h + (size_t)(token * a.K + r) * a.I, c0, c1, lane);
    o.run(hs, 0, 1);
    lo = fmaf(p, o.sum[0][0][0], lo);  // of the token in lane t = 0
    hi = fmaf(p, o.sum[0][1][0], hi);
    at += b1 - b0;
    routes &= routes - 1;
  }
  if (!waited) griddep_wait();
  griddep_launch_dependents();
  if (t == 0) {
    part[warp][g] = lo;
    part[warp][g + 8] = hi;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const size_t c = (size_t)token * a.H + r0 + threadIdx.x;
    float v = a.add ? bf(a.add[c]) : 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][threadIdx.x];
    a.y[c] = to_bf(v);
  }
}

// ------------------------------------------------------------------ several tokens
// What the grouping kernel leaves in the workspace: pieces of at most `most` routes
// of one expert, experts ascending, routes in their order. A route without an
// expert (an id outside 0..E-1), or to an expert that its token has named before,
// is in none.
constexpr int kMaxPieces = kMaxExperts + kMaxRoutes;
struct W4Groups {
  int32_t pieces;
  int32_t expert[kMaxPieces], first[kMaxPieces], count[kMaxPieces];  // first: its place in `order`
  int32_t order[kMaxRoutes];  // routes, sorted by expert
  int32_t used[kMaxRoutes];   // of each route: whether it is in a piece
  float prob[kMaxRoutes];     // the token's whole probability of the route's expert
};

__global__ void __launch_bounds__(kMaxExperts) w4_group_kernel(const int32_t* ids, const float* probs,
                                                               int R, int K, int E, int most, W4Groups* G) {
  __shared__ int16_t named[kMaxRoutes], id[kMaxRoutes], rank[kMaxRoutes];
  __shared__ int routes[kMaxExperts], scan[2][kMaxExperts / 32];
  __shared__ int16_t of_warp[kWarps][kMaxExperts];  // routes of an expert in a warp's share, then before it
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  for (int w = 0; w < kWarps; ++w) of_warp[w][tid] = 0;
  for (int i = tid; i < R; i += kMaxExperts) {
    const int e = ids[i];
    named[i] = (int16_t)(e < 0 || e >= E ? -1 : e);
  }
  __syncthreads();
  for (int i = tid; i < R; i += kMaxExperts) {
    const int r0 = i / K * K;
    int e = named[i];
    float p = e >= 0 ? probs[i] : 0.0f;
    for (int r = r0; r < r0 + K && e >= 0; ++r) {
      if (r == i || named[r] != e) continue;
      if (r < i) e = -1;
      else p += probs[r];
    }
    id[i] = (int16_t)e;
    G->used[i] = e >= 0;
    G->prob[i] = p;
  }
  __syncthreads();
  // each warp ranks its share of the routes within their experts, 32 at a time, in order
  const int part = ((R + kWarps - 1) / kWarps + 31) / 32 * 32, from = warp * part, to = min(R, from + part);
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < to ? id[i] : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int before = __popc(same & ((1u << lane) - 1u));
    const int had = e >= 0 ? of_warp[warp][e] : 0;
    __syncwarp();
    if (e >= 0 && before == 0) of_warp[warp][e] = (int16_t)(had + __popc(same));
    if (i < to) rank[i] = (int16_t)(had + before);
    __syncwarp();
  }
  __syncthreads();
  int n = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int v = of_warp[w][tid];
    of_warp[w][tid] = (int16_t)n;
    n += v;
  }
  // exclusive sums over the experts of their routes and of their pieces
  const int np = (n + most - 1) / most;
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
    scan[0][warp] = sn;
    scan[1][warp] = sp;
  }
  __syncthreads();
  int on = sn - n, op = sp - np;
  for (int w = 0; w < warp; ++w) {
    on += scan[0][w];
    op += scan[1][w];
  }
  routes[tid] = on;  // where the expert's routes begin
  for (int j = 0; j < np; ++j) {
    G->expert[op + j] = tid;
    G->first[op + j] = on + j * most;
    G->count[op + j] = min(most, n - j * most);
  }
  if (tid == kMaxExperts - 1) G->pieces = op + np;
  __syncthreads();
  for (int i = tid; i < R; i += kMaxExperts)
    if (id[i] >= 0) G->order[routes[id[i]] + of_warp[i / part][id[i]] + rank[i]] = i;
}

// The work is a list of items, those of the first piece, of the second, ...: kWarps / S
// tiles of 16 rows, S warps a tile, which split its columns. A block takes a run of
// the list, and a warp's stream of codes goes on from tile to tile of a piece. Gated:
// 8 features a tile, rows g their gate rows, rows g + 8 their up rows; h of each
// route, in the order of open_codes. Else 16 columns of the output a tile; each
// route's products, times its probability, in fp32.
template <bool GATED, int GROUP, int P>
__global__ void __launch_bounds__(kThreads, 2)
    w4_piece_kernel(const W4Args a, const W4Groups* G, float* o, const int S, const uint32_t stride) {
  using R = Rows<GROUP, P>;
  constexpr int kMost = R::kTok * P;
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float part[2][kWarps][16][kMost];
  __shared__ int route_s[kMost];
  __shared__ float prob_s[kMost];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int cols = GATED ? a.H : a.I, rows = GATED ? a.I : a.H, step = GATED ? 8 : 16;
  const int per = kWarps / S * step, items = (rows + per - 1) / per;  // rows of an item, items of a piece
  // The second product's pieces and weights were there before the first one began
  // (its kernel started after the grouping's had finished): only h has to wait.
  if (GATED) griddep_wait();
  griddep_launch_dependents();
  bool waited = GATED;
  const int64_t all = (int64_t)__ldcg(&G->pieces) * items;
  int at = (int)(all * blockIdx.x / gridDim.x);
  const int end = (int)(all * (blockIdx.x + 1) / gridDim.x);
  const int member = warp % S, c0 = share(member, S, cols), c1 = share(member + 1, S, cols);
  const uint32_t xs = smem_u32(dynamic) + (uint32_t)c0 * 2u;
  while (at < end) {
    const int piece = at / items, from = at - piece * items, to = min(items, from + end - at);
    at += to - from;
    const int e = __ldcg(&G->expert[piece]), first = __ldcg(&G->first[piece]), n = __ldcg(&G->count[piece]);
    const int row0 = from * per + warp / S * step;
    int tiles = to - from;  // this warp's: the last item may have fewer
    if (row0 + (tiles - 1) * per >= rows) --tiles;
    R r;  // not set up, and not used, in a warp without a tile
    if (tiles > 0)
      r.begin(GATED ? a.w13 : a.w2, GATED ? a.w13_scale : a.w2_scale,
              GATED ? (int64_t)e * 2 * a.I + row0 + g : (int64_t)e * a.H + row0 + g, GATED ? a.I : 8, cols, c0,
              c1, lane);
    if (!waited) {
      griddep_wait();
      waited = true;
    }
    // the piece's tokens (second product: their h), a warp a token at a time
    for (int k = warp; k < n; k += kWarps) {
      const int route = __ldcg(&G->order[first + k]);
      if (lane == 0) {
        route_s[k] = route;
        prob_s[k] = __ldcg(&G->prob[route]);
      }
      const uint16_t* x = GATED ? a.x + (size_t)(route / a.K) * cols : a.h + (size_t)route * cols;
      lay_out<!GATED>(smem_u32(dynamic) + (uint32_t)k * stride, x, 0, cols, lane);
    }
    __syncthreads();
    const auto put = [&](int tok, int row, float v, float u) {
      const int route = route_s[tok];
      if (GATED)
        a.h[(size_t)route * a.I + permuted(row)] = to_bf((a.activation ? act_fwd<1>(v) : act_fwd<0>(v)) * u);
      else
        o[(size_t)route * a.H + row] = prob_s[tok] * v;
    };
    for (int i = 0; i < to - from; ++i) {
      if (i < tiles) r.template run<true>(xs, stride, n, i + 1 < tiles, per, cols);
      if (S == 1) {
        if (i < tiles)
          r.each(n, [&](int tok, float v0, float v1) {
            const int row = row0 + i * per + g;
            put(tok, row, v0, v1);
            if (!GATED) put(tok, row + 8, v1, 0.0f);
          });
      } else {
        float(*mine)[16][kMost] = part[i & 1];
        if (i < tiles)
          r.each(n, [&](int tok, float v0, float v1) {
            mine[warp][g][tok] = v0;
            mine[warp][g + 8][tok] = v1;
          });
        __syncthreads();
        for (int j = threadIdx.x; j < per * n; j += kThreads) {
          const int in_item = j % per, tok = j / per, row = (from + i) * per + in_item;
          if (row >= rows) continue;
          const int w0 = in_item / step * S, in = in_item % step;
          float v = 0.0f, u = 0.0f;
          for (int w = w0; w < w0 + S; ++w) {
            v += mine[w][in][tok];
            if (GATED) u += mine[w][8 + in][tok];
          }
          put(tok, row, v, u);
        }
      }
      if (i < tiles) r.clear();
    }
    __syncthreads();  // before the next piece's x is laid out
  }
  if (!waited) griddep_wait();
}

// y[t] = add[t] + the products of t's routes, in their order: four columns a thread.
__global__ void __launch_bounds__(256) w4_sum_kernel(const W4Args a, const W4Groups* G, const float* o) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (c >= a.H) return;
  const size_t at = (size_t)t * a.H + c;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (a.add) {
    const uint2 b = *reinterpret_cast<const uint2*>(a.add + at);
    v = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                    __uint_as_float(b.y & 0xFFFF0000u));
  }
  for (int k = 0; k < a.K; ++k) {
    const int r = t * a.K + k;
    if (!G->used[r]) continue;
    const float4 b = *reinterpret_cast<const float4*>(o + (size_t)r * a.H + c);
    v.x += b.x;
    v.y += b.y;
    v.z += b.z;
    v.w += b.w;
  }
  *reinterpret_cast<uint2*>(a.y + at) =
      make_uint2((uint32_t)to_bf(v.x) | ((uint32_t)to_bf(v.y) << 16), (uint32_t)to_bf(v.z) | ((uint32_t)to_bf(v.w) << 16));
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

// A launch whose kernel takes up to `most` bytes of dynamic shared memory (asked
// for once per device).
template <typename... KArgs, typename... Args>
cudaError_t launch_ring(DeviceOnce& once, void (*kernel)(KArgs...), size_t most, dim3 grid,
                        dim3 block, size_t smem, cudaStream_t s, Args... args) {
  const cudaError_t err = once_per_device(once, nullptr, [&](int, int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  return err != cudaSuccess ? err : launch_pdl(kernel, grid, block, smem, s, args...);
}

cudaError_t sm_count(int* sms) {
  static DeviceOnce once;
  return once_per_device(once, sms, [](int dev, int* v) {
    return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
}

template <int GROUP, int TOK>
cudaError_t matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                   int cols, uint16_t* y, cudaStream_t s) {
  static DeviceOnce once;
  constexpr size_t smem = kWarps * Stream<GROUP, TOK>::kBytes + 128;
  return launch_ring(once, w4_matvec_kernel<GROUP, TOK>, smem,
                     dim3((rows + 15) / 16, (N + TOK - 1) / TOK), dim3(kThreads), smem, s, x, q, scale,
                     N, rows, cols, y);
}

template <int TOK>
cudaError_t matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                   int cols, int group, uint16_t* y, cudaStream_t s) {
  return group == 128  ? matvec<128, TOK>(x, q, scale, N, rows, cols, y, s)
         : group == 64 ? matvec<64, TOK>(x, q, scale, N, rows, cols, y, s)
                       : matvec<32, TOK>(x, q, scale, N, rows, cols, y, s);
}

// Several tokens. Routes of a piece: what x leaves room for in half of an SM's shared
// memory, at most 8. Warps a row tile: more where there are few items for the blocks
// (2 an SM) to share evenly, while a warp keeps eight blocks of columns: four tokens'
// experts of 7168 x 2048 145 us with kFill 4, 154 us with 2.
constexpr size_t kPieceBytes = 96 << 10;
constexpr int kFill = 4;

struct W4Layout {
  size_t groups, o, h, total;
};

W4Layout w4_layout(int N, int K, int H, int I) {
  W4Layout L{};
  const size_t R = (size_t)N * K;
  L.h = (sizeof(W4Groups) + 255) / 256 * 256;
  L.o = L.h + (R * I * 2 + 255) / 256 * 256;
  L.total = L.o + (R * H * 4 + 255) / 256 * 256;
  return L;
}

template <bool GATED, int GROUP, int P>
cudaError_t piece(const W4Args& a, const W4Groups* G, float* o, int most, int pieces, int sms, cudaStream_t s) {
  static DeviceOnce once;
  const int cols = GATED ? a.H : a.I, rows = GATED ? a.I / 8 : a.H / 16;
  // 64 bytes over a multiple of 128: two tokens' words in different banks
  const uint32_t stride = (uint32_t)((cols + 127) / 128 * 256 + 64);
  const int blocks = 2 * sms;
  int S = 1;
  while (S < 8 && (int64_t)((rows + 8 / S - 1) / (8 / S)) * pieces < kFill * (int64_t)blocks && cols / 128 >= 8 * S) S *= 2;
  const int64_t items = (int64_t)((rows + 8 / S - 1) / (8 / S)) * pieces;
  return launch_ring(once, w4_piece_kernel<GATED, GROUP, P>, kPieceBytes + 1024,
                     dim3((unsigned)(items < blocks ? items : blocks)), dim3(kThreads), (size_t)most * stride, s, a, G,
                     o, S, stride);
}

template <bool GATED, int GROUP>
cudaError_t piece(const W4Args& a, const W4Groups* G, float* o, int most, int pieces, int sms, cudaStream_t s) {
  constexpr int kTok = 8 / (128 / GROUP);
  if (most <= kTok) return piece<GATED, GROUP, 1>(a, G, o, most, pieces, sms, s);
  if constexpr (kTok < 8) return piece<GATED, GROUP, 2>(a, G, o, most, pieces, sms, s);
  return cudaErrorInvalidValue;
}

template <bool GATED>
cudaError_t piece(const W4Args& a, const W4Groups* G, float* o, int most, int pieces, int sms, cudaStream_t s) {
  return a.group == 128  ? piece<GATED, 128>(a, G, o, most, pieces, sms, s)
         : a.group == 64 ? piece<GATED, 64>(a, G, o, most, pieces, sms, s)
                         : piece<GATED, 32>(a, G, o, most, pieces, sms, s);
}

cudaError_t ffn_many(const W4Args& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const int wide = a.H > a.I ? a.H : a.I, R = a.N * a.K;
  int most = (int)(kPieceBytes / ((size_t)(wide + 127) / 128 * 256 + 64));
  const int experts = R < a.E ? R : a.E, one = 8 / (128 / a.group);  // routes of one MMA
  // Pieces of what one MMA takes: the second piece of an expert finds its weights in
  // L2. Of two MMAs' routes where experts have that many each: 16 experts of 4096 x
  // 1408, group 32, 2 routes an expert 54 us and 60, 4 83 and 80, 16 247 and 195; four
  // MMAs' 66, 82 and 213.
  const int take = one < 8 && R >= 2 * one * experts ? 2 * one : one;
  if (most > take) most = take;
  if (most > a.N) most = a.N;
  // pieces there may be: one more for every `most` routes beyond an expert's first
  const int pieces = experts + (R - experts) / most;
  const W4Layout L = w4_layout(a.N, a.K, a.H, a.I);
  uint8_t* ws = a.ws;
  W4Groups* G = reinterpret_cast<W4Groups*>(ws);
  float* o = reinterpret_cast<float*>(ws + L.o);
  err = launch_pdl(w4_group_kernel, dim3(1), dim3(kMaxExperts), 0, s, a.topk_ids, a.topk_p, R, a.K, a.E, most, G);
  if (err != cudaSuccess) return err;
  err = piece<true>(a, G, o, most, pieces, sms, s);
  if (err != cudaSuccess) return err;
  err = piece<false>(a, G, o, most, pieces, sms, s);
  if (err != cudaSuccess) return err;
  return launch_pdl(w4_sum_kernel, dim3((a.H + 1023) / 1024, a.N), dim3(256), 0, s, a, G, o);
}

// One token: x, or h of its routes, has to fit the block's shared memory next to
// six (three) more blocks on the SM.
constexpr size_t kOneBytes = 36 << 10;

template <int GROUP>
cudaError_t matvec_one(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int rows, int cols,
                       uint16_t* y, cudaStream_t s) {
  return launch_pdl(w4_matvec_one_kernel<GROUP>, dim3((rows + 15) / 16), dim3(kOneWarps * 32),
                    (size_t)(cols + 127) / 128 * 256, s, x, q, scale, rows, cols, y);
}

template <int GROUP>
cudaError_t ffn_one(const W4Args& a, cudaStream_t s) {
  const cudaError_t err = launch_pdl(w4_fc1_one_kernel<GROUP>, dim3(a.I / 8, a.K, a.N), dim3(kOneWarps * 32),
                                     (size_t)(a.H + 127) / 128 * 256, s, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(w4_fc2_one_kernel<GROUP>, dim3(a.H / 16, a.N), dim3(kThreads),
                    (size_t)a.K * ((a.I + 127) / 128) * 256, s, a);
}

}  // namespace

int launch_w4_matvec(const uint16_t* x, const uint8_t* q, const uint16_t* scale, int N, int rows,
                     int cols, int group, uint16_t* y, cudaStream_t s) {
  cudaError_t err;
  if (N == 1 && (size_t)cols * 2 <= kOneBytes)
    err = group == 128  ? matvec_one<128>(x, q, scale, rows, cols, y, s)
          : group == 64 ? matvec_one<64>(x, q, scale, rows, cols, y, s)
                        : matvec_one<32>(x, q, scale, rows, cols, y, s);
  else {
    // 16 tokens a block where that leaves every second SM a block: 13 tokens, 4104 x
    // 4096 7.5 us against 10.4, 720 x 6144 6.2 against 4.7
    int sms = 0;
    err = sm_count(&sms);
    if (err != cudaSuccess) return -(int)err;
    err = N <= 8 || 2 * (int64_t)((rows + 15) / 16) * ((N + 15) / 16) < sms
              ? matvec<8>(x, q, scale, N, rows, cols, group, y, s)
              : matvec<16>(x, q, scale, N, rows, cols, group, y, s);
  }
  return err != cudaSuccess ? -(int)err : 1;
}

int64_t w4_workspace_bytes(int N, int K, int H, int I) { return (int64_t)w4_layout(N, K, H, I).total; }

// Each token for itself, as if it were the only one: two launches instead of four, but
// an expert's weights are read for each token that names it. Where few routes share an
// expert (as many as E experts chosen evenly would give), or experts are small: 2 tokens
// of 128 experts of 2048 x 768, group 64, 15 us against 22, 6 (16.5 MB read again) 37.5
// and 39.8, 8 (30 MB) 47 and 44.5; 16 of 8 experts of 512 x 352 10 and 12.7.
constexpr int kAloneTokens = 32;
constexpr double kAloneBytes = 16 << 20;

static bool token_by_token(const W4Args& a) {
  if (a.N == 1) return true;
  if (a.N > kAloneTokens) return false;
  const int chosen = a.K < a.E ? a.K : a.E;  // experts of a token: it reads one named again once
  double none = 1.0;  // that no token names an expert
  for (int t = 0; t < a.N; ++t) none *= 1.0 - (double)chosen / a.E;
  const double again = (double)a.N * chosen - a.E * (1.0 - none);
  return again * 3.0 * a.H * a.I * (0.5 + 2.0 / a.group) <= kAloneBytes;
}

int launch_w4_ffn(const W4Args& args, cudaStream_t s) {
  W4Args a = args;
  a.h = reinterpret_cast<uint16_t*>(a.ws + w4_layout(a.N, a.K, a.H, a.I).h);
  cudaError_t err;
  if (token_by_token(a) && (size_t)a.H * 2 <= kOneBytes && (size_t)a.K * ((a.I + 127) / 128) * 256 <= kOneBytes) {
    err = a.group == 128 ? ffn_one<128>(a, s) : a.group == 64 ? ffn_one<64>(a, s) : ffn_one<32>(a, s);
    return err != cudaSuccess ? -(int)err : 2;
  }
  err = ffn_many(a, s);
  return err != cudaSuccess ? -(int)err : 4;
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
