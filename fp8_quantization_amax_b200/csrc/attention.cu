// Attention of one new token per request over a paged FP8 KV cache (fp8_attention_paged).
//
//   z_j = scale s_k(j) sum_d q_d K_jd,   o_d = sum_j 2^(z_j log2 e - m) s_v(j) V_jd / sum_j 2^(z_j log2 e - m)
//
// over the visible tokens j of a request, K and V the decoded codes, for each query head; `group`
// query heads share a key-value head.  One pass over K and V with the running maximum m and sum
// of the softmax.
//
// What bounds it: the codes, 2 heads head_dim bytes a token, are read once from HBM.  With a
// group of 8 every byte meets 8 multiply-adds, 52 T a second at the memory's rate, above the fp32
// pipes' 36 T: the products go to the tensor cores, m16n8k16 with f16 operands and fp32 sums.
// Every code is exact in f16, and so is a query (bf16) times a power of two of its row, but for elements
// below 2^-31 of the row's largest (off by at most 2^-39 of that).  The softmax weights are rounded to f16:
// half a step is 2^-11 of a weight, below the output's bf16 2^-8, and 2^-34 of the row's largest weight where
// that is more (kUp).  Query rows fill 8 of a tile's rows, so a 128-row tcgen05 tile would be 6 % full.
//
//   S^T (token x query): A = K (rows: 16 tokens), B = q (columns: 8 query heads)
//   O^T (dim x query):   A = V^T (rows: 16 dims),  B = P^T (columns: 8 query heads)
//
// Both results leave a thread (g = lane / 4, t = lane % 4) with columns 2t and 2t + 1: the running
// maximum and sum of its two heads, and the factors that rescale O, are its own.  The weights of
// tokens g, g + 8 become the second product's operand by a transposition of 8 x 8 halves (movmatrix).
// The order of the sum over dims and the dims' order in O^T are free, so thread t reads 16
// contiguous bytes of a K row per 64 dims, and thread g head_dim / 8 contiguous bytes of a V row.
// The maximum follows the scores only when one exceeds it by 2^6 (f16 holds weights to 2^16): a
// vote a tile instead of a reduction, and next to no rescaling.
//
// Each warp streams the tokens of one key-value head on its own through a private ring of
// 16-token stages (cp.async, no barrier between warps), across the requests of its block's share
// without draining; the warps of a block take adjacent heads of the same tokens, so a
// [token][head][dim] page is read in whole rows.  With fewer heads than warps several warps take
// every second, third ... tile of a head and are joined at a request's end through a free stage.
//
// All requests' tiles laid end to end, with what a change of request costs, are divided evenly over
// one wave of blocks (kv_pages.cuh), from the lengths on the device: ragged batches and one long
// request fill the machine alike.  A request whose tiles are shared leaves fp32 partial results,
// joined by a second launch in the blocks' order, so results do not depend on timing.
//
// Measured (us a call, calls back to back in a graph; HBM's floor at 6.53 TB/s):
//   64 requests of 2000 .. 8192 tokens, 64 + 2 * 8 heads of 128    112.3 (102.6: 91 %)
//   one request of 131072 tokens, a scale per token and head        57.1 (42.4)
//   16 requests of 130 .. 4096 tokens, 32 + 2 * 8 heads of 128      21.7 (9.3)
//   16 requests of up to 500 tokens, the same heads                  8.6 (1.7)
//   one request of 33 tokens                                         4.4
// The first runs at HBM's rate but for the 4 us before its first tile and the last blocks' end (350
// instructions for 16 tokens of a head, 53 % of the issue slots); the shorter the work, the more its
// fixed parts show: 4 us to the first tile (lengths, division, table, first copies), 1 us from the last
// block's end to the second launch, 4 us of that.  Copies of whole tiles by the tensor unit (a box of 16
// tokens of a head, a barrier a stage) were slower (116 / 62 us): the boxes are small, and what
// limits the copies is not their instructions.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8q_device.cuh"
#include "internal.h"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace fp8q {
namespace attn {

constexpr int kMaxWarps = 16;
constexpr int kMaxWorkers = 1024;             // blocks of the first launch (one per SM)
// least share of a block, in tiles (one request of 1500 tokens: 10.7 us, with 4 11.3)
constexpr int kMinTiles = 2;
constexpr int kWholeTiles = 8;                // requests of no more tiles a warp are not divided (shape_of)
constexpr int kSpreadRounds = 4;              // few requests of so many tiles a warp have their heads spread,
constexpr int kSpreadPhases = 12;             // with so many warps a head at most (shape_of)
constexpr int64_t kMaxCost = 0x7FFFFFFF;      // of all requests
// a change of request, in tiles of a phase (us at 0 / 1 / 2 / 3 / 5: 16 ragged requests 24.8 23.2 22.1 21.7 22.0, 64
// 113.7 112.5 112.0 112.2 113.2)
constexpr int kTurn = 3;
constexpr int kMaxTokens = 0x7FFFFFFF - 64;   // of one request: token numbers stay inside an int
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;
constexpr int kJoinBatch = 8;                 // parts whose loads are in flight together
// A weight is 1 at the running maximum m, which follows the scores when one exceeds it by 2^kSlack.  For f16
// (2^16 at most) weights are taken times kUp = 2^9, so a row's largest is 2^9 .. 2^(9 + kSlack) and what the
// rounding takes from small ones is at most 2^-34 of it (without the factor, 8192 tokens of weight
// 2^-26 beside one of V = 0 gave 0).  The sum l is of the weights themselves and m the maximum itself, so that
// lse does not lose the bits that a shifted score would have to give up.
// us at slacks 8 / 6 / 4 / 2: window 17.6 17.6 17.9 18.5, one kv head 27.1 26.8 27.4 27.5, the other cases alike.
constexpr float kUp = 512.0f, kDown = 1.0f / kUp, kSlack = 6.0f;
static_assert(kUp * 64.0f < 65504.0f, "weights fit f16");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  KvPages c;
  const uint16_t* q;
  int64_t q_stride;          // elements from request to request
  const int* table;
  const int* lens;
  int batch, max_pages, group;
  int window, sinks;
  float scale2;              // softmax scale times log2 e
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  int vheads, row_tiles;     // (key-value head, tile of query rows) pairs; query-row tiles per head
  int heads_per_block, phases;
  int turn;                  // tiles' worth of a change of request
  int workers;               // gridDim.x of the first launch
  int4* desc;                // per worker: the shared request that begins in its range
  float* part;               // per (worker, first or last request, vhead): a warp's registers
  uint32_t* err;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same on a zero sum
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// four codes -> two f16 pairs (exact)
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kE4M3) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e5m2x2 %0, l; cvt.rn.f16x2.e5m2x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// 2^x.  Results below 2^-126 become zero unless FULL: that takes four instructions in place of one.
// Without scales of single tokens the largest weight of a row is at least 1 and what
// vanishes does not show; a token's scale joins the reference, so with them all weights may be small.
template <bool FULL>
__device__ __forceinline__ float ex2(float x) {
  float y;
  if constexpr (FULL) asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  else asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_normal(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 8 x 8 f16: lane holds row lane / 4, columns 2 (lane % 4) + {0, 1}; the same of the transposed matrix
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 2^(a - b) with b = -inf standing for "nothing yet" (a is -inf too then)
template <bool FULL>
__device__ __forceinline__ float ex2_diff(float a, float b) {
  return b == -INFINITY ? 0.0f : ex2<FULL>(a - b);
}

__device__ __forceinline__ int clamped_len(const Params& p, int b) {
  const int n = p.lens[b];
  return (int)max((int64_t)0, min((int64_t)n, min((int64_t)p.max_pages * p.c.page_size, (int64_t)kMaxTokens)));
}

// Running softmax and product of a warp's query heads, as it lies in a thread's registers: heads
// 8 n + 2 t + e (e = 0, 1) have their reference (base 2) in m[n][e] and, over this thread's tokens
// until reduced, their sum in l[n][e]; o[n][i] holds dims VB g + 2 i (elements e) and VB g + 2 i + 1
// (elements 2 + e).
template <int DP, int NH>
struct State {
  static constexpr int kDimTiles = DP / 16;
  // a tile of 8 heads in memory: o[i] as the float4 32 i + lane, then 8 m, then 8 l
  static constexpr int kTileFloats = 128 * kDimTiles + 16;
  static constexpr int kImage = NH * kTileFloats;
  float m[NH][2], l[NH][2], o[NH][kDimTiles][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
    }
  }
  __device__ __forceinline__ void rescale(int n, float f0, float f1) {
    l[n][0] *= f0;
    l[n][1] *= f1;
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i) {
      o[n][i][0] *= f0;
      o[n][i][1] *= f1;
      o[n][i][2] *= f0;
      o[n][i][3] *= f1;
    }
  }
  __device__ __forceinline__ void reduce_sums() {
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], d);
  }
  __device__ __forceinline__ void store_tile(int n, float* image, int lane) const {
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i)
      reinterpret_cast<float4*>(image)[32 * i + lane] = make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]);
    if (lane < 4) {
      *reinterpret_cast<float2*>(image + 128 * kDimTiles + 2 * lane) = make_float2(m[n][0], m[n][1]);
      *reinterpret_cast<float2*>(image + 128 * kDimTiles + 8 + 2 * lane) = make_float2(l[n][0], l[n][1]);
    }
  }
  // add the heads of tile n over other tokens
  template <bool FULL>
  __device__ __forceinline__ void add_tile(int n, const float* image, int lane) {
    const float2 um = *reinterpret_cast<const float2*>(image + 128 * kDimTiles + 2 * (lane & 3));
    const float2 ul = *reinterpret_cast<const float2*>(image + 128 * kDimTiles + 8 + 2 * (lane & 3));
    const float m0 = fmaxf(m[n][0], um.x), m1 = fmaxf(m[n][1], um.y);
    const float u0 = ex2_diff<FULL>(um.x, m0), u1 = ex2_diff<FULL>(um.y, m1);
    rescale(n, ex2_diff<FULL>(m[n][0], m0), ex2_diff<FULL>(m[n][1], m1));
    m[n][0] = m0;
    m[n][1] = m1;
    l[n][0] += ul.x * u0;
    l[n][1] += ul.y * u1;
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i) {
      const float4 x = reinterpret_cast<const float4*>(image)[32 * i + lane];
      o[n][i][0] += x.x * u0;
      o[n][i][1] += x.y * u1;
      o[n][i][2] += x.z * u0;
      o[n][i][3] += x.w * u1;
    }
  }
};

// ln(2^m l).  With scales of tokens m and log l may be far from 0 and cancel: l's exponent meets m first, or the
// logarithm's error would be one of their size
template <bool TOKEN_SCALES>
__device__ __forceinline__ float lse_of(float m, float l) {
  if constexpr (TOKEN_SCALES) {
    const uint32_t bits = __float_as_uint(l), exponent = bits >> 23;
    if (exponent - 1u < 254u)                // neither 0, subnormal, infinite nor NaN
      return kLn2 * ((m + (float)((int)exponent - 127)) + lg2(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u)));
  }
  return l == 0.0f ? -INFINITY : kLn2 * (m + lg2(l));
}

// out[b][head][dim] and lse of a finished state; vs: V's scale where it is one for the head
template <int DP, int NH, bool TOKEN_SCALES>
__device__ __forceinline__ void write_rows(const Params& p, State<DP, NH>& s, int b, int vh, float vs, int lane) {
  constexpr int VB = DP / 8;
  const int g = lane >> 2, t = lane & 3;
  const int kvh = vh / p.row_tiles, r0 = (vh - kvh * p.row_tiles) * 8 * NH;
  const int D = p.c.head_dim;
#pragma unroll
  for (int n = 0; n < NH; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * n + 2 * t + e;
      if (r >= p.group) continue;
      const float l = s.l[n][e], f = vs * (kDown * rcp(l));
      if (p.lse && g == 0)
        p.lse[(int64_t)b * (p.c.heads * p.group) + kvh * p.group + r] = lse_of<TOKEN_SCALES>(s.m[n][e], l);
      uint16_t* dst = p.out + (int64_t)b * p.out_stride + (int64_t)(kvh * p.group + r) * D + g * VB;
#pragma unroll
      for (int c = 0; c < VB / 8; ++c) {
        if (g * VB + 8 * c >= D) continue;
        uint4 w;
        w.x = f32x2_to_bf16x2(s.o[n][4 * c + 0][e] * f, s.o[n][4 * c + 0][2 + e] * f);
        w.y = f32x2_to_bf16x2(s.o[n][4 * c + 1][e] * f, s.o[n][4 * c + 1][2 + e] * f);
        w.z = f32x2_to_bf16x2(s.o[n][4 * c + 2][e] * f, s.o[n][4 * c + 2][2 + e] * f);
        w.w = f32x2_to_bf16x2(s.o[n][4 * c + 3][e] * f, s.o[n][4 * c + 3][2 + e] * f);
        *reinterpret_cast<uint4*>(dst + 8 * c) = w;
      }
    }
  }
}

// Position of 16-byte piece `c` of row `row` in a stage: pieces are exchanged within a row so that
// the eight threads of a shared-memory access phase (rows g, g + 1 and pieces t of K; rows 2t and
// pieces g, g + 1 of V) fall on different banks for 128-byte rows.  Rows r and r + 8 are alike.
template <int DP>
__device__ __forceinline__ int swizzled(int row, int c) {
  if constexpr (DP == 64) {
    return c ^ (((row >> 1) & 1) << 1);
  } else {
    return c ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2));
  }
}

template <int DP>
constexpr int kStageBytes = 2 * kAttnTile * DP + 2 * kAttnTile * 4;

// One block per SM.  Up to 128 registers a thread 16 warps share an SM (us with 16 / with 8 warps: 64 requests of
// up to 8192 tokens 112.0 / 123.4, one of 131072 57.5 / 64.4, 16 of up to 4096 21.7 / 21.9); two row tiles of 128
// dims or one of 256 need more, and 8 warps.
__host__ __device__ constexpr int warps_of(int dp, int nh) { return dp * nh <= 128 ? 16 : 8; }
// Two row tiles of 256 dims leave no registers for the query fragments: they lie in shared memory, each
// thread's own, beside two stages.  Else as many stages as fit in about 200 KB, at most 6
__host__ __device__ constexpr bool shared_q(int dp, int nh) { return dp * nh > 256; }
// of a warp
__host__ __device__ constexpr int query_bytes(int dp, int nh) { return shared_q(dp, nh) ? 16 * nh * dp : 0; }
__host__ __device__ constexpr int stages_of(int dp, int nh) {
  return shared_q(dp, nh) ? 2
         : 204800 / (warps_of(dp, nh) * (2 * kAttnTile * dp + 2 * kAttnTile * 4)) < 6
             ? 204800 / (warps_of(dp, nh) * (2 * kAttnTile * dp + 2 * kAttnTile * 4)) : 6;
}

// Sum over the threads up to and including this one, and over the block (in *any: is `flag` set in any
// thread).  sh: kMaxWarps entries that no thread still reads
__device__ __forceinline__ int block_sum(int v, bool flag, int* sh, int* all, bool* any) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  if (lane == 31) sh[warp] = v;
  *any = __syncthreads_or(flag) != 0;
  const int warps = blockDim.x >> 5;
  int before = 0, total = 0;
#pragma unroll
  for (int k = 0; k < kMaxWarps; ++k) {
    const int x = k < warps ? sh[k] : 0;
    if (k < warp) before += x;
    total += x;
  }
  *all = total;
  return v + before;
}

// The tiles of one request that a block holds.
struct Cursor {
  int b;           // request; the batch size when there is none left
  int n;           // its tokens
  int first, end;  // its tiles [first, end) are the block's
  int left;        // the block's share from tile `first` on
  int tiles;       // all its tiles
};

__device__ __forceinline__ void enter(const Params& p, Cursor& c, int first) {
  c.n = clamped_len(p, c.b);
  c.tiles = attn_range(c.n, p.window, p.sinks).tiles;
  c.first = first;
  c.end = p.part ? min(c.tiles, first + c.left) : c.tiles;         // (undivided: see Shape)
}
// to the next request with tiles
__device__ __forceinline__ void advance(const Params& p, Cursor& c) {
  c.left -= c.tiles + p.turn - c.first;
  do {
    ++c.b;
    if (c.left <= 0) c.b = p.batch;
    if (c.b >= p.batch) {
      c.b = p.batch;
      c.n = c.first = c.end = c.tiles = 0;
      return;
    }
    enter(p, c, 0);
  } while (c.tiles == 0);
}

template <int FMT, int DP, int NH, bool TOKEN_SCALES>
__global__ void __launch_bounds__(32 * warps_of(DP, NH), 1) k_attention(const Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) int sh_sum[2][kMaxWarps];
  __shared__ int sh_base, sh_req;
  __shared__ int sh_free[kMaxWarps];         // each warp's free stage at a request's end
  constexpr int DPC = DP / 16;               // 16-byte pieces of a padded row
  constexpr int RPI = 32 / DPC;              // rows one warp-wide copy covers
  constexpr int VB = DP / 8;
  constexpr int kStages = stages_of(DP, NH);
  constexpr int kBytes = kStageBytes<DP>;
  using St = State<DP, NH>;
  static_assert(St::kTileFloats * 4 <= kBytes, "a stage holds the state of 8 heads");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int phase = warp / p.heads_per_block;
  const int vh = blockIdx.y * p.heads_per_block + warp % p.heads_per_block;
  const bool active = vh < p.vheads;         // the last group of heads may be short
  const int kvh = active ? vh / p.row_tiles : 0;
  const int r0 = active ? (vh - kvh * p.row_tiles) * 8 * NH : 0;
  const int D = p.c.head_dim;

  if (threadIdx.x == 0) sh_req = p.batch;
  if (p.batch > 0) prefetch_l2(p.lens + min((int)threadIdx.x, p.batch - 1));
  allow_dependent_launch();
  grid_dependency_wait();

  const int w = blockIdx.x;
  // a request without a visible token: zeros, and an empty sum
  auto write_empty = [&](int b) {
    if (!active || phase > 0) return;
    for (int r = r0; r < min(p.group, r0 + 8 * NH); ++r) {
      uint16_t* dst = p.out + (int64_t)b * p.out_stride + (int64_t)(kvh * p.group + r) * D;
      if (8 * lane < D) *reinterpret_cast<uint4*>(dst + 8 * lane) = make_uint4(0, 0, 0, 0);
      if (p.lse && lane == 0) p.lse[(int64_t)b * (p.c.heads * p.group) + kvh * p.group + r] = -INFINITY;
    }
  };
  int workers = p.workers, t_begin = 0, t_end = 1;
  AttnSplit split = {0, 0};
  if (!p.part && p.batch <= p.workers) {
    // ---- undivided requests, no more than blocks: each has its own
    if (w >= p.batch) return;
    if (clamped_len(p, w) == 0) {
      write_empty(w);
      return;
    }
    if (threadIdx.x == 0) sh_req = w, sh_base = 0;
  } else {
    // ---- the cost of all requests; this block's share of it, and the request it begins in.  With at
    // most one request a thread one sum over the block gives all.
    const bool single = p.batch <= (int)blockDim.x;
    int mine = 0;
    bool empty = false;
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
      const int n = attn_cost(attn_range(clamped_len(p, b), p.window, p.sinks).tiles, p.turn);
      mine += n;
      empty |= n == 0;
    }
    int total;
    bool any_empty;
    const int upto = block_sum(mine, empty, sh_sum[0], &total, &any_empty);
    workers = attn_workers(total, p.workers, kMinTiles);
    if (blockIdx.y == 0 && threadIdx.x == 0 && p.desc) p.desc[w] = make_int4(-1, 0, 0, 0);

    if (any_empty)
      for (int b = w; b < p.batch; b += p.workers)
        if (clamped_len(p, b) == 0) write_empty(b);
    if (w >= workers || total == 0) return;
    split = attn_split(total, workers);
    t_begin = attn_start(split, w);
    t_end = attn_start(split, w + 1);
    if (single) {
      if (mine > 0 && upto - mine <= t_begin && t_begin < upto) {
        sh_req = threadIdx.x;
        sh_base = upto - mine;
      }
    } else {
      int before = 0;
      for (int b0 = 0, turn = 1; b0 < p.batch; b0 += blockDim.x, turn ^= 1) {
        const int b = b0 + threadIdx.x;
        const int n = b < p.batch ? attn_cost(attn_range(clamped_len(p, b), p.window, p.sinks).tiles, p.turn) : 0;
        int all;
        bool any;
        const int incl = before + block_sum(n, false, sh_sum[turn], &all, &any);
        if (n > 0 && incl - n <= t_begin && t_begin < incl) {
          sh_req = b;
          sh_base = incl - n;
        }
        before += all;
        if (before > t_begin) break;           // the same for every thread
      }
    }
  }
  const uint32_t ring_u = smem_u32(smem) + (uint32_t)warp * (kStages * kBytes);
  // this thread's query fragments behind all rings, 16 bytes every 512
  constexpr bool kSharedQ = shared_q(DP, NH);
  const uint32_t q_u = smem_u32(smem) + (blockDim.x >> 5) * (kStages * kBytes) + (uint32_t)warp * query_bytes(DP, NH) +
                       16 * lane;
  if (D < DP) {
    // the pieces past head_dim stay zero: no copy writes them
    for (int i = lane; i < kStages * kBytes / 16; i += 32)
      *reinterpret_cast<uint4*>(smem + (size_t)warp * (kStages * kBytes) + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  if (!active || sh_req >= p.batch) return;

  float vscale = 1.0f, kscale = 1.0f;
  if constexpr (!TOKEN_SCALES) {
    const int i = p.c.gran == 0 ? 0 : kvh;
    kscale = p.c.ks[i];
    vscale = p.c.vs[i];
  }
  const uint8_t* kbase = p.c.k + (int64_t)kvh * p.c.head_stride;
  const uint8_t* vbase = p.c.v + (int64_t)kvh * p.c.head_stride;
  // tokens of a block that lies in one page: 16, 8, or 0 where pages do not divide into such
  const int sub = p.c.page_size % 16 == 0 ? 16 : p.c.page_size % 8 == 0 ? 8 : 0;
  const int row0 = lane / DPC, piece = lane % DPC;                 // this lane's first row and its piece in a copy
  const bool has_piece = 16 * piece < D;
  const uint32_t token16 = (uint32_t)(p.c.token_stride / 16), page16 = (uint32_t)(p.c.page_stride / 16);

  Cursor load, c;                            // of the copies, and of the products
  c.b = sh_req;
  c.left = t_end - t_begin;
  enter(p, c, t_begin - sh_base);
  // the share begins behind the request's last tile; undivided requests are their first tile's block's
  if (c.first >= c.tiles || (!p.part && c.first > 0)) advance(p, c);
  load = c;

  auto tile_token = [&](int i, int n) {
    if (p.window > 0) {
      const AttnRange r = attn_range(n, p.window, p.sinks);
      if (i >= r.head) i += r.skip;
    }
    return i * kAttnTile;
  };
  auto visible = [&](int tok, int n) { return tok < n && (p.window == 0 || tok >= n - p.window || tok < p.sinks); };
  auto all_visible = [&](int tok0, int n) {
    return tok0 + kAttnTile <= n && (p.window == 0 || tok0 >= n - p.window || tok0 + kAttnTile <= p.sinks);
  };
  auto prefetch_q = [&](int b) {
    const int bytes = min(8 * NH, p.group - r0) * D * 2;
    if (lane * 128 < bytes)
      prefetch_l2(p.q + (int64_t)b * p.q_stride + (int64_t)(kvh * p.group + r0) * D + lane * 64);
  };

  // this lane's scales, of K (lanes 0 .. 15) or V, and a slot's place among them (slots are below 2^31)
  const float* const scales = (lane < 16 ? p.c.ks : p.c.vs) +
                              (p.c.gran == 2 ? kvh : (int64_t)kvh * ((int64_t)p.c.num_pages * p.c.page_size));
  auto scale_at = [&](int slot) { return p.c.gran == 2 ? (int64_t)(slot >> 7) * p.c.heads : (int64_t)slot; };

  // ---- copies: `i_load` is the next tile to copy.  Where pages divide into blocks of `sub` tokens, lane l
  // holds the page of the l-th block from the tile i_load - used on, and its place in the page; else
  // those of this lane's token (lane % 16) of the next tile.  -1 where there is none
  int i_load = load.first + phase, pages = -1, offs = 0, used = 32;
  auto find_pages = [&]() {
    while (i_load >= load.end && load.b < p.batch) {
      advance(p, load);
      i_load = load.first + phase;
      used = 32;
      if (load.b < p.batch) prefetch_q(load.b);
    }
    if (load.b >= p.batch || (sub > 0 && used < 32)) return;
    int i = i_load, tok = lane & 15;
    if (sub == 16) i += lane * p.phases, tok = 0;
    if (sub == 8) i += (lane >> 1) * p.phases, tok = 8 * (lane & 1);
    pages = -1;
    if (i < load.end) {                      // (a place past the request's last tile may leave the tokens' range)
      tok += tile_token(i, load.n);
      const uint32_t col = div_u32((uint32_t)tok, p.c.page_div);
      offs = tok - (int)(col * (uint32_t)p.c.page_size);
      if (tok < load.n) pages = p.table[(int64_t)load.b * p.max_pages + col];
    }
    used = 0;
  };
  auto issue = [&](int slot_index) {
    if (load.b < p.batch) {
      const uint32_t dst = ring_u + slot_index * kBytes;
      const int tok_load = tile_token(i_load, load.n);
      bool whole = sub > 0 && all_visible(tok_load, load.n);
      int page = pages, off = offs, page8 = 0, off8 = 0;           // of the tile's tokens 0 .. 7 or 15, and of 8 .. 15
      if (sub > 0) {
        page = __shfl_sync(0xFFFFFFFFu, pages, used);
        off = __shfl_sync(0xFFFFFFFFu, offs, used++);
        page8 = page;
        off8 = off + 8;
        if (sub == 8) {
          page8 = __shfl_sync(0xFFFFFFFFu, pages, used);
          off8 = __shfl_sync(0xFFFFFFFFu, offs, used++);
        }
        whole = whole && (uint32_t)page < (uint32_t)p.c.num_pages && (uint32_t)page8 < (uint32_t)p.c.num_pages;
      }
      if (whole) {
        if (has_piece) {
          // places in units of 16 bytes fit 32 bits (checked on the host)
          uint32_t at = (uint32_t)page * page16 + (uint32_t)(off + row0) * token16 + piece;
          const uint32_t at8 = (uint32_t)page8 * page16 + (uint32_t)(off8 + row0) * token16 + piece;
#pragma unroll
          for (int k = 0; k < kAttnTile / RPI; ++k) {
            if (k * RPI == 8) at = at8;
            const uint32_t to = dst + row0 * DP + 16 * swizzled<DP>(k * RPI + row0, piece) + k * RPI * DP;
            cp_async16(to, kbase + (uint64_t)at * 16);
            cp_async16(to + kAttnTile * DP, vbase + (uint64_t)at * 16);
            at += RPI * token16;
          }
        }
        if constexpr (TOKEN_SCALES) {
          const int slot = ((lane & 8) ? page8 : page) * p.c.page_size + ((lane & 8) ? off8 : off) + (lane & 7);
          cp_async4(dst + 2 * kAttnTile * DP + 4 * lane, scales + scale_at(slot));
        }
      } else {
        // this lane's token, lane % 16
        if (sub > 0) {
          if (lane & 8) page = page8, off = off8;
          off += lane & 7;
        }
        const bool ok = (uint32_t)page < (uint32_t)p.c.num_pages;
        const bool see = visible(tok_load + (lane & 15), load.n);
        if (!ok && see) raise_device_error(p.err, kErrBadPage);
        const uint32_t place = (uint32_t)page * page16 + (uint32_t)off * token16;
        const uint32_t seen = __ballot_sync(0xFFFFFFFFu, ok && see);
#pragma unroll
        for (int k = 0; k < kAttnTile / RPI; ++k) {
          const int row = k * RPI + row0;
          const uint32_t at = __shfl_sync(0xFFFFFFFFu, place, row) + piece;
          const bool take = (seen >> row) & 1u;
          const uint64_t from = take ? (uint64_t)at * 16 : 0;
          const uint32_t to = dst + row0 * DP + 16 * swizzled<DP>(k * RPI + row0, piece) + k * RPI * DP;
          if (has_piece) {
            cp_async16_or_zero(to, kbase + from, take);
            cp_async16_or_zero(to + kAttnTile * DP, vbase + from, take);
          }
        }
        if constexpr (TOKEN_SCALES) {
          const bool take = (seen >> (lane & 15)) & 1u;
          cp_async4_or_zero(dst + 2 * kAttnTile * DP + 4 * lane,
                            scales + scale_at(take ? page * p.c.page_size + off : 0), take);
        }
      }
      i_load += p.phases;
    }
    cp_async_commit();
  };

  // ---- query heads: 16 dims of a row a thread, of the request c.b
  uint32_t qb[NH][DP / 64][8];
  auto load_q = [&](int b) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int r = r0 + 8 * h + g;
      const uint16_t* src = p.q + (int64_t)b * p.q_stride + (int64_t)(kvh * p.group + min(r, p.group - 1)) * D;
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        const int k = t + 4 * j;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (r < p.group && 16 * k < D) {
          x = *reinterpret_cast<const uint4*>(src + 16 * k);
          y = *reinterpret_cast<const uint4*>(src + 16 * k + 8);
        }
        qb[h][j][0] = x.x, qb[h][j][1] = x.y, qb[h][j][2] = x.z, qb[h][j][3] = x.w;
        qb[h][j][4] = y.x, qb[h][j][5] = y.y, qb[h][j][6] = y.z, qb[h][j][7] = y.w;
      }
    }
  };

  find_pages();
#pragma unroll 1
  for (int k = 0; k < kStages - 1; ++k) {
    issue(k);
    find_pages();
  }
  int stage = 0;                             // the next stage to be read; the one before it is free

  while (c.b < p.batch) {
    const int n = c.n;
    load_q(c.b);
    // ---- query heads as B fragments: f16 after a power of two that brings a head's largest element to
    // 2^14 .. 2^15; the inverse power joins the score's factor
    float qmul[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      uint32_t mx = 0;
#pragma unroll
      for (int j = 0; j < DP / 64; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = absmax2(mx, qb[h][j][i]);
      mx = absmax2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = absmax2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const uint32_t ex = __float_as_uint(packed_amax_to_f32(mx)) >> 23;   // biased exponent of the largest
      const uint32_t up = ex == 255u ? 127u : min(268u - ex, 253u);
      const float f = __uint_as_float(up << 23);
      const float back = __uint_as_float((254u - up) << 23) * p.scale2 * kscale;
      qmul[h][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * t);
      qmul[h][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) qb[h][j][i] = pack_f16(bf16_lo(qb[h][j][i]) * f, bf16_hi(qb[h][j][i]) * f);
        if constexpr (kSharedQ) {
          sts128(q_u + ((h * (DP / 64) + j) * 2) * 512, qb[h][j][0], qb[h][j][1], qb[h][j][2], qb[h][j][3]);
          sts128(q_u + ((h * (DP / 64) + j) * 2 + 1) * 512, qb[h][j][4], qb[h][j][5], qb[h][j][6], qb[h][j][7]);
        }
      }
    }

    St s;
    s.clear();
    for (int i = c.first + phase; i < c.end; i += p.phases) {
      cp_async_wait<kStages - 2>();
      __syncwarp();                          // the stage has landed for every lane; the one before is read out
      issue(stage == 0 ? kStages - 1 : stage - 1);
      find_pages();
      const uint32_t ks = ring_u + stage * kBytes;
      const uint32_t vs = ks + kAttnTile * DP;
      const uint32_t sc = vs + kAttnTile * DP;
      stage = stage == kStages - 1 ? 0 : stage + 1;

      // ---- S^T = K q^T: elements 0, 1 are token g, elements 2, 3 token g + 8
      float st[NH][4];
#pragma unroll
      for (int d = 0; d < DP / 64; ++d) {
        const uint32_t at = ks + g * DP + 16 * swizzled<DP>(g, t + 4 * d);
        const uint4 x = lds128(at), y = lds128(at + 8 * DP);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
        uint32_t qd[NH][8];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if constexpr (kSharedQ) {
            const uint32_t at_q = q_u + (h * (DP / 64) + d) * 1024;
            const uint4 q0 = lds128(at_q), q1 = lds128(at_q + 512);
            qd[h][0] = q0.x, qd[h][1] = q0.y, qd[h][2] = q0.z, qd[h][3] = q0.w;
            qd[h][4] = q1.x, qd[h][5] = q1.y, qd[h][6] = q1.z, qd[h][7] = q1.w;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) qd[h][k] = qb[h][d][k];
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t a0, a1, a2, a3;
          decode4<FMT>(xw[m], a0, a2);
          decode4<FMT>(yw[m], a1, a3);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            if (d == 0 && m == 0) mma_f16_first(st[h], a0, a1, a2, a3, qd[h][2 * m], qd[h][2 * m + 1]);
            else mma_f16(st[h], a0, a1, a2, a3, qd[h][2 * m], qd[h][2 * m + 1]);
          }
        }
      }

      // ---- softmax weights
      float vf[2], vl[2];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[h][e] *= qmul[h][e & 1];
      if constexpr (TOKEN_SCALES) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float kf = lds32(sc + 4 * (g + 8 * k));
          vf[k] = lds32(sc + 4 * (16 + g + 8 * k));
          vl[k] = lg2_normal(fmaxf(fabsf(vf[k]), 0x1.0p-60f));
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            st[h][2 * k] *= kf;
            st[h][2 * k + 1] *= kf;
          }
        }
      }
      const int tok0 = tile_token(i, n);
      if (!all_visible(tok0, n)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (!visible(tok0 + g + 8 * k, n)) {
#pragma unroll
            for (int h = 0; h < NH; ++h) st[h][2 * k] = st[h][2 * k + 1] = -INFINITY;
          }
      }
      // The magnitude of V's scale counts towards the reference, so that a weight times its scale fits f16
      // (one below 2^-60 counts as that: the weight itself, at most 2^66 then, has to fit fp32)
      bool above = false;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          above |= (TOKEN_SCALES ? st[h][e] + vl[e >> 1] : st[h][e]) > s.m[h][e & 1] + kSlack;
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float top[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = TOKEN_SCALES ? fmaxf(st[h][e] + vl[0], st[h][2 + e] + vl[1]) : fmaxf(st[h][e], st[h][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], d));
            top[e] = fmaxf(top[e], s.m[h][e]);
          }
          s.rescale(h, ex2_diff<TOKEN_SCALES>(s.m[h][0], top[0]), ex2_diff<TOKEN_SCALES>(s.m[h][1], top[1]));
          s.m[h][0] = top[0];
          s.m[h][1] = top[1];
        }
      }
      uint32_t pb[NH][2];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float m0 = s.m[h][0] == -INFINITY ? 0.0f : s.m[h][0], m1 = s.m[h][1] == -INFINITY ? 0.0f : s.m[h][1];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float a = ex2<TOKEN_SCALES>(st[h][2 * k] - m0), e = ex2<TOKEN_SCALES>(st[h][2 * k + 1] - m1);
          s.l[h][0] += a;
          s.l[h][1] += e;
          float2 w = make_float2(a, e);
          if constexpr (TOKEN_SCALES) w = __fmul2_rn(w, make_float2(vf[k], vf[k]));
          w = __fmul2_rn(w, make_float2(kUp, kUp));
          pb[h][k] = transpose8(pack_f16(w.x, w.y));
        }
      }

      // ---- O^T += V^T P^T
      constexpr int VW = VB / 4;             // words of a row a thread reads
      uint32_t v[4][VW];                     // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 2 * t + (k & 1);
        if constexpr (DP == 64) {
          const uint2 x = lds64(vs + r * DP + 16 * swizzled<DP>(r, g >> 1) + 8 * (g & 1) + 8 * (k >> 1) * DP);
          v[k][0] = x.x, v[k][1] = x.y;
        } else {
#pragma unroll
          for (int e = 0; e < VB / 16; ++e) {
            const uint4 x = lds128(vs + r * DP + 16 * swizzled<DP>(r, g * (VB / 16) + e) + 8 * (k >> 1) * DP);
            v[k][4 * e] = x.x, v[k][4 * e + 1] = x.y, v[k][4 * e + 2] = x.z, v[k][4 * e + 3] = x.w;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < VW; ++m) {
        // bytes of both tokens side by side: dims 4 m, 4 m + 1 and 4 m + 2, 4 m + 3
        uint32_t a0, a1, a2, a3;
        decode4<FMT>(__byte_perm(v[0][m], v[1][m], 0x5140), a0, a1);
        decode4<FMT>(__byte_perm(v[2][m], v[3][m], 0x5140), a2, a3);
#pragma unroll
        for (int h = 0; h < NH; ++h) mma_f16(s.o[h][2 * m], a0, a1, a2, a3, pb[h][0], pb[h][1]);
        decode4<FMT>(__byte_perm(v[0][m], v[1][m], 0x7362), a0, a1);
        decode4<FMT>(__byte_perm(v[2][m], v[3][m], 0x7362), a2, a3);
#pragma unroll
        for (int h = 0; h < NH; ++h) mma_f16(s.o[h][2 * m + 1], a0, a1, a2, a3, pb[h][0], pb[h][1]);
      }
    }

    // ---- the request's end: warps that shared a head's tiles meet, and the first adds up the others'
    // states from their free stages
    s.reduce_sums();
    if (p.phases > 1) {
      const uint32_t bar = 1 + warp % p.heads_per_block, threads = 32 * p.phases;
      const int free_stage = stage == 0 ? kStages - 1 : stage - 1;
      uint8_t* mine_at = smem + (size_t)warp * (kStages * kBytes) + free_stage * kBytes;
      if (lane == 0) sh_free[warp] = free_stage;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        __syncwarp();                        // every lane has read the stage
        if (phase > 0) s.store_tile(h, reinterpret_cast<float*>(mine_at), lane);
        named_barrier(bar, threads);
        if (phase == 0)
          for (int k = 1; k < p.phases; ++k) {
            const int other = warp + k * p.heads_per_block;
            const uint8_t* from = smem + ((size_t)other * kStages + sh_free[other]) * kBytes;
            s.template add_tile<TOKEN_SCALES>(h, reinterpret_cast<const float*>(from), lane);
          }
        named_barrier(bar, threads);         // the stages are read before they are written again
      }
      if (D < DP && phase > 0) {
        // the free stage's pieces past head_dim are zero again
        for (int i = lane; i < kBytes / 16; i += 32) reinterpret_cast<uint4*>(mine_at)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
    }
    const bool opens = c.first == 0, closes = c.end == c.tiles;
    const int place = c.left == t_end - t_begin ? 0 : 1;        // the block's first request, or a later one
    if (phase == 0) {
      if (opens && closes) {
        write_rows<DP, NH, TOKEN_SCALES>(p, s, c.b, vh, vscale, lane);
      } else {
#pragma unroll
        for (int h = 0; h < NH; ++h)
          s.store_tile(h, p.part + ((int64_t)(2 * w + place) * p.vheads + vh) * St::kImage + h * St::kTileFloats, lane);
      }
    }
    if (opens && !closes && blockIdx.y == 0 && threadIdx.x == 0)
      p.desc[w] = make_int4(c.b, place, w, min(workers - 1, attn_owner(split, t_end - c.left + c.tiles - 1)));
    advance(p, c);
  }
  cp_async_wait<0>();
}

// Second launch: adds up the parts of each shared request.  A unit is one dim tile of a row tile of
// one (request, vhead), 16 bytes of a part a thread.  Where units are few, several warps share one
// (each takes every wpu-th part) and are added in shared memory in their order.
template <int DP, int NH, bool TOKEN_SCALES>
__global__ void __launch_bounds__(kJoinThreads) k_attention_join(const Params p) {
  using St = State<DP, NH>;
  constexpr int kUnits = NH * St::kDimTiles;
  constexpr int VB = DP / 8;
  __shared__ int4 list[kMaxWorkers];
  __shared__ int sh_count[kJoinWarps];
  __shared__ float sh[kJoinWarps][8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  allow_dependent_launch();
  grid_dependency_wait();

  // ---- the shared requests, in the workers' order
  int count = 0;
  for (int w0 = 0; w0 < p.workers; w0 += kJoinThreads) {
    const int w = w0 + threadIdx.x;
    const int4 d = w < p.workers ? p.desc[w] : make_int4(-1, 0, 0, 0);
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, d.x >= 0);
    if (w0 > 0) __syncthreads();
    if (lane == 0) sh_count[warp] = __popc(has);
    __syncthreads();
    int at = count + __popc(has & ((1u << lane) - 1u));
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) {
      if (k < warp) at += sh_count[k];
      count += sh_count[k];
    }
    if (d.x >= 0) list[at] = d;
  }
  __syncthreads();
  // (at most kMaxWorkers requests of 65536 heads: below 2^31)
  const uint32_t pairs = (uint32_t)count * (uint32_t)p.vheads, units = pairs * kUnits;
  uint32_t wpu = 1;                          // warps a unit
  while (wpu < kJoinWarps && units * (2 * wpu) <= gridDim.x * kJoinWarps) wpu *= 2;
  const uint32_t per_block = kJoinWarps / wpu, mine = warp & (wpu - 1);
  const int64_t part_floats = (int64_t)p.vheads * St::kImage;      // of one (worker, first or last request)
  for (uint32_t u0 = blockIdx.x * per_block; u0 < units; u0 += gridDim.x * per_block) {
    const uint32_t u = u0 + warp / wpu;
    const bool live = u < units;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int4 e = make_int4(0, 0, 0, -1);
    int vh = 0, n = 0, tile = 0;
    if (live) {
      const uint32_t part = u % kUnits, v = u / kUnits, r = v / (uint32_t)p.vheads;
      vh = (int)(v - r * (uint32_t)p.vheads);
      e = list[r];
      n = part / St::kDimTiles;
      tile = part % St::kDimTiles;
      // a part's rows of this tile; the first worker holds them as its first or its last request's, the
      // others as their first
      const float* at = p.part + (int64_t)(2 * (e.z + (int)mine)) * part_floats + vh * St::kImage + n * St::kTileFloats;
      if (mine == 0) at += e.y * part_floats;
      for (int x0 = e.z + (int)mine; x0 <= e.w; x0 += wpu * kJoinBatch) {
        float2 um[kJoinBatch], ul[kJoinBatch];
        float4 uo[kJoinBatch];
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
          um[k] = make_float2(-INFINITY, -INFINITY);
          ul[k] = make_float2(0.0f, 0.0f);
          uo[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (x0 + k * (int)wpu <= e.w) {
            um[k] = *reinterpret_cast<const float2*>(at + 128 * St::kDimTiles + 2 * t);
            ul[k] = *reinterpret_cast<const float2*>(at + 128 * St::kDimTiles + 8 + 2 * t);
            uo[k] = reinterpret_cast<const float4*>(at)[32 * tile + lane];
            at += 2 * wpu * part_floats - (x0 + k == e.z ? e.y * part_floats : 0);
          }
        }
        float a0 = m0, a1 = m1;
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) a0 = fmaxf(a0, um[k].x), a1 = fmaxf(a1, um[k].y);
        const float f0 = ex2_diff<TOKEN_SCALES>(m0, a0), f1 = ex2_diff<TOKEN_SCALES>(m1, a1);
        m0 = a0;
        m1 = a1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] *= (j & 1) ? f1 : f0;
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
          const float h0 = ex2_diff<TOKEN_SCALES>(um[k].x, m0), h1 = ex2_diff<TOKEN_SCALES>(um[k].y, m1);
          l0 += ul[k].x * h0;
          l1 += ul[k].y * h1;
          o[0] += uo[k].x * h0;
          o[1] += uo[k].y * h1;
          o[2] += uo[k].z * h0;
          o[3] += uo[k].w * h1;
        }
      }
    }
    if (wpu > 1) {
      __syncthreads();                       // sh of the unit before has been read
      sh[warp][0][lane] = m0;
      sh[warp][1][lane] = m1;
      sh[warp][2][lane] = l0;
      sh[warp][3][lane] = l1;
#pragma unroll
      for (int j = 0; j < 4; ++j) sh[warp][4 + j][lane] = o[j];
      __syncthreads();
      if (mine == 0) {
#pragma unroll 1
        for (int k = warp + 1; k < warp + (int)wpu; ++k) {
          const float b0 = sh[k][0][lane], b1 = sh[k][1][lane];
          const float a0 = fmaxf(m0, b0), a1 = fmaxf(m1, b1);
          const float f0 = ex2_diff<TOKEN_SCALES>(m0, a0), f1 = ex2_diff<TOKEN_SCALES>(m1, a1);
          const float h0 = ex2_diff<TOKEN_SCALES>(b0, a0), h1 = ex2_diff<TOKEN_SCALES>(b1, a1);
          m0 = a0;
          m1 = a1;
          l0 = l0 * f0 + sh[k][2][lane] * h0;
          l1 = l1 * f1 + sh[k][3][lane] * h1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = (j & 1) ? o[j] * f1 + sh[k][4 + j][lane] * h1 : o[j] * f0 + sh[k][4 + j][lane] * h0;
        }
      }
    }
    if (live && mine == 0) {
      float vs = 1.0f;
      if constexpr (!TOKEN_SCALES) vs = p.c.vs[p.c.gran == 0 ? 0 : vh / p.row_tiles];
      const int kvh = vh / p.row_tiles, row = (vh - kvh * p.row_tiles) * 8 * NH + 8 * n + 2 * t;
      const int dim = g * VB + 2 * tile;     // o holds dims dim, dim + 1 of rows row, row + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (row + r >= p.group) continue;
        const float l = r ? l1 : l0, m = r ? m1 : m0, f = vs * (kDown * rcp(l));
        const int64_t head = kvh * p.group + row + r;
        if (p.lse && tile == 0 && g == 0)
          p.lse[(int64_t)e.x * (p.c.heads * p.group) + head] = lse_of<TOKEN_SCALES>(m, l);
        if (dim < p.c.head_dim)
          *reinterpret_cast<uint32_t*>(p.out + (int64_t)e.x * p.out_stride + head * p.c.head_dim + dim) =
              f32x2_to_bf16x2(o[r] * f, o[2 + r] * f);
      }
    }
  }
}

// ---------------------------------------------------------------- host

struct Shape {
  int dp, nh;              // padded head_dim, query-row tiles of 8 a warp holds
  int row_tiles, vheads;   // query-row groups per key-value head, pairs in all
  int heads_per_block, phases, groups, workers;
  int64_t image;           // floats of one partial result
  bool whole;              // requests are not divided over blocks: no second launch, no workspace
};

// head_dim is padded to 64, 128 or 256.  Groups above 8 query heads have two tiles of query rows a warp,
// so a tile's codes are read and decoded once for both.  us with two tiles / with one: 64 requests of
// up to 4096 tokens, 9 query heads a head of 128, 85 / 107, 12 a head of 64 54 / 68, 12 a head of 256 139 / 193;
// 16 requests, 16 a head of 128, 30 / 36; of one head of 256 in all, 16 query heads, 7 requests 27.4 / 28.1 and
// 64 of up to 16384 tokens 73 / 98.
inline Shape shape_of(int64_t batch, int64_t max_tokens, int heads, int group, int head_dim) {
  Shape s;
  s.dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  s.nh = group > 8 ? 2 : 1;
  s.row_tiles = (group + 8 * s.nh - 1) / (8 * s.nh);
  s.vheads = heads * s.row_tiles;
  const int warps = warps_of(s.dp, s.nh), sms = std::max(1, device_sm_count());
  // Heads are divided over the fewest groups of blocks; over more where that keeps a tenth more warps of
  // the machine at work (5 of 8 warps with 5 heads of two row tiles, all of them with one head a block: 64
  // requests of up to 4096 tokens 66 us against 81; 11 heads of 2 query heads 90 / 95)
  s.groups = (s.vheads + warps - 1) / warps;
  auto busy = [&](int groups) {              // warps at work, on average, of all SMs
    const int heads = (s.vheads + groups - 1) / groups;
    return (double)s.vheads * (warps / heads) * std::max(1, sms / groups);
  };
  for (int g = s.groups + 1; g <= std::min(s.vheads, 16); ++g)
    if (busy(g) > 1.1 * busy(s.groups)) s.groups = g;
  s.heads_per_block = (s.vheads + s.groups - 1) / s.groups;
  s.phases = warps / s.heads_per_block;
  const int64_t tiles = (max_tokens + kAttnTile - 1) / kAttnTile;
  // Requests that cannot have more than kWholeTiles tiles a warp stay with the block in whose share they
  // begin, and there is no second launch.  us whole / divided, heads x dims: 300 requests of up to 100 tokens, 8 x 128,
  // 22.3 / 25.2; of up to 250 33.5 / 34.5; 150 of up to 160 18.8 / 21.0, of up to 250 24.7 / 25.5, of up to 380 (12 tiles
  // a warp) 31.6 / 29.0; 900 of up to 250 70.8 / 73.0; 4 x 256, 400 of up to 160 30.6 / 33.6; 16 x 128, 150 of up to 100
  // 20.8 / 25.6.
  s.whole = tiles <= kWholeTiles * s.phases;
  // Where each request can have blocks of its own for one head or a few, its heads are spread over the machine
  // and it stays whole up to kSpreadRounds tiles of each of a head's warps: 48 tiles where a block has 16 warps,
  // 32 where it has 8.  us spread / else, by heads x query heads of a head x dims.  16 warps: 8 x 4 x 128, one request
  // of 33 tokens 4.4 / 7.0, 500 8.3 / 10.1, 750 9.7 / 10.5, 1000 11.6 / 10.7, 16 of up to 750 9.8 / 12.8; one of 750,
  // 1 x 8 x 128 9.6 / 10.3, 2 x 8 x 64 7.4 / 8.7, 32 x 1 x 128 9.6 / 12.3.  8 warps: 1 x 16 x 256, one of 500 14.4 / 14.4,
  // 750 16.9 / 12.4; 8 x 12 x 128, 500 10.4 / 11.2, 750 12.0 / 10.8 (but 16 of up to 750 12.1 / 14.1); 4 x 4 x 256, 250
  // 8.3 / 9.3, 500 10.9 / 9.5, 16 of up to 500 10.9 / 11.1, one of 750 13.1 / 9.9.  With at most 6 or 16 warps a head
  // nearly all take as long or longer (8 x 1 x 64, 16 of up to 500: 7.8 and 7.3 against 6.7).
  const int most_warps = std::min(warps, kSpreadPhases);
  if (tiles <= kSpreadRounds * most_warps)
    for (int heads = 1; heads <= s.heads_per_block; ++heads) {
      const int groups = (s.vheads + heads - 1) / heads;
      if (batch * groups > sms) continue;
      s.groups = groups;
      s.heads_per_block = heads;
      const int64_t most = std::min(warps / heads, kSpreadPhases);
      const int64_t rounds = std::max<int64_t>(1, (tiles + most - 1) / most);
      s.phases = (int)std::max<int64_t>(1, (tiles + rounds - 1) / rounds);     // rounds of even tiles
      s.whole = true;
      break;
    }
  s.workers = std::min(kMaxWorkers, std::max(1, sms / s.groups));
  s.image = s.nh * (8 * s.dp + 16);
  return s;
}

template <int FMT, int DP, int NH, bool TOKEN_SCALES>
cudaError_t launch(const Params& p, const Shape& s, bool join, cudaStream_t st) {
  const int warps = s.heads_per_block * s.phases;
  const size_t smem = (size_t)warps * (stages_of(DP, NH) * kStageBytes<DP> + query_bytes(DP, NH));
  auto* kernel = k_attention<FMT, DP, NH, TOKEN_SCALES>;
  cudaError_t e = ensure_dynamic_smem((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(s.workers, s.groups), dim3(32 * warps), smem, st, p);
  if (e != cudaSuccess || !join) return e;
  auto* joiner = k_attention_join<DP, NH, TOKEN_SCALES>;
  return launch_pdl(joiner, dim3(2 * std::max(1, device_sm_count())), dim3(kJoinThreads), 0, st, p);
}

template <int FMT, bool TOKEN_SCALES>
cudaError_t launch_dims(const Params& p, const Shape& s, bool join, cudaStream_t st) {
  if (s.dp == 64)
    return s.nh == 1 ? launch<FMT, 64, 1, TOKEN_SCALES>(p, s, join, st) : launch<FMT, 64, 2, TOKEN_SCALES>(p, s, join, st);
  if (s.dp == 128)
    return s.nh == 1 ? launch<FMT, 128, 1, TOKEN_SCALES>(p, s, join, st) : launch<FMT, 128, 2, TOKEN_SCALES>(p, s, join, st);
  return s.nh == 1 ? launch<FMT, 256, 1, TOKEN_SCALES>(p, s, join, st) : launch<FMT, 256, 2, TOKEN_SCALES>(p, s, join, st);
}

}  // namespace attn

// Walks every worker's share with the kernel's own functions, for several costs of a change of
// request: each tile of each request is held once, a worker holds parts of at most two shared
// requests (the first and the last of its share), and the workers named by a shared request's
// descriptor are those that hold its tiles.
static int check_split(const int* lens, int64_t batch, int window, int sinks, int most, int turn) {
  int64_t total = 0;
  for (int64_t b = 0; b < batch; ++b) total += attn_cost(attn_range(lens[b], window, sinks).tiles, turn);
  if (total == 0) return 0;
  if (total > attn::kMaxCost) return -1;
  const int workers = attn_workers((int)total, most, attn::kMinTiles);
  if (workers < 1 || workers > most) return 3;
  const AttnSplit s = attn_split((int)total, workers);
  int64_t expect = 0;
  for (int w = 0; w < workers; ++w) {
    if (attn_start(s, w) != expect) return 4;
    expect = attn_start(s, w + 1);
    if (expect <= attn_start(s, w)) return 5;                    // every worker has a share
    for (int64_t x = attn_start(s, w); x < expect; ++x)
      if (attn_owner(s, (int)x) != w) return 6;
  }
  if (expect != total) return 7;
  int64_t base = 0;
  for (int64_t b = 0; b < batch; ++b) {
    const int n = attn_range(lens[b], window, sinks).tiles;
    if (n == 0) continue;
    const int first = attn_owner(s, (int)base), last = attn_owner(s, (int)(base + n - 1));
    int64_t held = 0;
    for (int w = first; w <= last; ++w) {
      // as Cursor's enter() has it: `left` of the share from tile `from` on
      const int64_t from = std::max<int64_t>(0, attn_start(s, w) - base), left = attn_start(s, w + 1) - base - from;
      const int64_t to = std::min<int64_t>(n, from + left);
      if (from != held || from >= to) return 8;                  // a named worker without a part, a tile twice or never
      held = to;
      // place 0 is the part at the beginning of a share, place 1 the one at its end
      const bool at_begin = base + from == attn_start(s, w);
      if (first != last && !at_begin && base + to != attn_start(s, w + 1)) return 9;
      if (w > first && !at_begin) return 10;
    }
    if (held != n) return 11;
    base += attn_cost(n, turn);
  }
  return 0;
}

int check_attention_split(const int* lens, int64_t batch, int window, int sinks, int most) {
  if (batch < 0 || most < 1 || window < 0 || sinks < 0 || (batch > 0 && !lens)) return -1;
  for (int64_t b = 0; b < batch; ++b) {
    const AttnRange r = attn_range(lens[b], window, sinks);
    if (r.tiles < 0 || r.head > r.tiles || r.skip < 0) return 1;
    // the tiles in order hold every visible token and end with the last one's
    for (int tok = 0; tok < lens[b]; ++tok) {
      if (window > 0 && tok < lens[b] - window && tok >= sinks) continue;
      const int tile = tok / kAttnTile;
      const int i = tile < r.head ? tile : tile - r.skip;
      if (i < 0 || i >= r.tiles || (i < r.head ? i : i + r.skip) != tile) return 2;
    }
  }
  for (int phases : {1, 2, 5, attn::kMaxWarps}) {
    const int bad = check_split(lens, batch, window, sinks, most, attn::kTurn * phases);
    if (bad) return bad;
  }
  return 0;
}

size_t attention_workspace_bytes(int64_t batch, int64_t max_tokens, int heads, int group, int head_dim) {
  const attn::Shape s = attn::shape_of(batch, max_tokens, heads, group, head_dim);
  if (s.whole) return 0;
  return (size_t)s.workers * 16 + 256 + (size_t)2 * s.workers * s.vheads * s.image * 4;
}

cudaError_t launch_attention_paged(const KvPages& c, int fmt, const uint16_t* q, int64_t q_stride, int group,
                                   const int* table, int64_t batch, int64_t max_pages, const int* lens, float scale,
                                   int window, int sinks, uint16_t* out, int64_t out_stride, float* lse, void* ws,
                                   cudaStream_t st) {
  const attn::Shape s = attn::shape_of(batch, max_pages * c.page_size, c.heads, group, c.head_dim);
  attn::Params p;
  p.c = c;
  p.q = q;
  p.q_stride = q_stride;
  p.table = table;
  p.lens = lens;
  p.batch = (int)batch;
  p.max_pages = (int)max_pages;
  p.group = group;
  p.window = window;
  p.sinks = sinks;
  p.scale2 = scale * attn::kLog2e;
  p.out = out;
  p.out_stride = out_stride;
  p.lse = lse;
  p.vheads = s.vheads;
  p.row_tiles = s.row_tiles;
  p.heads_per_block = s.heads_per_block;
  p.phases = s.phases;
  p.turn = attn::kTurn * s.phases;
  p.workers = s.workers;
  const bool join = !s.whole;
  p.desc = join ? static_cast<int4*>(ws) : nullptr;
  uint8_t* parts = static_cast<uint8_t*>(ws) + ((size_t)s.workers * 16 + 255) / 256 * 256;
  p.part = join ? reinterpret_cast<float*>(parts) : nullptr;
  p.err = device_error_word();
  const bool token_scales = c.gran >= 2;
  if (fmt == kE4M3)
    return token_scales ? attn::launch_dims<kE4M3, true>(p, s, join, st) : attn::launch_dims<kE4M3, false>(p, s, join, st);
  return token_scales ? attn::launch_dims<kE5M2, true>(p, s, join, st) : attn::launch_dims<kE5M2, false>(p, s, join, st);
}

}  // namespace fp8q
