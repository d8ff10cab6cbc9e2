// New tokens into the paged FP8 KV cache (fp8_kv_append): per-head RMS norm and rotary positions
// of q and k, k and v quantized into their slots, q back as bf16, in one pass.
//
//   y = x rsqrt(mean(x^2) + eps) w                         (each head; left out without weights)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   (angle = position * frequency of the pair)
//   s given, or amax |y| / FMAX;  code = FP8(RN(y / s))
//
// What bounds it: 2 bytes read an element and 2 (q) or 1 (k, v) written, against about ten
// operations: HBM, once there are a few hundred tokens; below that the latency of one launch.
// Measured (us a call, back to back in a graph; floor at 6.53 TB/s): 16384 tokens of 64 + 2 * 8 heads of
// 128 without norm 111.7 (97.6: 87 %), 8192 tokens of 32 + 2 * 8 heads with norm and a scale per token
// 38.8 (28.3: 73 %; 99 instructions for 256 elements, 46 % of the issue slots, the rest is waiting for
// shuffles, shared memory and HBM at 24 warps an SM), 32 tokens 2.5.
//
// Angles: a frequency comes as a fraction of a turn in 64 bits, so position * frequency modulo one
// turn is one integer product, exact to 2^-32 of a turn at any position (in fp32 the angle itself
// is off by 0.06 at position 10^6).  sincospi of the signed fraction follows; each block computes
// the pairs of its tokens once, for all heads, into shared memory.
//
// A row (one head of one token) is cut into chunks of 8 elements, two to a thread (LPR threads a
// row, a power of two): chunk c is two runs of 4 elements, chosen so that both elements of a
// rotated pair are in it (halves layout: the runs at 4 c of either half; neighbours: 8 adjacent
// elements).  No exchange is needed but the sums over the row, and q may be rotated in place.
// A chunk lies in four fp32 pairs, first elements of rotated pairs beside first ones, so that norm,
// rotation and quotient take one instruction a pair.
//
// A block takes up to kTokens tokens and works out their angles and places first.  A warp then goes
// through the tokens with its heads (32 / LPR rows at a time): what it does (q, k or v) is settled
// once, its places move by a stride, and the loads of two tokens run ahead.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8q_device.cuh"
#include "internal.h"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace fp8q {
namespace append {

constexpr int kMaxWarps = 8;
constexpr int kSmWarps = 24;                // an SM holds this many at 80 registers a thread
constexpr int kMaxPairs = 128;              // rotated pairs of a row (head_dim <= 256)
constexpr int kTokens = 16;                 // tokens of a block

struct Params {
  KvPages c;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;     // elements from token to token
  const uint16_t *q_weight, *k_weight;      // bf16 [head_dim] or null
  float eps, inv_dim;
  const int64_t* slots;
  const int* positions;
  const unsigned long long* turns;          // [rot / 2]
  int rot;
  float gain;                               // factor of cos and sin
  uint16_t* q_out;
  int64_t q_out_stride;
  int tokens, q_heads;
  int q_units, kv_units;                    // warp steps for the q rows, the k rows (and the v rows)
  int block_tokens;
  uint32_t* err;
};

// A chunk of eight elements: a[0] holds the first elements of its rotated pairs 0, 1, a[1] of 2, 3;
// b the second ones.  Where nothing is rotated the same places hold the elements in that order.
struct Chunk {
  float2 a[2], b[2];
};

// NEXT: pairs are neighbours (r0, r1 are 8 adjacent elements), else r0 holds first elements and r1
// second ones
template <bool NEXT>
__device__ __forceinline__ Chunk unpack(uint2 r0, uint2 r1) {
  Chunk y;
  if constexpr (NEXT) {
    y.a[0] = make_float2(bf16_lo(r0.x), bf16_lo(r0.y));
    y.b[0] = make_float2(bf16_hi(r0.x), bf16_hi(r0.y));
    y.a[1] = make_float2(bf16_lo(r1.x), bf16_lo(r1.y));
    y.b[1] = make_float2(bf16_hi(r1.x), bf16_hi(r1.y));
  } else {
    y.a[0] = make_float2(bf16_lo(r0.x), bf16_hi(r0.x));
    y.a[1] = make_float2(bf16_lo(r0.y), bf16_hi(r0.y));
    y.b[0] = make_float2(bf16_lo(r1.x), bf16_hi(r1.x));
    y.b[1] = make_float2(bf16_lo(r1.y), bf16_hi(r1.y));
  }
  return y;
}
template <bool NEXT>
__device__ __forceinline__ void pack_bf16(const Chunk& y, uint2& r0, uint2& r1) {
  if constexpr (NEXT) {
    r0 = make_uint2(f32x2_to_bf16x2(y.a[0].x, y.b[0].x), f32x2_to_bf16x2(y.a[0].y, y.b[0].y));
    r1 = make_uint2(f32x2_to_bf16x2(y.a[1].x, y.b[1].x), f32x2_to_bf16x2(y.a[1].y, y.b[1].y));
  } else {
    r0 = make_uint2(f32x2_to_bf16x2(y.a[0].x, y.a[0].y), f32x2_to_bf16x2(y.a[1].x, y.a[1].y));
    r1 = make_uint2(f32x2_to_bf16x2(y.b[0].x, y.b[0].y), f32x2_to_bf16x2(y.b[1].x, y.b[1].y));
  }
}
template <int FMT, bool NEXT>
__device__ __forceinline__ uint2 pack_codes(const Chunk& y) {
  if constexpr (NEXT) {
    return make_uint2(__byte_perm(cvt2<FMT>(y.a[0].x, y.b[0].x), cvt2<FMT>(y.a[0].y, y.b[0].y), 0x5410),
                      __byte_perm(cvt2<FMT>(y.a[1].x, y.b[1].x), cvt2<FMT>(y.a[1].y, y.b[1].y), 0x5410));
  } else {
    return make_uint2(__byte_perm(cvt2<FMT>(y.a[0].x, y.a[0].y), cvt2<FMT>(y.a[1].x, y.a[1].y), 0x5410),
                      __byte_perm(cvt2<FMT>(y.b[0].x, y.b[0].y), cvt2<FMT>(y.b[1].x, y.b[1].y), 0x5410));
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// largest magnitude of the eight; any NaN gives NaN
__device__ __forceinline__ float top_of(const Chunk& y) {
  const float m0 = max_nan(fabsf(y.a[0].x), fabsf(y.a[0].y)), m1 = max_nan(fabsf(y.a[1].x), fabsf(y.a[1].y));
  const float m2 = max_nan(fabsf(y.b[0].x), fabsf(y.b[0].y)), m3 = max_nan(fabsf(y.b[1].x), fabsf(y.b[1].y));
  return max_nan(max_nan(m0, m1), max_nan(m2, m3));
}

// Scale and reciprocal as the codes need them.  fast: a divisor of ordinary size
struct Divisor {
  float d, r;
  bool fast;
};

// a given scale
__device__ __forceinline__ Divisor divisor_of(float s) {
  Divisor v;
  v.d = s;
  v.fast = s >= 0x1.0p-68f && s <= 0x1.0p119f;
  v.r = v.fast ? __frcp_rn(s) : 0.0f;
  return v;
}

// RN(x / d) with r = RN(1 / d) (Markstein's step, fp8q_device.cuh: correct for every bf16 x, and to
// the last place for other x), d of ordinary size; an overflowing quotient stays infinite and saturates,
// a zero keeps its sign
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q0 = __fmul_rn(x, r);
  const float q = __fmaf_rn(-__fmaf_rn(q0, d, -x), r, q0);
  return q0 != 0.0f && fabsf(q0) < 0x1.0p100f ? q : q0;
}

// Codes for any divisor, without a division: a tiny or huge one is moved to ordinary size by a power
// of two together with the elements (an element that leaves fp32's range that way has a quotient
// that saturates, or far below the smallest code).  0 gives signed zeros, infinity zeros but NaN
// for an infinite element, NaN gives NaN.
template <int FMT, bool NEXT>
__device__ __forceinline__ uint2 codes_any(Chunk y, float d) {
  const float m = fabsf(d);
  const bool zero = d == 0.0f, inf = m == __int_as_float(0x7F800000);
  const float by = m < 0x1.0p-60f ? 0x1.0p100f : m > 0x1.0p100f ? 0x1.0p-20f : 1.0f;
  const float ds = zero || inf ? 1.0f : d * by;
  const float rs = __frcp_rn(ds);
  auto one = [&](float& x) {
    x = zero ? copysignf(0.0f, x) : inf ? x * copysignf(0.0f, d) : quotient(x * by, ds, rs);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    one(y.a[i].x);
    one(y.a[i].y);
    one(y.b[i].x);
    one(y.b[i].y);
  }
  return pack_codes<FMT, NEXT>(y);
}

// Codes of y / d
template <int FMT, bool NEXT>
__device__ __forceinline__ uint2 codes_of(const Chunk& y, const Divisor& v) {
  // quant4_fast's three steps on negated pairs: p = -q0, f = the residual, n = -q
  const float2 d2 = make_float2(v.d, v.d), nr = make_float2(-v.r, -v.r);
  Chunk p, n;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p.a[i] = __fmul2_rn(y.a[i], nr);
    p.b[i] = __fmul2_rn(y.b[i], nr);
  }
  if (!v.fast || !(top_of(p) < 0x1.0p100f)) return codes_any<FMT, NEXT>(y, v.d);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    n.a[i] = __ffma2_rn(__ffma2_rn(p.a[i], d2, y.a[i]), nr, p.a[i]);
    n.b[i] = __ffma2_rn(__ffma2_rn(p.b[i], d2, y.b[i]), nr, p.b[i]);
  }
  const uint2 c = pack_codes<FMT, NEXT>(n);
  return make_uint2(c.x ^ 0x80808080u, c.y ^ 0x80808080u);
}

// 8 bytes that are read once (not by the read-only path, kv_pages.cuh; q may be rotated in place too)
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int LPR>
struct Shared {
  float cosine[kTokens][kMaxPairs], sine[kTokens][kMaxPairs];
  float weights[2][2][4 * 2 * LPR];         // of q and k: the chunks' first runs, their second ones
  int2 slots[kTokens];                      // slot (-1: not at all) and its place in units of 16 bytes
};

// Rows u * 32 / LPR .. of one kind (0 q, 1 k, 2 v) of tokens t0 .. t0 + nt - 1.  FULL: rows of 16 LPR
// elements, all of them rotated in halves, so a thread's runs lie at fixed distances
template <int FMT, int LPR, bool NEXT, bool FULL, int KIND>
__device__ __forceinline__ void rows(const Params& p, const Shared<LPR>& sh, int u, int t0, int nt, bool first) {
  const int lane = threadIdx.x & 31;
  const int li = lane % LPR, head = u * (32 / LPR) + lane / LPR;
  const int D = FULL ? 16 * LPR : p.c.head_dim;
  const bool own = head < (KIND == 0 ? p.q_heads : p.c.heads);
  bool live[2], rotated[2];
  int o0[2], o1[2];                         // a chunk's runs
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int at = li + c * LPR;
    live[c] = own && (FULL || 8 * at < D);
    rotated[c] = FULL || 8 * at < p.rot;
    const bool split = rotated[c] && !NEXT;
    o0[c] = split ? 4 * at : 8 * at;
    o1[c] = split ? (FULL ? 8 * LPR : p.rot / 2) + 4 * at : 8 * at + 4;
  }
  const int64_t stride = KIND == 0 ? p.q_stride : KIND == 1 ? p.k_stride : p.v_stride;
  const uint16_t* src = (KIND == 0 ? p.q : KIND == 1 ? p.k : p.v) + t0 * stride + (int64_t)head * D + o0[0];
  uint16_t* dst = KIND == 0 ? p.q_out + t0 * p.q_out_stride + (int64_t)head * D + o0[0] : nullptr;
  uint8_t* const codes_at = KIND == 0 ? nullptr : (KIND == 1 ? p.c.k : p.c.v) + (int64_t)head * p.c.head_stride + o0[0];
  const int64_t cache_slots = (int64_t)p.c.num_pages * p.c.page_size;
  float* const scales = (KIND == 1 ? p.c.ks : p.c.vs) + (p.c.gran == 3 ? head * cache_slots : 0);
  const bool norm = KIND != 2 && (KIND == 0 ? p.q_weight : p.k_weight) != nullptr;
  Divisor by;
  by.d = by.r = 1.0f;
  by.fast = true;
  if (KIND != 0 && p.c.gran != 3 && own) by = divisor_of(scales[p.c.gran == 0 ? 0 : head]);

  struct Raw {
    uint2 r[2][2];
  };
  auto load = [&](Raw& x) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (live[c]) {
        x.r[c][0] = load8(src + (o0[c] - o0[0]));
        x.r[c][1] = load8(src + (o1[c] - o0[0]));
      }
    src += stride;
  };
  // row j of the block's tokens, and the load of row j + 2 into its place
  auto row = [&](Raw& x, int j) {
    Chunk y[2] = {unpack<NEXT>(x.r[0][0], x.r[0][1]), unpack<NEXT>(x.r[1][0], x.r[1][1])};
    if (j + 2 < nt) load(x);
    if (norm) {
      float2 ss = __fmul2_rn(y[0].a[0], y[0].a[0]);
      ss = __ffma2_rn(y[0].a[1], y[0].a[1], ss);
      ss = __ffma2_rn(y[0].b[0], y[0].b[0], ss);
      ss = __ffma2_rn(y[0].b[1], y[0].b[1], ss);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ss = __ffma2_rn(y[1].a[i], y[1].a[i], ss);
        ss = __ffma2_rn(y[1].b[i], y[1].b[i], ss);
      }
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const float f = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
      const float2 f2 = make_float2(f, f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 wa = *reinterpret_cast<const float4*>(&sh.weights[KIND & 1][0][4 * (li + c * LPR)]);
        const float4 wb = *reinterpret_cast<const float4*>(&sh.weights[KIND & 1][1][4 * (li + c * LPR)]);
        y[c].a[0] = __fmul2_rn(__fmul2_rn(y[c].a[0], f2), make_float2(wa.x, wa.y));
        y[c].a[1] = __fmul2_rn(__fmul2_rn(y[c].a[1], f2), make_float2(wa.z, wa.w));
        y[c].b[0] = __fmul2_rn(__fmul2_rn(y[c].b[0], f2), make_float2(wb.x, wb.y));
        y[c].b[1] = __fmul2_rn(__fmul2_rn(y[c].b[1], f2), make_float2(wb.z, wb.w));
      }
    }
    if (KIND != 2) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!rotated[c]) continue;
        const float4 cs = *reinterpret_cast<const float4*>(&sh.cosine[j][4 * (li + c * LPR)]);
        const float4 sn = *reinterpret_cast<const float4*>(&sh.sine[j][4 * (li + c * LPR)]);
        const float2 cc[2] = {make_float2(cs.x, cs.y), make_float2(cs.z, cs.w)};
        const float2 sc[2] = {make_float2(sn.x, sn.y), make_float2(sn.z, sn.w)};
        const float2 minus = make_float2(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 a = y[c].a[i], b = y[c].b[i];
          y[c].a[i] = __ffma2_rn(a, cc[i], __fmul2_rn(b, __fmul2_rn(sc[i], minus)));
          y[c].b[i] = __ffma2_rn(b, cc[i], __fmul2_rn(a, sc[i]));
        }
      }
    }
    if constexpr (KIND == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint2 x0, x1;
        pack_bf16<NEXT>(y[c], x0, x1);
        if (live[c]) {
          *reinterpret_cast<uint2*>(dst + (o0[c] - o0[0])) = x0;
          *reinterpret_cast<uint2*>(dst + (o1[c] - o0[0])) = x1;
        }
      }
      dst += p.q_out_stride;
    } else {
      const int2 to = sh.slots[j];
      if (to.x < 0) return;                 // the same for the whole block
      Divisor d = by;
      if (p.c.gran == 3) {
        float top = max_nan(top_of(y[0]), top_of(y[1]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const GroupScale g = make_group_scale<FMT>(top);
        if (own && li == 0) scales[to.x] = g.s;
        d = Divisor{g.d, g.r, g.fast};
      }
      uint8_t* at = codes_at + (uint64_t)(uint32_t)to.y * 16;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint2 codes = codes_of<FMT, NEXT>(y[c], d);
        if (live[c]) {
          *reinterpret_cast<uint32_t*>(at + (o0[c] - o0[0])) = codes.x;
          *reinterpret_cast<uint32_t*>(at + (o1[c] - o0[0])) = codes.y;
        }
      }
    }
  };

  Raw a, b;                                 // places past head_dim stay zero
#pragma unroll
  for (int c = 0; c < 2; ++c) a.r[c][0] = a.r[c][1] = b.r[c][0] = b.r[c][1] = make_uint2(0, 0);
  load(a);
  if (nt > 1) load(b);
  if (first) __syncthreads();               // the shared part is complete; every warp passes this once
#pragma unroll 1
  for (int j = 0; j < nt; j += 2) {
    row(a, j);
    if (j + 1 < nt) row(b, j + 1);
  }
}

template <int FMT, int LPR, bool NEXT, bool FULL>
__global__ void __launch_bounds__(32 * kMaxWarps, kSmWarps / kMaxWarps) k_append(const Params p) {
  __shared__ __align__(16) Shared<LPR> sh;
  const int64_t cache_slots = (int64_t)p.c.num_pages * p.c.page_size;
  const int warps = blockDim.x >> 5;
  allow_dependent_launch();
  grid_dependency_wait();

  const int t0 = blockIdx.x * p.block_tokens;
  const int nt = min(p.block_tokens, p.tokens - t0);
  const int units = p.q_units + 2 * p.kv_units;
  int u = blockIdx.y * warps + (threadIdx.x >> 5);
  const int pairs = p.rot / 2;
  for (int i = threadIdx.x; i < nt * kMaxPairs; i += blockDim.x) {
    const int tk = i / kMaxPairs, f = i % kMaxPairs;
    if (f >= pairs) continue;
    const unsigned long long a = (unsigned long long)(long long)p.positions[t0 + tk] * p.turns[f];
    float sn, cs;
    sincospif((float)(int)(a >> 32) * 0x1.0p-31f, &sn, &cs);
    sh.cosine[tk][f] = cs * p.gain;
    sh.sine[tk][f] = sn * p.gain;
  }
  for (int i = threadIdx.x; i < 2 * 2 * LPR; i += blockDim.x) {
    const int which = i / (2 * LPR), at = i % (2 * LPR);
    const uint16_t* weight = which == 0 ? p.q_weight : p.k_weight;
    if (!weight) continue;
    // chunks past head_dim have zeros: their elements are zero, but times what lies here by chance
    // (NaN, infinity) they would not be, and a row's scale is taken over all its chunks
    float4 wa = make_float4(0.0f, 0.0f, 0.0f, 0.0f), wb = wa;
    if (8 * at < p.c.head_dim) {
      const bool split = 8 * at < p.rot && !NEXT;
      const Chunk w = unpack<NEXT>(*reinterpret_cast<const uint2*>(weight + (split ? 4 * at : 8 * at)),
                                   *reinterpret_cast<const uint2*>(weight + (split ? pairs + 4 * at : 8 * at + 4)));
      wa = make_float4(w.a[0].x, w.a[0].y, w.a[1].x, w.a[1].y);
      wb = make_float4(w.b[0].x, w.b[0].y, w.b[1].x, w.b[1].y);
    }
    *reinterpret_cast<float4*>(&sh.weights[which][0][4 * at]) = wa;
    *reinterpret_cast<float4*>(&sh.weights[which][1][4 * at]) = wb;
  }
  if (threadIdx.x < nt) {
    const int64_t slot = p.slots[t0 + threadIdx.x];
    if (slot >= cache_slots) raise_device_error(p.err, kErrBadPage);
    const uint32_t page = div_u32((uint32_t)slot, p.c.page_div);
    const uint32_t off = (uint32_t)slot - page * (uint32_t)p.c.page_size;
    // the last code's place fits 32 bits (checked on the host)
    sh.slots[threadIdx.x] = make_int2(slot >= 0 && slot < cache_slots ? (int)slot : -1,
                                      (int)(page * (uint32_t)(p.c.page_stride >> 4) + off * (uint32_t)(p.c.token_stride >> 4)));
  }
  if (u >= units) __syncthreads();
  for (bool first = true; u < units; u += gridDim.y * warps, first = false) {
    if (u < p.q_units) rows<FMT, LPR, NEXT, FULL, 0>(p, sh, u, t0, nt, first);
    else if (u < p.q_units + p.kv_units) rows<FMT, LPR, NEXT, FULL, 1>(p, sh, u - p.q_units, t0, nt, first);
    else rows<FMT, LPR, NEXT, FULL, 2>(p, sh, u - p.q_units - p.kv_units, t0, nt, first);
  }
}

template <int FMT, int LPR, bool NEXT>
cudaError_t launch(Params& p, cudaStream_t st) {
  constexpr int rpw = 32 / LPR;
  p.q_units = (p.q_heads + rpw - 1) / rpw;
  p.kv_units = (p.c.heads + rpw - 1) / rpw;
  const int units = p.q_units + 2 * p.kv_units;
  const int64_t sms = std::max(1, device_sm_count());
  // as many warps a block as leaves the fewest without a unit in the last turn
  int warps = std::min(units, kMaxWarps);
  for (int w = warps; w >= 4; --w)
    if ((units + w - 1) / w * w < (units + warps - 1) / warps * warps) warps = w;
  const int64_t room = sms * (kSmWarps / warps);
  // tokens a block so that the blocks fill whole waves; where there are fewer tokens than blocks of a
  // wave, several blocks a token
  const int64_t waves = (p.tokens + room * kTokens - 1) / (room * kTokens);
  p.block_tokens = (int)((p.tokens + room * waves - 1) / (room * waves));
  const unsigned x = (unsigned)((p.tokens + p.block_tokens - 1) / p.block_tokens);
  const unsigned y = (unsigned)std::min<int64_t>((units + warps - 1) / warps, std::max<int64_t>(1, room / p.tokens));
  // rows rotated whole in halves have fixed places: 36.4 us against 38.2 of the general form at 8192 tokens of
  // 32 + 2 * 8 heads of 128 with norm, 32 tokens 2.5 / 2.7 (neighbouring pairs gained nothing by it, 36.1 / 35.0)
  if constexpr (!NEXT)
    if (p.c.head_dim == 16 * LPR && p.rot == p.c.head_dim)
      return launch_pdl(k_append<FMT, LPR, false, true>, dim3(x, y), dim3(32 * warps), 0, st, p);
  return launch_pdl(k_append<FMT, LPR, NEXT, false>, dim3(x, y), dim3(32 * warps), 0, st, p);
}

template <int FMT>
cudaError_t launch_lanes(Params& p, bool next, cudaStream_t st) {
  if (p.c.head_dim <= 64) return next ? launch<FMT, 4, true>(p, st) : launch<FMT, 4, false>(p, st);
  if (p.c.head_dim <= 128) return next ? launch<FMT, 8, true>(p, st) : launch<FMT, 8, false>(p, st);
  return next ? launch<FMT, 16, true>(p, st) : launch<FMT, 16, false>(p, st);
}

}  // namespace append

cudaError_t launch_kv_append(const KvPages& c, int fmt, const KvAppend& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  append::Params p;
  p.c = c;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.eps = a.eps;
  p.inv_dim = 1.0f / (float)c.head_dim;
  p.slots = a.slots;
  p.positions = a.positions;
  p.turns = a.turns;
  p.rot = a.rot;
  p.gain = a.gain;
  p.q_out = a.q_out;
  p.q_out_stride = a.q_out_stride;
  p.tokens = (int)a.tokens;
  p.q_heads = a.q_heads;
  p.err = device_error_word();
  const bool next = a.interleaved || a.rot == 0;
  return fmt == kE4M3 ? append::launch_lanes<kE4M3>(p, next, st) : append::launch_lanes<kE5M2>(p, next, st);
}

}  // namespace fp8q
