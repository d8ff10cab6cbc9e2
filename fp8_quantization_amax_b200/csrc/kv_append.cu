// New tokens into the paged FP8 KV cache (fp8_kv_append): per-head RMS norm and rotary positions
// of q and k, k and v quantized into their slots, q back as bf16, in one pass.
//
//   y = x rsqrt(mean(x^2) + eps) w                         (each head; left out without weights)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   (angle = position * frequency of the pair)
//   s given, or amax |y| / FMAX;  code = FP8(RN(y / s))
//
// What bounds it: 2 bytes read an element and 2 (q) or 1 (k, v) written, against about ten
// operations: HBM, once there are a few hundred tokens; below that the latency of one launch.
//
// Angles: a frequency comes as a fraction of a turn in 64 bits, so position * frequency modulo one
// turn is one integer product, exact to 2^-32 of a turn at any position (in fp32 the angle itself
// is off by 0.06 at position 10^6).  sincospi of the signed fraction follows; each block computes
// the pairs of its tokens once, for all heads, into shared memory.
//
// A row (one head of one token) belongs to head_dim / 8 threads of a warp, padded to a power of
// two; each holds two runs of 4 elements, chosen so that both elements of a rotated pair are its
// own (halves layout: the runs at 4 i of either half; neighbours: 8 adjacent elements).  No
// exchange is needed but the sums over the row, and q may be rotated in place.  A thread's elements
// lie in four fp32 pairs, first elements of rotated pairs beside first ones, so that norm, rotation
// and quotient take one instruction a pair.
//
// A warp keeps its heads over the tokens of its block: what it does (q, k or v), its weights and
// scales are settled once, and the rows of kBatch tokens are loaded together.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8q_device.cuh"
#include "internal.h"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace fp8q {
namespace append {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;              // rotated pairs of a row (head_dim <= 256)
constexpr int kBatch = 4;                   // tokens of a block where there are many

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
  uint32_t* err;
};

// A thread's eight elements: a[0] holds the first elements of its rotated pairs 0, 1, a[1] of 2, 3;
// b the second ones.  Where nothing is rotated the same places hold the elements in that order.
struct Row {
  float2 a[2], b[2];
};

// NEXT: pairs are neighbours (r0, r1 are 8 adjacent elements), else r0 holds first elements and r1
// second ones
template <bool NEXT>
__device__ __forceinline__ Row unpack(uint2 r0, uint2 r1) {
  Row y;
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
__device__ __forceinline__ void pack_bf16(const Row& y, uint2& r0, uint2& r1) {
  if constexpr (NEXT) {
    r0 = make_uint2(f32x2_to_bf16x2(y.a[0].x, y.b[0].x), f32x2_to_bf16x2(y.a[0].y, y.b[0].y));
    r1 = make_uint2(f32x2_to_bf16x2(y.a[1].x, y.b[1].x), f32x2_to_bf16x2(y.a[1].y, y.b[1].y));
  } else {
    r0 = make_uint2(f32x2_to_bf16x2(y.a[0].x, y.a[0].y), f32x2_to_bf16x2(y.a[1].x, y.a[1].y));
    r1 = make_uint2(f32x2_to_bf16x2(y.b[0].x, y.b[0].y), f32x2_to_bf16x2(y.b[1].x, y.b[1].y));
  }
}
template <int FMT, bool NEXT>
__device__ __forceinline__ uint2 pack_codes(const Row& y) {
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
__device__ __forceinline__ float top_of(const Row& y) {
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
// the last place for other x), d of ordinary size; an overflowing quotient stays infinite and saturates
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q0 = __fmul_rn(x, r);
  const float q = __fmaf_rn(-__fmaf_rn(q0, d, -x), r, q0);
  return fabsf(q0) < 0x1.0p100f ? q : q0;
}

// Codes for any divisor, without a division: a tiny or huge one is moved to ordinary size by a power
// of two together with the elements (an element that leaves fp32's range that way has a quotient
// that saturates, or far below the smallest code).  0 gives signed zeros, infinity zeros but NaN
// for an infinite element, NaN gives NaN.
template <int FMT, bool NEXT>
__device__ __forceinline__ uint2 codes_any(Row y, float d) {
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

// Codes of y / d.  GIVEN: the quotients may overflow (a scale that does not come from the row)
template <int FMT, bool NEXT, bool GIVEN>
__device__ __forceinline__ uint2 codes_of(const Row& y, const Divisor& v) {
  // quant4_fast's three steps on negated pairs: p = -q0, f = the residual, n = -q
  const float2 d2 = make_float2(v.d, v.d), nr = make_float2(-v.r, -v.r);
  Row p, n;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p.a[i] = __fmul2_rn(y.a[i], nr);
    p.b[i] = __fmul2_rn(y.b[i], nr);
  }
  if (!v.fast || (GIVEN && !(top_of(p) < 0x1.0p100f))) return codes_any<FMT, NEXT>(y, v.d);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    n.a[i] = __ffma2_rn(__ffma2_rn(p.a[i], d2, y.a[i]), nr, p.a[i]);
    n.b[i] = __ffma2_rn(__ffma2_rn(p.b[i], d2, y.b[i]), nr, p.b[i]);
  }
  const uint2 c = pack_codes<FMT, NEXT>(n);
  return make_uint2(c.x ^ 0x80808080u, c.y ^ 0x80808080u);
}

// 8 bytes that are read once (q may be rotated in place, so not the read-only path)
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int FMT, int LPR, bool NEXT, int BT>
__global__ void __launch_bounds__(kThreads, 4) k_append(const Params p) {
  __shared__ __align__(16) float cosine[BT][kMaxPairs], sine[BT][kMaxPairs];
  constexpr int RPW = 32 / LPR;             // rows a warp takes at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPR, sub = lane / LPR;
  const int D = p.c.head_dim;
  const bool inside = 8 * li < D;
  const bool rotated = 8 * li < p.rot;
  const bool split = rotated && !NEXT;
  const int o0 = split ? 4 * li : 8 * li, o1 = split ? p.rot / 2 + 4 * li : 8 * li + 4;

  allow_dependent_launch();
  grid_dependency_wait();

  const int t0 = blockIdx.x * BT;
  const int nt = min(BT, p.tokens - t0);
  if (p.rot > 0) {
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < BT * kMaxPairs; i += kThreads) {
      const int tk = i / kMaxPairs, f = i % kMaxPairs;
      if (tk < nt && f < pairs) {
        const unsigned long long a = (unsigned long long)(long long)__ldg(p.positions + t0 + tk) * __ldg(p.turns + f);
        float sn, cs;
        sincospif((float)(int)(a >> 32) * 0x1.0p-31f, &sn, &cs);
        cosine[tk][f] = cs * p.gain;
        sine[tk][f] = sn * p.gain;
      }
    }
    __syncthreads();
  }

  const int units = p.q_units + 2 * p.kv_units;
  const int64_t cache_slots = (int64_t)p.c.num_pages * p.c.page_size;
  for (int unit = blockIdx.y * kWarps + warp; unit < units; unit += gridDim.y * kWarps) {
    int u = unit, kind = 0;                 // 0 q, 1 k, 2 v
    if (u >= p.q_units) {
      u -= p.q_units;
      kind = 1;
      if (u >= p.kv_units) {
        u -= p.kv_units;
        kind = 2;
      }
    }
    const int head = u * RPW + sub;
    const bool live = inside && head < (kind == 0 ? p.q_heads : p.c.heads);
    const int64_t stride = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    const uint16_t* src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t0 * stride + (int64_t)head * D;
    const uint16_t* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    uint2 r0[BT], r1[BT];
    int64_t slot[BT];
#pragma unroll
    for (int j = 0; j < BT; ++j) {
      r0[j] = r1[j] = make_uint2(0, 0);
      slot[j] = -1;
      if (j < nt) {
        if (live) {
          r0[j] = load8(src + j * stride + o0);
          r1[j] = load8(src + j * stride + o1);
        }
        if (kind != 0) slot[j] = __ldg(p.slots + t0 + j);
      }
    }
    Row w;
    if (weight) {
      uint2 w0 = make_uint2(0, 0), w1 = w0;
      if (inside) {
        w0 = __ldg(reinterpret_cast<const uint2*>(weight + o0));
        w1 = __ldg(reinterpret_cast<const uint2*>(weight + o1));
      }
      w = unpack<NEXT>(w0, w1);
    }
    float* scales = kind == 1 ? p.c.ks : p.c.vs;
    Divisor by;
    by.d = by.r = 1.0f;
    by.fast = true;
    if (kind != 0 && p.c.gran != 3 && live) by = divisor_of(__ldg(scales + (p.c.gran == 0 ? 0 : head)));

#pragma unroll
    for (int j = 0; j < BT; ++j) {
      if (j >= nt) break;
      if (kind != 0) {
        if (slot[j] < 0) continue;          // a padded row; the same for the whole warp
        if (slot[j] >= cache_slots) {
          raise_device_error(p.err, kErrBadPage);
          continue;
        }
      }
      Row y = unpack<NEXT>(r0[j], r1[j]);
      if (weight) {
        float2 ss = __fmul2_rn(y.a[0], y.a[0]);
        ss = __ffma2_rn(y.a[1], y.a[1], ss);
        ss = __ffma2_rn(y.b[0], y.b[0], ss);
        ss = __ffma2_rn(y.b[1], y.b[1], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float f = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y.a[i] = __fmul2_rn(__fmul2_rn(y.a[i], f2), w.a[i]);
          y.b[i] = __fmul2_rn(__fmul2_rn(y.b[i], f2), w.b[i]);
        }
      }
      if (kind != 2 && rotated) {
        const float4 cs = *reinterpret_cast<const float4*>(&cosine[j][4 * li]);
        const float4 sn = *reinterpret_cast<const float4*>(&sine[j][4 * li]);
        const float2 c[2] = {make_float2(cs.x, cs.y), make_float2(cs.z, cs.w)};
        const float2 s[2] = {make_float2(sn.x, sn.y), make_float2(sn.z, sn.w)};
        const float2 minus = make_float2(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 a = y.a[i], b = y.b[i];
          y.a[i] = __ffma2_rn(a, c[i], __fmul2_rn(b, __fmul2_rn(s[i], minus)));
          y.b[i] = __ffma2_rn(b, c[i], __fmul2_rn(a, s[i]));
        }
      }
      if (kind == 0) {
        if (live) {
          uint16_t* dst = p.q_out + (t0 + j) * p.q_out_stride + (int64_t)head * D;
          uint2 x0, x1;
          pack_bf16<NEXT>(y, x0, x1);
          *reinterpret_cast<uint2*>(dst + o0) = x0;
          *reinterpret_cast<uint2*>(dst + o1) = x1;
        }
        continue;
      }
      uint2 codes;
      if (p.c.gran == 3) {
        float top = top_of(y);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const GroupScale g = make_group_scale<FMT>(top);
        if (live && li == 0) scales[(int64_t)head * cache_slots + slot[j]] = g.s;
        codes = codes_of<FMT, NEXT, false>(y, Divisor{g.d, g.r, g.fast});
      } else {
        codes = codes_of<FMT, NEXT, true>(y, by);
      }
      if (live) {
        const uint32_t page = div_u32((uint32_t)slot[j], p.c.page_div);
        const uint32_t off = (uint32_t)slot[j] - page * (uint32_t)p.c.page_size;
        uint8_t* dst = (kind == 1 ? p.c.k : p.c.v) + (int64_t)page * p.c.page_stride + (int64_t)off * p.c.token_stride +
                       (int64_t)head * p.c.head_stride;
        *reinterpret_cast<uint32_t*>(dst + o0) = codes.x;
        *reinterpret_cast<uint32_t*>(dst + o1) = codes.y;
      }
    }
  }
}

template <int FMT, int LPR, bool NEXT>
cudaError_t launch(Params& p, cudaStream_t st) {
  constexpr int rpw = 32 / LPR;
  p.q_units = (p.q_heads + rpw - 1) / rpw;
  p.kv_units = (p.c.heads + rpw - 1) / rpw;
  const int units = p.q_units + 2 * p.kv_units;
  const int64_t sms = std::max(1, device_sm_count());
  // kBatch tokens a block once that leaves some waves of blocks, else one, and then as many blocks a
  // token as the machine has room for
  if (p.tokens >= sms * 4 * kBatch)
    return launch_pdl(k_append<FMT, LPR, NEXT, kBatch>, dim3((p.tokens + kBatch - 1) / kBatch), dim3(kThreads), 0, st, p);
  const int64_t most = (units + kWarps - 1) / kWarps, room = std::max<int64_t>(1, sms * 4 / p.tokens);
  return launch_pdl(k_append<FMT, LPR, NEXT, 1>, dim3(p.tokens, (unsigned)std::min(most, room)), dim3(kThreads), 0, st, p);
}

template <int FMT, bool NEXT>
cudaError_t launch_lanes(Params& p, cudaStream_t st) {
  if (p.c.head_dim <= 32) return launch<FMT, 4, NEXT>(p, st);
  if (p.c.head_dim <= 64) return launch<FMT, 8, NEXT>(p, st);
  if (p.c.head_dim <= 128) return launch<FMT, 16, NEXT>(p, st);
  return launch<FMT, 32, NEXT>(p, st);
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
  if (fmt == kE4M3)
    return a.interleaved ? append::launch_lanes<kE4M3, true>(p, st) : append::launch_lanes<kE4M3, false>(p, st);
  return a.interleaved ? append::launch_lanes<kE5M2, true>(p, st) : append::launch_lanes<kE5M2, false>(p, st);
}

}  // namespace fp8q
