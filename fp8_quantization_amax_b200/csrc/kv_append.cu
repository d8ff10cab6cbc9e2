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
// exchange is needed but the sums over the row, and q may be rotated in place.
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
constexpr int kMaxBlockTokens = 4;

struct Params {
  KvPages c;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;     // elements from token to token
  const uint16_t *q_weight, *k_weight;      // bf16 [head_dim] or null
  float eps;
  const int64_t* slots;
  const int* positions;
  const unsigned long long* turns;          // [rot / 2]
  int rot, interleaved;
  float gain;                               // factor of cos and sin
  uint16_t* q_out;
  int64_t q_out_stride;
  int tokens, q_heads;
  int block_tokens;
  int q_units, kv_units;                    // warp steps for the q rows, the k rows (and the v rows)
  FastDiv units;                            // division by the steps of a token
  uint32_t* err;
};

// RN(x / d) (correct for every bf16 x, and to the last place for other x) with r = RN(1 / d), for
// d of ordinary size; an overflowing quotient stays infinite and saturates in the cast
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q0 = __fmul_rn(x, r);
  const float q = __fmaf_rn(-__fmaf_rn(q0, d, -x), r, q0);
  return fabsf(q0) < 0x1.0p100f ? q : q0;
}

template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float (&y)[4], const GroupScale& g) {
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = g.fast ? quotient(y[i], g.d, g.r) : g.d == 0.0f ? copysignf(0.0f, y[i]) : __fdiv_rn(y[i], g.d);
  return __byte_perm(cvt2<FMT>(q[0], q[1]), cvt2<FMT>(q[2], q[3]), 0x5410);
}

// a given scale: the fast quotient's range is that of make_group_scale; 0 gives signed zeros
__device__ __forceinline__ GroupScale given_scale(float s) {
  GroupScale g;
  g.s = s;
  g.d = s;
  g.fast = s >= 0x1.0p-68f && s <= 0x1.0p119f;
  g.r = g.fast ? __frcp_rn(s) : 0.0f;
  return g;
}

__device__ __forceinline__ void unpack4(uint2 w, float (&x)[4]) {
  x[0] = bf16_lo(w.x);
  x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y);
  x[3] = bf16_hi(w.y);
}

template <int FMT, int LPR>
__global__ void __launch_bounds__(kThreads) k_append(const Params p) {
  __shared__ __align__(16) float2 turn[kMaxBlockTokens][kMaxPairs];
  constexpr int RPW = 32 / LPR;             // rows a warp takes at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPR, sub = lane / LPR;
  const int D = p.c.head_dim;
  const bool inside = 8 * li < D;
  const bool rotated = 8 * li < p.rot;
  const bool split = rotated && !p.interleaved;
  const int o0 = split ? 4 * li : 8 * li, o1 = split ? p.rot / 2 + 4 * li : 8 * li + 4;

  allow_dependent_launch();
  grid_dependency_wait();

  const int t0 = blockIdx.x * p.block_tokens;
  const int nt = min(p.block_tokens, p.tokens - t0);

  float wq[2][4], wk[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) wq[0][i] = wq[1][i] = wk[0][i] = wk[1][i] = 1.0f;
  if (p.q_weight && inside) {
    unpack4(__ldg(reinterpret_cast<const uint2*>(p.q_weight + o0)), wq[0]);
    unpack4(__ldg(reinterpret_cast<const uint2*>(p.q_weight + o1)), wq[1]);
  }
  if (p.k_weight && inside) {
    unpack4(__ldg(reinterpret_cast<const uint2*>(p.k_weight + o0)), wk[0]);
    unpack4(__ldg(reinterpret_cast<const uint2*>(p.k_weight + o1)), wk[1]);
  }

  if (p.rot > 0) {
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
      const int tk = i / pairs, f = i - tk * pairs;
      const unsigned long long a = (unsigned long long)(long long)__ldg(p.positions + t0 + tk) * __ldg(p.turns + f);
      float sn, cs;
      sincospif((float)(int)(a >> 32) * 0x1.0p-31f, &sn, &cs);
      turn[tk][f] = make_float2(cs * p.gain, sn * p.gain);
    }
    __syncthreads();
  }

  const int units = p.q_units + 2 * p.kv_units;
  for (int i = warp; i < nt * units; i += kWarps) {
    const int tk = (int)div_u32((uint32_t)i, p.units);
    int u = i - tk * units;
    const int64_t token = t0 + tk;
    int kind = 0;                           // 0 q, 1 k, 2 v
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
    int64_t slot = 0;
    if (kind != 0) {
      slot = __ldg(p.slots + token);
      if (slot < 0) continue;               // a padded row; the same for the whole warp
      if (slot >= (int64_t)p.c.num_pages * p.c.page_size) {
        raise_device_error(p.err, kErrBadPage);
        continue;
      }
    }
    const int a0 = kind == 2 ? 8 * li : o0, a1 = kind == 2 ? 8 * li + 4 : o1;
    const uint16_t* src = kind == 0 ? p.q + token * p.q_stride : kind == 1 ? p.k + token * p.k_stride
                                                                           : p.v + token * p.v_stride;
    src += (int64_t)head * D;
    uint2 r0 = make_uint2(0, 0), r1 = r0;
    if (live) {
      r0 = *reinterpret_cast<const uint2*>(src + a0);
      r1 = *reinterpret_cast<const uint2*>(src + a1);
    }
    float y[2][4];
    unpack4(r0, y[0]);
    unpack4(r1, y[1]);

    if (kind != 2) {
      if (kind == 0 ? p.q_weight != nullptr : p.k_weight != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss += y[0][e] * y[0][e] + y[1][e] * y[1][e];
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float f = __frsqrt_rn(ss / (float)D + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[0][e] = y[0][e] * f * (kind == 0 ? wq[0][e] : wk[0][e]);
          y[1][e] = y[1][e] * f * (kind == 0 ? wq[1][e] : wk[1][e]);
        }
      }
      if (rotated) {
        const float4 c0 = *reinterpret_cast<const float4*>(&turn[tk][4 * li]);
        const float4 c1 = *reinterpret_cast<const float4*>(&turn[tk][4 * li + 2]);
        const float cs[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = y[e >> 1][2 * (e & 1)], b = y[e >> 1][2 * (e & 1) + 1];
            y[e >> 1][2 * (e & 1)] = a * cs[e] - b * sn[e];
            y[e >> 1][2 * (e & 1) + 1] = b * cs[e] + a * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = y[0][e], b = y[1][e];
            y[0][e] = a * cs[e] - b * sn[e];
            y[1][e] = b * cs[e] + a * sn[e];
          }
        }
      }
    }

    if (kind == 0) {
      if (live) {
        uint16_t* dst = p.q_out + token * p.q_out_stride + (int64_t)head * D;
        *reinterpret_cast<uint2*>(dst + a0) = make_uint2(f32x2_to_bf16x2(y[0][0], y[0][1]), f32x2_to_bf16x2(y[0][2], y[0][3]));
        *reinterpret_cast<uint2*>(dst + a1) = make_uint2(f32x2_to_bf16x2(y[1][0], y[1][1]), f32x2_to_bf16x2(y[1][2], y[1][3]));
      }
      continue;
    }
    float* scales = kind == 1 ? p.c.ks : p.c.vs;
    GroupScale g;
    if (p.c.gran == 3) {
      float top = 0.0f;
      bool nan = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        top = fmaxf(top, fmaxf(fabsf(y[0][e]), fabsf(y[1][e])));
        nan |= y[0][e] != y[0][e] || y[1][e] != y[1][e];
      }
      if (nan) top = __int_as_float(0x7FC00000);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, o);
        top = top != top || other != other ? __int_as_float(0x7FC00000) : fmaxf(top, other);
      }
      g = make_group_scale<FMT>(top);
      if (live && li == 0) scales[(int64_t)head * ((int64_t)p.c.num_pages * p.c.page_size) + slot] = g.s;
    } else {
      g = given_scale(live ? __ldg(scales + (p.c.gran == 0 ? 0 : head)) : 1.0f);
    }
    if (live) {
      const uint32_t page = div_u32((uint32_t)slot, p.c.page_div);
      const uint32_t off = (uint32_t)slot - page * (uint32_t)p.c.page_size;
      uint8_t* dst = (kind == 1 ? p.c.k : p.c.v) + (int64_t)page * p.c.page_stride + (int64_t)off * p.c.token_stride +
                     (int64_t)head * p.c.head_stride;
      *reinterpret_cast<uint32_t*>(dst + a0) = codes4<FMT>(y[0], g);
      *reinterpret_cast<uint32_t*>(dst + a1) = codes4<FMT>(y[1], g);
    }
  }
}

template <int FMT, int LPR>
cudaError_t launch(Params& p, cudaStream_t st) {
  constexpr int rpw = 32 / LPR;
  p.q_units = (p.q_heads + rpw - 1) / rpw;
  p.kv_units = (p.c.heads + rpw - 1) / rpw;
  p.units = make_fastdiv((uint32_t)(p.q_units + 2 * p.kv_units));
  const int blocks = (p.tokens + p.block_tokens - 1) / p.block_tokens;
  return launch_pdl(k_append<FMT, LPR>, dim3(blocks), dim3(kThreads), 0, st, p);
}

template <int FMT>
cudaError_t launch_lanes(Params& p, cudaStream_t st) {
  if (p.c.head_dim <= 32) return launch<FMT, 4>(p, st);
  if (p.c.head_dim <= 64) return launch<FMT, 8>(p, st);
  if (p.c.head_dim <= 128) return launch<FMT, 16>(p, st);
  return launch<FMT, 32>(p, st);
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
  p.slots = a.slots;
  p.positions = a.positions;
  p.turns = a.turns;
  p.rot = a.rot;
  p.interleaved = a.interleaved;
  p.gain = a.gain;
  p.q_out = a.q_out;
  p.q_out_stride = a.q_out_stride;
  p.tokens = (int)a.tokens;
  p.q_heads = a.q_heads;
  // one token a block until the blocks fill the machine, then several share the block's set-up
  p.block_tokens = a.tokens >= (int64_t)device_sm_count() * 8 * append::kMaxBlockTokens ? append::kMaxBlockTokens : 1;
  p.err = device_error_word();
  return fmt == kE4M3 ? append::launch_lanes<kE4M3>(p, st) : append::launch_lanes<kE5M2>(p, st);
}

}  // namespace fp8q
