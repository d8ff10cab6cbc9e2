// The paged FP8 KV cache as the kernels see it, and the small pieces the paged operators share.
//
// The paged kernels read global memory with plain loads only, no __ldg or ld.global.nc: those ask for memory
// that nobody writes while the kernel lives, and as a programmatic dependent (sm100.cuh) it lives while
// the kernel before it still writes lengths, tables, slots, queries or scales.
#pragma once

#include <cstdint>

#include "internal.h"

namespace fp8q {

// Codes of page p, token t of the page, head h, element d of K and V sit at byte
// p * page_stride + t * token_stride + h * head_stride + d.  The slot of that token is
// p * page_size + t.
struct KvPages {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t page_stride, token_stride, head_stride;
  int num_pages, page_size, heads, head_dim;
  int gran;            // fp8q_kv_granularity
  FastDiv page_div;    // division by page_size
};

__device__ __forceinline__ uint32_t div_u32(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)__umulhi(n, f.m) + n) >> f.s);
}

// 4-, 16-byte asynchronous copies to shared memory; the or_zero forms read nothing and write zeros
// where !valid
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- division of the attention's work
//
// A request of n tokens is read in tiles of 16 tokens.  With a window only the tiles that hold a
// visible token count: those of the first `sinks` tokens and those from token n - window on.  A
// request costs its tiles and `turn` more, what a worker spends on ending one request and beginning
// the next; all requests' costs, laid end to end (below 2^31 in all), are divided evenly over the
// workers, and a worker holds the tiles that fall into its share.
constexpr int kAttnTile = 16;

struct AttnRange {
  int tiles;      // tiles to read
  int head;       // the first `head` of them begin at token 0 ...
  int skip;       // ... and the others this many tiles further on
};

__host__ __device__ __forceinline__ AttnRange attn_range(int n, int window, int sinks) {
  AttnRange r;
  r.tiles = (n + kAttnTile - 1) / kAttnTile;
  r.head = r.tiles;
  r.skip = 0;
  if (window > 0 && n > window) {
    const int first = (n - window) / kAttnTile;                    // tile of the window's first token
    const int front = ((sinks < n ? sinks : n) + kAttnTile - 1) / kAttnTile;
    if (first > front) {
      r.skip = first - front;
      r.head = front;
      r.tiles -= r.skip;
    }
  }
  return r;
}

__host__ __device__ __forceinline__ int attn_cost(int tiles, int turn) { return tiles == 0 ? 0 : tiles + turn; }

// workers that take part: a share of at least `least` each, so short work is not split without need
__host__ __device__ __forceinline__ int attn_workers(int cost, int most, int least) {
  const int w = cost / least;
  return w < 1 ? 1 : w < most ? w : most;
}

// The first `more` workers' shares are each + 1, the others' each: where worker w's begins, and the worker
// in whose share place x lies
struct AttnSplit {
  int each, more;
};
__host__ __device__ __forceinline__ AttnSplit attn_split(int cost, int workers) {
  const int each = (int)((uint32_t)cost / (uint32_t)workers);
  return AttnSplit{each, cost - each * workers};
}
__host__ __device__ __forceinline__ int attn_start(const AttnSplit& s, int w) {
  return w * s.each + (w < s.more ? w : s.more);
}
__host__ __device__ __forceinline__ int attn_owner(const AttnSplit& s, int x) {
  const int front = s.more * (s.each + 1);
  return x < front ? (int)((uint32_t)x / (uint32_t)(s.each + 1)) : s.more + (int)((uint32_t)(x - front) / (uint32_t)s.each);
}

}  // namespace fp8q
