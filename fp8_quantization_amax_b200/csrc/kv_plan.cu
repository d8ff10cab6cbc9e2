// Block tables, slots and positions from the requests' lengths (fp8_kv_pages_update): the page
// bookkeeping of one serving step on the device, so that lengths never travel to the host.
//
// Requests that end put their pages on the free list; then the others take the pages their new
// tokens need from its top.  Both are prefix sums over the requests in order, so the result does
// not depend on timing.  Table entries below zero (pages given away before) give nothing back: the
// entries go on the list as they are, and where such a one was among them a second pass over them with
// sums puts the pages alone.  What bounds it: 12 bytes written a token and a few words a request, a
// microsecond of traffic at most: the chain of dependent steps (lengths, two sums, table, slots)
// and the launches are what a call costs.
//
// One block of 1024 threads does the requests (kChunk at a time): one sum over the pages given back
// and the new tokens, one over the pages wanted.  Up to kInlineTokens tokens it goes on to the slots
// itself; above that a second launch over the whole machine does, from the per-request plan left in
// the workspace.  There a warp looks up the requests of its first and last token by 32-way
// searches (two dependent loads for 1024 requests), and its threads search between them.
//
// Measured (us a call, back to back in a graph): 256 decoding requests, 8 of which end, 5.9; prompts of 96
// requests, 295 thousand tokens, 7.3 to 7.5 (the floor of the traffic is 0.6).  One launch against two: 6.5 /
// 6.9 at 3000 tokens of 8 requests, 7.6 / 6.8 at 4800, 11.6 / 7.0 at 9000.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace fp8q {
namespace plan {

constexpr int kChunk = 1024;
constexpr int kInlineTokens = 4096;
constexpr int kCopies = 4;                   // pages given back that a thread copies at a time
constexpr int kSpreadThreads = 256;
constexpr int kSpreadTokens = 4;             // of a thread (us for 296 thousand tokens: 2 7.6, 4 7.1, 8 8.6)

struct Request {
  int old_len;     // tokens held before
  int from;        // number of its first new page among all new pages; -1: not served
};

struct Params {
  int* table;
  int max_pages;
  const int* lens;
  const int* added;
  int* lens_out;
  int* free;
  int num_pages;
  const int* free_count;
  int* free_count_out;
  int64_t* slots;
  int* positions;
  int* offsets;
  int* served;
  int batch, page_size, max_tokens;
  int inline_tokens;
  FastDiv page_div;
  Request* plan;   // [batch]; null when the slots are done in the same launch
  int* total;      // pages on the free list before any are taken
  uint32_t* err;
};

__device__ __forceinline__ int pages_of(int64_t tokens, const Params& p) {
  return (int)((tokens + p.page_size - 1) / p.page_size);
}

// Inclusive sums over the first n threads of the block; *all: over all of them.  Warps without a value
// take no part: shuffles of 32 warps would cost more than the steps between them.  sh: that no
// thread still reads
struct Pair {
  int64_t x, y;
};
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) { return Pair{a.x + b.x, a.y + b.y}; }
__device__ __forceinline__ Pair shuffle_up(const Pair& v, int o) {
  return Pair{__shfl_up_sync(0xFFFFFFFFu, v.x, o), __shfl_up_sync(0xFFFFFFFFu, v.y, o)};
}
__device__ __forceinline__ int64_t shuffle_up(int64_t v, int o) { return __shfl_up_sync(0xFFFFFFFFu, v, o); }

template <class T>
struct Sums {
  T before[kChunk / 32], all;
};
template <class T>
__device__ __forceinline__ T block_sum(T v, int n, Sums<T>& sh, T* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (n + 31) >> 5;
  const T own = v;
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T up = shuffle_up(v, o);
      if (lane >= o) v = v + up;
    }
    if (lane == 31) sh.before[warp] = v;
  }
  __syncthreads();
  if (warp == 0) {
    T w = T{};
    if (lane < warps) w = sh.before[lane];
    T upto = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T up = shuffle_up(upto, o);
      if (lane >= o) upto = upto + up;
    }
    const T below = shuffle_up(upto, 1);
    sh.before[lane] = lane == 0 ? T{} : below;
    if (lane == 31) sh.all = upto;
  }
  __syncthreads();
  *all = sh.all;
  return warp < warps ? v + sh.before[warp] : own + sh.all;
}

// largest i in [lo, hi) with first[i] <= x (first[lo] <= x)
template <class T>
__device__ __forceinline__ int find(const T* first, int lo, int hi, T x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same in [0, n) by a whole warp, 32 places at a time.
__device__ __forceinline__ int find_by_warp(const int* first, int n, int x) {
  int lo = 0, hi = n;                        // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int span = (hi - lo + 31) / 32, at = lo + (int)(threadIdx.x & 31) * span;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && first[at] <= x);
    lo += (31 - __clz(below | 1u)) * span;
    hi = min(hi, lo + span);
  }
  return lo;
}

// slot and position of token i of request b, whose first one is `first`, and the table entry where it
// is the first of a new page.  Below zero where that holds no page
__device__ __forceinline__ int place_token(const Params& p, int i, int b, int first, const Request& r, int total) {
  const int64_t pos = (int64_t)r.old_len + (i - first);
  int64_t slot = -1;
  int page = 0;
  if (r.from >= 0) {
    const int col = (int)div_u32((uint32_t)pos, p.page_div);
    const int off = (int)(pos - (int64_t)col * p.page_size);
    const int held = pages_of(r.old_len, p);
    int* entry = p.table + (int64_t)b * p.max_pages + col;
    if (col < held) {
      page = *entry;
    } else {
      page = max(-1, p.free[total - 1 - r.from - (col - held)]);
      if (off == 0) *entry = page;
    }
    slot = page < 0 ? -1 : (int64_t)page * p.page_size + off;
  }
  p.slots[i] = slot;
  p.positions[i] = (int)pos;
  return page;
}

// entry i of those that the ending requests give back
__device__ __forceinline__ int back_page(const int* table, int max_pages, const int* first, const int* ending, int givers,
                                         int i) {
  const int k = find(first, 0, givers, i);
  return table[(int64_t)ending[k] * max_pages + (i - first[k])];
}

// The pages among the `given` entries, in order, to `list`, what does not fit dropped; how many there are.  By
// the whole block.  Not inlined: the kernel runs through its code once, and code that it jumps over costs too
// (256 decoding requests 5.85 us against 5.91, 1000 of which 500 end 127.5 against 129.0)
__device__ __noinline__ int pages_alone(const int* table, int max_pages, int given, int givers, const int* first,
                                        const int* ending, int* list, int room, Sums<int64_t>& sh) {
  int kept = 0;
  for (uint32_t i0 = 0; i0 < (uint32_t)given; i0 += kChunk) {
    const uint32_t i = i0 + threadIdx.x;
    const int page = i < (uint32_t)given ? back_page(table, max_pages, first, ending, givers, (int)i) : -1;
    int64_t pages;
    const int at = kept + (int)block_sum<int64_t>(page >= 0 ? 1 : 0, kChunk, sh, &pages) - 1;
    if (page >= 0 && at < room) list[at] = page;
    kept += (int)pages;
    __syncthreads();                         // sh has been read
  }
  return kept;
}

__global__ void __launch_bounds__(kChunk) k_pages_plan(const Params p) {
  __shared__ Sums<Pair> sh_pair;
  __shared__ Sums<int64_t> sh;
  __shared__ int first[kChunk];              // first given-back page of each request that ends; first token of each
  __shared__ int ending[kChunk];             // requests that end
  __shared__ Request sh_plan[kChunk];
  __shared__ int sh_used;
  const int tid = threadIdx.x;
  if (tid == 0) sh_used = 0;
  allow_dependent_launch();
  grid_dependency_wait();

  const int count = *p.free_count;
  const int64_t row_tokens = (int64_t)p.max_pages * p.page_size;
  int64_t total = max(0, min(count, p.num_pages)), tokens = 0;
  if (tid == 0 && total != count) raise_device_error(p.err, kErrBadPage);

  struct Row {
    int64_t len, more;                       // tokens held and new
    bool ends;
  };
  auto row = [&](int b, bool report) {
    Row r = {0, 0, false};
    if (b < p.batch) {
      const int len = p.lens[b], n = p.added[b];
      if (report && (len < 0 || len > row_tokens)) raise_device_error(p.err, kErrBadPage);
      r.len = max((int64_t)0, min((int64_t)len, row_tokens));
      r.ends = n < 0;
      r.more = max(0, n);
    }
    return r;
  };

  // ---- requests that end: their pages go on the free list, in order.  The sums: pages given back
  // (x, less than 2^31 in all) with the number of requests that give some above bit 32, new tokens (y)
  Row r;
  int64_t end = 0;                           // this thread's request's last token + 1 among the new ones
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    if (b0 > 0) __syncthreads();             // sh_pair has been read
    r = row(b0 + tid, true);
    const int back = r.ends ? pages_of(r.len, p) : 0;
    Pair all;
    const Pair upto = block_sum(Pair{back > 0 ? (int64_t(1) << 32) | back : 0, r.more}, min(kChunk, p.batch - b0), sh_pair, &all);
    end = tokens + upto.y;
    if (p.batch > kChunk) tokens = 0;        // summed up again below
    else tokens = all.y;
    const int given = (int)(uint32_t)all.x, givers = (int)(all.x >> 32);
    if (given == 0) continue;                // the same for every thread
    if (back > 0) {
      const int k = (int)(upto.x >> 32) - 1;
      first[k] = (int)(uint32_t)upto.x - back;
      ending[k] = b0 + tid;
    }
    const int64_t room = (int64_t)p.num_pages - total;
    const uint32_t most = (uint32_t)min((int64_t)given, room);
    __syncthreads();
    bool marked = false;
    for (uint32_t i0 = tid; i0 < most; i0 += kCopies * kChunk) {
      int page[kCopies];                     // in flight together
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        const uint32_t i = i0 + c * kChunk;
        page[c] = i < most ? back_page(p.table, p.max_pages, first, ending, givers, (int)i) : 0;
      }
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        marked |= page[c] < 0;
        if (i0 + c * kChunk < most) p.free[total + i0 + c * kChunk] = page[c];
      }
    }
    if (!__syncthreads_or(marked || (uint32_t)given > most)) {
      total += given;
      continue;
    }
    const int kept = pages_alone(p.table, p.max_pages, given, givers, first, ending, p.free + total, (int)room, sh);
    if (kept > room && tid == 0) raise_device_error(p.err, kErrBadPage);
    total += min((int64_t)kept, room);
  }
  __syncthreads();                           // the list is complete

  // ---- the others: pages wanted, served in order while they last
  int64_t wanted = 0, used = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    const int b = b0 + tid;
    int64_t all;
    const int n = min(kChunk, p.batch - b0);
    if (p.batch > kChunk) {
      __syncthreads();                       // sh has been read
      r = row(b, false);
      end = tokens + block_sum(r.more, n, sh, &all);
      tokens += all;
      __syncthreads();
    }
    int64_t need = 0;
    const bool fits = b < p.batch && !r.ends && r.len + r.more <= row_tokens && end <= p.max_tokens;
    if (fits) need = pages_of(r.len + r.more, p) - pages_of(r.len, p);
    const int64_t upto = wanted + block_sum(need, n, sh, &all);
    wanted += all;
    const bool ok = fits && (need == 0 || upto <= total);
    if (b < p.batch) {
      const Request q = {(int)r.len, ok ? (int)(upto - need) : -1};
      const int off = (int)min(end - r.more, (int64_t)0x7FFFFFFF);
      if (p.plan) {
        p.plan[b] = q;
      } else {
        sh_plan[tid] = q;
        first[tid] = off;
      }
      p.offsets[b] = off;
      p.served[b] = ok ? 1 : 0;
      p.lens_out[b] = (int)(r.ends ? 0 : ok ? r.len + r.more : r.len);
    }
    // the pages of the served requests are the first `used`: upto grows with b, and is at most total
    // (below 2^31) where a request that needs pages is served
    const int top = __reduce_max_sync(0xFFFFFFFFu, ok && need > 0 ? (int)upto : 0);
    if ((tid & 31) == 0 && top > 0) atomicMax(&sh_used, top);
  }
  __syncthreads();
  used = sh_used;
  if (tid == 0) {
    p.offsets[p.batch] = (int)min(tokens, (int64_t)0x7FFFFFFF);
    *p.free_count_out = (int)(total - used);
    if (p.total) *p.total = (int)total;
  }
  if (!p.inline_tokens) return;

  // ---- slots and positions
  const int n = (int)min(tokens, (int64_t)p.max_tokens);
  int bad = 0;
#pragma unroll 2
  for (int i = tid; i < p.max_tokens; i += kChunk) {
    if (i < n) {
      const int b = find(first, 0, p.batch, i);
      bad |= place_token(p, i, b, first[b], sh_plan[b], (int)total);
    } else {
      p.slots[i] = -1;
      p.positions[i] = 0;
    }
  }
  if (bad < 0) raise_device_error(p.err, kErrBadPage);
}

__global__ void __launch_bounds__(kSpreadThreads) k_pages_spread(const Params p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int n = min(p.offsets[p.batch], p.max_tokens), total = *p.total;
  const int lane = threadIdx.x & 31;
  const int64_t begin = ((int64_t)blockIdx.x * (kSpreadThreads / 32) + (threadIdx.x >> 5)) * (32 * kSpreadTokens);
  if (begin >= p.max_tokens) return;
  int lo = 0, hi = 0;
  if (begin < n) {
    lo = find_by_warp(p.offsets, p.batch, (int)begin);
    hi = find_by_warp(p.offsets, p.batch, (int)min(begin + 32 * kSpreadTokens, (int64_t)n) - 1);
  }
  int bad = 0;
#pragma unroll
  for (int k = 0; k < kSpreadTokens; ++k) {
    const int64_t i = begin + 32 * k + lane;
    if (i < n) {
      const int b = find(p.offsets, lo, hi + 1, (int)i);
      bad |= place_token(p, (int)i, b, p.offsets[b], p.plan[b], total);
    } else if (i < p.max_tokens) {
      p.slots[i] = -1;
      p.positions[i] = 0;
    }
  }
  if (bad < 0) raise_device_error(p.err, kErrBadPage);
}

}  // namespace plan

namespace {
bool plan_inline(int64_t batch, int64_t max_tokens) {
  return batch <= plan::kChunk && max_tokens <= plan::kInlineTokens;
}
}  // namespace

size_t pages_workspace_bytes(int64_t batch, int64_t max_tokens) {
  return plan_inline(batch, max_tokens) ? 0 : (size_t)batch * sizeof(plan::Request) + 16;
}

cudaError_t launch_pages_update(const PagesUpdate& u, cudaStream_t st) {
  plan::Params p;
  p.table = u.table;
  p.max_pages = (int)u.max_pages;
  p.lens = u.lens;
  p.added = u.added;
  p.lens_out = u.lens_out;
  p.free = u.free_pages;
  p.num_pages = (int)u.num_pages;
  p.free_count = u.free_count;
  p.free_count_out = u.free_count_out;
  p.slots = u.slots;
  p.positions = u.positions;
  p.offsets = u.offsets;
  p.served = u.served;
  p.batch = (int)u.batch;
  p.page_size = (int)u.page_size;
  p.max_tokens = (int)u.max_tokens;
  p.inline_tokens = plan_inline(u.batch, u.max_tokens) ? 1 : 0;
  p.page_div = make_fastdiv((uint32_t)u.page_size);
  p.total = p.inline_tokens ? nullptr : static_cast<int*>(u.ws);
  p.plan = p.inline_tokens ? nullptr : reinterpret_cast<plan::Request*>(static_cast<uint8_t*>(u.ws) + 16);
  p.err = device_error_word();
  const cudaError_t e = launch_pdl(plan::k_pages_plan, dim3(1), dim3(plan::kChunk), 0, st, p);
  if (e != cudaSuccess || p.inline_tokens || u.max_tokens == 0) return e;
  const int64_t per_block = plan::kSpreadThreads * plan::kSpreadTokens;
  const int blocks = (int)((u.max_tokens + per_block - 1) / per_block);
  return launch_pdl(plan::k_pages_spread, dim3(blocks), dim3(plan::kSpreadThreads), 0, st, p);
}

}  // namespace fp8q
