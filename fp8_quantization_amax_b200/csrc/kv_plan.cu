// Block tables, slots and positions from the requests' lengths (fp8_kv_pages_update): the page
// bookkeeping of one serving step on the device, so that lengths never travel to the host.
//
// Requests that end put their pages on the free list; then the others take the pages their new
// tokens need from its top.  Both are prefix sums over the requests in order, so the result does
// not depend on timing.  What bounds it: 12 bytes written a token and a few words a request, a
// microsecond of traffic at most: the chain of dependent steps (lengths, two sums, table, slots)
// and the launches are what a call costs.
//
// One block of 1024 threads does the requests (kChunk at a time).  Up to kInlineTokens tokens it
// goes on to the slots itself; above that a second launch over the whole machine does, from the
// per-request plan left in the workspace.
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
constexpr int kSpreadThreads = 256;

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

// inclusive sum over the block's threads; *all: the block's sum
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sh, int64_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int k = 0; k < kChunk / 32; ++k) {
    const int64_t x = sh[k];
    if (k < warp) before += x;
    total += x;
  }
  *all = total;
  return v + before;
}

// largest i in [0, n) with first[i] <= x (first[0] <= x)
template <class T>
__device__ __forceinline__ int find(const T* first, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// slot and position of token i, and the table entry where it is the first of a new page
__device__ __forceinline__ void place_token(const Params& p, int i, const int* offsets, const Request* plan, int total) {
  const int b = find(offsets, p.batch, i);
  const Request r = plan[b];
  const int64_t pos = (int64_t)r.old_len + (i - offsets[b]);
  int64_t slot = -1;
  if (r.from >= 0) {
    const int col = (int)div_u32((uint32_t)pos, p.page_div);
    const int off = (int)(pos - (int64_t)col * p.page_size);
    const int held = pages_of(r.old_len, p);
    int* entry = p.table + (int64_t)b * p.max_pages + col;
    int page;
    if (col < held) {
      page = *entry;
    } else {
      page = p.free[total - 1 - r.from - (col - held)];
      if (off == 0) *entry = page;
    }
    slot = (int64_t)page * p.page_size + off;
  }
  p.slots[i] = slot;
  p.positions[i] = (int)pos;
}

__global__ void __launch_bounds__(kChunk) k_pages_plan(const Params p) {
  __shared__ int64_t sh[kChunk / 32];
  __shared__ int first[kChunk + 1];          // first given-back page, later first token, of each request
  __shared__ Request sh_plan[kChunk];
  const int tid = threadIdx.x;
  allow_dependent_launch();
  grid_dependency_wait();

  int count = *p.free_count;
  if (count < 0 || count > p.num_pages) {
    if (tid == 0) raise_device_error(p.err, kErrBadPage);
    count = max(0, min(count, p.num_pages));
  }
  const int64_t row_tokens = (int64_t)p.max_pages * p.page_size;

  // ---- requests that end: their pages go on the free list, in order
  int64_t total = count;
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    const int b = b0 + tid;
    int64_t back = 0;
    if (b < p.batch) {
      const int64_t len = p.lens[b];
      if (len < 0 || len > row_tokens) raise_device_error(p.err, kErrBadPage);
      if (p.added[b] < 0) back = pages_of(max((int64_t)0, min(len, row_tokens)), p);
    }
    int64_t all;
    const int64_t incl = block_sum(back, sh, &all);
    if (all == 0) continue;                  // the same for every thread
    int64_t room = (int64_t)p.num_pages - total;
    if (all > room && tid == 0) raise_device_error(p.err, kErrBadPage);
    if (all < room) room = all;              // what does not fit on the list is dropped
    first[tid] = (int)(incl - back);         // at most the table's entries: checked on the host
    __syncthreads();
    const int nb = min(kChunk, p.batch - b0);
    for (int i = tid; i < room; i += kChunk) {
      // among requests that start at the same page (all but the last give none back) the last
      const int r = find(first, nb, i);
      p.free[total + i] = p.table[(int64_t)(b0 + r) * p.max_pages + (i - first[r])];
    }
    total += room;
    __syncthreads();
  }
  __syncthreads();                           // the list is complete

  // ---- the others: pages wanted, served in order while they last
  int64_t wanted = 0, tokens = 0, used = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    const int b = b0 + tid;
    int64_t len = 0, more = 0, need = 0;
    bool fits = false, ends = false;
    if (b < p.batch) {
      len = max((int64_t)0, min((int64_t)p.lens[b], row_tokens));
      const int n = p.added[b];
      ends = n < 0;
      more = max(0, n);
      fits = !ends && len + more <= row_tokens;
    }
    int64_t all;
    const int64_t end = tokens + block_sum(more, sh, &all);
    tokens += all;
    fits = fits && end <= p.max_tokens;
    if (fits) need = pages_of(len + more, p) - pages_of(len, p);
    const int64_t upto = wanted + block_sum(need, sh, &all);
    wanted += all;
    const bool ok = fits && (need == 0 || upto <= total);
    if (b < p.batch) {
      const Request r = {(int)len, ok ? (int)(upto - need) : -1};
      if (p.plan) p.plan[b] = r;
      else sh_plan[tid] = r;
      const int off = (int)min(end - more, (int64_t)0x7FFFFFFF);
      if (!p.plan) first[tid] = off;
      p.offsets[b] = off;
      p.served[b] = ok ? 1 : 0;
      p.lens_out[b] = (int)(ends ? 0 : ok ? len + more : len);
    }
    // the pages of the served requests are the first `used`: upto grows with b
    const int64_t mine = ok ? upto : 0;
    int64_t top = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    __syncthreads();
    if ((tid & 31) == 0) sh[tid >> 5] = top;
    __syncthreads();
    for (int k = 0; k < kChunk / 32; ++k) used = max(used, sh[k]);
  }
  if (tid == 0) {
    p.offsets[p.batch] = (int)min(tokens, (int64_t)0x7FFFFFFF);
    *p.free_count_out = (int)(total - used);
    if (p.total) *p.total = (int)total;
  }
  if (!p.inline_tokens) return;

  // ---- slots and positions
  __syncthreads();
  const int n = (int)min(tokens, (int64_t)p.max_tokens);
  for (int i = tid; i < p.max_tokens; i += kChunk) {
    if (i < n) {
      place_token(p, i, first, sh_plan, (int)total);
    } else {
      p.slots[i] = -1;
      p.positions[i] = 0;
    }
  }
}

__global__ void __launch_bounds__(kSpreadThreads) k_pages_spread(const Params p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int n = p.offsets[p.batch];
  const int i = blockIdx.x * kSpreadThreads + threadIdx.x;
  if (i >= p.max_tokens) return;
  if (i < n) {
    place_token(p, i, p.offsets, p.plan, *p.total);
  } else {
    p.slots[i] = -1;
    p.positions[i] = 0;
  }
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
  if (e != cudaSuccess || p.inline_tokens) return e;
  const int blocks = (int)((u.max_tokens + plan::kSpreadThreads - 1) / plan::kSpreadThreads);
  return launch_pdl(plan::k_pages_spread, dim3(blocks), dim3(plan::kSpreadThreads), 0, st, p);
}

}  // namespace fp8q
