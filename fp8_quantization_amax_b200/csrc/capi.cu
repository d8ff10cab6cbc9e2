// C-ABI entry points declared in include/fp8q.h: argument validation, sizes and dispatch.
// Every check happens on the host before anything is launched.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp8q.h"
#include "internal.h"
#include "kv_pages.cuh"

namespace fp8q {
cudaError_t launch_selftest_wait(cudaStream_t st);
}

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 33;   // 32-bit indexing of 16-byte pieces of two tensors
constexpr int64_t kMaxHistory = int64_t(1) << 20;   // amax history entries per group (the kernels index with int)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool valid_fmt(int f) { return f == FP8Q_E4M3 || f == FP8Q_E5M2; }
bool valid_gran(int g) { return g == FP8Q_PER_TENSOR || g == FP8Q_GROUP_1x128 || g == FP8Q_BLOCK_128x128; }
bool valid_kv_gran(int g) {
  return g == FP8Q_KV_PER_TENSOR || g == FP8Q_KV_PER_HEAD || g == FP8Q_KV_PER_HEAD_TOK128;
}
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// rows * cols without overflow; -1 when it does not fit the library's indexing
int64_t checked_elems(int64_t a, int64_t b) {
  if (a < 0 || b < 0) return -1;
  if (a == 0 || b == 0) return 0;
  if (a > kMaxElems / b) return -1;
  return a * b;
}

constexpr int64_t kMaxTableTokens = (int64_t(1) << 31) - 65;   // token numbers and slots fit an int

constexpr int64_t kMaxSpan = int64_t(1) << 36;                 // bytes of a paged K or V

// A paged cache from the caller's description; FP8Q_OK and *out, or the reason why not.
fp8q_status paged_cache(const fp8q_kv_pages* c, fp8q::KvPages* out) {
  if (!c || !valid_fmt(c->f) || c->g < FP8Q_KV_PER_TENSOR || c->g > FP8Q_KV_PER_TOKEN) return FP8Q_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 0 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1) return FP8Q_ERR_INVALID_ARGUMENT;
  // strides of dimensions of one entry are not used
  const int64_t page_stride = c->num_pages > 1 ? c->page_stride : 0, token_stride = c->page_size > 1 ? c->token_stride : 0,
                head_stride = c->heads > 1 ? c->head_stride : 0;
  if (c->head_dim % 16 != 0 || page_stride % 16 != 0 || token_stride % 16 != 0 || head_stride % 16 != 0)
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (c->head_dim > 256 || c->heads > 65536 || c->page_size > kMaxTableTokens ||
      (c->num_pages > 0 && c->page_size > kMaxTableTokens / c->num_pages))
    return FP8Q_ERR_UNSUPPORTED;
  // the last code's place, in units of 16 bytes, fits 32 bits (64 GB a tensor)
  if (page_stride > kMaxSpan || token_stride > kMaxSpan || head_stride > kMaxSpan ||
      page_stride * (double)c->num_pages + token_stride * (double)c->page_size + head_stride * (double)c->heads >
          (double)kMaxSpan)
    return FP8Q_ERR_UNSUPPORTED;
  // places of different tokens, heads and pages do not overlap: taken by their strides, each dimension steps
  // over all that lies within one entry of it
  struct Dim {
    int64_t stride, n;
  } dims[3] = {{page_stride, c->num_pages}, {token_stride, c->page_size}, {head_stride, c->heads}};
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t within = c->head_dim;              // bytes from the first to the last code of an entry
  for (const Dim& d : dims) {
    if (d.n <= 1) continue;
    if (d.stride < within) return FP8Q_ERR_INVALID_ARGUMENT;
    within += (d.n - 1) * d.stride;          // (at most kMaxSpan)
  }
  if (!c->k_scales || !c->v_scales || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (c->num_pages > 0 && (!c->k_codes || !c->v_codes || !aligned(c->k_codes, 16) || !aligned(c->v_codes, 16)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  out->k = c->k_codes;
  out->v = c->v_codes;
  out->ks = c->k_scales;
  out->vs = c->v_scales;
  out->page_stride = page_stride;
  out->token_stride = token_stride;
  out->head_stride = head_stride;
  out->num_pages = (int)c->num_pages;
  out->page_size = (int)c->page_size;
  out->heads = (int)c->heads;
  out->head_dim = (int)c->head_dim;
  out->gran = c->g;
  out->page_div = fp8q::make_fastdiv((uint32_t)c->page_size);
  return FP8Q_OK;
}

fp8q_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA; }

}  // namespace

extern "C" {

const char* fp8q_status_string(fp8q_status status) {
  switch (status) {
    case FP8Q_OK: return "ok";
    case FP8Q_ERR_INVALID_ARGUMENT: return "invalid argument";
    case FP8Q_ERR_UNSUPPORTED: return "unsupported";
    case FP8Q_ERR_WORKSPACE: return "workspace missing or too small";
    case FP8Q_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

int fp8q_version(void) { return 100; }

uint32_t fp8q_device_status(void) { return fp8q::read_and_clear_device_error(); }

fp8q_status fp8q_selftest_wait_timeout(fp8q_stream_t stream) {
  return from_cuda(fp8q::launch_selftest_wait((cudaStream_t)stream));
}

int fp8q_check_tile_walk(int64_t M, int64_t N, int64_t K) { return fp8q::check_tile_walk(M, N, K); }

int fp8q_check_decode_split(int64_t M, int64_t N, int64_t K, int sms) {
  return fp8q::check_decode_split(M, N, K, sms);
}

size_t fp8q_num_scales(int64_t rows, int64_t cols, fp8q_granularity g) {
  if (rows < 0 || cols < 0 || !valid_gran(g)) return 0;
  if (g == FP8Q_PER_TENSOR) return 1;
  if (g == FP8Q_GROUP_1x128) return (size_t)(cdiv(cols, 128) * rows);
  return (size_t)(cdiv(rows, 128) * cdiv(cols, 128));
}

size_t fp8q_workspace_bytes(int64_t rows, int64_t cols, fp8q_granularity g) {
  if (rows < 0 || cols < 0 || !valid_gran(g)) return 0;
  return g == FP8Q_PER_TENSOR ? fp8q::two_pass_workspace_bytes(1, 1) : 0;
}

size_t fp8q_kv_num_scales(int64_t tokens, int64_t heads, fp8q_kv_granularity g) {
  if (tokens < 0 || heads < 0 || !valid_kv_gran(g)) return 0;
  if (g == FP8Q_KV_PER_TENSOR) return 1;
  if (g == FP8Q_KV_PER_HEAD) return (size_t)heads;
  return (size_t)(cdiv(tokens, 128) * heads);
}

size_t fp8q_kv_workspace_bytes(int64_t tokens, int64_t heads, int64_t head_dim, fp8q_kv_granularity g) {
  if (tokens < 0 || heads < 0 || head_dim < 0 || !valid_kv_gran(g)) return 0;
  if (g == FP8Q_KV_PER_TENSOR) return fp8q::two_pass_workspace_bytes(2, 1);
  if (g == FP8Q_KV_PER_HEAD) return fp8q::two_pass_workspace_bytes(2, heads);
  return 0;
}

size_t fp8q_linear_act_workspace_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || K % 128 != 0 || checked_elems(M, K) < 0) return 0;
  return fp8q::linear_act_workspace_bytes(M, K);
}

size_t fp8q_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return 0;
  return fp8q::gemm_workspace_bytes(M, N, K);
}

fp8q_status fp8_encode(const float* q, int64_t n, fp8q_format f, uint8_t* codes, fp8q_stream_t stream) {
  if (n < 0 || n > kMaxElems || !valid_fmt(f)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n == 0) return FP8Q_OK;
  if (!q || !codes || !aligned(q, 16) || !aligned(codes, 16)) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_encode(q, n, f, codes, (cudaStream_t)stream));
}

fp8q_status fp8_decode(const uint8_t* codes, int64_t n, fp8q_format f, float* out, fp8q_stream_t stream) {
  if (n < 0 || n > kMaxElems || !valid_fmt(f)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n == 0) return FP8Q_OK;
  if (!codes || !out || !aligned(codes, 16) || !aligned(out, 16)) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_decode(codes, n, f, out, (cudaStream_t)stream));
}

fp8q_status fp8_quantize(const void* x, int64_t rows, int64_t cols, fp8q_format f, fp8q_granularity g,
                         uint8_t* codes, float* scales, void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || !valid_gran(g) || cols % 8 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (n > 0 && (!x || !codes || !aligned(x, 16) || !aligned(codes, 16))) return FP8Q_ERR_INVALID_ARGUMENT;
  if ((n > 0 || g == FP8Q_PER_TENSOR) && (!scales || !aligned(scales, 4))) return FP8Q_ERR_INVALID_ARGUMENT;
  const cudaStream_t st = (cudaStream_t)stream;
  const uint16_t* xs = static_cast<const uint16_t*>(x);
  if (g == FP8Q_PER_TENSOR) {
    const size_t need = fp8q_workspace_bytes(rows, cols, g);
    if (!ws || ws_bytes < need || !aligned(ws, 4)) return FP8Q_ERR_WORKSPACE;
    return from_cuda(fp8q::launch_quant_two_pass(xs, nullptr, codes, nullptr, scales, nullptr, 1, rows, 1, cols, f,
                                                 static_cast<float*>(ws), st));
  }
  if (n == 0) return FP8Q_OK;
  if (g == FP8Q_GROUP_1x128) return from_cuda(fp8q::launch_quant_1x128(xs, rows, cols, f, codes, scales, st));
  return from_cuda(
      fp8q::launch_quant_tiles(xs, nullptr, codes, nullptr, scales, nullptr, 1, rows, cols, cols, 128, f, st));
}

fp8q_status fp8_quantize_many(const fp8q_quant_tensor* tensors, int n, fp8q_format f, fp8q_stream_t stream) {
  if (!tensors || n < 1 || n > fp8q::kMaxManyJobs || !valid_fmt(f)) return FP8Q_ERR_INVALID_ARGUMENT;
  fp8q::QuantJob jobs[fp8q::kMaxManyJobs];
  for (int j = 0; j < n; ++j) {
    const fp8q_quant_tensor& t = tensors[j];
    const int64_t e = checked_elems(t.rows, t.cols);
    if (t.rows < 0 || t.cols < 0 || !valid_gran(t.g) || t.cols % 8 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
    if (t.g == FP8Q_PER_TENSOR) return FP8Q_ERR_UNSUPPORTED;
    if (e < 0) return FP8Q_ERR_UNSUPPORTED;
    if (e > 0 && (!t.x || !t.codes || !t.scales || !aligned(t.x, 16) || !aligned(t.codes, 16) ||
                  !aligned(t.scales, 4)))
      return FP8Q_ERR_INVALID_ARGUMENT;
    jobs[j].x = static_cast<const uint16_t*>(t.x);
    jobs[j].rows = t.rows;
    jobs[j].cols = t.cols;
    jobs[j].block = t.g == FP8Q_BLOCK_128x128 ? 1 : 0;
    jobs[j].codes = t.codes;
    jobs[j].scales = t.scales;
  }
  return from_cuda(fp8q::launch_quant_many(jobs, n, f, (cudaStream_t)stream));
}

fp8q_status fp8_quantize_mx(const void* x, int64_t rows, int64_t cols, fp8q_format f, uint8_t* codes,
                            uint8_t* scales, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || cols % 32 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16)) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_quant_mx(static_cast<const uint16_t*>(x), rows, cols, f, codes, scales, 0,
                                         (cudaStream_t)stream));
}

size_t fp8q_mx_blocked_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return (size_t)(cdiv(rows, 128) * cdiv(cols, 128) * 512);
}

fp8q_status fp8_quantize_mx_blocked(const void* x, int64_t rows, int64_t cols, fp8q_format f, uint8_t* codes,
                                    uint8_t* scales, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || cols % 32 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16)) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_quant_mx(static_cast<const uint16_t*>(x), rows, cols, f, codes, scales, 1,
                                         (cudaStream_t)stream));
}

fp8q_status fp8_dequantize_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, fp8q_format f,
                              void* y, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || cols % 32 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(y, 16)) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_dequant(codes, reinterpret_cast<const float*>(scales), rows, cols, f, 3,
                                        static_cast<uint16_t*>(y), (cudaStream_t)stream));
}

fp8q_status fp8_quantize_delayed(const void* x, int64_t rows, int64_t cols, fp8q_format f, float* amax_history,
                                 int64_t history_len, int64_t step, uint8_t* codes, float* scale,
                                 unsigned long long* counts, void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || cols % 8 != 0 || history_len < 1 || step < 0)
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0 || history_len > kMaxHistory) return FP8Q_ERR_UNSUPPORTED;
  if (n > 0 && (!x || !codes || !aligned(x, 16) || !aligned(codes, 16))) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!scale || !aligned(scale, 4) || !amax_history || !aligned(amax_history, 4)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (counts && !aligned(counts, 8)) return FP8Q_ERR_INVALID_ARGUMENT;
  const size_t need = fp8q_workspace_bytes(rows, cols, FP8Q_PER_TENSOR);
  if (!ws || ws_bytes < need || !aligned(ws, 4)) return FP8Q_ERR_WORKSPACE;
  return from_cuda(fp8q::launch_quant_delayed(static_cast<const uint16_t*>(x), nullptr, codes, nullptr, scale, nullptr,
                                              1, rows, 1, cols, f, amax_history, nullptr, history_len, step, counts,
                                              static_cast<float*>(ws), (cudaStream_t)stream));
}

fp8q_status fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, fp8q_format f,
                           fp8q_granularity g, void* y, fp8q_stream_t stream) {
  const int64_t n = checked_elems(rows, cols);
  if (rows < 0 || cols < 0 || !valid_fmt(f) || !valid_gran(g) || cols % 8 != 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(y, 16) || !aligned(scales, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_dequant(codes, scales, rows, cols, f, g, static_cast<uint16_t*>(y),
                                        (cudaStream_t)stream));
}

fp8q_status fp8_kv_quantize(const void* k, const void* v, int64_t tokens, int64_t heads, int64_t head_dim,
                            fp8q_format f, fp8q_kv_granularity g, uint8_t* k_codes, uint8_t* v_codes,
                            float* k_scales, float* v_scales, void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  if (tokens < 0 || heads < 0 || head_dim < 0 || !valid_fmt(f) || !valid_kv_gran(g) || head_dim % 8 != 0)
    return FP8Q_ERR_INVALID_ARGUMENT;
  const int64_t row = checked_elems(heads, head_dim);
  const int64_t n = row < 0 ? -1 : checked_elems(tokens, row);
  if (n < 0) return FP8Q_ERR_UNSUPPORTED;
  if (g == FP8Q_KV_PER_HEAD_TOK128 && head_dim > 256) return FP8Q_ERR_UNSUPPORTED;
  if (g == FP8Q_KV_PER_HEAD && (heads > 128 || head_dim > 256)) return FP8Q_ERR_UNSUPPORTED;
  const size_t nsc = fp8q_kv_num_scales(tokens, heads, g);
  if (n > 0 && (!k || !v || !k_codes || !v_codes || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_codes, 16) ||
                !aligned(v_codes, 16)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (nsc > 0 && (!k_scales || !v_scales || !aligned(k_scales, 4) || !aligned(v_scales, 4)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const cudaStream_t st = (cudaStream_t)stream;
  const uint16_t* ks = static_cast<const uint16_t*>(k);
  const uint16_t* vs = static_cast<const uint16_t*>(v);
  if (g == FP8Q_KV_PER_HEAD_TOK128) {
    if (n == 0) return FP8Q_OK;
    return from_cuda(fp8q::launch_quant_tiles(ks, vs, k_codes, v_codes, k_scales, v_scales, 2, tokens, row, row,
                                              (int)head_dim, f, st));
  }
  if (nsc == 0) return FP8Q_OK;   // no heads: nothing to write
  const size_t need = fp8q_kv_workspace_bytes(tokens, heads, head_dim, g);
  if (!ws || ws_bytes < need || !aligned(ws, 4)) return FP8Q_ERR_WORKSPACE;
  const int64_t h = g == FP8Q_KV_PER_TENSOR ? 1 : heads;
  const int64_t d = g == FP8Q_KV_PER_TENSOR ? row : head_dim;
  return from_cuda(fp8q::launch_quant_two_pass(ks, vs, k_codes, v_codes, k_scales, v_scales, 2, tokens, h, d, f,
                                               static_cast<float*>(ws), st));
}

fp8q_status fp8_kv_quantize_delayed(const void* k, const void* v, int64_t tokens, int64_t heads, int64_t head_dim,
                                    fp8q_format f, fp8q_kv_granularity g, float* k_history, float* v_history,
                                    int64_t history_len, int64_t step, uint8_t* k_codes, uint8_t* v_codes,
                                    float* k_scales, float* v_scales, unsigned long long* counts, void* ws,
                                    size_t ws_bytes, fp8q_stream_t stream) {
  if (tokens < 0 || heads < 0 || head_dim < 0 || !valid_fmt(f) || !valid_kv_gran(g) || head_dim % 8 != 0 ||
      history_len < 1 || step < 0)
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (g == FP8Q_KV_PER_HEAD_TOK128) return FP8Q_ERR_UNSUPPORTED;   // already one pass: no history to keep
  const int64_t row = checked_elems(heads, head_dim);
  const int64_t n = row < 0 ? -1 : checked_elems(tokens, row);
  if (n < 0 || history_len > kMaxHistory) return FP8Q_ERR_UNSUPPORTED;
  if (g == FP8Q_KV_PER_HEAD && (heads > 128 || head_dim > 256)) return FP8Q_ERR_UNSUPPORTED;
  const size_t nsc = fp8q_kv_num_scales(tokens, heads, g);
  if (n > 0 && (!k || !v || !k_codes || !v_codes || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_codes, 16) ||
                !aligned(v_codes, 16)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (nsc > 0 && (!k_scales || !v_scales || !aligned(k_scales, 4) || !aligned(v_scales, 4) || !k_history ||
                  !v_history || !aligned(k_history, 4) || !aligned(v_history, 4)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (counts && !aligned(counts, 8)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (nsc == 0) return FP8Q_OK;   // no heads: nothing to write
  const size_t need = fp8q_kv_workspace_bytes(tokens, heads, head_dim, g);
  if (!ws || ws_bytes < need || !aligned(ws, 4)) return FP8Q_ERR_WORKSPACE;
  const int64_t h = g == FP8Q_KV_PER_TENSOR ? 1 : heads;
  const int64_t d = g == FP8Q_KV_PER_TENSOR ? row : head_dim;
  return from_cuda(fp8q::launch_quant_delayed(static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                                              k_codes, v_codes, k_scales, v_scales, 2, tokens, h, d, f, k_history,
                                              v_history, history_len, step, counts, static_cast<float*>(ws),
                                              (cudaStream_t)stream));
}

fp8q_status fp8_gemm_blockscaled(const uint8_t* A, const float* sA, fp8q_granularity gA, const uint8_t* B,
                                 const float* sB, fp8q_granularity gB, int64_t M, int64_t N, int64_t K, void* C,
                                 void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gA == FP8Q_GROUP_1x128 || gA == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gB == FP8Q_BLOCK_128x128 || gB == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (!A || !B || !C || !sA || !sB || !aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(sA, 4) ||
      !aligned(sB, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const size_t need = fp8q::gemm_workspace_bytes(M, N, K);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return FP8Q_ERR_WORKSPACE;
  const cudaError_t e = fp8q::launch_gemm(A, sA, gA, B, false, sB, gB, M, N, K, static_cast<uint16_t*>(C), ws,
                                          ws_bytes, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8Q_ERR_UNSUPPORTED;
  return from_cuda(e);
}

fp8q_status fp8_scale_histogram(const void* scales, int64_t n, fp8q_scale_kind kind, uint32_t* hist,
                                fp8q_stream_t stream) {
  if (n < 0 || !(kind == FP8Q_SCALES_F32 || kind == FP8Q_SCALES_MX)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n > kMaxElems) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!scales || !hist || !aligned(hist, 4) || (kind == FP8Q_SCALES_F32 && !aligned(scales, 4)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_scale_histogram(scales, n, kind, hist, (cudaStream_t)stream));
}

fp8q_status fp8_count_underflow(const void* x, const uint8_t* codes, int64_t n, unsigned long long* count,
                                fp8q_stream_t stream) {
  if (n < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (n > kMaxElems) return FP8Q_ERR_UNSUPPORTED;
  if (n == 0) return FP8Q_OK;
  if (!x || !codes || !count || !aligned(x, 16) || !aligned(codes, 16) || !aligned(count, 8))
    return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_count_underflow(static_cast<const uint16_t*>(x), codes, n, count,
                                                (cudaStream_t)stream));
}

fp8q_status fp8_gemm_blockscaled_to_fp8(const uint8_t* A, const float* sA, fp8q_granularity gA, const uint8_t* B,
                                        const float* sB, fp8q_granularity gB, int64_t M, int64_t N, int64_t K,
                                        uint8_t* codes, float* scales, fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gA == FP8Q_GROUP_1x128 || gA == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gB == FP8Q_BLOCK_128x128 || gB == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (M <= 64) return FP8Q_ERR_UNSUPPORTED;   // decode shapes: the decode kernel has no such epilogue
  if (!A || !B || !codes || !sA || !sB || !scales || !aligned(A, 16) || !aligned(B, 16) || !aligned(codes, 16) ||
      !aligned(sA, 4) || !aligned(sB, 4) || !aligned(scales, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const cudaError_t e = fp8q::launch_gemm_to_fp8(A, sA, gA, B, false, sB, gB, M, N, K, codes, scales,
                                                 (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8Q_ERR_UNSUPPORTED;
  return from_cuda(e);
}

fp8q_status fp8_pack_b_tiles(const uint8_t* B, int64_t N, int64_t K, uint8_t* packed, fp8q_stream_t stream) {
  if (N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(N, K) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (!B || !packed || !aligned(B, 16) || !aligned(packed, 16) || B == packed) return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_pack_b_tiles(B, N, K, packed, (cudaStream_t)stream));
}

fp8q_status fp8_gemm_blockscaled_packed(const uint8_t* A, const float* sA, fp8q_granularity gA, const uint8_t* Bp,
                                        const float* sB, fp8q_granularity gB, int64_t M, int64_t N, int64_t K,
                                        void* C, void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gA == FP8Q_GROUP_1x128 || gA == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gB == FP8Q_BLOCK_128x128 || gB == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (!A || !Bp || !C || !sA || !sB || !aligned(A, 16) || !aligned(Bp, 16) || !aligned(C, 16) || !aligned(sA, 4) ||
      !aligned(sB, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const size_t need = fp8q::gemm_workspace_bytes(M, N, K);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return FP8Q_ERR_WORKSPACE;
  const cudaError_t e = fp8q::launch_gemm(A, sA, gA, Bp, true, sB, gB, M, N, K, static_cast<uint16_t*>(C), ws,
                                          ws_bytes, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8Q_ERR_UNSUPPORTED;
  return from_cuda(e);
}

fp8q_status fp8_linear_dynamic(const void* X, int64_t M, int64_t N, int64_t K, const uint8_t* B, const float* sB,
                               fp8q_granularity gB, void* C, void* act_ws, size_t act_ws_bytes, void* gemm_ws,
                               size_t gemm_ws_bytes, fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gB == FP8Q_BLOCK_128x128 || gB == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (!X || !B || !C || !sB || !aligned(X, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(sB, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (!act_ws || act_ws_bytes < fp8q::linear_act_workspace_bytes(M, K) || !aligned(act_ws, 16))
    return FP8Q_ERR_WORKSPACE;
  const size_t need = fp8q::gemm_workspace_bytes(M, N, K);
  if (need > 0 && (!gemm_ws || gemm_ws_bytes < need || !aligned(gemm_ws, 16))) return FP8Q_ERR_WORKSPACE;
  const cudaError_t e = fp8q::launch_linear(static_cast<const uint16_t*>(X), B, sB, gB, M, N, K,
                                            static_cast<uint16_t*>(C), act_ws, gemm_ws, gemm_ws_bytes,
                                            (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8Q_ERR_UNSUPPORTED;
  return from_cuda(e);
}

size_t fp8q_linear_fused_workspace_bytes(int64_t M, int64_t K) {
  if (M <= 64 || K <= 0 || K % 128 != 0 || checked_elems(M, K) < 0) return 0;
  return fp8q::linear_fused_workspace_bytes(M, K);
}

fp8q_status fp8_linear_dynamic_fused(const void* X, int64_t M, int64_t N, int64_t K, const uint8_t* B, const float* sB,
                                     fp8q_granularity gB, void* C, void* act_ws, size_t act_ws_bytes,
                                     fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (!(gB == FP8Q_BLOCK_128x128 || gB == FP8Q_PER_TENSOR)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (M <= 64) return FP8Q_ERR_UNSUPPORTED;   // decode shapes: fp8_linear_dynamic
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (!X || !B || !C || !sB || !aligned(X, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(sB, 4))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (!act_ws || act_ws_bytes < fp8q::linear_fused_workspace_bytes(M, K) || !aligned(act_ws, 256))
    return FP8Q_ERR_WORKSPACE;
  const cudaError_t e = fp8q::launch_linear_fused(static_cast<const uint16_t*>(X), B, sB, gB, M, N, K,
                                                  static_cast<uint16_t*>(C), act_ws, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported || e == cudaErrorCooperativeLaunchTooLarge) return FP8Q_ERR_UNSUPPORTED;
  return from_cuda(e);
}

fp8q_status fp8_gemm_mx(const uint8_t* A, const uint8_t* sA, fp8q_format fa, const uint8_t* B, const uint8_t* sB,
                        fp8q_format fb, int64_t M, int64_t N, int64_t K, void* C, fp8q_stream_t stream) {
  if (M < 0 || N < 0 || K < 0 || !valid_fmt(fa) || !valid_fmt(fb)) return FP8Q_ERR_INVALID_ARGUMENT;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (N % 128 != 0 || K % 128 != 0 || K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (checked_elems(M, K) < 0 || checked_elems(N, K) < 0 || checked_elems(M, N) < 0) return FP8Q_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 31) - 1 || N > (int64_t(1) << 31) - 1) return FP8Q_ERR_UNSUPPORTED;
  if (!A || !B || !C || !sA || !sB || !aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(sA, 16) ||
      !aligned(sB, 16))
    return FP8Q_ERR_INVALID_ARGUMENT;
  return from_cuda(fp8q::launch_gemm_mx(A, sA, fa, B, sB, fb, M, N, K, static_cast<uint16_t*>(C),
                                        (cudaStream_t)stream));
}

// ------------------------------------------------------------------ paged KV cache

size_t fp8q_pages_workspace_bytes(int64_t batch, int64_t max_tokens) {
  if (batch < 0 || max_tokens < 0) return 0;
  return fp8q::pages_workspace_bytes(batch, max_tokens);
}

fp8q_status fp8_kv_pages_update(int32_t* block_table, int64_t batch, int64_t max_pages, int64_t page_size,
                                const int32_t* lens, const int32_t* added, int32_t* lens_out, int32_t* free_pages,
                                int64_t num_pages, const int32_t* free_count, int32_t* free_count_out,
                                int64_t max_tokens, int64_t* slots, int32_t* positions, int32_t* offsets,
                                int32_t* served, void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  if (batch < 0 || max_pages < 0 || page_size < 1 || num_pages < 0 || max_tokens < 0) return FP8Q_ERR_INVALID_ARGUMENT;
  if (page_size > kMaxTableTokens || batch > kMaxTableTokens || max_tokens > kMaxTableTokens ||
      (max_pages > 0 && page_size > kMaxTableTokens / max_pages) ||
      (batch > 0 && max_pages > kMaxTableTokens / batch) || (num_pages > 0 && page_size > kMaxTableTokens / num_pages))
    return FP8Q_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !offsets || !aligned(free_count, 4) || !aligned(free_count_out, 4) ||
      !aligned(offsets, 4) || (num_pages > 0 && (!free_pages || !aligned(free_pages, 4))))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!lens || !added || !lens_out || !served || !aligned(lens, 4) || !aligned(added, 4) ||
                    !aligned(lens_out, 4) || !aligned(served, 4) ||
                    (max_pages > 0 && (!block_table || !aligned(block_table, 4)))))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (max_tokens > 0 && (!slots || !positions || !aligned(slots, 8) || !aligned(positions, 4)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const size_t need = fp8q::pages_workspace_bytes(batch, max_tokens);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return FP8Q_ERR_WORKSPACE;
  fp8q::PagesUpdate u;
  u.table = block_table;
  u.batch = batch;
  u.max_pages = max_pages;
  u.page_size = page_size;
  u.lens = lens;
  u.added = added;
  u.lens_out = lens_out;
  u.free_pages = free_pages;
  u.num_pages = num_pages;
  u.free_count = free_count;
  u.free_count_out = free_count_out;
  u.max_tokens = max_tokens;
  u.slots = slots;
  u.positions = positions;
  u.offsets = offsets;
  u.served = served;
  u.ws = ws;
  return from_cuda(fp8q::launch_pages_update(u, (cudaStream_t)stream));
}

fp8q_status fp8q_rope_turns(int64_t rot_dim, double base, fp8q_rope_kind kind, double factor, double original_len,
                            double low, double high, uint64_t* turns, float* gain) {
  if (rot_dim < 0 || rot_dim > 256 || rot_dim % 8 != 0 || !(base > 0.0) || !std::isfinite(base) ||
      kind < FP8Q_ROPE_PLAIN || kind > FP8Q_ROPE_RAMP || !gain || (rot_dim > 0 && !turns))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (kind != FP8Q_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return FP8Q_ERR_INVALID_ARGUMENT;
  if (kind >= FP8Q_ROPE_SMOOTH &&
      (!(original_len > 0.0) || !std::isfinite(original_len) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (kind == FP8Q_ROPE_RAMP && !(base > 1.0)) return FP8Q_ERR_INVALID_ARGUMENT;
  const double two_pi = 6.283185307179586476925;
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot_dim);    // radians per position
    const double periods = original_len * f / two_pi;                 // turns over the original length
    if (kind == FP8Q_ROPE_LINEAR) {
      f /= factor;
    } else if (kind == FP8Q_ROPE_SMOOTH) {
      const double keep = std::fmin(1.0, std::fmax(0.0, (periods - low) / (high - low)));
      f = (1.0 - keep) * f / factor + keep * f;
    } else if (kind == FP8Q_ROPE_RAMP) {
      // pair numbers whose turns over the original length are `high` and `low`, to whole pairs
      const double half = 0.5 * (double)rot_dim / std::log(base);
      const double from = std::fmax(0.0, std::floor(half * std::log(original_len / (high * two_pi))));
      double to = std::fmin((double)(rot_dim - 1), std::ceil(half * std::log(original_len / (low * two_pi))));
      if (to <= from) to = from + 0.001;
      const double stretch = std::fmin(1.0, std::fmax(0.0, ((double)i - from) / (to - from)));
      f = (1.0 - stretch) * f + stretch * f / factor;
    }
    if (!std::isfinite(f)) return FP8Q_ERR_INVALID_ARGUMENT;         // (base below 1e-300 or so)
    const double turn = f / two_pi;
    // the fraction of a turn in units of 2^-64 (positions are whole numbers: whole turns vanish)
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(turn - std::floor(turn), 64));
  }
  *gain = kind == FP8Q_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return FP8Q_OK;
}

fp8q_status fp8_kv_append(const fp8q_kv_pages* cache, const void* q, int64_t q_stride, int64_t q_heads, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens, const int64_t* slots,
                          const int32_t* positions, const uint64_t* turns, int64_t rot_dim, int interleaved, float gain,
                          const void* q_weight, const void* k_weight, float eps, void* q_out, int64_t q_out_stride,
                          fp8q_stream_t stream) {
  fp8q::KvPages c;
  const fp8q_status st = paged_cache(cache, &c);
  if (st != FP8Q_OK) return st;
  if (tokens < 0 || q_heads < 0 || rot_dim < 0 || rot_dim % 8 != 0 || rot_dim > cache->head_dim || !(eps >= 0.0f))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (cache->g == FP8Q_KV_PER_HEAD_TOK128) return FP8Q_ERR_UNSUPPORTED;   // a block's amax needs all its tokens
  if (tokens > kMaxTableTokens || q_heads > 65536) return FP8Q_ERR_UNSUPPORTED;
  if (tokens == 0) return FP8Q_OK;
  const int64_t kv_row = cache->heads * cache->head_dim, q_row = q_heads * cache->head_dim;
  if (!k || !v || !slots || !aligned(k, 8) || !aligned(v, 8) || !aligned(slots, 8) || k_stride % 4 != 0 ||
      v_stride % 4 != 0 || (tokens > 1 && (k_stride < kv_row || v_stride < kv_row)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (q_heads > 0 && (!q || !q_out || !aligned(q, 8) || !aligned(q_out, 8) || q_stride % 4 != 0 ||
                      q_out_stride % 4 != 0 || (tokens > 1 && (q_stride < q_row || q_out_stride < q_row))))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (rot_dim > 0 && (!positions || !turns || !aligned(positions, 4) || !aligned(turns, 8)))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if ((q_weight && !aligned(q_weight, 8)) || (k_weight && !aligned(k_weight, 8))) return FP8Q_ERR_INVALID_ARGUMENT;
  fp8q::KvAppend a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_heads = (int)q_heads;
  a.tokens = tokens;
  a.slots = slots;
  a.positions = positions;
  a.turns = reinterpret_cast<const unsigned long long*>(turns);
  a.rot = (int)rot_dim;
  a.interleaved = interleaved != 0;
  a.gain = gain;
  a.q_weight = static_cast<const uint16_t*>(q_weight);
  a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.eps = eps;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_out_stride = q_out_stride;
  return from_cuda(fp8q::launch_kv_append(c, cache->f, a, (cudaStream_t)stream));
}

size_t fp8q_attention_workspace_bytes(int64_t batch, int64_t max_tokens, int64_t q_heads, int64_t kv_heads,
                                      int64_t head_dim) {
  if (batch <= 0 || max_tokens <= 0 || q_heads < 1 || kv_heads < 1 || kv_heads > 65536 || q_heads > 65536 ||
      q_heads % kv_heads != 0 || head_dim < 1 || head_dim > 256 || batch > kMaxTableTokens ||
      max_tokens > kMaxTableTokens)
    return 0;
  return fp8q::attention_workspace_bytes(batch, max_tokens, (int)kv_heads, (int)(q_heads / kv_heads), (int)head_dim);
}

int fp8q_check_attention_split(const int32_t* lens, int64_t batch, int64_t window, int64_t sinks, int workers) {
  if (window > kMaxTableTokens || sinks > kMaxTableTokens || (batch > 0 && !lens)) return -1;
  for (int64_t b = 0; b < batch; ++b)
    if (lens[b] < 0 || lens[b] > kMaxTableTokens) return -1;
  return fp8q::check_attention_split(lens, batch, (int)window, (int)sinks, workers);
}

fp8q_status fp8_attention_paged(const fp8q_kv_pages* cache, const void* q, int64_t q_stride, int64_t q_heads,
                                const int32_t* block_table, int64_t batch, int64_t max_pages, const int32_t* lens,
                                float scale, int64_t window, int64_t sinks, void* out, int64_t out_stride, float* lse,
                                void* ws, size_t ws_bytes, fp8q_stream_t stream) {
  fp8q::KvPages c;
  const fp8q_status st = paged_cache(cache, &c);
  if (st != FP8Q_OK) return st;
  if (batch < 0 || max_pages < 0 || q_heads < 1 || q_heads % cache->heads != 0 || window < 0 || sinks < 0 ||
      !(scale > 0.0f) || !std::isfinite(scale))
    return FP8Q_ERR_INVALID_ARGUMENT;
  if (q_heads > 65536 || batch > kMaxTableTokens || (max_pages > 0 && cache->page_size > kMaxTableTokens / max_pages))
    return FP8Q_ERR_UNSUPPORTED;
  // all requests' tiles of 16 tokens, and up to 48 more for each request, are counted in an int
  if (batch * ((max_pages * cache->page_size + 15) / 16 + 48) > kMaxTableTokens) return FP8Q_ERR_UNSUPPORTED;
  if (batch == 0) return FP8Q_OK;
  const int64_t row = q_heads * cache->head_dim;
  if (!q || !out || !lens || !aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || q_stride % 8 != 0 ||
      out_stride % 8 != 0 || (batch > 1 && (q_stride < row || out_stride < row)) || (lse && !aligned(lse, 4)) ||
      (max_pages > 0 && (!block_table || !aligned(block_table, 4))))
    return FP8Q_ERR_INVALID_ARGUMENT;
  const size_t need = fp8q_attention_workspace_bytes(batch, max_pages * cache->page_size, q_heads, cache->heads,
                                                     cache->head_dim);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return FP8Q_ERR_WORKSPACE;
  const int64_t limit = kMaxTableTokens;
  return from_cuda(fp8q::launch_attention_paged(
      c, cache->f, static_cast<const uint16_t*>(q), q_stride, (int)(q_heads / cache->heads), block_table, batch,
      max_pages, lens, scale, (int)(window < limit ? window : limit), (int)(sinks < limit ? sinks : limit),
      static_cast<uint16_t*>(out), out_stride, lse, ws, (cudaStream_t)stream));
}

}  // extern "C"
