// api.cu -- the C ABI declared in include/molora.h: host-side argument validation, then
// kernel selection and launch.  Nothing here allocates, frees or synchronises.
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace molora {

int num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool valid_dtype(molora_dtype d) { return d == MOLORA_F32 || d == MOLORA_BF16; }
static molora_status launched(cudaError_t e) { return e == cudaSuccess ? MOLORA_OK : MOLORA_ERR_CUDA; }

// Smallest slot count (N*k) at which the grouped tensor-core apply beats the scalar apply,
// measured on GB300 with the decode sweep (d = 4096, top-1, batch 1..2048, K = 4..64 hot-set
// adapters drawn uniformly and Zipf(1.1); vocabulary routing -> scalar apply against routing with
// dispatch -> grouped apply; calls back to back in one CUDA graph, the decode steady state with
// the hot set in L2).  The scalar path re-reads its token's A_a and B_a (d_in r + r d_out
// elements) from L2 for every token, so the crossover falls as the rank grows:
//   r <= 16: 768 tokens up to 8 adapters, 1024 with 16, 2048 with 32; scalar at every batch
//            measured with 64;
//   r = 32:  768 up to 16 adapters, 1536 with 32 (768 under uniform draws, 1536 under Zipf),
//            2048 with 64;
//   r = 64:  160 up to 8 adapters (Figures 5 and 9 put it near batch 160 for 8 adapters of rank
//            64), 512 with 16, 768 with 32, 1024 with 64.
static int64_t crossover_tokens(int32_t K, int32_t r) {
  if (r >= 64) {
    if (K <= 8) return 160;
    if (K <= 16) return 512;
    if (K <= 32) return 768;
    return 1024;
  }
  if (r >= 32) {
    if (K <= 16) return 768;
    if (K <= 32) return 1536;
    return 2048;
  }
  if (K <= 8) return 768;
  if (K <= 16) return 1024;
  if (K <= 32) return 2048;
  return 4096;
}

static molora_status check_apply_sizes(molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out, int32_t K,
                                       int32_t r, int32_t k) {
  if (!valid_dtype(dtype) || N < 0 || d_in < 1 || d_out < 1 || K < 1 || K > kMaxAdapters || k < 1 || k > K)
    return MOLORA_ERR_INVALID_ARG;
  if (!(r == 8 || r == 16 || r == 32 || r == 64)) return MOLORA_ERR_INVALID_ARG;
  if (N > INT32_MAX || N * (int64_t)k > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  return MOLORA_OK;
}

static molora_status check_apply_args(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                      const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids,
                                      int32_t k, const void* y) {
  const molora_status st = check_apply_sizes(dtype, N, d_in, d_out, K, r, k);
  if (st != MOLORA_OK || N == 0) return st;
  if (!x || !A || !B || !ids || !y) return MOLORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(y)) return MOLORA_ERR_INVALID_ARG;
  return MOLORA_OK;
}

// The best path that needs no workspace (AUTO without one, or with the adapter table of the
// indirect layout, which only the scalar and grouped kernels read).
static molora_path select_without_ws(molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out, int32_t K,
                                     int32_t r, int32_t k, bool table) {
  if (!table && k >= 2 && dense_preferred(dtype, N, d_in, d_out, K, r)) return MOLORA_PATH_DENSE;
  if (!grouped_supported(dtype, N, d_in, d_out, K, r, k)) return MOLORA_PATH_SCALAR;
  return N * (int64_t)k >= crossover_tokens(K, r) ? MOLORA_PATH_GROUPED : MOLORA_PATH_SCALAR;
}

// Workspace convention (include/molora.h): ws_bytes == NULL -> none; ws == NULL -> query;
// else a buffer of *ws_bytes bytes.  `need` is what the chosen path needs.
static molora_status check_ws(void* ws, size_t* ws_bytes, size_t need, bool* query) {
  *query = ws_bytes != nullptr && ws == nullptr;
  if (*query) {
    *ws_bytes = need;
    return MOLORA_OK;
  }
  if (need == 0) return MOLORA_OK;
  if (!ws || !ws_bytes || *ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOLORA_ERR_INVALID_ARG;
  return MOLORA_OK;
}

static molora_status apply_impl(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids, const float* w,
                                int32_t k, const int32_t* counts, const int32_t* offsets, const int32_t* perm,
                                float scale, void* y, bool y_bf16, int32_t* err_word, molora_path path,
                                cudaStream_t stream, const AdapterTable* table = nullptr, void* ws = nullptr,
                                size_t* ws_bytes = nullptr) {
  const bool have_ws = ws_bytes != nullptr;
  const bool query = have_ws && ws == nullptr;  // sizes only: no pointer is looked at
  const molora_status st = query ? check_apply_sizes(dtype, N, d_in, d_out, K, r, k)
                                 : check_apply_args(x, dtype, N, d_in, d_out, A, B, K, r, ids, k, y);
  if (st != MOLORA_OK) return st;
  if (path == MOLORA_PATH_AUTO) {
    if (table) {
      // the adapter table is read by the scalar and grouped kernels only: choose between them
      path = select_without_ws(dtype, N, d_in, d_out, K, r, k, true);
    } else {
      path = molora_select_path(dtype, N, d_in, d_out, K, r, k);
      if (path == MOLORA_PATH_STACKED && (!have_ws || y_bf16 || !stacked_supported(dtype, N, d_in, d_out, K, r, false)))
        path = select_without_ws(dtype, N, d_in, d_out, K, r, k, false);
    }
    // AUTO takes the grouped path only with the dispatch outputs it reads; without them, the
    // fastest path that needs none (the stacked pair if its workspace was given)
    if (path == MOLORA_PATH_GROUPED && !query && (!counts || !offsets || !perm)) {
      const bool ws_fits = have_ws && ws != nullptr && *ws_bytes >= stacked_workspace_bytes(N, K, r);
      if (!table && !y_bf16 && ws_fits && stacked_supported(dtype, N, d_in, d_out, K, r, false))
        path = MOLORA_PATH_STACKED;
      else if (!table && k >= 2 && dense_supported(dtype, N, d_in, d_out, K, r))
        path = MOLORA_PATH_DENSE;
      else
        path = MOLORA_PATH_SCALAR;
    }
  }
  if (path == MOLORA_PATH_STACKED) {
    if (!have_ws) return N == 0 ? MOLORA_OK : MOLORA_ERR_INVALID_ARG;
    if (table || y_bf16 || !stacked_supported(dtype, N, d_in, d_out, K, r, false)) return MOLORA_ERR_UNSUPPORTED;
    bool is_query = false;
    const molora_status ws_st = check_ws(ws, ws_bytes, stacked_workspace_bytes(N, K, r), &is_query);
    if (ws_st != MOLORA_OK || is_query || N == 0) return ws_st;
    return launched(launch_lora_stacked(x, N, d_in, d_out, A, B, K, r, ids, w, k, scale, static_cast<float*>(y), ws,
                                        err_word, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                        stream));
  }
  if (path < MOLORA_PATH_AUTO || path > MOLORA_PATH_STACKED) return MOLORA_ERR_INVALID_ARG;
  if (query) {  // the other paths need no workspace
    *ws_bytes = 0;
    return MOLORA_OK;
  }
  if (N == 0) return MOLORA_OK;
  if (path == MOLORA_PATH_SCALAR)
    return launched(launch_lora_scalar(x, dtype, N, d_in, d_out, A, B, K, r, ids, w, k, scale, y, y_bf16, -1,
                                       err_word, stream, table));
  if (path == MOLORA_PATH_DENSE) {
    if (table || !dense_supported(dtype, N, d_in, d_out, K, r)) return MOLORA_ERR_UNSUPPORTED;
    return launched(launch_lora_dense(x, N, d_in, d_out, A, B, K, r, ids, w, k, scale, y, y_bf16, err_word, stream));
  }
  if (path != MOLORA_PATH_GROUPED) return MOLORA_ERR_INVALID_ARG;
  if (!grouped_supported(dtype, N, d_in, d_out, K, r, k)) return MOLORA_ERR_UNSUPPORTED;
  if (!counts || !offsets || !perm) return MOLORA_ERR_INVALID_ARG;
  return launched(launch_lora_grouped(x, N, d_in, d_out, A, B, K, r, ids, w, k, counts, offsets, perm, scale, y,
                                      y_bf16, -1, err_word, stream, table));
}

static size_t size_of(molora_dtype d) { return d == MOLORA_F32 ? 4 : d == MOLORA_BF16 ? 2 : 1; }
// Whether a pointer (NULL included) starts on a boundary of its element's size: kernels read whole elements.
static bool on_element(const void* p, size_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }
// The most rows, and columns, of the norm's and the product's arrays: kernels count to a tile past the end
// in 32 bits.
static constexpr int32_t kMostSize = INT32_MAX - 1023;

// Rows x columns of `size` bytes at p.  An absent or empty array shares nothing with another.
struct Span {
  const void* p;
  unsigned __int128 first, last;
  Span(const void* at, int64_t rows, int64_t cols, size_t size)
      : p(at), first(reinterpret_cast<uintptr_t>(at)), last(at && rows && cols ? first + (unsigned __int128)rows * cols * size : 0) {}
  bool shares(const Span& o) const { return first < o.last && o.first < last; }
  // as an output that may be the other array itself
  bool shares_part(const Span& o) const { return p != o.p && shares(o); }
};

// molora_linear's checks.  With N == 0 no pointer is looked at.
static molora_status check_linear(const LinearArgs& a) {
  if (!(valid_dtype(a.dtype) || a.dtype == MOLORA_E4M3) || a.N < 0 || a.N > kMostSize || a.d_in < 1 ||
      a.d_in > kMostSize || a.d_out < 1 || a.d_out > kMostSize || a.act < MOLORA_ACT_NONE || a.act > MOLORA_ACT_GELU_TANH)
    return MOLORA_ERR_INVALID_ARG;
  if (a.N == 0) return MOLORA_OK;
  if (!a.x || !a.W || !a.y) return MOLORA_ERR_INVALID_ARG;
  if ((a.dtype == MOLORA_E4M3) != (a.x_scale != nullptr) || (a.dtype == MOLORA_E4M3) != (a.w_scale != nullptr))
    return MOLORA_ERR_INVALID_ARG;
  const size_t e = size_of(a.dtype), ye = a.y_bf16 ? 2 : 4;
  if (!on_element(a.x, e) || !on_element(a.W, e) || !on_element(a.y, ye) || !on_element(a.residual, ye) ||
      !on_element(a.bias, 4) || !on_element(a.x_scale, 4) || !on_element(a.w_scale, 4))
    return MOLORA_ERR_INVALID_ARG;
  const Span y = {a.y, a.N, a.d_out, ye};
  if (y.shares({a.x, a.N, a.d_in, e}) || y.shares({a.W, a.d_out, a.d_in, e}) || y.shares({a.x_scale, a.N, 1, 4}) ||
      y.shares({a.w_scale, a.d_out, 1, 4}) || y.shares({a.bias, a.d_out, 1, 4}) ||
      y.shares_part({a.residual, a.N, a.d_out, ye}))
    return MOLORA_ERR_INVALID_ARG;
  return MOLORA_OK;
}

static molora_status linear_impl(const LinearArgs& a, cudaStream_t stream) {
  const molora_status st = check_linear(a);
  if (st != MOLORA_OK || a.N == 0) return st;
  return launched(launch_linear(a, stream));
}

static molora_status check_rmsnorm(const void* x, molora_dtype dtype, int64_t N, int32_t d, const void* residual,
                                   const void* sum_out, const void* weight, float eps, const void* out,
                                   const void* out8, const float* scale8) {
  if (!valid_dtype(dtype) || N < 0 || N > kMostSize || d < 1 || d > kMostSize || !(eps > 0.f) || !(eps <= 3.4e38f))
    return MOLORA_ERR_INVALID_ARG;
  if (N == 0) return MOLORA_OK;
  if (!x || !weight || (!out && !out8) || (out8 != nullptr) != (scale8 != nullptr) || (sum_out && !residual))
    return MOLORA_ERR_INVALID_ARG;
  const size_t e = size_of(dtype);
  if (!on_element(x, e) || !on_element(residual, e) || !on_element(sum_out, e) || !on_element(weight, e) ||
      !on_element(out, e) || !on_element(scale8, 4))
    return MOLORA_ERR_INVALID_ARG;
  const Span xs = {x, N, d, e}, rs = {residual, N, d, e}, ws = {weight, 1, d, e}, ss = {sum_out, N, d, e}, os = {out, N, d, e},
             os8 = {out8, N, d, 1}, sc = {scale8, N, 1, 4};
  for (const Span& o : {ss, os})
    if (o.shares_part(xs) || o.shares_part(rs) || o.shares(ws) || o.shares(os8) || o.shares(sc)) return MOLORA_ERR_INVALID_ARG;
  for (const Span& o : {os8, sc})
    if (o.shares(xs) || o.shares(rs) || o.shares(ws)) return MOLORA_ERR_INVALID_ARG;
  return ss.shares(os) || os8.shares(sc) ? MOLORA_ERR_INVALID_ARG : MOLORA_OK;
}

}  // namespace molora

using namespace molora;

extern "C" {

molora_status molora_route_vocab_ex(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K,
                                    int32_t* adapter, int32_t* err_word, uint32_t flags, cudaStream_t stream) {
  if (flags & ~(uint32_t)MOLORA_INPUTS_READY) return MOLORA_ERR_INVALID_ARG;
  if (N < 0 || K < 1 || K > kMaxAdapters) return MOLORA_ERR_INVALID_ARG;
  if (N == 0) return MOLORA_OK;
  if (!tok || !starts || !adapter) return MOLORA_ERR_INVALID_ARG;
  const int early = (flags & MOLORA_INPUTS_READY) ? 1 : 0;
  return launched(launch_route_vocab(tok, N, starts, K, adapter, err_word, early, stream));
}

molora_status molora_route_vocab(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K, int32_t* adapter,
                                 int32_t* err_word, cudaStream_t stream) {
  return molora_route_vocab_ex(tok, N, starts, K, adapter, err_word, 0u, stream);
}

molora_status molora_router_topk(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, const void* W1,
                                 const float* b1, const void* W2, const float* b2, int32_t K, int32_t k,
                                 float* logits, int32_t* ids, float* w, cudaStream_t stream) {
  if (!valid_dtype(dtype) || N < 0 || d_in < 1 || K < 1 || K > kMaxAdapters || k < 1 || k > K)
    return MOLORA_ERR_INVALID_ARG;
  if (N > INT32_MAX || N * (int64_t)K > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  if (N == 0) return MOLORA_OK;
  if (!x || !W1 || !W2 || !ids || !w) return MOLORA_ERR_INVALID_ARG;
  if (router_tc_supported(dtype, N, d_in, K, k)) {
    if (!aligned16(x) || !aligned16(W1)) return MOLORA_ERR_INVALID_ARG;
    return launched(launch_router_tc(x, N, d_in, W1, b1, W2, b2, K, k, logits, ids, w, stream));
  }
  return launched(launch_router_scalar(x, dtype, N, d_in, W1, b1, W2, b2, K, k, logits, ids, w, stream));
}

molora_status molora_dispatch(const int32_t* ids, int64_t N, int32_t k, int32_t K, int32_t* counts, int32_t* offsets,
                              int32_t* perm, int32_t* err_word, cudaStream_t stream) {
  if (N < 0 || k < 1 || K < 1 || K > kMaxAdapters || k > K) return MOLORA_ERR_INVALID_ARG;
  if (N * (int64_t)k > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  if (!counts || !offsets || (N > 0 && (!ids || !perm))) return MOLORA_ERR_INVALID_ARG;
  return launched(launch_dispatch(ids, N, k, K, counts, offsets, perm, err_word, stream));
}

molora_status molora_route_vocab_dispatch(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K,
                                          int32_t* adapter, int32_t* counts, int32_t* offsets, int32_t* perm,
                                          int32_t* err_word, cudaStream_t stream) {
  if (N < 0 || K < 1 || K > kMaxAdapters || N > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  if (!starts || !counts || !offsets || (N > 0 && (!tok || !adapter || !perm))) return MOLORA_ERR_INVALID_ARG;
  return launched(launch_route_vocab_dispatch(tok, N, starts, K, adapter, counts, offsets, perm, err_word, 0, stream));
}

molora_status molora_route_vocab_dispatch_ex(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K,
                                             int32_t* adapter, int32_t* counts, int32_t* offsets, int32_t* perm,
                                             int32_t* err_word, uint32_t flags, cudaStream_t stream) {
  if (flags & ~(uint32_t)MOLORA_INPUTS_READY) return MOLORA_ERR_INVALID_ARG;
  if (N < 0 || K < 1 || K > kMaxAdapters || N > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  if (!starts || !counts || !offsets || (N > 0 && (!tok || !adapter || !perm))) return MOLORA_ERR_INVALID_ARG;
  const int early = (flags & MOLORA_INPUTS_READY) ? 1 : 0;
  return launched(launch_route_vocab_dispatch(tok, N, starts, K, adapter, counts, offsets, perm, err_word, early, stream));
}

molora_status molora_route_vocab_lora_apply_ex(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K,
                                               const void* x, molora_dtype dtype, int32_t d_in, int32_t d_out,
                                               const void* A, const void* B, int32_t r, float scale, void* y,
                                               int32_t y_bf16, int32_t* adapter, int32_t* counts, int32_t* offsets,
                                               int32_t* perm, int32_t* err_word, uint32_t flags, cudaStream_t stream) {
  if (flags & ~(uint32_t)MOLORA_INPUTS_READY) return MOLORA_ERR_INVALID_ARG;
  const molora_status st = check_apply_args(x, dtype, N, d_in, d_out, A, B, K, r, tok, 1, y);
  if (st != MOLORA_OK) return st;
  if (!starts || !counts || !offsets || (N > 0 && (!adapter || !perm))) return MOLORA_ERR_INVALID_ARG;
  const int early = (flags & MOLORA_INPUTS_READY) ? 1 : 0;
  if (N == 0)  // the empty histogram, as molora_route_vocab_dispatch writes it
    return launched(launch_route_vocab_dispatch(tok, 0, starts, K, adapter, counts, offsets, perm, err_word, early,
                                                stream));
  const molora_path path = select_without_ws(dtype, N, d_in, d_out, K, r, 1, false);
  if (launch_route_vocab_dispatch(tok, N, starts, K, adapter, counts, offsets, perm, err_word, early, stream) !=
      cudaSuccess)
    return MOLORA_ERR_CUDA;
  return apply_impl(x, dtype, N, d_in, d_out, A, B, K, r, adapter, nullptr, 1, counts, offsets, perm, scale, y,
                    y_bf16 != 0, err_word, path, stream);
}

molora_status molora_route_vocab_lora_apply(const int32_t* tok, int64_t N, const int32_t* starts, int32_t K,
                                            const void* x, molora_dtype dtype, int32_t d_in, int32_t d_out,
                                            const void* A, const void* B, int32_t r, float scale, void* y,
                                            int32_t y_bf16, int32_t* adapter, int32_t* counts, int32_t* offsets,
                                            int32_t* perm, int32_t* err_word, cudaStream_t stream) {
  return molora_route_vocab_lora_apply_ex(tok, N, starts, K, x, dtype, d_in, d_out, A, B, r, scale, y, y_bf16,
                                          adapter, counts, offsets, perm, err_word, 0u, stream);
}

molora_path molora_select_path(molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out, int32_t K, int32_t r,
                               int32_t k) {
  if (stacked_preferred(dtype, N, d_in, d_out, K, r, k, false)) return MOLORA_PATH_STACKED;
  return select_without_ws(dtype, N, d_in, d_out, K, r, k, false);
}

molora_status molora_lora_apply_ex(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                   const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids,
                                   const float* w, int32_t k, const int32_t* counts, const int32_t* offsets,
                                   const int32_t* perm, float scale, float* y, void* ws, size_t* ws_bytes,
                                   int32_t* err_word, molora_path path, cudaStream_t stream) {
  return molora::apply_impl(x, dtype, N, d_in, d_out, A, B, K, r, ids, w, k, counts, offsets, perm, scale, y, false,
                            err_word, path, stream, nullptr, ws, ws_bytes);
}

molora_status molora_lora_apply_bf16y(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                      const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids,
                                      const float* w, int32_t k, const int32_t* counts, const int32_t* offsets,
                                      const int32_t* perm, float scale, void* y, int32_t* err_word,
                                      molora_path path, cudaStream_t stream) {
  return molora::apply_impl(x, dtype, N, d_in, d_out, A, B, K, r, ids, w, k, counts, offsets, perm, scale, y, true,
                            err_word, path, stream);
}

molora_status molora_lora_apply_indirect(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                         const void* const* A_ptrs, const void* const* B_ptrs, int32_t K, int32_t r,
                                         const int32_t* ids, const float* w, int32_t k, const int32_t* counts,
                                         const int32_t* offsets, const int32_t* perm, float scale, void* y,
                                         int32_t y_bf16, int32_t* err_word, molora_path path, cudaStream_t stream) {
  if (!A_ptrs || !B_ptrs || K < 1 || K > kMaxAdapters) return MOLORA_ERR_INVALID_ARG;
  molora::AdapterTable table;
  for (int i = 0; i < kMaxAdapters; ++i) table.a[i] = table.b[i] = nullptr;
  for (int32_t i = 0; i < K; ++i) {
    if (!A_ptrs[i] || !B_ptrs[i] || !aligned16(A_ptrs[i]) || !aligned16(B_ptrs[i])) return MOLORA_ERR_INVALID_ARG;
    table.a[i] = A_ptrs[i];
    table.b[i] = B_ptrs[i];
  }
  return molora::apply_impl(x, dtype, N, d_in, d_out, A_ptrs[0], B_ptrs[0], K, r, ids, w, k, counts, offsets, perm,
                            scale, y, y_bf16 != 0, err_word, path, stream, &table);
}

molora_status molora_router_lora_apply(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                       const void* W1, const float* b1, const void* W2, const float* b2,
                                       const void* A, const void* B, int32_t K, int32_t r, int32_t k, float scale,
                                       float* logits, int32_t* ids, float* w, void* y, int32_t y_bf16, void* ws,
                                       size_t* ws_bytes, int32_t* err_word, cudaStream_t stream) {
  const bool query = ws_bytes != nullptr && ws == nullptr;  // sizes only: no pointer is looked at
  const molora_status st = query ? check_apply_sizes(dtype, N, d_in, d_out, K, r, k)
                                 : check_apply_args(x, dtype, N, d_in, d_out, A, B, K, r, ids, k, y);
  if (st != MOLORA_OK) return st;
  if (N * (int64_t)K > INT32_MAX) return MOLORA_ERR_INVALID_ARG;
  if (!query && N > 0 && (!W1 || !W2 || !w || !aligned16(W1))) return MOLORA_ERR_INVALID_ARG;
  // A query sizes the preferred family: the stacked pair where it applies and either wins or is
  // the only one.  A call given a buffer runs the stacked pair wherever it applies.
  const bool one_kernel = router_dense_supported(dtype, N, d_in, d_out, K, r);
  const bool stacked_ok = y_bf16 == 0 && stacked_supported(dtype, N, d_in, d_out, K, r, true);
  const bool stacked = stacked_ok && ws_bytes != nullptr &&
                       (query ? !one_kernel || stacked_preferred(dtype, N, d_in, d_out, K, r, k, true) : true);
  if (stacked) {
    bool is_query = false;
    const molora_status ws_st = check_ws(ws, ws_bytes, stacked_workspace_bytes(N, K, r), &is_query);
    if (ws_st != MOLORA_OK || is_query || N == 0) return ws_st;
    return launched(launch_lora_stacked(x, N, d_in, d_out, A, B, K, r, nullptr, nullptr, k, scale,
                                        static_cast<float*>(y), ws, err_word, W1, b1, W2, b2, logits, ids, w, stream));
  }
  if (query) {  // the one-kernel path needs no workspace
    *ws_bytes = 0;
    return one_kernel || N == 0 ? MOLORA_OK : MOLORA_ERR_UNSUPPORTED;
  }
  if (N == 0) return MOLORA_OK;
  if (!one_kernel) return MOLORA_ERR_UNSUPPORTED;
  return launched(launch_router_lora_dense(x, N, d_in, d_out, W1, b1, W2, b2, A, B, K, r, k, scale, logits, ids, w, y,
                                           y_bf16 != 0, err_word, stream));
}

molora_status molora_lora_apply(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids, const float* w,
                                int32_t k, const int32_t* counts, const int32_t* offsets, const int32_t* perm,
                                float scale, float* y, void* ws, size_t* ws_bytes, int32_t* err_word,
                                cudaStream_t stream) {
  return molora_lora_apply_ex(x, dtype, N, d_in, d_out, A, B, K, r, ids, w, k, counts, offsets, perm, scale, y, ws,
                              ws_bytes, err_word, MOLORA_PATH_AUTO, stream);
}

molora_status molora_lora_apply_masked_pass(const void* x, molora_dtype dtype, int64_t N, int32_t d_in,
                                            int32_t d_out, const void* A, const void* B, int32_t K, int32_t r,
                                            const int32_t* adapter_of, int32_t a, float scale, float* y,
                                            int32_t* err_word, molora_path path, cudaStream_t stream) {
  const molora_status st = check_apply_args(x, dtype, N, d_in, d_out, A, B, K, r, adapter_of, 1, y);
  if (st != MOLORA_OK) return st;
  if (a < 0 || a >= K) return MOLORA_ERR_INVALID_ARG;
  if (N == 0) return MOLORA_OK;
  // a masked pass takes no workspace: AUTO chooses between the scalar and grouped kernels
  if (path == MOLORA_PATH_AUTO) path = select_without_ws(dtype, N, d_in, d_out, K, r, 1, false);
  if (path == MOLORA_PATH_SCALAR)
    return launched(launch_lora_scalar(x, dtype, N, d_in, d_out, A, B, K, r, adapter_of, nullptr, 1, scale, y, false,
                                       a, err_word, stream));
  if (path != MOLORA_PATH_GROUPED) return MOLORA_ERR_INVALID_ARG;
  if (!grouped_supported(dtype, N, d_in, d_out, K, r, 1)) return MOLORA_ERR_UNSUPPORTED;
  return launched(launch_lora_grouped(x, N, d_in, d_out, A, B, K, r, adapter_of, nullptr, 1, nullptr, nullptr,
                                      nullptr, scale, y, false, a, err_word, stream));
}

molora_status molora_lora_apply_static_ws(const void* x, molora_dtype dtype, int64_t N, int32_t d_in, int32_t d_out,
                                          const void* A, const void* B, int32_t K, int32_t r, const int32_t* ids,
                                          const float* w, int32_t k, float scale, float* y, int32_t* err_word,
                                          cudaStream_t stream) {
  const molora_status st = check_apply_args(x, dtype, N, d_in, d_out, A, B, K, r, ids, k, y);
  if (st != MOLORA_OK || N == 0) return st;
  if (!stacked_supported(dtype, N, d_in, d_out, K, r, false)) return MOLORA_ERR_UNSUPPORTED;
  const size_t need = stacked_workspace_bytes(N, K, r);
  if (need > stacked_static_scratch_bytes() || stacked_static_scratch_bytes() != MOLORA_STATIC_SCRATCH_BYTES)
    return MOLORA_ERR_SCRATCH_TOO_SMALL;
  void* scratch = nullptr;
  if (stacked_static_scratch(&scratch) != cudaSuccess) return MOLORA_ERR_CUDA;
  return launched(launch_lora_stacked(x, N, d_in, d_out, A, B, K, r, ids, w, k, scale, y, scratch, err_word, nullptr,
                                      nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, stream));
}

molora_status molora_rmsnorm(const void* x, molora_dtype dtype, int64_t N, int32_t d, const void* residual, void* sum_out,
                             const void* weight, float eps, void* out, void* out8, float* scale8,
                             cudaStream_t stream) {
  const molora_status st = check_rmsnorm(x, dtype, N, d, residual, sum_out, weight, eps, out, out8, scale8);
  if (st != MOLORA_OK || N == 0) return st;
  return launched(launch_rmsnorm(x, dtype, N, d, residual, sum_out, weight, eps, out, out8, scale8, stream));
}

molora_status molora_gate_topk(const void* logits, molora_dtype dtype, int64_t N, int32_t K, molora_score score,
                               const float* bias, int32_t groups, int32_t keep_groups, int32_t group_top, int32_t k,
                               int32_t renormalise, float scale, int32_t* ids, float* w, int32_t* err_word,
                               cudaStream_t stream) {
  if (!valid_dtype(dtype) || N < 0 || N > INT32_MAX || K < 1 || K > MOLORA_MAX_EXPERTS ||
      (score != MOLORA_SCORE_SOFTMAX && score != MOLORA_SCORE_SIGMOID) || groups < 1 || groups > MOLORA_MAX_GROUPS ||
      K % groups || keep_groups < 1 || keep_groups > groups || (group_top != 1 && group_top != 2) ||
      K / groups < group_top || k < 1 || k > MOLORA_MAX_GATE_K || k > keep_groups * (K / groups) ||
      !(scale >= -3.4e38f && scale <= 3.4e38f))
    return MOLORA_ERR_INVALID_ARG;
  if (N == 0) return MOLORA_OK;
  if (!logits || !ids || !w || !on_element(logits, size_of(dtype)) || !on_element(bias, 4) || !on_element(ids, 4) ||
      !on_element(w, 4))
    return MOLORA_ERR_INVALID_ARG;
  const Span ls = {logits, N, K, size_of(dtype)}, bs = {bias, 1, K, 4}, is = {ids, N, k, 4}, ws = {w, N, k, 4};
  if (is.shares(ls) || is.shares(bs) || is.shares(ws) || ws.shares(ls) || ws.shares(bs)) return MOLORA_ERR_INVALID_ARG;
  return launched(launch_gate_topk(logits, dtype, N, K, score == MOLORA_SCORE_SIGMOID, bias, groups, keep_groups,
                                   group_top, k, renormalise != 0, scale, ids, w, err_word, stream));
}

molora_status molora_linear(const void* x, molora_dtype dtype, const float* x_scale, int64_t N, int32_t d_in,
                            const void* W, const float* w_scale, int32_t d_out, const float* bias,
                            molora_activation act, const void* residual, void* y, int32_t y_bf16, int32_t* err_word,
                            cudaStream_t stream) {
  const LinearArgs a = {x, dtype, x_scale, N, d_in, W, w_scale, d_out, bias, act, residual, y, y_bf16 != 0, err_word};
  return linear_impl(a, stream);
}

molora_status molora_norm_linear_lora_apply(const void* x, molora_dtype dtype, int64_t N, int32_t d_in,
                                            const void* residual, void* sum_out, const void* norm_weight, float eps,
                                            void* h, void* h8, float* scale8, const void* W, molora_dtype w_dtype,
                                            const float* w_scale, int32_t d_out, const float* bias, const void* A,
                                            const void* B, int32_t K, int32_t r, const int32_t* ids, const float* w,
                                            int32_t k, const int32_t* counts, const int32_t* offsets,
                                            const int32_t* perm, float scale, void* y, int32_t y_bf16, void* ws,
                                            size_t* ws_bytes, int32_t* err_word, cudaStream_t stream) {
  const bool fp8 = w_dtype == MOLORA_E4M3;
  if (!fp8 && w_dtype != dtype) return MOLORA_ERR_INVALID_ARG;
  const LinearArgs lin = {fp8 ? h8 : h, w_dtype, scale8, N, d_in, W, w_scale, d_out, bias, MOLORA_ACT_NONE, nullptr, y,
                          y_bf16 != 0, err_word};
  const bool query = ws_bytes && !ws;
  molora_status st = query ? check_apply_sizes(dtype, N, d_in, d_out, K, r, k) : MOLORA_OK;
  if (st != MOLORA_OK) return st;
  // every argument of the three steps is checked before the first of them is enqueued
  if (!query) {
    st = check_rmsnorm(x, dtype, N, d_in, residual, sum_out, norm_weight, eps, h, h8, scale8);
    if (st == MOLORA_OK) st = check_linear(lin);
    if (st == MOLORA_OK) st = check_apply_args(h, dtype, N, d_in, d_out, A, B, K, r, ids, k, y);
    if (st != MOLORA_OK || N == 0) return st;
    if (ws && (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOLORA_ERR_INVALID_ARG;
    // what a step writes shares nothing with what a later one reads, nor with another output
    const size_t e = size_of(dtype);
    const Span ys = {y, N, d_out, y_bf16 ? size_t(2) : size_t(4)}, hs = {h, N, d_in, e}, sums = {sum_out, N, d_in, e},
               h8s = {h8, N, d_in, 1}, scales = {scale8, N, 1, 4},
               wss = {ws_bytes ? ws : nullptr, 1, ws_bytes ? (int64_t)*ws_bytes : 0, 1};
    const Span read[] = {{W, d_out, d_in, size_of(w_dtype)}, {w_scale, d_out, 1, 4}, {bias, d_out, 1, 4},
                         {A, (int64_t)K * d_in, r, e}, {B, (int64_t)K * r, d_out, e}, {ids, N, k, 4}, {w, N, k, 4},
                         {counts, K, 1, 4}, {offsets, K + 1, 1, 4}, {perm, N, k, 4}};
    for (const Span& in : read)
      for (const Span* out : {&ys, &hs, &sums, &h8s, &scales, &wss})
        if (out->shares(in)) return MOLORA_ERR_INVALID_ARG;
    if (ys.shares(hs) || ys.shares(sums)) return MOLORA_ERR_INVALID_ARG;  // (h8 and scale8 are the product's inputs)
    for (const Span* out : {&ys, &hs, &sums, &h8s, &scales})
      if (wss.shares(*out)) return MOLORA_ERR_INVALID_ARG;
  }
  // With more than 256 tokens the product takes the adapters' update along (y is then written, and
  // rounded, once), if its two planes fit the workspace: K*r/32 more K blocks of 64 against a pass over y.
  const size_t plane = lora_update_bytes(N, K * r), stacked = stacked_workspace_bytes(N, K, r);
  const bool update = N > 0 && ws_bytes && K * r <= 512 && linear_takes_update(lin, B, K * r) &&
                      lora_update_supported(dtype, N, d_in, K, r);
  if (query) {
    *ws_bytes = update ? 2 * plane : 0;
    if (update || y_bf16) return MOLORA_OK;
    return apply_impl(nullptr, dtype, N, d_in, d_out, nullptr, nullptr, K, r, nullptr, nullptr, k, nullptr, nullptr,
                      nullptr, scale, nullptr, false, nullptr, MOLORA_PATH_AUTO, stream, nullptr, nullptr, ws_bytes);
  }
  if (ws_bytes && *ws_bytes < (update ? 2 * plane
                               : !y_bf16 && molora_select_path(dtype, N, d_in, d_out, K, r, k) == MOLORA_PATH_STACKED
                                   ? stacked
                                   : 0))
    return MOLORA_ERR_INVALID_ARG;
  if (launch_rmsnorm(x, dtype, N, d_in, residual, sum_out, norm_weight, eps, h, h8, scale8, stream) != cudaSuccess)
    return MOLORA_ERR_CUDA;
  if (update) {
    void* lo = static_cast<uint8_t*>(ws) + plane;
    if (launch_lora_update(h, N, d_in, A, K, r, ids, w, k, scale, ws, lo, err_word, stream) != cudaSuccess)
      return MOLORA_ERR_CUDA;
    const LinearUpdate u = {ws, lo, B, K * r};
    return launched(launch_linear(lin, stream, &u));
  }
  st = linear_impl(lin, stream);
  if (st != MOLORA_OK) return st;
  return apply_impl(h, dtype, N, d_in, d_out, A, B, K, r, ids, w, k, counts, offsets, perm, scale, y, y_bf16 != 0,
                    err_word, MOLORA_PATH_AUTO, stream, nullptr, y_bf16 ? nullptr : ws, y_bf16 ? nullptr : ws_bytes);
}

const char* molora_status_string(molora_status status) {
  switch (status) {
    case MOLORA_OK:
      return "ok";
    case MOLORA_ERR_INVALID_ARG:
      return "invalid argument";
    case MOLORA_ERR_UNSUPPORTED:
      return "unsupported shape for this path";
    case MOLORA_ERR_CUDA:
      return "CUDA launch error";
    case MOLORA_ERR_SCRATCH_TOO_SMALL:
      return "problem too large for the fixed scratch buffer (N * K * r too large)";
  }
  return "unknown status";
}

int32_t molora_version(void) { return 100; }

molora_status molora_selftest_bounded_wait(uint32_t limit_us, int32_t* err_word, cudaStream_t stream) {
  if (!err_word || limit_us == 0 || limit_us > 1000000u) return MOLORA_ERR_INVALID_ARG;
  return launched(launch_bounded_wait_selftest((uint64_t)limit_us * 1000ull, err_word, stream));
}

}  // extern "C"
