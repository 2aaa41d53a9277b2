// tk_attend.cu -- attention of new and drafted tokens over the paged cache
// (tk_kv_attend): o = sum_j softmax_j(scale q.k_j) v_j over the keys j that a
// token sees.
#include <new>

#include "tk_kv.cuh"

namespace tk {

struct AttendArgs {
  const void* q;
  int64_t q_stride;
  int hq, hk;
  const int64_t* off;
  int64_t R, T, max_new;
  const int32_t* len;
  const int32_t* table;
  int64_t table_stride, table_width;
  const int64_t* mask;
  float scale;
  void* out;
  float* lse;
  KvStatus* status;
  const void* k;
  const void* v;
  int64_t n_blocks, s_block, s_head, s_token;
  int log2_bs;
};

// One warp per token and query head; a lane holds D / 32 elements of the
// query, the key, the value and the output.  Softmax by a running maximum and
// sum in fp32.
template <class T, int D>
__global__ void __launch_bounds__(128) k_kv_attend(AttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 5;
  const int64_t t = w / a.hq;
  const int h = (int)(w - t * a.hq);
  if (t >= a.T || t >= a.off[a.R]) return;
  int64_t lo = 0, hi = a.R;  // the request: off[r] <= t < off[r + 1]
  while (hi - lo > 1) {
    const int64_t m = (lo + hi) >> 1;
    if (a.off[m] <= t) lo = m;
    else hi = m;
  }
  const int64_t r = lo, n = a.off[r + 1] - a.off[r], i = t - a.off[r], len = a.len[r], ctx = len - n;
  const bool good = n <= a.max_new && (!a.mask || n <= KV_TREE_MAX) && ctx >= 0 && i >= 0 &&
                    len <= a.table_width << a.log2_bs;
  if (!good && lane == 0 && h == 0 && i == 0 && atomicCAS(&a.status->code, 0, TK_E_LIMIT) == 0)
    a.status->request = r;
  const uint64_t mask = a.mask ? (uint64_t)a.mask[t] : 0;
  const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)h * D + lane * E;
  float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) x[e] = (float)q[e] * a.scale;
  const int64_t end = good ? (a.mask ? len : ctx + i + 1) : 0;
  for (int64_t j = 0; j < end; j++) {
    if (a.mask && j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
    const int64_t b = a.table[r * a.table_stride + (j >> a.log2_bs)];
    const bool in = b >= 0 && b < a.n_blocks;
    const int64_t at = b * a.s_block + (h / (a.hq / a.hk)) * a.s_head + (j & ((1 << a.log2_bs) - 1)) * a.s_token + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) s += x[e] * (in ? (float)static_cast<const T*>(a.k)[at + e] : 0.f);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float top = fmaxf(m, s);
    const float p = s == -INFINITY ? 0.f : expf(s - top), c = m == -INFINITY ? 0.f : expf(m - top);
    m = top;
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] = o[e] * c + p * (in ? (float)static_cast<const T*>(a.v)[at + e] : 0.f);
  }
  T* out = static_cast<T*>(a.out) + (t * a.hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e++) out[e] = (T)(l == 0.f ? 0.f : o[e] / l);
  if (a.lse && lane == 0) a.lse[t * a.hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace tk

static int attend_arg(const char* where, const char* what) {
  tk_set_error("%s: %s", where, what);
  return TK_E_ARG;
}

extern "C" int tk_kv_workspace_create(tk_kv_workspace** out) {
  using namespace tk;
  const char* where = "tk_kv_workspace_create";
  if (!out) return attend_arg(where, "null pointer");
  *out = nullptr;
  tk_kv_workspace* ws = new (std::nothrow) tk_kv_workspace();
  if (!ws) {
    tk_set_error("%s: out of memory", where);
    return TK_E_NOMEM;
  }
  cudaError_t e = cudaGetDevice(&ws->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&ws->sms, cudaDevAttrMultiProcessorCount, ws->device);
  if (e == cudaSuccess) e = cudaMalloc(&ws->status, sizeof(KvStatus));
  if (e == cudaSuccess) e = cudaMemset(ws->status, 0, sizeof(KvStatus));
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    tk_kv_workspace_free(ws);
    return e == cudaErrorMemoryAllocation ? TK_E_NOMEM : TK_E_CUDA;
  }
  *out = ws;
  return TK_OK;
}

extern "C" void tk_kv_workspace_free(tk_kv_workspace* ws) {
  if (!ws) return;
  cudaFree(ws->status);
  delete ws;
}

extern "C" int tk_kv_status(tk_kv_workspace* ws, int64_t* h_request, void* cuda_stream) {
  using namespace tk;
  if (h_request) *h_request = -1;
  if (!ws) return attend_arg("tk_kv_status", "null workspace");
  KvStatus s = {};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  cudaError_t e = cudaMemcpyAsync(&s, ws->status, sizeof(s), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && s.code) e = cudaMemsetAsync(ws->status, 0, sizeof(s), st);
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_status: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  if (s.code) {
    if (h_request) *h_request = s.request;
    tk_set_error("tk_kv_attend: request %lld: lengths outside the call's limits", (long long)s.request);
  }
  return s.code;
}

extern "C" int tk_kv_attend(const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                            int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new,
                            const int32_t* d_len, const int32_t* d_table, int64_t table_stride, int64_t table_width,
                            const int64_t* d_mask, float scale, void* d_out, float* d_lse, void* cuda_stream) {
  using namespace tk;
  const char* where = "tk_kv_attend";
  if (!cache || !ws) return attend_arg(where, "null cache or workspace");
  if (ws->device != cache->device) return attend_arg(where, "cache and workspace are on different devices");
  if (cache->head_dim != 64 && cache->head_dim != 128) return attend_arg(where, "head_dim is neither 64 nor 128");
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % cache->n_heads)
    return attend_arg(where, "n_q_heads is no multiple of the cache's heads up to 1,024");
  if (R < 0 || T < 0 || R > INT32_MAX || T > 1 << 26 || max_new < 0 || table_width < 0 || table_stride < table_width)
    return attend_arg(where, "bad size");
  if (q_stride < (int64_t)n_q_heads * cache->head_dim || q_stride % 8)
    return attend_arg(where, "q_stride is below a token's elements or no multiple of 8");
  if (!(scale > 0.f) || scale > 3e38f) return attend_arg(where, "scale is not a positive number");
  if (T == 0 || R == 0) return TK_OK;
  if (!d_q || !d_off || !d_len || !d_out || (table_width > 0 && !d_table)) return attend_arg(where, "null pointer");
  if ((((uintptr_t)d_q | (uintptr_t)d_out) & 15) != 0) return attend_arg(where, "a buffer is not 16-byte aligned");
  AttendArgs a = {d_q, q_stride, n_q_heads, cache->n_heads, d_off, R, T, max_new, d_len, d_table, table_stride,
                  table_width, d_mask, scale, d_out, d_lse, ws->status, cache->k, cache->v, cache->n_blocks,
                  cache->stride[0], cache->stride[1], cache->stride[2], cache->log2_block};
  const unsigned grid = (unsigned)((T * n_q_heads + 3) / 4);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const bool bf = cache->type == TK_BF16;
  if (cache->head_dim == 64) {
    if (bf) k_kv_attend<__nv_bfloat16, 64><<<grid, 128, 0, st>>>(a);
    else k_kv_attend<__half, 64><<<grid, 128, 0, st>>>(a);
  } else {
    if (bf) k_kv_attend<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(a);
    else k_kv_attend<__half, 128><<<grid, 128, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}
