// tk_attend.cu -- tk_kv_attend, tk_kv_attend_window and their workspace; the kernels are in
// tk_attend_mma.cuh and tk_attend8.cu.
#include <algorithm>
#include <new>

#include "tk_attend_mma.cuh"

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
  // one allocation: the partial outputs of two pieces of every stream, its counters, the status
  const size_t part = sizeof(float) * 2 * 2 * 128 * (128 + 2) * (size_t)ws->sms,
               counters = sizeof(unsigned) * 2 * 2 * (size_t)ws->sms;
  uint8_t* mem = nullptr;
  if (e == cudaSuccess) e = cudaMalloc(&mem, part + counters + 64 + sizeof(KvStatus));
  if (e == cudaSuccess) {
    ws->part = reinterpret_cast<float*>(mem);
    ws->counters = reinterpret_cast<unsigned*>(mem + part);
    ws->status = reinterpret_cast<KvStatus*>(mem + (part + counters + 63) / 64 * 64);
    e = cudaMemset(ws->counters, 0, counters + 64 + sizeof(KvStatus));
    // a first call on a stream that does not wait for the legacy one would find them as they were
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
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
  cudaFree(ws->part);
  delete ws;
}

extern "C" int tk_kv_status(tk_kv_workspace* ws, int64_t* h_request, void* cuda_stream) {
  using namespace tk;
  if (h_request) *h_request = -1;
  if (!ws) return attend_arg("tk_kv_status", "null workspace");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != ws->device)
    return attend_arg("tk_kv_status", "the current device is not the workspace's");
  KvStatus s = {};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  cudaError_t e = cudaMemcpyAsync(&s, ws->status, sizeof(s), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && s.code) e = cudaMemsetAsync(ws->status, 0, sizeof(s), st);
  // a call that gave up may have left counts behind
  if (e == cudaSuccess && s.code == TK_E_TIMEOUT) e = cudaMemsetAsync(ws->counters, 0, sizeof(unsigned) * 4 * ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_status: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  if (s.code) {
    if (h_request) *h_request = s.request;
    if (s.code == TK_E_TIMEOUT) tk_set_error("tk_kv_attend: a wait on the device gave up");
    else if (s.request < 0) tk_set_error("tk_kv_attend: more work than one call takes, or offsets that contradict each other");
    else tk_set_error("tk_kv_attend: request %lld: lengths outside the call's limits", (long long)s.request);
  }
  return s.code;
}

// window: INT32_MAX for none
static int kv_attend(const char* where, const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                     int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new, const int32_t* d_len,
                     const int32_t* d_table, int64_t table_stride, int64_t table_width, const int64_t* d_mask, int window,
                     int sinks, float scale, void* d_out, float* d_lse, void* cuda_stream) {
  using namespace tk;
  if (!cache || !ws) return attend_arg(where, "null cache or workspace");
  if (ws->device != cache->device) return attend_arg(where, "cache and workspace are on different devices");
  if (cache->head_dim != 64 && cache->head_dim != 128) return attend_arg(where, "head_dim is neither 64 nor 128");
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % cache->n_heads)
    return attend_arg(where, "n_q_heads is no multiple of the cache's heads up to 1,024");
  if (R < 0 || T < 0 || R > 1 << 20 || T > 1 << 26 || max_new < 0 || table_width < 0 || table_stride < table_width)
    return attend_arg(where, "bad size");
  if (q_stride < (int64_t)n_q_heads * cache->head_dim || q_stride % 8)
    return attend_arg(where, "q_stride is below a token's elements or no multiple of 8");
  if (!(scale > 0.f && scale < 1e38f)) return attend_arg(where, "scale is not a positive number below 1e38");
  if (T * n_q_heads > INT32_MAX) return attend_arg(where, "T times n_q_heads is above 2^31");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != cache->device) return attend_arg(where, "the current device is not the cache's");
  if (T == 0) return TK_OK;
  if (!d_q || !d_out || (R > 0 && (!d_off || !d_len || (table_width > 0 && !d_table)))) return attend_arg(where, "null pointer");
  if ((((uintptr_t)d_q | (uintptr_t)d_out) & 15) != 0) return attend_arg(where, "a buffer is not 16-byte aligned");
  const int group = n_q_heads / cache->n_heads;
  AttendArgs a = {d_q, q_stride, n_q_heads, cache->n_heads, group, d_off, R, T, max_new, d_len, d_table, table_stride,
                  table_width, d_mask, scale * 1.4426950408889634f, d_out, d_lse, ws->status,
                  cache->v, cache->n_blocks, cache->stride[0], cache->stride[1],
                  cache->stride[2], cache->log2_block, ws->part, ws->counters, window, sinks, cache->k_scale, cache->v_scale,
                  group == 1 ? 0 : UINT64_MAX / group + 1};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int64_t rows = std::min(max_new, T) * group;  // of a request and key head
  const cudaError_t e = cache->k_scale ? attend8(a, cache, rows, ws->sms, st)
                        : window < INT32_MAX ? attend_windowed(a, cache, rows, ws->sms, st)
                                             : attend_types<false>(a, cache, rows, ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}

extern "C" int tk_kv_attend(const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                            int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new,
                            const int32_t* d_len, const int32_t* d_table, int64_t table_stride, int64_t table_width,
                            const int64_t* d_mask, float scale, void* d_out, float* d_lse, void* cuda_stream) {
  return kv_attend("tk_kv_attend", cache, ws, d_q, q_stride, n_q_heads, d_off, R, T, max_new, d_len, d_table, table_stride,
                   table_width, d_mask, INT32_MAX, 0, scale, d_out, d_lse, cuda_stream);
}

extern "C" int tk_kv_attend_window(const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                                   int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new,
                                   const int32_t* d_len, const int32_t* d_table, int64_t table_stride, int64_t table_width,
                                   const int64_t* d_mask, int64_t window, int64_t sinks, float scale, void* d_out,
                                   float* d_lse, void* cuda_stream) {
  using namespace tk;
  const char* where = "tk_kv_attend_window";
  if (window < 1 || sinks < 0) return attend_arg(where, "window is below 1 or sinks below 0");
  if (d_mask && window < KV_TREE_MAX) return attend_arg(where, "a window under masks is below 64, the most tokens of a tree");
  // a request has less than 2^31 places
  const int w = (int)std::min<int64_t>(window, INT32_MAX), s = (int)std::min<int64_t>(sinks, INT32_MAX - 128);
  return kv_attend(where, cache, ws, d_q, q_stride, n_q_heads, d_off, R, T, max_new, d_len, d_table, table_stride, table_width,
                   d_mask, w, s, scale, d_out, d_lse, cuda_stream);
}
