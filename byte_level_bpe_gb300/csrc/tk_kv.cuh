// tk_kv.cuh -- the paged key/value cache: definitions shared by tk_kv.cu and tk_attend.cu.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tk_internal.cuh"

namespace tk {

constexpr int KV_TREE_MAX = 64;  // drafted tokens of one request: one mask word

// Status of the attention calls on a workspace, cleared by tk_kv_status.
struct KvStatus {
  int32_t code;     // first error met (TK_E_*), 0 = none
  int32_t pad;
  int64_t request;  // the request it was met at
};

inline bool kv_block_size_ok(int bs) { return bs >= 16 && bs <= 128 && (bs & (bs - 1)) == 0; }
inline int kv_log2(int bs) {
  int l = 0;
  while ((1 << l) < bs) l++;
  return l;
}

template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static constexpr bool BF = true;
  static __device__ float2 up(type x) { return __bfloat1622float2(x); }
  static __device__ type down(float a, float b) { return __floats2bfloat162_rn(a, b); }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static constexpr bool BF = false;
  static __device__ float2 up(type x) { return __half22float2(x); }
  static __device__ type down(float a, float b) { return __floats2half2_rn(a, b); }
};

}  // namespace tk

struct tk_kv_cache {
  int device, sms;
  int type;
  int64_t n_blocks;
  int n_heads, block_size, log2_block, head_dim;
  int64_t stride[3];  // block, head, token, in elements
  void* k;
  void* v;
  float* k_scale;  // [n_blocks][n_heads] of a cache in 8 bits, else null
  float* v_scale;
  CUtensorMap map_k, map_v;  // for tk_kv_attend; head_dim 64 and 128 only
  CUtensorMap map_k16, map_v16;  // in 8 bits: boxes of 16 tokens
};

struct tk_kv_workspace {
  int device;
  int sms;
  float* part;         // partial outputs of divided units (the allocation's start)
  unsigned* counters;  // their finished pieces
  tk::KvStatus* status;
};
