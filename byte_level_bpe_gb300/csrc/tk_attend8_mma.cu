// tk_attend8_mma.cu -- the kernels of tk_attend_mma.cuh over a cache in 8 bits, for more than 16 rows.
// Up to 128 rows are units of a stream of their own, more go 256 to a pair: four prompts of 2,000 tokens with a window of
// 1,024 take 420 us so and 444 as units of 128.
#include "tk_attend_mma.cuh"

namespace tk {

template <class T, int D, bool WIN>
static cudaError_t attend8_rows(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  return rows <= 128 ? attend_launch<T, D, 1, true, WIN, true>(a, cache, grid, st) : attend_launch<T, D, 2, true, WIN, true>(a, cache, grid, st);
}

template <class T, int D>
static cudaError_t attend8_win(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  return a.window < INT32_MAX ? attend8_rows<T, D, true>(a, cache, rows, grid, st) : attend8_rows<T, D, false>(a, cache, rows, grid, st);
}

cudaError_t attend8_many(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (cache->type == TK_BF16)
    return cache->head_dim == 64 ? attend8_win<__nv_bfloat16, 64>(a, cache, rows, grid, st)
                                 : attend8_win<__nv_bfloat16, 128>(a, cache, rows, grid, st);
  return cache->head_dim == 64 ? attend8_win<__half, 64>(a, cache, rows, grid, st) : attend8_win<__half, 128>(a, cache, rows, grid, st);
}

}  // namespace tk
