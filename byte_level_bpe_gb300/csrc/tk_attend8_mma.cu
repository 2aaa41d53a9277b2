// tk_attend8_mma.cu -- the kernels of tk_attend_mma.cuh over a cache in 8 bits, for more than 16 rows.
// Units of 128 rows for each stream, or for more rows of head_dim 128 of 256 for the pair (us, 256 and 128 rows):
// 64 drafted tokens over 131k 247 and 338, chunks of 700 over 9k 275 and 322, four prompts of 2,000 tokens with a window
// of 1,024 403 and 437, 94 trees of up to 56 tokens, 448 rows, 442 and 459, the same in fp16 432 and 423.  Of head_dim 64, whose
// products are short beside what a unit's start and end take, the same are 215 and 235, 219 and 212, 354 and 312, and the trees in
// fp16 362 and 274.
#include "tk_attend_mma.cuh"

namespace tk {

template <class T, int D, bool WIN>
static cudaError_t attend8_rows(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if constexpr (D == 128) {
    if (rows > 128) return attend_launch<T, D, 2, true, WIN, true>(a, cache, grid, st);
  }
  return attend_launch<T, D, 1, true, WIN, true>(a, cache, grid, st);
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
