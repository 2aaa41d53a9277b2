// tk_attend_window.cu -- the kernels of tk_attend_mma.cuh for calls with a window, over a cache in 16 bits.
#include "tk_attend_mma.cuh"

namespace tk {

cudaError_t attend_windowed(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  return attend_types<true>(a, cache, rows, grid, st);
}

}  // namespace tk
