// loss_rows_f16.cu -- the row kernels of the training losses for __half scores.
#include "loss_row.cuh"

namespace semicrf {

cudaError_t launch_rows_f16(int mode, const RowArgs& a, cudaStream_t st) {
  return rows_of<__half>(mode, a, st);
}

}  // namespace semicrf
