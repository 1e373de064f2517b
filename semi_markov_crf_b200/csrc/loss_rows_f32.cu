// loss_rows_f32.cu -- the row kernels of the training losses for float scores.
#include "loss_row.cuh"

namespace semicrf {

cudaError_t launch_rows_f32(int mode, const RowArgs& a, cudaStream_t st) {
  return rows_of<float>(mode, a, st);
}

}  // namespace semicrf
