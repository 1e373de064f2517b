// loss_rows_bf16.cu -- the row kernels of the training losses for __nv_bfloat16 scores.
#include "loss_row.cuh"

namespace semicrf {

cudaError_t launch_rows_bf16(int mode, const RowArgs& a, cudaStream_t st) {
  return rows_of<__nv_bfloat16>(mode, a, st);
}

}  // namespace semicrf
