// extend_split_d64.cu -- the kernels of extend_split.cuh for head dimension 64.
#include "extend_split.cuh"

namespace ekv {

cudaError_t launch_extend_split_64(const CUtensorMap (&tm)[3], const ExtSplitParams& p, int vm, int grid,
                                   cudaStream_t st) {
  return launch_ext_split_d<64>(tm, p, vm, grid, st);
}

}  // namespace ekv
