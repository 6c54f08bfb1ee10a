// extend_split_d128.cu -- the kernels of extend_split.cuh for head dimension 128.
#include "extend_split.cuh"

namespace ekv {

cudaError_t launch_extend_split_128(const CUtensorMap (&tm)[3], const ExtSplitParams& p, int vm, int grid,
                                   cudaStream_t st) {
  return launch_ext_split_d<128>(tm, p, vm, grid, st);
}

}  // namespace ekv
