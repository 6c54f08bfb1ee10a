// extend_tc05_d128.cu -- the kernels of extend_tc05.cuh for head dimension 128.
#include "extend_tc05.cuh"

namespace ekv {

cudaError_t launch_extend_tc05_128(const ExtTcMaps& m, const ExtTcParams& p, int vm, int grid, cudaStream_t st) {
  return launch_ext_tc_d<128>(m, p, vm, grid, st);
}

}  // namespace ekv
