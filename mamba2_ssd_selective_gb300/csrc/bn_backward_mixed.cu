#include "block_norm.cuh"

namespace ssd {

template void launch_bn_backward<__nv_bfloat16, float>(const BnProblem &, int, cudaStream_t);

}  // namespace ssd
