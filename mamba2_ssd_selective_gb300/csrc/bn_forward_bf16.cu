#include "block_norm.cuh"

namespace ssd {

template void launch_bn_forward<__nv_bfloat16, __nv_bfloat16>(const BnProblem &, int, cudaStream_t);

}  // namespace ssd
