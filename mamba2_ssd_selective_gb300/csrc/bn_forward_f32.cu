#include "block_norm.cuh"

namespace ssd {

template void launch_bn_forward<float, float>(const BnProblem &, int, cudaStream_t);

}  // namespace ssd
