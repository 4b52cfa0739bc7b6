// Group norm with an activation: the backward kernels for f32 tensors.
#include "group_norm.cuh"

namespace ssd {

template <>
void run_gn_backward<float>(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  if (p.act == SSD_ACT_GATE)
    gn::backward<float, true>(p, pl, ws, s);
  else
    gn::backward<float, false>(p, pl, ws, s);
}

}  // namespace ssd
