// Group norm with an activation: the forward kernels for f32 tensors.
#include "group_norm.cuh"

namespace ssd {

template <>
void run_gn_forward<float>(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  if (p.act == SSD_ACT_GATE)
    gn::forward<float, true>(p, pl, ws, s);
  else
    gn::forward<float, false>(p, pl, ws, s);
}

}  // namespace ssd
