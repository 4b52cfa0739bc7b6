// Group norm with an activation: the forward kernels for bf16 tensors.
#include "group_norm.cuh"

namespace ssd {

template <>
void run_gn_forward<__nv_bfloat16>(const GnProblem &p, const GnPlan &pl, char *ws, cudaStream_t s) {
  if (p.act == SSD_ACT_GATE)
    gn::forward<__nv_bfloat16, true>(p, pl, ws, s);
  else
    gn::forward<__nv_bfloat16, false>(p, pl, ws, s);
}

}  // namespace ssd
