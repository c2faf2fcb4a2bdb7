// Distillation kernels for f32 logits.
#include "fm_distill.h"

namespace fm {

int distill_forward_f32(const DistillArgs& a) { return distill_forward_t<float>(a); }
int distill_backward_f32(const DistillArgs& a) { return distill_backward_t<float>(a); }

}  // namespace fm
