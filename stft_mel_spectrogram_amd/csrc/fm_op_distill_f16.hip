// Distillation kernels for f16 logits.
#include "fm_distill.h"

namespace fm {

int distill_forward_f16(const DistillArgs& a) { return distill_forward_t<f16_t>(a); }
int distill_backward_f16(const DistillArgs& a) { return distill_backward_t<f16_t>(a); }

}  // namespace fm
