// Distillation kernels for bf16 logits.
#include "fm_distill.h"

namespace fm {

int distill_forward_bf16(const DistillArgs& a) { return distill_forward_t<bf16_t>(a); }
int distill_backward_bf16(const DistillArgs& a) { return distill_backward_t<bf16_t>(a); }

}  // namespace fm
