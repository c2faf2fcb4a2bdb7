// Layer norm kernels for f32 rows.
#include "fm_norm.h"

namespace fm {

int norm_forward_f32(const NormForward& a) { return norm_forward_t<float, float>(a); }
int norm_backward_f32(const NormBackward& a) { return norm_backward_t<float, float>(a); }

}  // namespace fm
