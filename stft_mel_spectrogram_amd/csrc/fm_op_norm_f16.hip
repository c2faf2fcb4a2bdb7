// Layer norm kernels for f16 rows.
#include "fm_norm.h"

namespace fm {

int norm_forward_f16(const NormForward& a, bool w32) {
  return w32 ? norm_forward_t<f16_t, float>(a) : norm_forward_t<f16_t, f16_t>(a);
}
int norm_backward_f16(const NormBackward& a, bool w32) {
  return w32 ? norm_backward_t<f16_t, float>(a) : norm_backward_t<f16_t, f16_t>(a);
}

}  // namespace fm
