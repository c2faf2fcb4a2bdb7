// Layer norm kernels for bf16 rows.
#include "fm_norm.h"

namespace fm {

int norm_forward_bf16(const NormForward& a, bool w32) {
  return w32 ? norm_forward_t<bf16_t, float>(a) : norm_forward_t<bf16_t, bf16_t>(a);
}
int norm_backward_bf16(const NormBackward& a, bool w32) {
  return w32 ? norm_backward_t<bf16_t, float>(a) : norm_backward_t<bf16_t, bf16_t>(a);
}

}  // namespace fm
