// Root-mean-square norm kernels for bf16 rows.
#include "fm_rms.h"

namespace fm {

int rms_forward_bf16(const RmsForward& a, bool w32) {
  return w32 ? rms_forward_t<bf16_t, float>(a) : rms_forward_t<bf16_t, bf16_t>(a);
}
int rms_backward_bf16(const RmsBackward& a, bool w32) {
  return w32 ? rms_backward_t<bf16_t, float>(a) : rms_backward_t<bf16_t, bf16_t>(a);
}

}  // namespace fm
