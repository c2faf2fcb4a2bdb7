// Root-mean-square norm kernels for f16 rows.
#include "fm_rms.h"

namespace fm {

int rms_forward_f16(const RmsForward& a, bool w32) {
  return w32 ? rms_forward_t<f16_t, float>(a) : rms_forward_t<f16_t, f16_t>(a);
}
int rms_backward_f16(const RmsBackward& a, bool w32) {
  return w32 ? rms_backward_t<f16_t, float>(a) : rms_backward_t<f16_t, f16_t>(a);
}

}  // namespace fm
