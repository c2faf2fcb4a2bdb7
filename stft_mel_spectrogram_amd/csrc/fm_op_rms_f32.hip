// Root-mean-square norm kernels for f32 rows.
#include "fm_rms.h"

namespace fm {

int rms_forward_f32(const RmsForward& a) { return rms_forward_t<float, float>(a); }
int rms_backward_f32(const RmsBackward& a) { return rms_backward_t<float, float>(a); }

}  // namespace fm
