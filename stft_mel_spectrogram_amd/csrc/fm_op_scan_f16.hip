// Gated recurrence kernels for f16 frames.
#include "fm_scan.h"

namespace fm {

int scan_forward_f16(const ScanArgs& a, void* stream) { return scan_forward_t<f16_t>(a, stream); }
int scan_backward_f16(const ScanArgs& a, void* stream) { return scan_backward_t<f16_t>(a, stream); }

}  // namespace fm
