// Gated recurrence kernels for f32 frames.
#include "fm_scan.h"

namespace fm {

int scan_forward_f32(const ScanArgs& a, void* stream) { return scan_forward_t<float>(a, stream); }
int scan_backward_f32(const ScanArgs& a, void* stream) { return scan_backward_t<float>(a, stream); }

}  // namespace fm
