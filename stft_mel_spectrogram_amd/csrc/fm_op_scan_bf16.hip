// Gated recurrence kernels for bf16 frames.
#include "fm_scan.h"

namespace fm {

int scan_forward_bf16(const ScanArgs& a, void* stream) { return scan_forward_t<bf16_t>(a, stream); }
int scan_backward_bf16(const ScanArgs& a, void* stream) { return scan_backward_t<bf16_t>(a, stream); }

}  // namespace fm
