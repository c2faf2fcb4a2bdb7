// Adjusted-logits kernels for f16 logits.
#include "fm_adjust.h"

namespace fm {

int adjust_f16(const AdjustArgs& a, void* stream) { return adjust_t<f16_t>(a, stream); }

}  // namespace fm
