// Adjusted-logits kernels for f32 logits.
#include "fm_adjust.h"

namespace fm {

int adjust_f32(const AdjustArgs& a, void* stream) { return adjust_t<float>(a, stream); }

}  // namespace fm
