// Adjusted-logits kernels for bf16 logits.
#include "fm_adjust.h"

namespace fm {

int adjust_bf16(const AdjustArgs& a, void* stream) { return adjust_t<bf16_t>(a, stream); }

}  // namespace fm
