// Attention backward kernels for f16.
#include "fm_attn_bwd.h"

namespace fm {

int attn_backward_f16(const AttnArgs& a, void* stream) { return attn_backward_t<f16_t>(a, stream); }

}  // namespace fm
