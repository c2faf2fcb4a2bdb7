// Attention backward kernels for f32.
#include "fm_attn_bwd.h"

namespace fm {

int attn_backward_f32(const AttnArgs& a, void* stream) { return attn_backward_t<float>(a, stream); }

}  // namespace fm
