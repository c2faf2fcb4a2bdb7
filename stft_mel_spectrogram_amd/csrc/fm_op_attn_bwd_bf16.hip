// Attention backward kernels for bf16.
#include "fm_attn_bwd.h"

namespace fm {

int attn_backward_bf16(const AttnArgs& a, void* stream) { return attn_backward_t<bf16_t>(a, stream); }

}  // namespace fm
