// Attention forward kernels for bf16.
#include "fm_attn_fwd.h"

namespace fm {

int attn_forward_bf16(const AttnArgs& a, void* stream) { return attn_forward_t<bf16_t>(a, stream); }

}  // namespace fm
