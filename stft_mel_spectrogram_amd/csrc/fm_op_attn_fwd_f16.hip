// Attention forward kernels for f16.
#include "fm_attn_fwd.h"

namespace fm {

int attn_forward_f16(const AttnArgs& a, void* stream) { return attn_forward_t<f16_t>(a, stream); }

}  // namespace fm
