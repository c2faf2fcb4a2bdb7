// Attention forward kernels for f32.
#include "fm_attn_fwd.h"

namespace fm {

int attn_forward_f32(const AttnArgs& a, void* stream) { return attn_forward_t<float>(a, stream); }

}  // namespace fm
