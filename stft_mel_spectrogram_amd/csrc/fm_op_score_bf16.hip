// Token log probability kernels for bf16 logits.
#include "fm_score.h"

namespace fm {

int score_forward_bf16(const ScoreForward& a) { return score_forward_t<bf16_t>(a); }
int score_backward_bf16(const ScoreBackward& a) { return score_backward_t<bf16_t>(a); }

}  // namespace fm
