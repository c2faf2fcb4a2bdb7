// Token log probability kernels for f16 logits.
#include "fm_score.h"

namespace fm {

int score_forward_f16(const ScoreForward& a) { return score_forward_t<f16_t>(a); }
int score_backward_f16(const ScoreBackward& a) { return score_backward_t<f16_t>(a); }

}  // namespace fm
