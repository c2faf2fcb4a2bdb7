// Token log probability kernels for f32 logits.
#include "fm_score.h"

namespace fm {

int score_forward_f32(const ScoreForward& a) { return score_forward_t<float>(a); }
int score_backward_f32(const ScoreBackward& a) { return score_backward_t<float>(a); }

}  // namespace fm
