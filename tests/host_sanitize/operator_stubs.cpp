// Host-only stand-ins for the operators' launches (fm_op_*.hip).  Each writes
// every element of the workspace that the kernels' indexing can reach, so that
// a workspace smaller than what a call uses is an invalid write here.
// Test infrastructure: never linked into the library.
#include "fm_ops.h"

namespace fm {
namespace {

void fill(float* p, int64_t n) {
  for (int64_t i = 0; i < n; ++i) p[i] = 1.f;
}

int norm_backward(const NormBackward& a, int ve) {
  const int parts = norm_parts(a.rows, a.width, ve);
  if (a.dw && a.rows > 0 && !norm_single(a.rows, a.width, ve))
    fill(static_cast<float*>(a.workspace), int64_t(parts) * 2 * a.width);
  return FM_OK;
}

int score_forward(const ScoreForward& a, int ve) {
  const ScoreSplit p = score_split(a.rows, a.vocab, ve, a.top);
  if (int64_t(p.segs) * p.seg_len < a.vocab || int64_t(p.segs - 1) * p.seg_len >= a.vocab)
    return set_error(FM_E_HIP, "segments do not cover the row");
  if (p.segs == 1) return FM_OK;
  fill(static_cast<float*>(a.workspace), a.rows * p.segs * 3);
  auto* keys = reinterpret_cast<uint64_t*>(static_cast<char*>(a.workspace) + score_part_bytes(a.rows, p.segs));
  for (int64_t i = 0; i < a.rows * p.segs * a.top; ++i) keys[i] = 1;
  return FM_OK;
}

int attn_forward(const AttnArgs& a) {
  if (a.splits < 1 || a.splits > kAttnMaxSplits) return set_error(FM_E_HIP, "splits out of range");
  if (a.splits > 1) {
    fill(a.part_o, a.splits * attn_rows(a) * a.dim);
    fill(a.part_lse, a.splits * attn_rows(a));
  }
  return FM_OK;
}

int attn_backward(const AttnArgs& a, bool f16) {
  fill(a.delta, attn_rows(a));
  if (f16) fill(a.amax, attn_rows(a));
  if (a.d_table) {
    fill(a.table_part, int64_t(a.batch) * a.heads * attn_query_blocks(a) * a.dq_splits * bias_window(a.far));
    fill(a.table_dist, int64_t(a.heads) * bias_window(a.far));
  }
  if (a.dq_splits < 1) return set_error(FM_E_HIP, "no ranges");
  if (a.dq_splits > 1) {
    fill(a.part_dq, a.dq_splits * attn_rows(a) * a.dim);
    fill(a.part_row, a.dq_splits * attn_rows(a) * 3);
  }
  if (a.dkv_splits < 1) return set_error(FM_E_HIP, "no shares");
  if (a.dkv_splits > 1) fill(a.part_dkv, int64_t(a.dkv_splits) * a.batch * a.kv_heads * a.k_len * 2 * a.dim);
  return FM_OK;
}

}  // namespace

int norm_forward_f32(const NormForward&) { return FM_OK; }
int norm_forward_f16(const NormForward&, bool) { return FM_OK; }
int norm_forward_bf16(const NormForward&, bool) { return FM_OK; }
int norm_backward_f32(const NormBackward& a) { return norm_backward(a, 4); }
int norm_backward_f16(const NormBackward& a, bool) { return norm_backward(a, 8); }
int norm_backward_bf16(const NormBackward& a, bool) { return norm_backward(a, 8); }
int score_forward_f32(const ScoreForward& a) { return score_forward(a, 4); }
int score_forward_f16(const ScoreForward& a) { return score_forward(a, 8); }
int score_forward_bf16(const ScoreForward& a) { return score_forward(a, 8); }
int score_backward_f32(const ScoreBackward&) { return FM_OK; }
int score_backward_f16(const ScoreBackward&) { return FM_OK; }
int score_backward_bf16(const ScoreBackward&) { return FM_OK; }
int attn_forward_f32(const AttnArgs& a, void*) { return attn_forward(a); }
int attn_forward_f16(const AttnArgs& a, void*) { return attn_forward(a); }
int attn_forward_bf16(const AttnArgs& a, void*) { return attn_forward(a); }
int attn_backward_f32(const AttnArgs& a, void*) { return attn_backward(a, false); }
int attn_backward_f16(const AttnArgs& a, void*) { return attn_backward(a, true); }
int attn_backward_bf16(const AttnArgs& a, void*) { return attn_backward(a, false); }

}  // namespace fm
