// Internal declarations of the distillation loss and of adjusted logits: the
// arguments that the C ABI (fm_logit.cpp) has checked, the rules that split work,
// and the launches per element type (fm_op_distill_*.hip, fm_op_adjust_*.hip).
// No HIP types, so that host-only builds can include it.
#pragma once

#include "fm_ops.h"

namespace fm {

struct DistillArgs {
  const void* x;
  int64_t x_stride, x_inner, x_outer;
  const int64_t* ids;  // [rows, top]
  const float* lps;    // [rows, top]
  float* loss;         // forward
  float* stats;        // [rows, 4]
  const float* grad;   // backward
  void* dx;
  void* workspace;
  int64_t rows;
  int vocab, top;
  float temperature;
  int rest;
  void* stream;
};
constexpr int kDistillMaxTop = 64;  // one entry per lane of a wave

// Rows are split like those of the token log probabilities without alternatives.
inline int64_t distill_workspace(int64_t rows, int vocab, int ve) {
  const ScoreSplit p = score_split(rows, vocab, ve, 0);
  return p.segs == 1 ? 0 : rows * p.segs * 2 * (int64_t)sizeof(float);
}

// Also the kernels' argument.
struct AdjustArgs {
  const void* x;
  void* out;
  int64_t x_stride;
  const void* history;
  int64_t history_stride;
  int history64;
  int history_len;
  const int32_t* history_lengths;
  const int32_t* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  float repetition_value, frequency_value, presence_value;
  const int64_t* bias_ids;
  const float* bias;
  int biases;
  const uint8_t* allowed;
  int64_t allowed_stride;  // bytes
  int64_t rows;
  int vocab, segs;
};
constexpr int kAdjustMaxBiases = 1024;

// 16-byte groups of a lane: a workgroup of 256 lanes takes a segment of a row.
inline int adjust_vecs(int64_t rows, int vocab, int ve) {
  for (int v : {4, 2})
    if (rows * ((vocab + 256 * ve * v - 1) / (256 * ve * v)) >= 512) return v;
  return 1;
}
inline int adjust_segments(int64_t rows, int vocab, int ve) {
  const int n = 256 * ve * adjust_vecs(rows, vocab, ve);
  return (int)(((int64_t)vocab + n - 1) / n);
}

int distill_forward_f32(const DistillArgs& a);
int distill_forward_f16(const DistillArgs& a);
int distill_forward_bf16(const DistillArgs& a);
int distill_backward_f32(const DistillArgs& a);
int distill_backward_f16(const DistillArgs& a);
int distill_backward_bf16(const DistillArgs& a);
int adjust_f32(const AdjustArgs& a, void* stream);
int adjust_f16(const AdjustArgs& a, void* stream);
int adjust_bf16(const AdjustArgs& a, void* stream);

}  // namespace fm
