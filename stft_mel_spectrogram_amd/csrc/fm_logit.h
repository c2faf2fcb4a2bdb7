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
constexpr int kAdjustMaxHistory = 1 << 20;  // a count takes 20 bits of a slot
constexpr int kAdjustThreads = 512;

// 16-byte groups of a lane: a workgroup takes a segment of a row, of 8192 tokens
// while there are 512 of them, two per compute unit, since each reads the row's
// history again (history 4000, 300 biases, us: 256 x 131072 f16 52, segments of 4096 tokens
// 69; f32 72, 4096 tokens 78, 2048 106; 64 x 131072 f32 24, 24, 26).  Fewer tokens where
// there are fewer workgroups (8 x 50001 bf16: 4096 tokens 5.2, 8192 6.2).
inline int adjust_vecs(int64_t rows, int vocab, int ve) {
  int v = 16 / ve;
  for (; v > 1; v /= 2) {
    const int n = kAdjustThreads * ve * v;
    if (rows * (((int64_t)vocab + n - 1) / n) >= 512) break;
  }
  return v;
}
inline int adjust_segments(int64_t rows, int vocab, int ve) {
  const int n = kAdjustThreads * ve * adjust_vecs(rows, vocab, ve);
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
