// C ABI of the distillation loss and of adjusted logits (declared in
// include/fm.h): argument checks on the host, then the launches of the type.
#include "fm_logit.h"

#include <cmath>
#include <cstdint>

#include "fm_check.h"

namespace fm {
namespace {

int bad(const char* what) { return set_error(FM_E_INVAL, what); }

constexpr int64_t kVocabMost = (int64_t(1) << 31) - 65536;

int check_distill_size(int64_t rows, int64_t vocab, int dtype) {
  if (!elem_bytes(dtype)) return bad("distillation: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (rows < 0) return bad("distillation: rows must be >= 0");
  if (vocab < 1 || vocab >= kVocabMost) return bad("distillation: vocab must be in [1, 2^31 - 65536)");
  const ScoreSplit p = score_split(rows, static_cast<int>(vocab), 16 / elem_bytes(dtype), 0);
  if (rows >= (int64_t(1) << 31) / p.segs) return bad("distillation: too many rows for one launch");
  return FM_OK;
}

// What both directions share; ids and lps are looked at by the kernels.
int check_distill(const DistillArgs& a, int64_t vocab, double temperature, int dtype) {
  if (int st = check_distill_size(a.rows, vocab, dtype)) return st;
  if (a.top < 1 || a.top > kDistillMaxTop) return bad("distillation: top must be in [1, 64]");
  if (!(temperature >= 0x1p-10 && temperature <= 0x1p10))
    return bad("distillation: temperature must be in [2^-10, 2^10]");
  if (a.rest && temperature != 1.0) return bad("distillation: the rest needs a temperature of 1");
  if (a.rows == 0) return FM_OK;
  if (!a.x || !a.ids || !a.lps) return bad("distillation: x, ids and lps must not be NULL");
  if (a.rows > 1 && a.x_stride < 0) return bad("distillation: x_stride must be >= 0");
  if (a.x_inner < 0 || a.x_inner >= int64_t(1) << 31 || (a.x_inner > 0 && a.x_outer < 0))
    return bad("distillation: x_inner must be in [0, 2^31) and x_outer >= 0");
  const int es = elem_bytes(dtype);
  if (!aligned_to(a.x, es) || !aligned_to(a.dx, es) || !aligned_to(a.ids, 8) || !aligned_to(a.lps, 4) ||
      !aligned_to(a.loss, 4) || !aligned_to(a.stats, 4) || !aligned_to(a.grad, 4))
    return bad("distillation: misaligned pointer");
  return FM_OK;
}

}  // namespace
}  // namespace fm

using fm::bad;

extern "C" {

int64_t fm_distill_workspace(int64_t rows, int64_t vocab, int dtype) try {
  if (int st = fm::check_distill_size(rows, vocab, dtype)) return st;
  return fm::distill_workspace(rows, static_cast<int>(vocab), 16 / fm::elem_bytes(dtype));
} catch (...) {
  return FM_E_NOMEM;
}

int fm_distill(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer, const int64_t* ids,
               const float* lps, float* loss, float* stats, void* workspace, int64_t rows, int64_t vocab, int top,
               double temperature, int rest, int dtype, void* stream) try {
  fm::DistillArgs a = {};
  a.x = x, a.x_stride = x_stride, a.x_inner = x_inner, a.x_outer = x_outer;
  a.ids = ids, a.lps = lps, a.loss = loss, a.stats = stats, a.workspace = workspace;
  a.rows = rows, a.top = top, a.rest = rest != 0, a.stream = stream;
  if (int st = fm::check_distill(a, vocab, temperature, dtype)) return st;
  a.vocab = static_cast<int>(vocab);
  a.temperature = static_cast<float>(temperature);
  if (rows == 0) return FM_OK;
  if (!loss) return bad("distillation: loss must not be NULL");
  if (fm::distill_workspace(rows, a.vocab, 16 / fm::elem_bytes(dtype)) > 0 &&
      (!workspace || !fm::aligned_to(workspace, 16)))
    return bad("distillation: the workspace must be 16-byte aligned device memory");
  if (dtype == FM_F32) return fm::distill_forward_f32(a);
  return dtype == FM_F16 ? fm::distill_forward_f16(a) : fm::distill_forward_bf16(a);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_distill_backward(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer, const int64_t* ids,
                        const float* lps, const float* stats, const float* grad_loss, void* dx, int64_t rows,
                        int64_t vocab, int top, double temperature, int rest, int dtype, void* stream) try {
  fm::DistillArgs a = {};
  a.x = x, a.x_stride = x_stride, a.x_inner = x_inner, a.x_outer = x_outer;
  a.ids = ids, a.lps = lps, a.stats = const_cast<float*>(stats), a.grad = grad_loss, a.dx = dx;
  a.rows = rows, a.top = top, a.rest = rest != 0, a.stream = stream;
  if (int st = fm::check_distill(a, vocab, temperature, dtype)) return st;
  a.vocab = static_cast<int>(vocab);
  a.temperature = static_cast<float>(temperature);
  if (rows == 0) return FM_OK;
  if (!stats || !grad_loss || !dx) return bad("distillation: stats, grad_loss and dx must not be NULL");
  if (dtype == FM_F32) return fm::distill_backward_f32(a);
  return dtype == FM_F16 ? fm::distill_backward_f16(a) : fm::distill_backward_bf16(a);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_adjust_logits(const fm_adjust_args* p, void* stream) try {
  if (!p) return bad("adjusted logits: args must not be NULL");
  const int es = fm::elem_bytes(p->dtype);
  if (!es) return bad("adjusted logits: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (p->rows < 0 || p->rows >= int64_t(1) << 31) return bad("adjusted logits: rows must be in [0, 2^31)");
  if (p->vocab < 1 || p->vocab >= fm::kVocabMost)
    return bad("adjusted logits: vocab must be in [1, 2^31 - 65536)");
  if (p->history_len < 0) return bad("adjusted logits: history_len must be >= 0");
  if (p->history_len >= fm::kAdjustMaxHistory)
    return fm::set_error(FM_E_UNSUPPORTED, "adjusted logits: history_len must be < 2^20");
  if (p->history_bits != 64 && p->history_bits != 32) return bad("adjusted logits: history_bits must be 32 or 64");
  if (p->biases < 0) return bad("adjusted logits: biases must be >= 0");
  if (p->biases > fm::kAdjustMaxBiases)
    return fm::set_error(FM_E_UNSUPPORTED, "adjusted logits: at most 1024 biases per row");
  // as the kernels take them
  const float rep = static_cast<float>(p->repetition_value);
  if (!p->repetition && !(rep > 0.f && std::isfinite(rep) && std::isfinite(1.f / rep)))
    return bad("adjusted logits: repetition must be > 0, and finite in float32 like its reciprocal");
  if ((!p->frequency && !std::isfinite(static_cast<float>(p->frequency_value))) ||
      (!p->presence && !std::isfinite(static_cast<float>(p->presence_value))))
    return bad("adjusted logits: frequency and presence must be finite in float32");
  fm::AdjustArgs a = {};
  a.rows = p->rows;
  a.vocab = static_cast<int>(p->vocab);
  a.segs = fm::adjust_segments(a.rows, a.vocab, 16 / es);
  if (a.rows >= (int64_t(1) << 22) / a.segs) return bad("adjusted logits: too many rows for one launch");
  if (a.rows == 0) return FM_OK;
  const bool history = p->history_len > 0;
  if (!p->x || !p->out) return bad("adjusted logits: x and out must not be NULL");
  if (history && !p->history) return bad("adjusted logits: history must not be NULL");
  if (p->biases > 0 && (!p->bias_ids || !p->bias)) return bad("adjusted logits: bias_ids and bias must not be NULL");
  if (a.rows > 1 && (p->x_stride < 0 || (history && p->history_stride < 0)))
    return bad("adjusted logits: strides must be >= 0");
  if (p->allowed && p->allowed_stride < 0) return bad("adjusted logits: strides must be >= 0");
  if (!fm::aligned_to(p->x, es) || !fm::aligned_to(p->out, es) ||
      !fm::aligned_to(p->history, p->history_bits / 8) || !fm::aligned_to(p->history_lengths, 4) ||
      !fm::aligned_to(p->prompt_lengths, 4) || !fm::aligned_to(p->repetition, 4) ||
      !fm::aligned_to(p->frequency, 4) || !fm::aligned_to(p->presence, 4) || !fm::aligned_to(p->bias_ids, 8) ||
      !fm::aligned_to(p->bias, 4) || !fm::aligned_to(p->allowed, 4))
    return bad("adjusted logits: misaligned pointer");
  a.x = p->x;
  a.out = p->out;
  a.x_stride = p->x_stride;
  a.history = p->history;
  a.history_stride = p->history_stride;
  a.history64 = p->history_bits == 64;
  a.history_len = static_cast<int>(p->history_len);
  a.history_lengths = p->history_lengths;
  a.prompt_lengths = p->prompt_lengths;
  a.repetition = p->repetition;
  a.frequency = p->frequency;
  a.presence = p->presence;
  a.repetition_value = rep;
  a.frequency_value = static_cast<float>(p->frequency_value);
  a.presence_value = static_cast<float>(p->presence_value);
  a.bias_ids = p->bias_ids;
  a.bias = p->bias;
  a.biases = static_cast<int>(p->biases);
  a.allowed = reinterpret_cast<const uint8_t*>(p->allowed);
  a.allowed_stride = p->allowed_stride * 4;
  if (p->dtype == FM_F32) return fm::adjust_f32(a, stream);
  return p->dtype == FM_F16 ? fm::adjust_f16(a, stream) : fm::adjust_bf16(a, stream);
} catch (...) {
  return FM_E_NOMEM;
}

}  // extern "C"
