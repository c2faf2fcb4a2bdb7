// Drives the C ABI of the recurrence, the RMS norm, the distillation and the
// adjusted logits over a grid of shapes and random ones, each with a workspace of
// exactly the size that is asked for.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "fm.h"

namespace {

int failures = 0;
void expect(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0) {
  if (ok) return;
  ++failures;
  std::printf("FAILED %s (%lld %lld %lld): %s\n", what, a, b, c, fm_last_error());
}

struct Scratch {  // exactly n bytes, from malloc's 16-byte alignment
  void* p;
  explicit Scratch(int64_t n) : p(n > 0 ? std::malloc(static_cast<size_t>(n)) : nullptr) {}
  ~Scratch() { std::free(p); }
};

alignas(256) char dummy[4096];
float* const f = reinterpret_cast<float*>(dummy);
int64_t* const ids = reinterpret_cast<int64_t*>(dummy);

void recurrence(int64_t b, int64_t t, int64_t c, int dtype) {
  fm_recurrence_args a = {};
  a.dtype = dtype;
  a.batch = b, a.time = t, a.channels = c;
  a.x = a.forget = a.gate = a.grad_y = dummy;
  a.y = a.grad_x = a.grad_forget = a.grad_gate = dummy;
  a.state = a.grad_last = f;
  a.last_state = a.grad_state = a.saved = f;
  for (int backward = 0; backward < 2; ++backward) {
    const int64_t n = fm_gated_recurrence_workspace(&a, backward);
    expect(n >= 0, "recurrence workspace", b, t, c);
    Scratch ws(n);
    expect((backward ? fm_gated_recurrence_backward(&a, ws.p, nullptr) : fm_gated_recurrence_forward(&a, ws.p, nullptr)) ==
               FM_OK, backward ? "recurrence backward" : "recurrence", b, t, c);
    a.saved = backward ? f : nullptr;
    expect(fm_gated_recurrence_forward(&a, ws.p, nullptr) == FM_OK || backward, "recurrence alone", b, t, c);
    a.saved = f;
  }
}

void rms(int64_t rows, int64_t width, int dtype) {
  const int64_t n = fm_rms_norm_backward_workspace(rows, width, dtype);
  expect(n >= 0, "rms workspace", rows, width, dtype);
  Scratch ws(n);
  expect(fm_rms_norm_forward(dummy, width, dummy, width, dummy, dummy, dummy, f, rows, width, 1e-6, dtype, dtype,
                             nullptr) == FM_OK, "rms", rows, width, dtype);
  expect(fm_rms_norm_quantized(dummy, width, nullptr, 0, nullptr, dummy, f, nullptr, rows, width, 0.0, dtype, FM_F32,
                               FM_I8, nullptr) == FM_OK, "rms 8 bits", rows, width, dtype);
  expect(fm_rms_norm_backward(dummy, width, dummy, width, dummy, width, dummy, f, dummy, dummy, ws.p, rows, width, dtype,
                              FM_F32, nullptr) == FM_OK, "rms backward", rows, width, dtype);
}

void logits(int64_t rows, int64_t vocab, int dtype) {
  const int64_t n = fm_distill_workspace(rows, vocab, dtype);
  expect(n >= 0, "distillation workspace", rows, vocab, dtype);
  Scratch ws(n);
  expect(fm_distill(dummy, vocab, 0, 0, ids, f, f, f, ws.p, rows, vocab, 64, 1.0, 1, dtype, nullptr) == FM_OK,
         "distillation", rows, vocab, dtype);
  expect(fm_distill_backward(dummy, vocab, 0, 0, ids, f, f, f, dummy, rows, vocab, 1, 2.0, 0, dtype, nullptr) == FM_OK,
         "distillation backward", rows, vocab, dtype);
  fm_adjust_args a = {};
  a.dtype = dtype, a.history_bits = 64;
  a.rows = rows, a.vocab = vocab;
  a.x = a.out = dummy;
  a.repetition_value = 1.0;
  expect(fm_adjust_logits(&a, nullptr) == FM_OK, "adjusted logits", rows, vocab, dtype);
}

}  // namespace

int main() {
  const int types[] = {FM_F32, FM_F16, FM_BF16};
  std::mt19937 rng(7);
  const auto pick = [&](int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); };
  for (int t : types) {
    for (int64_t b : {0, 1, 3, 64, 300})
      for (int64_t time : {0, 1, 8, 9, 63, 64, 65, 128, 129, 256, 513, 2000, 9001})
        for (int64_t c : {1, 3, 4, 32, 65, 400}) recurrence(b, time, c, t);
    recurrence(1, 1000003, 16, t);
    recurrence(2, 100000000, 1, t);
    for (int64_t rows : {0, 1, 3, 16, 17, 64, 257, 2049, 9000})
      for (int64_t width : {1, 63, 64, 129, 513, 2048, 2049, 4097, 8192, 8193}) rms(rows, width, t);
    for (int64_t rows : {0, 1, 7, 255, 256, 300, 641, 1281})
      for (int64_t vocab : {1, 65, 1024, 1025, 2049, 8193, 50001, 131073}) logits(rows, vocab, t);
    logits(1, (int64_t(1) << 31) - 65537, t);
    for (int i = 0; i < 200; ++i) {
      recurrence(pick(0, 40), pick(0, 5000), pick(1, 600), t);
      rms(pick(0, 4000), pick(1, 9000), t);
      logits(pick(0, 700), pick(1, 140000), t);
    }
  }
  // refusals leave a message and do nothing
  expect(fm_gated_recurrence_forward(nullptr, nullptr, nullptr) < 0, "NULL args");
  expect(fm_gated_recurrence_workspace(nullptr, 1) < 0, "NULL args");
  expect(fm_adjust_logits(nullptr, nullptr) < 0, "NULL args");
  expect(fm_rms_norm_backward_workspace(-1, 8, FM_F32) < 0, "negative rows");
  expect(fm_distill_workspace(4, 0, FM_F32) < 0, "no vocabulary");
  std::printf("%s\n", failures ? "failed" : "frame operators: all calls passed");
  return failures != 0;
}
