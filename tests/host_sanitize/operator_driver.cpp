// Drives the operators' C ABI over a grid of shapes and random ones, each with
// a workspace of exactly the size that is asked for.
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

void norm(int64_t rows, int64_t width, int dtype) {
  const int64_t n = fm_layer_norm_backward_workspace(rows, width, dtype);
  expect(n >= 0, "layer norm workspace", rows, width, dtype);
  Scratch ws(n);
  float* f = reinterpret_cast<float*>(dummy);
  expect(fm_layer_norm_forward(dummy, width, dummy, dummy, dummy, f, f, rows, width, 1e-5, dtype, dtype,
                               nullptr) == FM_OK, "layer norm", rows, width, dtype);
  expect(fm_layer_norm_backward(dummy, width, dummy, width, dummy, f, f, dummy, dummy, dummy, ws.p, rows, width,
                                dtype, FM_F32, nullptr) == FM_OK, "layer norm backward", rows, width, dtype);
}

void score(int64_t rows, int64_t vocab, int top, int dtype) {
  const int64_t n = fm_token_logprobs_workspace(rows, vocab, top, dtype);
  expect(n >= 0, "scores workspace", rows, vocab, top);
  Scratch ws(n);
  float* f = reinterpret_cast<float*>(dummy);
  int64_t* ids = reinterpret_cast<int64_t*>(dummy);
  expect(fm_token_logprobs(dummy, vocab, dummy, 64, f, f, f, ids, f, ws.p, rows, vocab, top, dtype, nullptr) == FM_OK,
         "scores", rows, vocab, top);
  expect(fm_token_logprobs_backward(dummy, vocab, dummy, 32, f, f, f, f, ids, top ? f : nullptr, dummy, rows, vocab, top, dtype,
                                    nullptr) == FM_OK, "scores backward", rows, vocab, top);
}

void attention(int64_t b, int64_t h, int64_t hk, int64_t tq, int64_t tk, int64_t d, int far, int dtype) {
  fm_attention_args a = {};
  a.dtype = a.table_dtype = dtype;
  a.far = far;
  a.num_buckets = 32;
  a.batch = b, a.heads = h, a.kv_heads = hk, a.q_len = tq, a.k_len = tk, a.head_dim = d;
  a.scale = 0.125;
  a.q = a.k = a.v = a.table = a.grad_o = dummy;
  a.bucket_map = reinterpret_cast<int32_t*>(dummy);
  a.o = a.grad_q = a.grad_k = a.grad_v = a.grad_table = dummy;
  a.lse = reinterpret_cast<float*>(dummy);
  for (int backward = 0; backward < 2; ++backward) {
    const int64_t n = fm_attention_workspace(&a, backward);
    expect(n >= 0, "attention workspace", tq, tk, d);
    Scratch ws(n);
    expect((backward ? fm_attention_backward(&a, ws.p, nullptr) : fm_attention_forward(&a, ws.p, nullptr)) == FM_OK,
           backward ? "attention backward" : "attention", tq, tk, d);
  }
}

}  // namespace

int main() {
  const int types[] = {FM_F32, FM_F16, FM_BF16};
  std::mt19937 rng(7);
  const auto pick = [&](int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); };
  for (int t : types) {
    for (int64_t rows : {0, 1, 3, 16, 17, 64, 255, 256, 257, 2049, 9000})
      for (int64_t width : {1, 63, 64, 129, 513, 2048, 2049, 4097, 8192, 8193}) norm(rows, width, t);
    for (int64_t rows : {0, 1, 7, 255, 256, 300, 639, 641, 1281})
      for (int64_t vocab : {1, 65, 1024, 1025, 2049, 8193, 50001, 131073})
        for (int top : {0, 1, 20, 64})
          if (top <= vocab) score(rows, vocab, top, t);
    for (int64_t tq : {0, 1, 16, 32, 33, 128, 129, 700})
      for (int64_t tk : {0, 1, 256, 257, 1023, 1024, 2048, 4100})
        for (int64_t h : {1, 4})
          for (int far : {0, 128, 1024}) attention(2, h, 1, tq, tk, 40, far, t);
    for (int i = 0; i < 150; ++i) {
      const int64_t hk = pick(1, 8);
      attention(pick(0, 5), hk * pick(1, 6), hk, pick(0, 400), pick(0, 3000), pick(1, 128), int(pick(0, 1024)), t);
      norm(pick(0, 4000), pick(1, 9000), t);
      const int64_t vocab = pick(1, 140000);
      score(pick(0, 700), vocab, int(pick(0, vocab < 64 ? vocab : 64)), t);
    }
  }
  // refusals leave a message and do nothing
  expect(fm_attention_forward(nullptr, nullptr, nullptr) < 0, "NULL args");
  expect(fm_attention_workspace(nullptr, 1) < 0, "NULL args");
  expect(fm_layer_norm_backward_workspace(-1, 8, FM_F32) < 0, "negative rows");
  expect(fm_token_logprobs_workspace(4, 100, 65, FM_F32) < 0, "too many alternatives");
  expect(fm_token_logprobs(dummy, 50001, dummy, 64, nullptr, nullptr, nullptr, reinterpret_cast<int64_t*>(dummy),
                           reinterpret_cast<float*>(dummy), nullptr, 8, 50001, 5, FM_BF16, nullptr) < 0,
         "a workspace that is missing");
  std::printf("%s\n", failures ? "failed" : "operators: all calls passed");
  return failures != 0;
}
