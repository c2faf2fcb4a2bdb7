// Rows in launches that a grid takes, and attention's refusals of grids that
// no launch takes.
#include <cstdio>

#include "fm.h"
#include "fm_ops.h"

int main() {
  int failures = 0;
  const auto expect = [&](bool ok, const char* what, long long n = 0) {
    if (!ok) {
      ++failures;
      std::printf("FAILED %s (%lld)\n", what, n);
    }
  };
  for (int threads : {16, 64, 256, 1024})
    for (int64_t rows : {int64_t(0), int64_t(1), (int64_t(1) << 22) + 1, int64_t(1) << 25, (int64_t(1) << 26) + 5,
                         (int64_t(1) << 31) - 1}) {
      int64_t next = 0;
      const int st = fm::by_rows(rows, fm::kGridThreads / threads, [&](int64_t at, int64_t n) {
        expect(at == next && n > 0 && n * threads < (int64_t(1) << 32), "range of rows", at);
        next = at + n;
        return FM_OK;
      });
      expect(st == FM_OK && next == rows, "all rows", rows);
    }
  int calls = 0;
  expect(fm::by_rows(10, 3, [&](int64_t at, int64_t) { return ++calls, at == 3 ? FM_E_HIP : FM_OK; }) == FM_E_HIP &&
             calls == 2, "the first failure ends it");

  // attention: workgroups of 256 threads, of 1024 for few queries of 16 bits
  const auto workspace = [&](int64_t batch, int64_t heads, int64_t q_len, int64_t k_len, int dtype) {
    fm_attention_args a = {};
    a.dtype = a.table_dtype = dtype;
    a.far = 4, a.num_buckets = 4, a.batch = batch, a.heads = a.kv_heads = heads, a.q_len = q_len, a.k_len = k_len;
    a.head_dim = 8, a.scale = 1.0;
    return fm_attention_workspace(&a, 0);
  };
  expect(workspace((1 << 20) - 1, 16, 40, 40, FM_BF16) >= 0, "the most query blocks");
  expect(workspace(1 << 20, 16, 40, 40, FM_BF16) == FM_E_INVAL, "too many query blocks");
  expect(workspace(1 << 19, 16, 40, 300, FM_BF16) == FM_E_INVAL, "too many key blocks");
  expect(workspace((1 << 18) - 1, 16, 1, 300, FM_BF16) >= 0, "the most single tokens");
  expect(workspace(1 << 18, 16, 1, 300, FM_BF16) == FM_E_INVAL, "too many single tokens");
  expect(workspace(1 << 18, 16, 1, 300, FM_F32) >= 0, "fewer threads for float32");
  expect(workspace((1 << 30) - 1, 65535, (1 << 30) - 1, (1 << 30) - 1, FM_BF16) == FM_E_INVAL, "far too many");
  return failures != 0;
}
