// The row segments of the token log probabilities near the ends of the
// documented range, with the kernels' own index arithmetic: every entry of a
// row lies in exactly one segment, and no int overflows on the way.
#include <cstdint>
#include <cstdio>

#include "fm_ops.h"

int main() {
  const int64_t most = (int64_t(1) << 31) - 65537;  // the longest vocabulary
  int failures = 0, checked = 0;
  for (int ve : {4, 8})
    for (int top : {0, 5})
      for (int64_t rows : {1, 2, 3, 5, 7, 31, 255, 256, 300, 639, 641})
        for (int64_t vocab : {most, most - 1, most - 8191, most - 700001, int64_t(2146225813), int64_t(2145389604),
                              int64_t(2140000000), int64_t(1500000000), int64_t(1) << 30, int64_t(50001), int64_t(9000)}) {
          const fm::ScoreSplit p = fm::score_split(rows, int(vocab), ve, top);
          int64_t at = 0;
          bool ok = true;
          for (int seg = 0; seg < p.segs; ++seg) {
            const int beg = seg * p.seg_len, end = fm::score_segment_end(beg, p.seg_len, int(vocab));
            ok = ok && beg == at && end > beg && end <= vocab;
            at = end;
          }
          ++checked;
          if (ok && at == vocab) continue;
          ++failures;
          std::printf("FAILED rows %lld vocab %lld ve %d: %d segments of %d end at %lld\n", (long long)rows,
                      (long long)vocab, ve, p.segs, p.seg_len, (long long)at);
        }
  std::printf("%d splits, %d failures\n", checked, failures);
  return failures != 0;
}
