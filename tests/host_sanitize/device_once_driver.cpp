// DeviceOnce: work runs once on every device, and again after a failure.
#include <cstdio>

#include "fm_ops.h"

int main() {
  int failures = 0;
  const auto expect = [&](bool ok, const char* what) {
    if (!ok) {
      ++failures;
      std::printf("FAILED %s\n", what);
    }
  };
  fm::DeviceOnce once;
  int runs[70] = {};
  const auto run = [&](int device, int status) {
    return once(device, [&] {
      ++runs[device];
      return status;
    });
  };
  expect(run(0, FM_E_HIP) == FM_E_HIP && run(0, FM_OK) == FM_OK && runs[0] == 2, "a failure is tried again");
  expect(run(0, FM_E_HIP) == FM_OK && runs[0] == 2, "done work does not run again");
  for (int d : {1, 2, 7, 63}) {
    expect(run(d, FM_OK) == FM_OK && run(d, FM_OK) == FM_OK && runs[d] == 1, "another device runs it once");
  }
  expect(run(69, FM_OK) == FM_OK && run(69, FM_OK) == FM_OK && runs[69] == 2, "beyond 64 devices it runs every time");
  fm::DeviceOnce other;
  int n = 0;
  other(0, [&] { return ++n, FM_OK; });
  expect(n == 1, "each set of kernels has its own");
  return failures != 0;
}
