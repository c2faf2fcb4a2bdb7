// Host-side checks that the operators' C entries share.
#pragma once

#include <cstdint>

#include "fm_internal.h"

namespace fm {

inline int elem_bytes(int dtype) {
  return dtype == FM_F32 ? 4 : (dtype == FM_F16 || dtype == FM_BF16) ? 2 : 0;
}
inline bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

}  // namespace fm
