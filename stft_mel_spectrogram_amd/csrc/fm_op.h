// Device helpers shared by the speech-model operators (layer norm, relative
// attention, token log probabilities): element types, 16-byte vectors from
// any element alignment, wave reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>
#include <tuple>
#include <utility>

#include "fm_ops.h"

namespace fm {

// Launches `kernel` on `stream`; FM_OK or FM_E_HIP with a message.
template <class... P, std::size_t... I>
int launch_packed(const char* what, void (*kernel)(P...), dim3 grid, dim3 block, size_t lds,
                  void* stream, std::tuple<P...>& args, std::index_sequence<I...>) {
  void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&std::get<I>(args)))...};
  const hipError_t e =
      hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, lds,
                      static_cast<hipStream_t>(stream));
  if (e == hipSuccess) return FM_OK;
  return set_error(FM_E_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

template <class... P, class... A>
int launch(const char* what, void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, void* stream,
           const A&... a) {
  std::tuple<P...> args{static_cast<P>(a)...};
  return launch_packed(what, kernel, grid, block, lds, stream, args,
                       std::index_sequence_for<P...>{});
}

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Lets a kernel use `bytes` of dynamic LDS (over 64 KiB needs this) on the current
// device.
template <class K>
int lds_opt_in(K kernel, size_t bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes)) == hipSuccess
             ? FM_OK
             : FM_E_HIP;
}
// `opt_in()` of a set of kernels, once on each device that launches them.
template <class F>
int opted_in(DeviceOnce& once, F opt_in) {
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess) return set_error(FM_E_HIP, "no current device");
  return once(device, opt_in) == FM_OK ? FM_OK : set_error(FM_E_HIP, "attention: LDS size refused");
}

// What the wave's lanes have stored in LDS is seen by its reads below, and what
// they have read above is not yet overwritten.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A 16-byte group of elements.  Loads and stores take any element-aligned
// address: gfx950 runs with unaligned global access on, so one dwordx4
// access serves rows of odd widths too.
template <class T>
struct Vec16 {
  static constexpr int n = 16 / sizeof(T);
  T v[n];
};

template <class T>
__device__ __forceinline__ Vec16<T> load16(const T* p) {
  Vec16<T> r;
  __builtin_memcpy(&r, p, 16);
  return r;
}

template <class T>
__device__ __forceinline__ void store16(T* p, const Vec16<T>& r) {
  __builtin_memcpy(p, &r, 16);
}

// The first `have` elements of a group at p (none if have <= 0), the rest
// `fill`.
template <class T>
__device__ __forceinline__ Vec16<T> load16_part(const T* p, int have, T fill) {
  Vec16<T> r;
  if (have >= Vec16<T>::n) {
    r = load16(p);
  } else {
#pragma unroll
    for (int e = 0; e < Vec16<T>::n; ++e) r.v[e] = e < have ? p[e] : fill;
  }
  return r;
}

// N elements from any element-aligned address, of which `have` exist.
template <class W, int N>
struct Group {
  W v[N];
};
template <class W, int N>
__device__ __forceinline__ Group<W, N> load_group(const W* p, int have, W fill) {
  Group<W, N> r;
  if (have >= N) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) r.v[e] = e < have ? p[e] : fill;
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store16_part(T* p, const Vec16<T>& r, int have) {
  if (have >= Vec16<T>::n) {
    store16(p, r);
  } else {
#pragma unroll
    for (int e = 0; e < Vec16<T>::n; ++e)
      if (e < have) p[e] = r.v[e];
  }
}

// Reductions over aligned groups of LANES (16, 32 or 64) lanes; every lane gets
// the result, and the order of the operations is fixed.  Within 16 lanes by
// rotations, beyond by exchanges of rows: vector instructions only.
template <int ROT>
__device__ __forceinline__ float lanes_rotate(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(v), 0x120 + ROT, 0xf, 0xf, false));
}
template <int LANES, class F>
__device__ __forceinline__ float lanes_reduce(float v, F f) {
  v = f(v, lanes_rotate<8>(v));
  v = f(v, lanes_rotate<4>(v));
  v = f(v, lanes_rotate<2>(v));
  v = f(v, lanes_rotate<1>(v));
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<LANES>(v, [](float a, float b) { return a + b; });
}
// The largest of the wave's unsigned integers.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  const float r = lanes_reduce<64>(__uint_as_float(v), [](float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  });
  return __float_as_uint(r);
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_reduce<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace fm
