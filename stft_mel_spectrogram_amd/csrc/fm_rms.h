// Root-mean-square norm over the last axis, of x or of x + residual, forward and
// backward, and with an output in 8 bits.
//
//   s = x + r, rounded to the rows' type (it is the next layer's residual),
//   rstd = 1 / sqrt(mean(s^2) + eps), u = s rstd, y = u w
//   g = dy w, dx = dr = rstd (g - u mean(g u)) + ds, dw = sum over rows of dy u
//   8 bits: scale = max |y| / 448 (e4m3) or 127 (int8) per row, y / scale rounded
//   to nearest from the unrounded y, whose steps are single float32 operations:
//   s / sqrt(..), its product with w, the quotient by the scale.  Sums and scales
//   are float32.
//
// The lane layouts are layer norm's: a row stays in the registers of LPR lanes,
// VPL groups of 16 bytes each, so that every tensor moves once; wider rows are
// swept again from the cache.  The backward adds dw up in registers over the rows
// that a workgroup walks, one partial row per workgroup and a second launch.  Memory
// bound: 96064 x 1024 bf16 with the residual, 787 MB each way, forward 180 us (4.4 TB/s),
// backward 167 (4.7) and 5 for the partial rows (a large copy runs at 5.12); 24016 x 4096
// bf16 in e4m3 147 (4.7), int8 154 (4.5); 48032 x 1024 f32 with the residual 141 (5.6) and
// 163 (4.8).
#pragma once

#include "fm_norm.h"
#include "fm_seq.h"

namespace fm {

// A row's largest |v|, as bits: a NaN is larger than any number.
template <int LPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, uint32_t* red) {
  constexpr int L = LPR < 64 ? LPR : 64;
  v = __float_as_uint(lanes_reduce<L>(__uint_as_float(v), [](float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  }));
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < LPR / 64; ++w) v = v > red[w] ? v : red[w];
  }
  return v;
}

// OUT 1: e4m3, 2: int8; `most` the row's largest |y|.  The smallest scale keeps
// its reciprocal finite; a row of zeros has scale 1.
template <int OUT>
__device__ __forceinline__ float rms_scale(uint32_t most) {
  if (most == 0) return 1.f;
  const float m = __uint_as_float(most) / (OUT == 1 ? 448.f : 127.f);
  return m < 0x1p-126f ? 0x1p-126f : m;
}
// v / d, rounded once: the product with 1 / d, then what it misses.  Short numbers
// often have quotients right between two 8-bit values (one in 10^4 of bfloat16 rows),
// which one rounding more would decide.  What v / inf gives is 0.
struct RmsDivisor {
  float inv, d;
  __device__ __forceinline__ explicit RmsDivisor(float by) : inv(1.f / by), d(by == INFINITY ? 0.f : by) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * inv;
    return fmaf(fmaf(-q, d, v), inv, q);
  }
};
template <int OUT, int N>
__device__ __forceinline__ void rms_store8(uint8_t* p, const float (&y)[N], RmsDivisor scale, int have) {
  uint32_t v[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = scale(y[4 * i + e]);
    if constexpr (OUT == 1) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
      v[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
    } else {
      v[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[i] |= ((uint32_t)(int)fminf(fmaxf(rintf(z[e]), -127.f), 127.f) & 255u) << (8 * e);
    }
  }
  if (have >= N) {
    __builtin_memcpy(p, v, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < have) p[e] = (uint8_t)(v[e / 4] >> (8 * (e % 4)));
  }
}

template <class T>
__device__ __forceinline__ Vec16<T> rms_add(const Vec16<T>& a, const Vec16<T>& b) {
  Vec16<T> r;
#pragma unroll
  for (int e = 0; e < Vec16<T>::n; ++e) r.v[e] = (T)((float)a.v[e] + (float)b.v[e]);
  return r;
}

template <class T, class W, int LPR, int VPL, int OUT>
__global__ __launch_bounds__(norm_threads(LPR)) void rms_forward_kernel(
    const T* __restrict__ x, int64_t x_stride, const T* residual, int64_t r_stride, const W* __restrict__ w,
    void* __restrict__ y, float* __restrict__ scale, T* sum, float* __restrict__ rstd, int64_t rows, int width,
    float eps) {
  constexpr int VE = Vec16<T>::n;
  constexpr int RPB = norm_threads(LPR) / LPR;
  constexpr int SLOTS = LPR > 64 ? LPR / 64 : 0;
  __shared__ float2 red[2 * SLOTS + 1];
  __shared__ uint32_t umax[2 * SLOTS + 1];
  bool odd = false;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const float n = (float)width;
  Group<W, VE> wv[VPL];
  bool first = true;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + sub;
    const int have_all = row < rows ? width : 0;
    Vec16<T> s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      s[i] = load16_part(x + row * x_stride + c, have_all - c, (T)0.f);
    }
    if (residual) {
      Vec16<T> r[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        r[i] = load16_part(residual + row * r_stride + c, have_all - c, (T)0.f);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        s[i] = rms_add(s[i], r[i]);
        if (have_all - c > 0) store16_part(sum + row * width + c, s[i], have_all - c);
      }
    }
    if (first) {
      first = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        wv[i] = load_group<W, VE>(w + c, w ? width - c : 0, (W)1.f);
      }
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) q = fmaf((float)s[i].v[e], (float)s[i].v[e], q);
    const float root = sqrtf(row_sum<LPR>(q, red + (odd ? SLOTS : 0)) / n + eps);
    if constexpr (OUT == 0) {
      const float rs = 1.f / root;
      if (rstd && lane == 0 && row < rows) rstd[row] = rs;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        if (have_all - c > 0) {
          Vec16<T> out;
#pragma unroll
          for (int e = 0; e < VE; ++e) out.v[e] = (T)((float)s[i].v[e] * rs * (float)wv[i].v[e]);
          store16_part((T*)y + row * width + c, out, have_all - c);
        }
      }
    } else {
      const RmsDivisor by(root);
      uint32_t most = 0;
      float v[VPL][VE];
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          // past the end s is 0 and w 1
          v[i][e] = by((float)s[i].v[e]) * (float)wv[i].v[e];
          const uint32_t b = __float_as_uint(v[i][e]) & 0x7fffffffu;
          most = b > most ? b : most;
        }
      const float sc = rms_scale<OUT>(row_umax<LPR>(most, umax + (odd ? SLOTS : 0)));
      if (lane == 0 && row < rows) scale[row] = sc;
      const RmsDivisor to(sc);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        if (have_all - c > 0) rms_store8<OUT, VE>((uint8_t*)y + row * width + c, v[i], to, have_all - c);
      }
    }
    odd = !odd;
  }
}

// Rows too wide for the registers: one workgroup of 1024 lanes per row; with a
// residual the sum is read back by the lane that wrote it.
template <class T, class W, int OUT>
__global__ __launch_bounds__(kNormWide) void rms_forward_wide_kernel(
    const T* x, int64_t x_stride, const T* residual, int64_t r_stride, const W* __restrict__ w,
    void* __restrict__ y, float* __restrict__ scale, T* sum, float* __restrict__ rstd, int64_t rows, int width,
    float eps) {
  constexpr int VE = Vec16<T>::n;
  __shared__ float2 red[kNormWide / 64];
  __shared__ uint32_t umax[kNormWide / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * x_stride;
  const T* rr = residual ? residual + row * r_stride : nullptr;
  T* sr = residual ? sum + row * width : nullptr;
  const float n = (float)width;
  float q = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    Vec16<T> v = load16_part(xr + c, width - c, (T)0.f);
    if (rr) {
      v = rms_add(v, load16_part(rr + c, width - c, (T)0.f));
      store16_part(sr + c, v, width - c);
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) q = fmaf((float)v.v[e], (float)v.v[e], q);
  }
  const float root = sqrtf(row_sum<kNormWide>(q, red) / n + eps);
  const float rs = 1.f / root;
  if (rstd && threadIdx.x == 0) rstd[row] = rs;
  const T* from = rr ? sr : xr;
  const RmsDivisor by(root);
  const auto value = [&](const Vec16<T>& v, int c, int e) {
    const int ce = c + e < width ? c + e : c;
    const float u = OUT == 0 ? (float)v.v[e] * rs : by((float)v.v[e]);
    return u * (w ? (float)w[ce] : 1.f);
  };
  float sc = 1.f;
  if constexpr (OUT != 0) {
    uint32_t most = 0;
#pragma unroll 1
    for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
      const Vec16<T> v = load16_part(from + c, width - c, (T)0.f);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint32_t b = c + e < width ? __float_as_uint(value(v, c, e)) & 0x7fffffffu : 0u;
        most = b > most ? b : most;
      }
    }
    sc = rms_scale<OUT>(row_umax<kNormWide>(most, umax));
    if (threadIdx.x == 0) scale[row] = sc;
  }
  const RmsDivisor to(sc);
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    Vec16<T> v = load16_part(from + c, width - c, (T)0.f);
    if constexpr (OUT == 0) {
#pragma unroll
      for (int e = 0; e < VE; ++e) v.v[e] = (T)value(v, c, e);
      store16_part((T*)y + row * width + c, v, width - c);
    } else {
      float z[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) z[e] = value(v, c, e);
      rms_store8<OUT, VE>((uint8_t*)y + row * width + c, z, to, width - c);
    }
  }
}

// PARTS: also add up dw (part: one row of width floats per workgroup; a single
// workgroup writes dw itself).
template <class T, class W, int LPR, int VPL, bool PARTS>
__global__ __launch_bounds__(norm_threads(LPR)) void rms_backward_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ s, int64_t s_stride,
    const T* __restrict__ ds, int64_t ds_stride, const W* __restrict__ w, const float* __restrict__ rstd,
    T* __restrict__ dx, float* __restrict__ part, W* __restrict__ dw, int64_t rows, int width) {
  constexpr int VE = Vec16<T>::n;
  constexpr int NT = norm_threads(LPR);
  constexpr int RPB = NT / LPR;
  constexpr int SLOTS = LPR > 64 ? LPR / 64 : 0;
  __shared__ float2 red[2 * SLOTS + 1];
  bool odd = false;
  const int lane = threadIdx.x % LPR;
  const int sub = threadIdx.x / LPR;
  const float inv_n = 1.f / (float)width;
  float aw[PARTS ? VPL * VE : 1];
  if constexpr (PARTS) {
#pragma unroll
    for (int i = 0; i < VPL * VE; ++i) aw[i] = 0.f;
  }
  Group<W, VE> wv[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = (i * LPR + lane) * VE;
    wv[i] = load_group<W, VE>(w + c, w ? width - c : 0, (W)1.f);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + sub;
    const int have_all = row < rows ? width : 0;
    Vec16<T> sv[VPL], gv[VPL], ev[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      sv[i] = load16_part(s + row * s_stride + c, have_all - c, (T)0.f);
      gv[i] = load16_part(dy + row * dy_stride + c, have_all - c, (T)0.f);
    }
    if (ds) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        ev[i] = load16_part(ds + row * ds_stride + c, have_all - c, (T)0.f);
      }
    }
    const float rs = row < rows ? rstd[row] : 0.f;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        // past the end dy is 0
        const float d = (float)gv[i].v[e], u = (float)sv[i].v[e] * rs;
        m = fmaf(d * (float)wv[i].v[e], u, m);
        if constexpr (PARTS) aw[i * VE + e] = fmaf(d, u, aw[i * VE + e]);
      }
    m = row_sum<LPR>(m, red + (odd ? SLOTS : 0)) * inv_n;
    odd = !odd;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      if (have_all - c > 0) {
        Vec16<T> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float u = (float)sv[i].v[e] * rs;
          const float d = rs * ((float)gv[i].v[e] * (float)wv[i].v[e] - u * m);
          out.v[e] = (T)(ds ? d + (float)ev[i].v[e] : d);
        }
        store16_part(dx + row * width + c, out, have_all - c);
      }
    }
  }
  if constexpr (PARTS) {
    const auto put = [&](int c, float v) {
      if (c >= width) return;
      if (gridDim.x > 1)
        part[(int64_t)blockIdx.x * width + c] = v;
      else
        dw[c] = (W)v;
    };
    // lanes of the same columns: RPB groups of LPR lanes
    if constexpr (RPB > 1) {
      __shared__ float col[RPB > 1 ? NT * VE : 1];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VE; ++e) col[threadIdx.x * VE + e] = aw[i * VE + e];
        __syncthreads();
        for (int t = threadIdx.x; t < LPR * VE; t += NT) {
          float v = 0.f;
#pragma unroll
          for (int r = 0; r < RPB; ++r) v += col[r * LPR * VE + t];
          put(i * LPR * VE + t, v);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) put((i * LPR + lane) * VE + e, aw[i * VE + e]);
    }
  }
}

template <class T, class W>
__global__ __launch_bounds__(kNormWide) void rms_backward_wide_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ s, int64_t s_stride,
    const T* __restrict__ ds, int64_t ds_stride, const W* __restrict__ w, const float* __restrict__ rstd,
    T* __restrict__ dx, int64_t rows, int width) {
  constexpr int VE = Vec16<T>::n;
  __shared__ float2 red[kNormWide / 64];
  const int64_t row = blockIdx.x;
  const T* sr = s + row * s_stride;
  const T* gr = dy + row * dy_stride;
  const T* er = ds ? ds + row * ds_stride : nullptr;
  const float rs = rstd[row];
  float m = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> sv = load16_part(sr + c, width - c, (T)0.f);
    const Vec16<T> gv = load16_part(gr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int ce = c + e < width ? c + e : c;
      m = fmaf((float)gv.v[e] * (w ? (float)w[ce] : 1.f), (float)sv.v[e] * rs, m);
    }
  }
  m = row_sum<kNormWide>(m, red) / (float)width;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> sv = load16_part(sr + c, width - c, (T)0.f);
    Vec16<T> gv = load16_part(gr + c, width - c, (T)0.f);
    Vec16<T> ev = {};
    if (er) ev = load16_part(er + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int ce = c + e < width ? c + e : c;
      const float d = rs * ((float)gv.v[e] * (w ? (float)w[ce] : 1.f) - (float)sv.v[e] * rs * m);
      gv.v[e] = (T)(er ? d + (float)ev.v[e] : d);
    }
    store16_part(dx + row * width + c, gv, width - c);
  }
}

// Column sums of dy * u for widths whose accumulators do not fit the registers.
template <class T>
__global__ __launch_bounds__(kNormThreads) void rms_columns_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ s, int64_t s_stride,
    const float* __restrict__ rstd, float* __restrict__ part, int64_t rows, int width) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= width) return;
  float aw = 0.f;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    aw = fmaf((float)dy[r * dy_stride + c], (float)s[r * s_stride + c] * rstd[r], aw);
  part[(int64_t)blockIdx.y * width + c] = aw;
}

// Adds the workgroups' partial rows: 64 columns per workgroup, 16 sets of lanes
// that take every 16th partial, then over the sets.
template <class W>
__global__ __launch_bounds__(1024) void rms_reduce_kernel(const float* __restrict__ part, int parts,
                                                          W* __restrict__ dw, int width) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, set = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float v = 0.f;
  if (c < width) {
    const float* q = part + c;
    const int64_t row = width;
    int p = set;
    // eight loads on their way at a time
    for (; p + 112 < parts; p += 128) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = q[(p + 16 * k) * row];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += t[k];
    }
    for (; p < parts; p += 16) v += q[p * row];
  }
  red[set][lane] = v;
  __syncthreads();
  if (set == 0 && c < width) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += red[k][lane];
    dw[c] = (W)t;
  }
}

template <class T, class W, int OUT>
int rms_forward_out(const RmsForward& a) {
  constexpr int VE = Vec16<T>::n;
  const NormShape s = norm_shape(a.width, VE);
#define FM_RMS_FWD(L, V)                                                                        \
  if constexpr (V * VE <= norm_most(L))                                                         \
    if (s.lpr == L && s.vpl == V) {                                                             \
      const int64_t need = (a.rows + norm_rows(L) - 1) / norm_rows(L);                          \
      return launch("rms norm", rms_forward_kernel<T, W, L, V, OUT>,                            \
                    dim3((unsigned)(need < kNormBlocks ? need : kNormBlocks)),                  \
                    dim3(norm_threads(L)), 0, a.stream, (const T*)a.x, a.x_stride,              \
                    (const T*)a.residual, a.r_stride, (const W*)a.weight, a.y, a.scale,         \
                    (T*)a.sum, a.rstd, a.rows, a.width, a.eps);                                 \
    }
  FM_NORM_SHAPES(FM_RMS_FWD)
#undef FM_RMS_FWD
  return by_rows(a.rows, kGridThreads / kNormWide, [&](int64_t at, int64_t rows) {
    return launch("rms norm", rms_forward_wide_kernel<T, W, OUT>, dim3((unsigned)rows), dim3(kNormWide), 0,
                  a.stream, (const T*)a.x + at * a.x_stride, a.x_stride,
                  a.residual ? (const T*)a.residual + at * a.r_stride : nullptr, a.r_stride,
                  (const W*)a.weight, (char*)a.y + at * a.width * (OUT ? 1 : (int)sizeof(T)),
                  a.scale ? a.scale + at : nullptr, a.sum ? (T*)a.sum + at * a.width : nullptr,
                  a.rstd ? a.rstd + at : nullptr, rows, a.width, a.eps);
  });
}
template <class T, class W>
int rms_forward_t(const RmsForward& a) {
  return a.out == 0 ? rms_forward_out<T, W, 0>(a)
                    : a.out == 1 ? rms_forward_out<T, W, 1>(a) : rms_forward_out<T, W, 2>(a);
}

template <class T, class W>
int rms_backward_t(const RmsBackward& a) {
  constexpr int VE = Vec16<T>::n;
  const NormShape s = norm_shape(a.width, VE);
  const int parts = norm_parts(a.rows, a.width, VE);
  const bool want = a.dw != nullptr;
  float* part = (float*)a.workspace;
  if (a.rows > 0) {
    int st = FM_OK;
    if (s.vpl == 0)
      st = by_rows(a.rows, kGridThreads / kNormWide, [&](int64_t at, int64_t rows) {
        return launch("rms norm backward", rms_backward_wide_kernel<T, W>, dim3((unsigned)rows), dim3(kNormWide), 0,
                      a.stream, (const T*)a.dy + at * a.dy_stride, a.dy_stride, (const T*)a.s + at * a.s_stride,
                      a.s_stride, a.ds ? (const T*)a.ds + at * a.ds_stride : nullptr, a.ds_stride,
                      (const W*)a.weight, a.rstd + at, (T*)a.dx + at * a.width, rows, a.width);
      });
#define FM_RMS_BWD(L, V)                                                                         \
  if constexpr (V * VE <= norm_most(L))                                                          \
    if (s.lpr == L && s.vpl == V)                                                                \
      st = launch("rms norm backward",                                                           \
                  want ? rms_backward_kernel<T, W, L, V, true> : rms_backward_kernel<T, W, L, V, false>, \
                  dim3((unsigned)parts), dim3(norm_threads(L)), 0, a.stream, (const T*)a.dy,     \
                  a.dy_stride, (const T*)a.s, a.s_stride, (const T*)a.ds, a.ds_stride,           \
                  (const W*)a.weight, a.rstd, (T*)a.dx, part, (W*)a.dw, a.rows, a.width);
    FM_NORM_SHAPES(FM_RMS_BWD)
#undef FM_RMS_BWD
    if (st != FM_OK) return st;
    if (want && s.vpl == 0) {
      st = launch("rms norm backward columns", rms_columns_kernel<T>,
                  dim3((a.width + kNormThreads - 1) / kNormThreads, parts), dim3(kNormThreads), 0, a.stream,
                  (const T*)a.dy, a.dy_stride, (const T*)a.s, a.s_stride, a.rstd, part, a.rows, a.width);
      if (st != FM_OK) return st;
    }
  }
  if (!want || norm_single(a.rows, a.width, VE)) return FM_OK;
  return launch("rms norm backward sums", rms_reduce_kernel<W>, dim3((unsigned)((a.width + 63) / 64)), dim3(1024), 0,
                a.stream, part, a.rows > 0 ? parts : 0, (W*)a.dw, a.width);
}

}  // namespace fm
