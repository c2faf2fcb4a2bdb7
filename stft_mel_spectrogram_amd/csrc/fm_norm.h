// Layer norm over the last axis, forward and backward.
//
//   u = (x - mean(x)) * rstd,  rstd = 1 / sqrt(var(x) + eps),  y = u * w + b
//   g = dy * w,  dx = rstd * (g - mean(g) - u * mean(g u))
//   dw = sum over rows of dy * u,  db = sum over rows of dy
//
// The variance is the mean square of the centred row (two sweeps over the
// row's registers, no difference of large sums); all sums are in float32.
//
// One row is held in registers by LPR lanes, VPL groups of 16 bytes each, so
// x (and dy) are read from memory once per pass; a wave takes 64 / LPR rows
// where LPR < 64.  Memory bound: workgroups walk over rows and keep their
// columns' weight and bias in registers; the backward adds dw and db up there
// too, writes one partial row per workgroup and a second launch adds the
// partials in a fixed order.  96064 x 1024 bf16: forward 96 us (4.1 TB/s),
// backward 131 (4.5 TB/s) and 5 for the partials; 24008 x 128 f32: 7.6, 8 and 4.5
// (a large copy runs at 5.06 TB/s).
#pragma once

#include "fm_op.h"

namespace fm {

// Sum over the LPR lanes that hold a row: within a wave by lane exchange, over
// several waves through LDS (`red`; successive calls take two slot sets in turn,
// so that one barrier each does).
template <int LPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red) {
  constexpr int L = LPR < 64 ? LPR : 64;
  v.x = lanes_sum<L>(v.x);
  v.y = lanes_sum<L>(v.y);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < LPR / 64; ++w) {
      v.x += red[w].x;
      v.y += red[w].y;
    }
  }
  return v;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v, float2* red) {
  return row_sum2<LPR>(make_float2(v, 0.f), red).x;
}

template <class T, class W, int LPR, int VPL>
__global__ __launch_bounds__(norm_threads(LPR)) void norm_forward_kernel(
    const T* __restrict__ x, int64_t x_stride, const W* __restrict__ w, const W* __restrict__ b,
    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width,
    float eps) {
  constexpr int VE = Vec16<T>::n;
  constexpr int RPB = norm_threads(LPR) / LPR;
  constexpr int SLOTS = LPR > 64 ? LPR / 64 : 0;
  __shared__ float2 red[2 * SLOTS + 1];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  // divided, not multiplied by 1 / n: a constant row has exactly that mean
  const float n = (float)width;
  Group<W, VE> wv[VPL], bv[VPL];
  bool first = true;
  // rows past the end (whole lane groups; a workgroup of one row has none) run
  // on an empty width
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + sub;
    const int have_all = row < rows ? width : 0;
    const T* xr = x + row * x_stride;
    Vec16<T> raw[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      raw[i] = load16_part(xr + c, have_all - c, (T)0.f);
    }
    if (first) {
      first = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = (i * LPR + lane) * VE;
        wv[i] = load_group<W, VE>(w + c, w ? width - c : 0, (W)1.f);
        bv[i] = load_group<W, VE>(b + c, b ? width - c : 0, (W)0.f);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) s += (float)raw[i].v[e];
    const float mu = row_sum<LPR>(s, red) / n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = c + e < width ? (float)raw[i].v[e] - mu : 0.f;
        q = fmaf(d, d, q);
      }
    }
    const float rs = 1.f / sqrtf(row_sum<LPR>(q, red + SLOTS) / n + eps);
    if (lane == 0 && row < rows) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    T* yr = y + row * width;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      if (have_all - c > 0) {
        Vec16<T> out;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          out.v[e] = (T)fmaf(((float)raw[i].v[e] - mu) * rs, (float)wv[i].v[e], (float)bv[i].v[e]);
        store16_part(yr + c, out, have_all - c);
      }
    }
  }
}

// PARTS: also add up dw and db (part: one row of [dw | db], 2 * width floats,
// per workgroup; a single workgroup writes dw and db themselves).
template <class T, class W, int LPR, int VPL, bool PARTS>
__global__ __launch_bounds__(norm_threads(LPR)) void norm_backward_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ x, int64_t x_stride,
    const W* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
    T* __restrict__ dx, float* __restrict__ part, W* __restrict__ dw, W* __restrict__ db,
    int64_t rows, int width) {
  constexpr int VE = Vec16<T>::n;
  constexpr int NT = norm_threads(LPR);
  constexpr int RPB = NT / LPR;
  constexpr int SLOTS = LPR > 64 ? LPR / 64 : 0;
  __shared__ float2 red[2 * SLOTS + 1];
  bool odd = false;
  const int lane = threadIdx.x % LPR;
  const int sub = threadIdx.x / LPR;
  const float inv_n = 1.f / (float)width;
  float aw[PARTS ? VPL * VE : 1], ab[PARTS ? VPL * VE : 1];
  if constexpr (PARTS) {
#pragma unroll
    for (int i = 0; i < VPL * VE; ++i) aw[i] = ab[i] = 0.f;
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
    const T* xr = x + row * x_stride;
    const T* gr = dy + row * dy_stride;
    Vec16<T> xv[VPL], gv[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      xv[i] = load16_part(xr + c, have_all - c, (T)0.f);
      gv[i] = load16_part(gr + c, have_all - c, (T)0.f);
    }
    const float mu = row < rows ? mean[row] : 0.f;
    const float rs = row < rows ? rstd[row] : 0.f;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        // past the end dy is 0
        const float d = (float)gv[i].v[e];
        const float u = ((float)xv[i].v[e] - mu) * rs;
        const float g = d * (float)wv[i].v[e];
        s.x += g;
        s.y = fmaf(g, u, s.y);
        if constexpr (PARTS) {
          aw[i * VE + e] = fmaf(d, u, aw[i * VE + e]);
          ab[i * VE + e] += d;
        }
      }
    s = row_sum2<LPR>(s, red + (odd ? SLOTS : 0));
    odd = !odd;
    const float m1 = s.x * inv_n, m2 = s.y * inv_n;
    T* dr = dx + row * width;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = (i * LPR + lane) * VE;
      if (have_all - c > 0) {
        Vec16<T> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float u = ((float)xv[i].v[e] - mu) * rs;
          const float g = (float)gv[i].v[e] * (float)wv[i].v[e];
          out.v[e] = (T)(rs * (g - m1 - u * m2));
        }
        store16_part(dr + c, out, have_all - c);
      }
    }
  }
  if constexpr (PARTS) {
    const auto put = [&](int k, int c, float s) {
      if (c >= width) return;
      if (gridDim.x > 1)
        part[((int64_t)blockIdx.x * 2 + k) * width + c] = s;
      else if (k == 0)
        dw[c] = (W)s;
      else if (db)
        db[c] = (W)s;
    };
    // lanes of the same columns: RPB groups of LPR lanes
    if constexpr (RPB > 1) {
      __shared__ float col[RPB > 1 ? NT * VE : 1];
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < VE; ++e)
            col[threadIdx.x * VE + e] = k ? ab[i * VE + e] : aw[i * VE + e];
          __syncthreads();
          for (int t = threadIdx.x; t < LPR * VE; t += NT) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < RPB; ++r) s += col[r * LPR * VE + t];
            put(k, i * LPR * VE + t, s);
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int c = (i * LPR + lane) * VE + e;
          put(0, c, aw[i * VE + e]);
          put(1, c, ab[i * VE + e]);
        }
    }
  }
}

// Rows too wide for the registers: one workgroup of 1024 lanes per row, the
// row read once from memory and twice more from the cache.  Memory bound too.
constexpr int kNormWide = 1024;

template <class T, class W>
__global__ __launch_bounds__(kNormWide) void norm_forward_wide_kernel(
    const T* __restrict__ x, int64_t x_stride, const W* __restrict__ w, const W* __restrict__ b,
    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int width,
    float eps) {
  constexpr int VE = Vec16<T>::n;
  __shared__ float2 red[2 * kNormWide / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * x_stride;
  T* yr = y + row * width;
  const float n = (float)width;
  float s = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> v = load16_part(xr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) s += (float)v.v[e];
  }
  const float mu = row_sum<kNormWide>(s, red) / n;
  float q = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> v = load16_part(xr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float d = c + e < width ? (float)v.v[e] - mu : 0.f;
      q = fmaf(d, d, q);
    }
  }
  const float rs = 1.f / sqrtf(row_sum<kNormWide>(q, red + kNormWide / 64) / n + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    Vec16<T> v = load16_part(xr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int ce = c + e < width ? c + e : c;
      float u = ((float)v.v[e] - mu) * rs;
      if (w) u = fmaf(u, (float)w[ce], b ? (float)b[ce] : 0.f);
      v.v[e] = (T)u;
    }
    store16_part(yr + c, v, width - c);
  }
}

template <class T, class W>
__global__ __launch_bounds__(kNormWide) void norm_backward_wide_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ x, int64_t x_stride,
    const W* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
    T* __restrict__ dx, int64_t rows, int width) {
  constexpr int VE = Vec16<T>::n;
  __shared__ float2 red[2 * kNormWide / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * x_stride;
  const T* gr = dy + row * dy_stride;
  T* dr = dx + row * width;
  const float inv_n = 1.f / (float)width, mu = mean[row], rs = rstd[row];
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> xv = load16_part(xr + c, width - c, (T)0.f);
    const Vec16<T> gv = load16_part(gr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if (c + e < width) {
        const float g = (float)gv.v[e] * (w ? (float)w[c + e] : 1.f);
        s.x += g;
        s.y = fmaf(g, ((float)xv.v[e] - mu) * rs, s.y);
      }
    }
  }
  s = row_sum2<kNormWide>(s, red);
  const float m1 = s.x * inv_n, m2 = s.y * inv_n;
#pragma unroll 1
  for (int c = threadIdx.x * VE; c < width; c += kNormWide * VE) {
    const Vec16<T> xv = load16_part(xr + c, width - c, (T)0.f);
    Vec16<T> gv = load16_part(gr + c, width - c, (T)0.f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int ce = c + e < width ? c + e : c;
      const float g = (float)gv.v[e] * (w ? (float)w[ce] : 1.f);
      gv.v[e] = (T)(rs * (g - m1 - ((float)xv.v[e] - mu) * rs * m2));
    }
    store16_part(dr + c, gv, width - c);
  }
}

// Column sums of dy * u and dy for widths whose accumulators do not fit the
// registers beside the row: one thread per column, a block of rows per
// workgroup, the same partial layout.
template <class T>
__global__ __launch_bounds__(kNormThreads) void norm_columns_kernel(
    const T* __restrict__ dy, int64_t dy_stride, const T* __restrict__ x, int64_t x_stride,
    const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part,
    int64_t rows, int width) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= width) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const float d = (float)dy[r * dy_stride + c];
    aw = fmaf(d, ((float)x[r * x_stride + c] - mean[r]) * rstd[r], aw);
    ab += d;
  }
  part[((int64_t)blockIdx.y * 2 + 0) * width + c] = aw;
  part[((int64_t)blockIdx.y * 2 + 1) * width + c] = ab;
}

// Adds the workgroups' partial rows: 64 columns of [dw | db] per workgroup,
// 16 lanes sets of every 16th partial, then over the sets.
template <class W>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part,
                                                           int parts, W* __restrict__ dw,
                                                           W* __restrict__ db, int width) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, set = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const bool in = c < 2 * (int64_t)width;
  float s = 0.f;
  if (in) {
    const float* q = part + c;
    const int64_t row = 2 * (int64_t)width;
    int p = set;
    // eight loads on their way at a time
    for (; p + 112 < parts; p += 128) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = q[(p + 16 * k) * row];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; p < parts; p += 16) s += q[p * row];
  }
  red[set][lane] = s;
  __syncthreads();
  if (set == 0 && in) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += red[k][lane];
    if (c < width)
      dw[c] = (W)t;
    else if (db)
      db[c - width] = (W)t;
  }
}

template <class T, class W>
int norm_forward_t(const NormForward& a) {
  constexpr int VE = Vec16<T>::n;
  const NormShape s = norm_shape(a.width, VE);
#define FM_NORM_FWD(L, V)                                                                     \
  if constexpr (V * VE <= norm_most(L))                                                                 \
    if (s.lpr == L && s.vpl == V) {                                                           \
      const int64_t need = (a.rows + norm_rows(L) - 1) / norm_rows(L);                        \
      return launch("layer norm forward", norm_forward_kernel<T, W, L, V>,                    \
                    dim3((unsigned)(need < kNormBlocks ? need : kNormBlocks)),                \
                    dim3(norm_threads(L)), 0, a.stream, (const T*)a.x, a.x_stride,            \
                    (const W*)a.weight, (const W*)a.bias, (T*)a.y, a.mean, a.rstd, a.rows,    \
                    a.width, a.eps);                                                          \
    }
  FM_NORM_SHAPES(FM_NORM_FWD)
#undef FM_NORM_FWD
  return by_rows(a.rows, kGridThreads / kNormWide, [&](int64_t at, int64_t rows) {
    return launch("layer norm forward", norm_forward_wide_kernel<T, W>, dim3((unsigned)rows),
                  dim3(kNormWide), 0, a.stream, (const T*)a.x + at * a.x_stride, a.x_stride,
                  (const W*)a.weight, (const W*)a.bias, (T*)a.y + at * a.width,
                  a.mean ? a.mean + at : nullptr, a.rstd ? a.rstd + at : nullptr, rows, a.width, a.eps);
  });
}

template <class T, class W>
int norm_backward_t(const NormBackward& a) {
  constexpr int VE = Vec16<T>::n;
  const NormShape s = norm_shape(a.width, VE);
  const int parts = norm_parts(a.rows, a.width, VE);
  const bool want = a.dw != nullptr;
  float* part = (float*)a.workspace;
  if (a.rows > 0) {
    int st = FM_OK;
    if (s.vpl == 0)
      st = by_rows(a.rows, kGridThreads / kNormWide, [&](int64_t at, int64_t rows) {
        return launch("layer norm backward", norm_backward_wide_kernel<T, W>, dim3((unsigned)rows),
                      dim3(kNormWide), 0, a.stream, (const T*)a.dy + at * a.dy_stride, a.dy_stride,
                      (const T*)a.x + at * a.x_stride, a.x_stride, (const W*)a.weight, a.mean + at,
                      a.rstd + at, (T*)a.dx + at * a.width, rows, a.width);
      });
#define FM_NORM_BWD(L, V)                                                                      \
  if constexpr (V * VE <= norm_most(L))                                                                  \
    if (s.lpr == L && s.vpl == V)                                                              \
      st = launch("layer norm backward",                                                       \
                  want ? norm_backward_kernel<T, W, L, V, true>                                \
                       : norm_backward_kernel<T, W, L, V, false>,                              \
                  dim3((unsigned)parts), dim3(norm_threads(L)), 0, a.stream, (const T*)a.dy,   \
                  a.dy_stride, (const T*)a.x, a.x_stride, (const W*)a.weight, a.mean, a.rstd,  \
                  (T*)a.dx, part, (W*)a.dw, (W*)a.db, a.rows, a.width);
    FM_NORM_SHAPES(FM_NORM_BWD)
#undef FM_NORM_BWD
    if (st != FM_OK) return st;
    if (want && s.vpl == 0) {
      st = launch("layer norm backward columns", norm_columns_kernel<T>,
                  dim3((a.width + kNormThreads - 1) / kNormThreads, parts), dim3(kNormThreads), 0,
                  a.stream, (const T*)a.dy, a.dy_stride, (const T*)a.x, a.x_stride, a.mean, a.rstd,
                  part, a.rows, a.width);
      if (st != FM_OK) return st;
    }
  }
  if (!want || norm_single(a.rows, a.width, VE)) return FM_OK;
  const int64_t cols = 2 * (int64_t)a.width;
  return launch("layer norm backward sums", norm_reduce_kernel<W>, dim3((unsigned)((cols + 63) / 64)),
                dim3(1024), 0, a.stream, part, a.rows > 0 ? parts : 0, (W*)a.dw, (W*)a.db, a.width);
}

}  // namespace fm
