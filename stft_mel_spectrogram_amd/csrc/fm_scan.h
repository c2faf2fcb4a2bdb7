// Gated linear recurrence over time, forward and backward.
//
//   a = sigmoid(f), h_t = a_t h_{t-1} + (1 - a_t) x_t, y_t = h_t silu(g_t)
//   e_t = dy_t silu(g_t), d_t = e_t + m_{t+1}, m_t = a_t d_t (m past the end: the
//   last state's gradient), dx = (1 - a) d, df = dx a (h_{t-1} - x), dg = dy h silu'(g),
//   dstate = m_0.  (a (h_{t-1} - x) is h - x too, but as a difference of two nearly equal
//   numbers where a is small.)
//
// Both directions are the recurrence z = a z' + u, and two successive ranges of
// frames join as (A1, U1), (A2, U2) -> (A1 A2, A2 U1 + U2).  A workgroup takes
// four channels times LC lanes through time, a tile of frames at a time:
// a lane walks R frames, the lanes of a wave that hold the same channels join by
// exchange, the 8 waves through LDS (one barrier a tile), and a second walk with
// what came before writes the results.  So every tensor is read and written once.
// The next tile's loads are on their way while this one is computed.  The
// backward computes h again from the state that the forward kept every 64
// frames.  Few channels are cut into time ranges: a first launch joins each
// range's (A, U), the second one starts from the ranges before.
//
// A group of channels that would cross the end is read four channels before the
// end instead; its lane stores only the channels that are its own.
//
// 16 x 1501 x 2048 bf16 (ragged, with gates): forward 84 us, 328 MB, 3.9 TB/s, the
// vector units busy 61% of the time; backward 170 us, 590 MB, 3.5 TB/s, 58%: memory,
// with the exponentials and the joins of a tile between its loads and its stores.  8 x
// 1501 x 1024: 26 and 54.  In time ranges x and forget cross memory twice: 1 x 100003 x
// 256 f16 22 + 41 us.  1 x 101 x 128 f32: 4.9 and 6.3, one tile; 8 x 1 x 1024 bf16: 3.3.
#pragma once

#include <type_traits>

#include "fm_op.h"
#include "fm_seq.h"

namespace fm {

__device__ __forceinline__ float from_lane(int byte_lane, float v) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(byte_lane, __float_as_int(v)));
}

// exp(-v), off by 2^-24 (1.25 |v| + 2) of itself; the product's rounding (the |v|) is made
// good for inputs in 32 bits, not for gates that have 8 or 11 bits themselves.
template <class T>
__device__ __forceinline__ float exp_minus(float v) {
  const float y = v * -kLog2e;
  float e = __builtin_amdgcn_exp2f(y);
  if constexpr (sizeof(T) == 4) {
    const float lo = fmaf(v, -kLog2e, -y) + v * -1.925963033500649e-8f;  // log2 e in two parts
    // not where e is infinite or 0
    e = fabsf(y) < 126.f ? fmaf(e, lo * kLn2, e) : e;
  }
  return e;
}
// sigmoid and one minus it, each to its own precision (the reciprocal's 2^-23 included).
template <class T>
__device__ __forceinline__ void sigmoids(float v, float& s, float& rest) {
  const float e = exp_minus<T>(v);
  s = __builtin_amdgcn_rcpf(1.f + e);
  rest = e < 1.f ? e * s : 1.f - s;
}

// Four channels of a lane: read from `base`, [own, end) of them written.
constexpr int kScanChannels = 4;
template <class T>
using Quad = Group<T, kScanChannels>;

struct ScanChannels {
  int base, own, end;
  __device__ __forceinline__ ScanChannels(int c, int channels) {
    constexpr int n = kScanChannels;
    const bool whole = channels >= n;
    base = !whole ? 0 : c + n <= channels ? c : channels - n;
    own = c < channels ? c - base : n;
    end = whole ? n : channels;
  }
};
template <class T>
__device__ __forceinline__ Quad<T> scan_pick(bool real, const Quad<T>& v) {
  Quad<T> r;
#pragma unroll
  for (int e = 0; e < kScanChannels; ++e) r.v[e] = real ? v.v[e] : (T)0.f;
  return r;
}

// Four channels as loaded: whole words, which stay as they are while on their way
// (as elements of 16 bits they would take a register each).
template <class T>
struct ScanRaw {
  static constexpr int N = sizeof(T);
  uint32_t w[N];
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[e]);
    } else {
      const uint32_t u = w[e / 2];
      if constexpr (std::is_same<T, bf16_t>::value) {
        return __uint_as_float(e % 2 ? u & 0xffff0000u : u << 16);
      } else {
        const uint16_t h = (uint16_t)(e % 2 ? u >> 16 : u);
        T v;
        __builtin_memcpy(&v, &h, sizeof(v));
        return (float)v;
      }
    }
  }
  // What was made of the words is to be made again.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(w[i]));
  }
  // 0, or +inf, where the frame is not real
  __device__ __forceinline__ void pick(bool real, bool inf) {
    constexpr uint32_t kInf = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, bf16_t>::value ? 0x7f807f80u : 0x7c007c00u;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = real ? w[i] : inf ? kInf : 0u;
  }
};

// A lane's frames of a tensor, tile by tile: a uniform address that moves, and 32
// bits of the lane's own.  TINY: fewer than four channels.
template <class T, bool TINY>
struct ScanRows {
  T* tile;  // first frame of the tile
  int64_t stride;
  uint32_t own;  // elements to the lane's first frame and its channels
  int have;
  __device__ __forceinline__ ScanRows(const void* p, int64_t entry, int64_t entry_stride, int64_t time_stride, int t0,
                                      int mine, int channel, int channels)
      : tile((T*)p + entry * entry_stride + t0 * time_stride), stride(time_stride),
        own((uint32_t)mine * (uint32_t)time_stride + (uint32_t)channel), have(channels - channel) {}
  __device__ __forceinline__ void move(int frames) { tile += frames * stride; }
  __device__ __forceinline__ ScanRaw<T> at(const T* p) const {
    ScanRaw<T> r;
    if constexpr (TINY) {
      const Quad<T> q = load_group<T, kScanChannels>(p, have, (T)0.f);
      __builtin_memcpy(&r, &q, sizeof(r));
    } else {
      __builtin_memcpy(&r, p, sizeof(r));
    }
    return r;
  }
  // the lane's frame r; where it is `past` frames after the last one, that one
  __device__ __forceinline__ ScanRaw<T> load(int r) const { return at(tile + r * stride + own); }
  __device__ __forceinline__ ScanRaw<T> load_last(int r, int past) const {
    return at(tile + r * stride + ((int64_t)own - (past > 0 ? past : 0) * stride));
  }
  __device__ __forceinline__ void store(int r, const Quad<T>& v, const ScanChannels& ch, bool ragged) const {
    T* p = tile + r * stride + own;
    if (!TINY && !ragged) {
      __builtin_memcpy(p, &v, sizeof(v));
    } else {
#pragma unroll
      for (int e = 0; e < kScanChannels; ++e)
        if (e >= ch.own && e < ch.end) p[e] = v.v[e];
    }
  }
};

// Workgroup -> (block of channels, time range, entry).  Blocks of 64-byte rows
// that share a 128-byte line go to the same XCD: workgroups b and b + 8.
template <int ROW>
__device__ __forceinline__ int64_t scan_unit() {
  const unsigned b = blockIdx.x;
  if (ROW == 64 && (b | 15u) < gridDim.x) return (b & ~15u) + 2 * (b & 7u) + (b >> 3 & 1u);
  return b;
}

// What every scan kernel knows about its place.
template <class T, int ROW, int R>
struct ScanPlace {
  static constexpr int VE = kScanChannels, LC = ROW / (int)(VE * sizeof(T)), K = LC * VE, SW = 64 / LC, SPAN = SW * R;
  static constexpr int NW = kScanWaves, TILE = NW * SPAN;
  int lane, wave, slot, time, len, entry, range, beg, end, c0;
  ScanChannels ch;
  bool ragged;    // the block crosses the last channel
  int64_t part;   // of (entry, range 0) and this block's first channel
  int64_t pitch;  // from range to range
  // role of a lane in the carried sums: channel k of the block
  int k, kc;
  bool kown;
  __device__ __forceinline__ explicit ScanPlace(const ScanArgs& a)
      : lane(threadIdx.x & 63), wave(threadIdx.x >> 6), slot(lane / LC), time(a.time), ch(0, 1) {
    const int blocks = (a.channels + K - 1) / K;
    const int64_t unit = scan_unit<ROW>();
    const int64_t at = unit / blocks;
    const int blk = (int)(unit - at * blocks);
    entry = (int)(at / a.splits);
    range = (int)(at - (int64_t)entry * a.splits);
    c0 = blk * K;
    ragged = c0 + K > a.channels;
    ch = ScanChannels(c0 + lane % LC * VE, a.channels);
    len = time;
    if (a.lengths) {
      len = a.lengths[entry];
      len = len < 0 ? 0 : len < time ? len : time;
    }
    beg = range * a.chunk;
    end = time - beg < a.chunk ? time : beg + a.chunk;
    pitch = (int64_t)blocks * K;
    part = (int64_t)entry * a.splits * pitch + c0;
    k = lane < K ? lane : 0;
    const ScanChannels mine(c0 + k / VE * VE, a.channels);
    kc = mine.base + k % VE;
    if (kc >= a.channels) kc = a.channels - 1;
    kown = lane < K && k % VE >= mine.own && k % VE < mine.end;
  }
  __device__ __forceinline__ int64_t state_at(const ScanArgs& a) const { return (int64_t)entry * a.channels + kc; }
};

// Joins ranges 0 .. n - 1 of `part` (A, U), from z = 0 on: threads / K sets of lanes
// a part of the list each.
template <class P>
__device__ __forceinline__ float scan_before(const P& p, const float* part, int n, float2* lds) {
  constexpr int K = P::K, SETS = 64 * P::NW / K;
  const int k = threadIdx.x % K, set = threadIdx.x / K;
  const int per = (n + SETS - 1) / SETS;
  const int lo = set * per, hi = lo + per < n ? lo + per : n;
  float A = 1.f, U = 0.f;
  const float2* q = (const float2*)part + p.part + k;
  for (int i = lo; i < hi; i += 4) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < hi ? q[(i + j) * p.pitch] : make_float2(1.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      U = fmaf(v[j].x, U, v[j].y);
      A *= v[j].x;
    }
  }
  lds[set * K + k] = make_float2(A, U);
  __syncthreads();
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < SETS; ++i) z = fmaf(lds[i * K + p.k].x, z, lds[i * K + p.k].y);
  __syncthreads();
  return z;
}

// Inclusive join over the wave's slots, in time's order (UP) or against it.
template <int LC, int VE, bool UP>
__device__ __forceinline__ void scan_slots(int lane, float (&A)[VE], float (&U)[VE]) {
#pragma unroll
  for (int d = LC; d < 64; d *= 2) {
    const int from = (UP ? lane - d : lane + d) * 4;
    float pa[VE], pu[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      pa[e] = from_lane(from, A[e]);
      pu[e] = from_lane(from, U[e]);
    }
    if (UP ? lane >= d : lane + d < 64) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        U[e] = fmaf(A[e], pu[e], U[e]);
        A[e] *= pa[e];
      }
    }
  }
}
// z of the slots before (UP) or after this one, from z at the wave's border.
template <int LC, int VE, bool UP>
__device__ __forceinline__ void scan_enter(int lane, const float (&A)[VE], const float (&U)[VE],
                                           const float (&border)[VE], float (&z)[VE]) {
  const bool edge = UP ? lane < LC : lane >= 64 - LC;
  const int from = (UP ? lane - LC : lane + LC) * 4;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const float pa = from_lane(from, A[e]), pu = from_lane(from, U[e]);
    z[e] = edge ? border[e] : fmaf(pa, border[e], pu);
  }
}

// a, u (and silu(g)) of a lane's frames, the next tile's loads issued behind each.
// WHOLE: all ranges, writing y; otherwise the sums of all ranges but the last.
template <class T, int ROW, int R, bool GATE, bool WHOLE, bool TINY>
__global__ __launch_bounds__(64 * kScanWaves, (sizeof(T) == 2 && ROW == 128 ? 4 : 1)) void scan_forward_kernel(const ScanArgs a) {
  using P = ScanPlace<T, ROW, R>;
  constexpr int VE = P::VE, LC = P::LC, K = P::K, NW = P::NW;
  const P p(a);
  if (!WHOLE && p.range == a.splits - 1) return;
  __shared__ float2 tot[2][NW][K];
  __shared__ __attribute__((aligned(16))) float cin[NW][K];
  __shared__ float2 sets[WHOLE ? 64 * NW : 1];
  const int mine = p.wave * P::SPAN + p.slot * R;
  using Rows = ScanRows<T, TINY>;
  int t0 = p.beg;
  Rows x(a.x, p.entry, a.xs[0], a.xs[1], t0, mine, p.ch.base, a.channels);
  Rows f(a.f, p.entry, a.fs[0], a.fs[1], t0, mine, p.ch.base, a.channels);
  Rows g(a.g, p.entry, a.gs[0], a.gs[1], t0, mine, p.ch.base, a.channels);
  Rows y(a.y, p.entry, (int64_t)a.time * a.channels, a.channels, t0, mine, p.ch.base, a.channels);

  const int stop = p.len < p.end ? p.len : p.end;
  ScanRaw<T> xv[R], fv[R], gv[R];
  const auto load = [&](int r) {
    xv[r] = x.load(r);
    fv[r] = f.load(r);
    if constexpr (GATE && WHOLE) gv[r] = g.load(r);
  };
  // of the tile at t, which may cross the end
  const auto load_last = [&](int t, int r) {
    const int past = t + mine + r - (stop - 1);
    xv[r] = x.load_last(r, past);
    fv[r] = f.load_last(r, past);
    if constexpr (GATE && WHOLE) gv[r] = g.load_last(r, past);
  };
  const auto move = [&]() {
    x.move(P::TILE);
    f.move(P::TILE);
    g.move(P::TILE);
  };
  if (t0 < stop) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_last(t0, r);
  }
  move();

  // in the role of channel k: the state before the tile, or the range's (A, U) so far
  float carry, carryA = 1.f;
  if (!WHOLE) {
    carry = 0.f;
    // the first state joins the list, so that no workgroup reads it while another writes the last one
    if (p.range == 0 && p.wave == 0 && p.lane < K)
      ((float2*)a.part)[p.part + p.k] = make_float2(0.f, a.state ? a.state[p.state_at(a)] : 0.f);
  } else if (a.splits == 1) {
    carry = a.state ? a.state[p.state_at(a)] : 0.f;
  } else {
    carry = scan_before(p, a.part, p.range + 1, sets);
  }

  int buf = 0;
  // MORE: this tile and the next one are whole
  const auto tile = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;
    float av[R][VE], uv[R][VE], gs[R][GATE && WHOLE ? VE : 1];
    float A[VE], U[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      A[e] = 1.f;
      U[e] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (!MORE) {
        // frames past the end keep the state: a = 1, u = 0
        const bool real = t0 + mine + r < stop;
        xv[r].pick(real, false);
        fv[r].pick(real, true);
        if constexpr (GATE && WHOLE) gv[r].pick(real, false);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float rest;
        sigmoids<T>(fv[r].get(e), av[r][e], rest);
        uv[r][e] = rest * xv[r].get(e);
        U[e] = fmaf(av[r][e], U[e], uv[r][e]);
        A[e] *= av[r][e];
        if constexpr (GATE && WHOLE) {
          const float gg = gv[r].get(e);
          gs[r][e] = gg * __builtin_amdgcn_rcpf(1.f + exp_minus<T>(gg));
        }
      }
      if constexpr (MORE) load(r);
    }
    if constexpr (!MORE) {
      if (t0 + P::TILE < stop) {
#pragma unroll
        for (int r = 0; r < R; ++r) load_last(t0 + P::TILE, r);
      }
    }
    move();
    scan_slots<LC, VE, true>(p.lane, A, U);
    if (p.slot == P::SW - 1) {
#pragma unroll
      for (int e = 0; e < VE; ++e) tot[buf][p.wave][p.lane % LC * VE + e] = make_float2(A[e], U[e]);
    }
    __syncthreads();
    float before = 0.f;
#pragma unroll 2
    for (int w = 0; w < NW; ++w) {
      const float2 v = tot[buf][w][p.k];
      if (w == p.wave) before = carry;
      carry = fmaf(v.x, carry, v.y);
      if (!WHOLE) carryA *= v.x;
    }
    if constexpr (WHOLE) {
      const int first = t0 + p.wave * P::SPAN;
      if (a.saved && p.kown && first % kScanSave == 0 && first < p.time)
        a.saved[((int64_t)p.entry * ((a.time + kScanSave - 1) / kScanSave) + first / kScanSave) * a.channels + p.kc] =
            before;
      wave_lds_fence();
      if (p.lane < K) cin[p.wave][p.k] = before;
      wave_lds_fence();
      float border[VE], h[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) border[e] = cin[p.wave][p.lane % LC * VE + e];
      scan_enter<LC, VE, true>(p.lane, A, U, border, h);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int t = t0 + mine + r;
        Quad<T> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          h[e] = fmaf(av[r][e], h[e], uv[r][e]);
          float o = h[e];
          if constexpr (GATE) o *= gs[r][e];
          out.v[e] = (T)o;
        }
        if constexpr (MORE)
          y.store(r, out, p.ch, p.ragged);
        else if (t < p.end)
          y.store(r, scan_pick(t < stop, out), p.ch, p.ragged);
      }
      y.move(P::TILE);
    }
    buf ^= 1;
    t0 += P::TILE;
  };
  while (t0 + 2 * P::TILE <= stop) tile(std::true_type{});
  while (t0 < stop) tile(std::false_type{});
  if constexpr (WHOLE) {
    // tiles past the length
    Quad<T> zero;
#pragma unroll
    for (int e = 0; e < VE; ++e) zero.v[e] = (T)0.f;
    for (; t0 < p.end; t0 += P::TILE) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (t0 + mine + r < p.end) y.store(r, zero, p.ch, p.ragged);
      y.move(P::TILE);
    }
    if (p.range == a.splits - 1 && p.wave == 0 && p.kown) a.last[p.state_at(a)] = carry;
  } else {
    if (p.wave == 0 && p.lane < K)
      ((float2*)a.part)[p.part + (p.range + 1) * p.pitch + p.k] = make_float2(carryA, carry);
  }
}

// One thread takes four channels of an entry through all frames.
template <class T>
__global__ __launch_bounds__(64) void scan_step_kernel(const ScanArgs a) {
  constexpr int VE = kScanChannels;
  const int groups = (a.channels + VE - 1) / VE;
  const int64_t at = (int64_t)blockIdx.x * 64 + threadIdx.x;
  const int64_t entry = at / groups;
  if (entry >= a.batch) return;
  const int c = (int)(at - entry * groups) * VE, have = a.channels - c;
  int len = a.time;
  if (a.lengths) {
    len = a.lengths[entry];
    len = len < 0 ? 0 : len < a.time ? len : a.time;
  }
  const T* x = (const T*)a.x + entry * a.xs[0] + c;
  const T* f = (const T*)a.f + entry * a.fs[0] + c;
  const T* g = a.g ? (const T*)a.g + entry * a.gs[0] + c : nullptr;
  T* y = (T*)a.y + entry * a.time * a.channels + c;
  Group<float, VE> h = load_group<float, VE>(a.state + entry * a.channels + c, a.state ? have : 0, 0.f);
  for (int t = 0; t < a.time; ++t) {
    const int n = t < len ? have : 0;
    const Quad<T> xv = load_group<T, VE>(x + t * a.xs[1], n, (T)0.f), fv = load_group<T, VE>(f + t * a.fs[1], n, (T)INFINITY);
    Quad<T> gv = {};
    if (g) gv = load_group<T, VE>(g + t * a.gs[1], n, (T)0.f);
    Quad<T> out;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      float s, rest;
      sigmoids<T>((float)fv.v[e], s, rest);
      h.v[e] = fmaf(s, h.v[e], rest * (float)xv.v[e]);
      float o = h.v[e];
      if (g) {
        const float gg = (float)gv.v[e];
        o *= gg * __builtin_amdgcn_rcpf(1.f + exp_minus<T>(gg));
      }
      out.v[e] = (T)(t < len ? o : 0.f);
    }
    T* to = y + (int64_t)t * a.channels;
    if (have >= VE) {
      __builtin_memcpy(to, &out, sizeof(out));
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e < have) to[e] = out.v[e];
    }
  }
  float* last = a.last + entry * a.channels + c;
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (e < have) last[e] = h.v[e];
}

// WHOLE: the gradients; otherwise the sums (A, m) of all ranges but the first.
// Ranges count from the end of time.
template <class T, int ROW, int R, bool GATE, bool WHOLE, bool TINY>
__global__ __launch_bounds__(64 * kScanWaves, (sizeof(T) == 2 && ROW == 128 ? 4 : 1)) void scan_backward_kernel(const ScanArgs a) {
  using P = ScanPlace<T, ROW, R>;
  constexpr int VE = P::VE, LC = P::LC, K = P::K, NW = P::NW;
  static_assert(P::TILE % kScanSave == 0, "a tile starts where a state was kept");
  const P p(a);
  if (!WHOLE && p.range == 0) return;
  const int back = a.splits - 1 - p.range;
  __shared__ float2 tot[2][NW][K];
  __shared__ float totm[2][NW][K];
  __shared__ __attribute__((aligned(16))) float cin[NW][2][K];
  __shared__ float2 sets[WHOLE ? 64 * NW : 1];
  const int mine = p.wave * P::SPAN + p.slot * R;
  using Rows = ScanRows<T, TINY>;
  const int stop = p.len < p.end ? p.len : p.end;
  const int tiles = stop > p.beg ? (stop - p.beg + P::TILE - 1) / P::TILE : 0;
  int t0 = p.beg + tiles * P::TILE;  // behind the last tile
  const int64_t whole = (int64_t)a.time * a.channels;
  Rows dx(a.dx, p.entry, whole, a.channels, t0, mine, p.ch.base, a.channels);
  Rows df(a.df, p.entry, whole, a.channels, t0, mine, p.ch.base, a.channels);
  Rows dg(a.dg, p.entry, whole, a.channels, t0, mine, p.ch.base, a.channels);
  const auto put = [&](int r, const Quad<T>& ox, const Quad<T>& of, const Quad<T>& og) {
    dx.store(r, ox, p.ch, p.ragged);
    df.store(r, of, p.ch, p.ragged);
    if constexpr (GATE) dg.store(r, og, p.ch, p.ragged);
  };
  const auto move_out = [&](int frames) {
    dx.move(frames);
    df.move(frames);
    dg.move(frames);
  };
  if constexpr (WHOLE) {
    // tiles past the length
    Quad<T> zero;
#pragma unroll
    for (int e = 0; e < VE; ++e) zero.v[e] = (T)0.f;
    int t = t0;
    for (; t < p.end; t += P::TILE) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (t + mine + r < p.end) put(r, zero, zero, zero);
      move_out(P::TILE);
    }
    move_out(t0 - t);
  }

  // in the role of channel k: m behind the tile
  float carry, carryA = 1.f;
  if (!WHOLE) {
    carry = 0.f;
    if (back == 0 && p.wave == 0 && p.lane < K)
      ((float2*)a.part)[p.part + p.k] = make_float2(0.f, a.dlast ? a.dlast[p.state_at(a)] : 0.f);
  } else if (a.splits == 1) {
    carry = a.dlast ? a.dlast[p.state_at(a)] : 0.f;
  } else {
    carry = scan_before(p, a.part, back + 1, sets);
  }

  t0 -= P::TILE;
  move_out(-P::TILE);
  Rows x(a.x, p.entry, a.xs[0], a.xs[1], t0, mine, p.ch.base, a.channels);
  Rows f(a.f, p.entry, a.fs[0], a.fs[1], t0, mine, p.ch.base, a.channels);
  Rows g(a.g, p.entry, a.gs[0], a.gs[1], t0, mine, p.ch.base, a.channels);
  Rows dy(a.dy, p.entry, a.dys[0], a.dys[1], t0, mine, p.ch.base, a.channels);
  const float* saved = a.saved + (int64_t)p.entry * ((a.time + kScanSave - 1) / kScanSave) * a.channels;
  ScanRaw<T> xv[R], fv[R], gv[R], dv[R];
  float kept = 0.f;
  const auto load = [&](int r) {
    if constexpr (WHOLE) xv[r] = x.load(r);
    fv[r] = f.load(r);
    if constexpr (GATE) gv[r] = g.load(r);
    dv[r] = dy.load(r);
  };
  const auto move = [&]() {
    x.move(-P::TILE);
    f.move(-P::TILE);
    g.move(-P::TILE);
    dy.move(-P::TILE);
  };
  if (tiles > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int past = t0 + mine + r - (stop - 1);
      if constexpr (WHOLE) xv[r] = x.load_last(r, past);
      fv[r] = f.load_last(r, past);
      if constexpr (GATE) gv[r] = g.load_last(r, past);
      dv[r] = dy.load_last(r, past);
    }
    if constexpr (WHOLE) kept = (saved + (int64_t)(t0 / kScanSave) * a.channels)[(uint32_t)p.kc];
  }
  move();
  int buf = 0;
  // FULL: all frames of this tile; only the first one may have fewer
  const auto tile = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    float av[R][VE], rest[R][VE], ev[R][VE], gd[R][GATE ? VE : 1];
    ScanRaw<T> xr[R];
    float A[VE], U[VE], B[VE], M[VE];
    const float state = kept;
    const bool more = t0 > p.beg;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (!FULL) {
        const bool real = t0 + mine + r < stop;
        if constexpr (WHOLE) xv[r].pick(real, false);
        fv[r].pick(real, true);
        if constexpr (GATE) gv[r].pick(real, false);
        dv[r].pick(real, false);
      }
      if constexpr (WHOLE) xr[r] = xv[r];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        sigmoids<T>(fv[r].get(e), av[r][e], rest[r][e]);
        const float d = dv[r].get(e);
        ev[r][e] = d;
        if constexpr (GATE) {
          const float gg = gv[r].get(e);
          const float sg = __builtin_amdgcn_rcpf(1.f + exp_minus<T>(gg));
          const float sl = gg * sg;
          ev[r][e] = d * sl;
          gd[r][e] = d * fmaf(sl, 1.f - sg, sg);  // dy silu'(g)
        }
      }
    }
    if (more) {
#pragma unroll
      for (int r = 0; r < R; ++r) load(r);
      if constexpr (WHOLE) kept = (saved + (int64_t)((t0 - P::TILE) / kScanSave) * a.channels)[(uint32_t)p.kc];
    }
    move();
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      A[e] = 1.f;
      U[e] = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (WHOLE) U[e] = fmaf(av[r][e], U[e], rest[r][e] * xr[r].get(e));
        A[e] *= av[r][e];
      }
      B[e] = A[e];
    }
    if constexpr (WHOLE) {
      scan_slots<LC, VE, true>(p.lane, A, U);
      if (p.slot == P::SW - 1) {
#pragma unroll
        for (int e = 0; e < VE; ++e) tot[buf][p.wave][p.lane % LC * VE + e] = make_float2(A[e], U[e]);
      }
      // one direction after the other: both at once take more registers than there are
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      M[e] = 0.f;
#pragma unroll
      for (int r = R - 1; r >= 0; --r) M[e] = av[r][e] * (ev[r][e] + M[e]);
    }
    scan_slots<LC, VE, false>(p.lane, B, M);
    if (p.slot == 0) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (!WHOLE) tot[buf][p.wave][p.lane % LC * VE + e].x = B[e];
        totm[buf][p.wave][p.lane % LC * VE + e] = M[e];
      }
    }
    __syncthreads();
    float behind = 0.f;
#pragma unroll 1
    for (int w = NW - 1; w >= 0; --w) {
      const float va = tot[buf][w][p.k].x;
      if (w == p.wave) behind = carry;
      carry = fmaf(va, carry, totm[buf][w][p.k]);
      if (!WHOLE) carryA *= va;
    }
    if constexpr (WHOLE) {
      float before = state;
#pragma unroll 1
      for (int w = 0; w < p.wave; ++w) {
        const float2 v = tot[buf][w][p.k];
        if (w < p.wave) before = fmaf(v.x, before, v.y);
      }
      wave_lds_fence();
      if (p.lane < K) {
        cin[p.wave][0][p.k] = before;
        cin[p.wave][1][p.k] = behind;
      }
      wave_lds_fence();
      float border[VE], h[VE], m[VE], hs[R][VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) border[e] = cin[p.wave][0][p.lane % LC * VE + e];
      scan_enter<LC, VE, true>(p.lane, A, U, border, h);
#pragma unroll
      for (int e = 0; e < VE; ++e) border[e] = cin[p.wave][1][p.lane % LC * VE + e];
      scan_enter<LC, VE, false>(p.lane, B, M, border, m);
      // x is unpacked again rather than kept in registers since the first walk
#pragma unroll
      for (int r = 0; r < R; ++r) xr[r].forget();
      // hs: a (h - x) of the state before the frame, and dg in place of dy silu'(g)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float xe = xr[r].get(e);
          hs[r][e] = av[r][e] * (h[e] - xe);
          h[e] = fmaf(av[r][e], h[e], rest[r][e] * xe);
          if constexpr (GATE) gd[r][e] *= h[e];
        }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        const int t = t0 + mine + r;
        Quad<T> ox, of, og;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float d = ev[r][e] + m[e];
          const float u = rest[r][e] * d;
          m[e] = av[r][e] * d;
          ox.v[e] = (T)u;
          of.v[e] = (T)(u * hs[r][e]);
          if constexpr (GATE) og.v[e] = (T)gd[r][e];
        }
        if constexpr (FULL) {
          put(r, ox, of, og);
        } else if (t < p.end) {
          // rest is 0 past the end, but the state need not be finite
          const bool real = t < stop;
          put(r, scan_pick(real, ox), scan_pick(real, of), GATE ? scan_pick(real, og) : ox);
        }
      }
      move_out(-P::TILE);
    }
    buf ^= 1;
    t0 -= P::TILE;
  };
  if (tiles > 0 && t0 + P::TILE > stop) tile(std::false_type{});
  while (t0 >= p.beg) tile(std::true_type{});
  if constexpr (WHOLE) {
    if (a.dstate && p.range == 0 && p.wave == 0 && p.kown) a.dstate[p.state_at(a)] = carry;
  } else {
    if (p.wave == 0 && p.lane < K)
      ((float2*)a.part)[p.part + (back + 1) * p.pitch + p.k] = make_float2(carryA, carry);
  }
}

template <class T>
int scan_forward_t(ScanArgs a, void* stream) {
  constexpr int VE = kScanChannels;
  if (scan_steps(a)) {
    const int64_t n = (int64_t)a.batch * ((a.channels + VE - 1) / VE);
    return launch("gated recurrence", scan_step_kernel<T>, dim3((unsigned)((n + 63) / 64)), dim3(64), 0, stream, a);
  }
  const ScanSplit s = scan_split(a.batch, a.time, a.channels, sizeof(T), false);
  a.splits = s.splits;
  a.chunk = s.chunk;
  const int64_t units = a.batch * scan_blocks(a.channels, s.row, sizeof(T));
  const auto go = [&](auto kernel) {
    return launch("gated recurrence", kernel, dim3((unsigned)(units * s.splits)), dim3(64 * kScanWaves), 0, stream, a);
  };
#define FM_SCAN_FWD(L, R, TINY)                                                     \
  if (s.row == L && s.frames == R && (a.channels < kScanChannels) == TINY) {        \
    if (s.splits > 1)                                                               \
      if (int st = go(scan_forward_kernel<T, L, R, false, false, TINY>)) return st; \
    return a.g ? go(scan_forward_kernel<T, L, R, true, true, TINY>)                 \
               : go(scan_forward_kernel<T, L, R, false, true, TINY>);               \
  }
  FM_SCAN_FWD(128, 2, false)
  FM_SCAN_FWD(128, 4, false)
  if constexpr (sizeof(T) == 4) {
    FM_SCAN_FWD(64, 2, false)
  } else {
    FM_SCAN_FWD(64, 4, false)
  }
  FM_SCAN_FWD(64, 1, true)
#undef FM_SCAN_FWD
  return set_error(FM_E_UNSUPPORTED, "gated recurrence: no kernel for this shape");
}

template <class T>
int scan_backward_t(ScanArgs a, void* stream) {
  const ScanSplit s = scan_split(a.batch, a.time, a.channels, sizeof(T), true);
  a.splits = s.splits;
  a.chunk = s.chunk;
  const int64_t units = a.batch * scan_blocks(a.channels, s.row, sizeof(T));
  const auto go = [&](auto kernel) {
    return launch("gated recurrence backward", kernel, dim3((unsigned)(units * s.splits)), dim3(64 * kScanWaves), 0,
                  stream, a);
  };
#define FM_SCAN_BWD(L, R, TINY)                                                 \
  if (s.row == L && s.frames == R && (a.channels < kScanChannels) == TINY) {    \
    if (s.splits > 1)                                                           \
      if (int st = a.g ? go(scan_backward_kernel<T, L, R, true, false, TINY>)   \
                       : go(scan_backward_kernel<T, L, R, false, false, TINY>)) \
        return st;                                                              \
    return a.g ? go(scan_backward_kernel<T, L, R, true, true, TINY>)            \
               : go(scan_backward_kernel<T, L, R, false, true, TINY>);          \
  }
  FM_SCAN_BWD(128, 2, false)
  if constexpr (sizeof(T) == 4) {
    FM_SCAN_BWD(64, 2, false)
  }
  FM_SCAN_BWD(64, 1, true)
#undef FM_SCAN_BWD
  return set_error(FM_E_UNSUPPORTED, "gated recurrence: no kernel for this shape");
}

}  // namespace fm
