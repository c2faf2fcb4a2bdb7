// Log probabilities of given tokens with entropy and top alternatives, and
// the logits' gradient.
//
//   lse = log sum exp(x),  lp_t = x_t - lse,  H = lse - sum p x = log s - t / s
//   with s = sum exp(x - m), t = sum exp(x - m) (x - m), m = max x
//   dx_j = sum of g over the named tokens equal to j - p_j (sum of all g)
//          - g_H p_j (lp_j + H)
//
// One pass over the logits: every lane keeps a running maximum with the two
// sums in float32 and rescales them when a register chunk raises it; the
// lanes' triples are joined in a fixed order.  Entries of -inf have p = 0 and
// add nothing to the entropy; NaN anywhere in a row makes its results NaN.
// A row of -inf only has lp = -inf, H = 0 and a zero gradient.
//
// Top alternatives: entries are 64-bit keys (value in an ordered integer, then
// the complement of the index, so that ties go to the lower index).  A wave
// collects candidates in LDS: of its first chunk those that reach a value which
// at least `top` of its lanes' maxima reach, of later ones those that beat the
// last one kept.  From time to time each candidate counts the larger ones, which
// is its place in the sorted list; the first `top` stay.
//
// Memory bound.  A row that 16 or 64 lanes hold in registers is read once, its
// maximum taken first.  Longer rows go through 4 waves chunk by chunk (8 waves
// per SIMD hide the loads better than a chunk fetched ahead: 75 us against 80 at
// 4096 x 32000 bf16); few of them are cut into segments, one workgroup each,
// whose partial results a second launch joins.  4096 x 32000 bf16: forward 73 us
// (3.6 TB/s), with 5 and 20 alternatives 74 and 92, backward 115 (4.6 TB/s); 24008 x
// 129 f32: 5.4 and 8.3 us.
#pragma once

#include "fm_op.h"

namespace fm {

typedef unsigned long long key_t;

__device__ __forceinline__ key_t score_key(float x, int idx) {
  uint32_t b = __float_as_uint(x);
  if (x == 0.f) b = 0;  // -0 ranks as 0
  b = (b >> 31) ? ~b : (b | 0x80000000u);
  return ((key_t)b << 32) | (uint32_t)~(uint32_t)idx;
}
__device__ __forceinline__ float key_value(key_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b >> 31) ? (b & 0x7fffffffu) : ~b);
}
__device__ __forceinline__ int key_index(key_t k) { return (int)~(uint32_t)k; }

// The candidates of a wave for the `top` largest keys.
struct TopKeys {
  static constexpr int kRoom = 128;
  static constexpr int kSize = kRoom + 4;  // keys of LDS
  key_t* buf;
  int top, lane;
  int count = 0;
  key_t last = 0;                // the least key kept, once there are `top`
  float bar = -INFINITY;         // entries below it need not be looked at

  // Sorts what there is and keeps the first `top`.
  __device__ __forceinline__ void prune() {
    if (lane < 4) buf[count + lane] = 0;
    wave_lds_fence();
    const key_t a = lane < count ? buf[lane] : 0, b = 64 + lane < count ? buf[64 + lane] : 0;
    int ra = 0, rb = 0;
    for (int i = 0; i < count; i += 4) {
      key_t k[4];
      __builtin_memcpy(k, buf + i, sizeof(k));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ra += k[j] > a;
        rb += k[j] > b;
      }
    }
    wave_lds_fence();
    if (a != 0 && ra < top) buf[ra] = a;
    if (b != 0 && rb < top) buf[rb] = b;
    wave_lds_fence();
    if (count < top) return;
    count = top;
    last = buf[top - 1];
    // later entries have higher indices: they have to be larger
    const uint32_t hi = (uint32_t)(last >> 32) + 1;
    bar = key_value((key_t)hi << 32);
  }
  __device__ __forceinline__ void push(bool real, key_t key) {
    const bool in = real && key > last;
    const uint64_t who = __ballot(in);
    if (who == 0) return;
    const int at = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in) buf[at] = key;
    count += __popcll(who);
    if (count > kRoom - 64) prune();
  }
  __device__ __forceinline__ key_t listed() {
    prune();
    return lane < count ? buf[lane] : 0;
  }
};

// A value (as the upper half of a key) that at least `top` of the wave's values
// reach, and few more.
__device__ __forceinline__ uint32_t top_bound(uint32_t o, int top) {
  uint32_t most = wave_umax(o), lo = ~wave_umax(~o);
  if (top == 1) return most;
  uint32_t span = most - lo;  // fewer than `top` reach lo + span + 1
  while (span > 0) {
    const uint32_t step = span / 2 + 1;
    const int n = __popcll(__ballot(o >= lo + step));
    if (n >= top) {
      lo += step;
      span -= step;
      if (n <= top + top / 4 + 2) break;
    } else {
      span = step - 1;
    }
  }
  return lo;
}

// m = max x, s = sum exp2(y), t = sum exp2(y) y of a set of entries, y = (x - m)
// log2 e (x log2 e alone would overflow for masks of the type's lowest value).
// The distance of two maxima is cut at -300: the factor is 0 there, and so must
// its product with the distance be.
struct ScoreSum {
  float m, s, t;
};
__device__ __forceinline__ float score_shift(float from, float to) {
  // a set of -inf has s = t = 0
  return from == -INFINITY ? 0.f : fmaxf((from - to) * kLog2e, -300.f);
}
__device__ __forceinline__ ScoreSum score_join(ScoreSum a, ScoreSum b) {
  const float m = fmaxf(a.m, b.m);
  const float da = score_shift(a.m, m), db = score_shift(b.m, m);
  const float ra = __builtin_amdgcn_exp2f(da), rb = __builtin_amdgcn_exp2f(db);
  return {m, a.s * ra + b.s * rb, (a.t + a.s * da) * ra + (b.t + b.s * db) * rb};
}

// Where a row's logits lie: rows at one stride, or groups of `inner` rows at one
// and the groups at another (a slice of positions out of every entry).
template <class T>
struct ScoreIn {
  const T* x;
  int64_t stride, outer, first;  // row 0 of this launch is row `first`
  uint32_t inner;
  __device__ __forceinline__ const T* row(int64_t r) const {
    r += first;
    if (inner == 0) return x + r * stride;
    const uint32_t g = (uint32_t)r / inner;
    return x + g * outer + (int64_t)((uint32_t)r - g * inner) * stride;
  }
};
template <class T, class A>
ScoreIn<T> score_in(const A& a, int64_t first) {
  return {(const T*)a.x, a.x_stride, a.x_outer, first, (uint32_t)a.x_inner};
}

struct ScoreOut {
  float* lp;
  float* ent;
  float* lse;
  int64_t* top_ids;
  float* top_lp;
};

// Joins the triples of LANES lanes around their common maximum.
template <int LANES>
__device__ __forceinline__ ScoreSum score_join_lanes(ScoreSum a) {
  const float m = lanes_max<LANES>(a.m);
  const float d = score_shift(a.m, m);
  const float r = __builtin_amdgcn_exp2f(d);
  return {m, lanes_sum<LANES>(a.s * r), lanes_sum<LANES>((a.t + a.s * d) * r)};
}

// Writes a row's results: lane 0, and lane i the i-th of the `top` keys.
template <class T>
__device__ __forceinline__ void score_finish(const ScoreSum& r, const T* xr, int64_t row, int vocab,
                                             const void* tokens, int tok64, key_t list, int top,
                                             const ScoreOut& o, int lane) {
  const float log_s = logf(r.s);
  // nothing but -inf; NaN if there was one
  const bool empty = r.m == -INFINITY && r.s == 0.f;
  const auto log_prob = [&](float v) { return empty ? -INFINITY : (v - r.m) - log_s; };
  if (lane == 0) {
    const int64_t t = tok64 ? ((const int64_t*)tokens)[row] : ((const int32_t*)tokens)[row];
    // no token asked for, or none that exists
    if (o.lp) o.lp[row] = t < 0 ? 0.f : t >= vocab ? NAN : log_prob((float)xr[t]);
    if (o.ent) o.ent[row] = empty ? 0.f : fmaf(r.t / r.s, -kLn2, log_s);
    if (o.lse) o.lse[row] = empty ? -INFINITY : r.m == -INFINITY ? NAN : r.m + log_s;
  }
  if (lane < top) {
    o.top_ids[row * top + lane] = key_index(list);
    o.top_lp[row * top + lane] = log_prob(key_value(list));
  }
}

// A register chunk added to s and t, m finite; entries of -inf add 0.
template <class T, int V>
__device__ __forceinline__ void score_add(const Vec16<T> (&v)[V], float m, float& s, float& t) {
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < Vec16<T>::n; ++e) {
      const float y = ((float)v[i].v[e] - m) * kLog2e;
      const float p = __builtin_amdgcn_exp2f(y);
      s += p;
      // p is 0 long before -300, where the product with -inf would be NaN
      t = fmaf(p, fmaxf(y, -300.f), t);
    }
}
template <class T, int V>
__device__ __forceinline__ float score_max(const Vec16<T> (&v)[V]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < Vec16<T>::n; ++e) m = fmaxf(m, (float)v[i].v[e]);
  return m;
}

// A chunk's entries into the candidates (group i starts at c0 + (i * nt + tid) *
// VE), m the lane's largest: marked by a bit each where they pass the bar, then
// read again, every lane's first one, second one, ... at a time.
template <class T, int V>
__device__ __forceinline__ void score_top(const Vec16<T> (&v)[V], const T* xr, float m, int c0, int nt,
                                          int tid, int end, TopKeys& keys) {
  constexpr int VE = Vec16<T>::n;
  if (keys.count == 0) {
    keys.bar = key_value((key_t)top_bound((uint32_t)(score_key(m, 0) >> 32), keys.top) << 32);
  } else if (__ballot(!(m < keys.bar)) == 0) {
    return;
  }
  uint32_t marks = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < VE; ++e)
      marks |= !((float)v[i].v[e] < keys.bar) ? 1u << (i * VE + e) : 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int have = end - (c0 + (i * nt + tid) * VE);
    if (have < VE) marks &= ~(((1u << VE) - (1u << (have > 0 ? have : 0))) << (i * VE));
  }
  while (__ballot(marks != 0)) {
    const int j = marks ? __builtin_ctz(marks) : 0;
    const int c = c0 + (j / VE * nt + tid) * VE + j % VE;
    keys.push(marks != 0, marks ? score_key((float)xr[c], c) : 0);
    marks &= marks - 1;
  }
  if (keys.last == 0 ? keys.count >= keys.top : keys.count >= keys.top + 16) keys.prune();
}

// Rows that L lanes hold, V groups each.
template <class T, int L, int V, bool TOP>
__global__ __launch_bounds__(256) void score_row_kernel(const ScoreIn<T> x,
                                                        const void* __restrict__ tokens, int tok64,
                                                        ScoreOut out, int64_t rows, int vocab,
                                                        int top) {
  constexpr int VE = Vec16<T>::n;
  const int lane = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const T* __restrict__ xr = x.row(row);
  const int end = row < rows ? vocab : 0;
  Vec16<T> v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * L + lane) * VE;
    v[i] = load16_part(xr + c, end - c, (T)-INFINITY);
  }
  ScoreSum r;
  const float most = score_max(v);
  r.m = lanes_max<L>(most);
  float s = 0.f, t = 0.f;
  score_add(v, r.m == -INFINITY ? 0.f : r.m, s, t);
  r.s = lanes_sum<L>(s);
  r.t = lanes_sum<L>(t);
  key_t list = 0;
  if constexpr (TOP) {
    __shared__ __attribute__((aligned(16))) key_t buf[256 / L][TopKeys::kSize];
    TopKeys keys = {buf[threadIdx.x / L], top, lane};
    score_top(v, xr, most, 0, L, lane, end, keys);
    list = keys.listed();
  }
  if (row < rows) score_finish(r, xr, row, vocab, tokens, tok64, list, TOP ? top : 0, out, lane);
}

// 4 waves per row segment.  With several segments, `part` gets (m, s, t) and
// the keys of each.
template <class T, int V, bool TOP>
__global__ __launch_bounds__(256) void score_forward_kernel(
    const ScoreIn<T> x, const void* __restrict__ tokens, int tok64,
    ScoreOut out, float* __restrict__ part, key_t* __restrict__ part_keys, int vocab, int top,
    int seg_len, int segs) {
  constexpr int VE = Vec16<T>::n;
  constexpr int NT = 256, CH = NT * VE * V;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t unit = blockIdx.x;
  const int64_t row = unit / segs;
  const int seg = (int)(unit - row * segs);
  const T* __restrict__ xr = x.row(row);
  const int beg = seg * seg_len;
  const int end = score_segment_end(beg, seg_len, vocab);

  ScoreSum acc = {-INFINITY, 0.f, 0.f};
  __shared__ __attribute__((aligned(16))) key_t buf[TOP ? 4 : 1][TopKeys::kSize];
  TopKeys keys = {buf[TOP ? wave : 0], top, lane};
  for (int c0 = beg; c0 < end; c0 += CH) {
    Vec16<T> v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + (i * NT + tid) * VE;
      v[i] = load16_part(xr + c, end - c, (T)-INFINITY);
    }
    const float most = score_max(v);
    const float m = fmaxf(acc.m, most);
    const float d0 = score_shift(acc.m, m);
    const float r0 = __builtin_amdgcn_exp2f(d0);
    float s = 0.f, t = 0.f;
    score_add(v, m == -INFINITY ? 0.f : m, s, t);
    acc.t = (acc.t + acc.s * d0) * r0 + t;
    acc.s = acc.s * r0 + s;
    acc.m = m;
    if constexpr (TOP) score_top(v, xr, most, c0, NT, tid, end, keys);
  }
  acc = score_join_lanes<64>(acc);
  __shared__ ScoreSum sums[4];
  __shared__ key_t lists[TOP ? 256 : 1];
  if (lane == 0) sums[wave] = acc;
  if constexpr (TOP) lists[tid] = keys.listed();
  __syncthreads();
  if (wave != 0) return;
  acc = sums[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) acc = score_join(acc, sums[w]);
  key_t list = 0;
  if constexpr (TOP) {
    for (int w = 1; w < 4; ++w) keys.push(lists[w * 64 + lane] != 0, lists[w * 64 + lane]);
    list = keys.listed();
  }
  if (segs == 1) {
    score_finish(acc, xr, row, vocab, tokens, tok64, list, TOP ? top : 0, out, lane);
  } else {
    if (lane == 0) {
      part[unit * 3 + 0] = acc.m;
      part[unit * 3 + 1] = acc.s;
      part[unit * 3 + 2] = acc.t;
    }
    if (TOP && lane < top) part_keys[unit * top + lane] = list;
  }
}

// One wave per row: joins the segments in order.
template <class T>
__global__ __launch_bounds__(64) void score_join_kernel(
    const ScoreIn<T> x, const void* __restrict__ tokens, int tok64,
    ScoreOut out, const float* __restrict__ part, const key_t* __restrict__ part_keys, int vocab,
    int top, int segs) {
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  ScoreSum acc = {-INFINITY, 0.f, 0.f};
  for (int s = lane; s < segs; s += 64) {
    const float* p = part + (row * segs + s) * 3;
    acc = score_join(acc, ScoreSum{p[0], p[1], p[2]});
  }
  acc = score_join_lanes<64>(acc);
  key_t list = 0;
  if (top > 0) {
    __shared__ __attribute__((aligned(16))) key_t buf[TopKeys::kSize];
    TopKeys keys = {buf, top, lane};
    const int n = segs * top;
    const key_t* from = part_keys + row * n;
    uint32_t first = 0;  // the segments' best
    for (int s = lane; s < segs; s += 64) {
      const uint32_t hi = (uint32_t)(from[s * top] >> 32);
      first = hi > first ? hi : first;
    }
    const key_t least = (key_t)top_bound(first, top) << 32;
    for (int i0 = 0; i0 < n; i0 += 256) {
      key_t k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = i0 + 64 * j + lane < n ? from[i0 + 64 * j + lane] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) keys.push(k[j] != 0 && k[j] >= least, k[j]);
    }
    list = keys.listed();
  }
  score_finish(acc, x.row(row), row, vocab, tokens, tok64, list, top, out, lane);
}

// dx of one row segment (L = 256), or of whole rows that L < 256 lanes hold
// with V groups each; see the formula above.
template <class T, int L, int V>
__global__ __launch_bounds__(256) void score_backward_kernel(
    const ScoreIn<T> x, const void* __restrict__ tokens, int tok64,
    const float* __restrict__ lse_, const float* __restrict__ ent, const float* __restrict__ g_lp,
    const float* __restrict__ g_ent, const int64_t* __restrict__ top_ids,
    const float* __restrict__ g_top, T* __restrict__ dx, int64_t rows, int vocab, int top,
    int seg_len, int segs) {
  constexpr int VE = Vec16<T>::n;
  const int tid = threadIdx.x % L;
  const int64_t unit = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int64_t row = L == 256 ? unit / segs : unit;
  const int seg = L == 256 ? (int)(unit - row * segs) : 0;
  if (row >= rows) return;
  const T* __restrict__ xr = x.row(row);
  T* dr = dx + row * vocab;
  const int beg = seg * seg_len;
  const int end = score_segment_end(beg, seg_len, vocab);
  Vec16<T> v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = beg + (i * L + tid) * VE;
    v[i] = load16_part(xr + c, end - c, (T)0.f);
  }
  const float lse = lse_[row];
  const bool empty = lse == -INFINITY;
  const float ls = empty ? 0.f : lse;
  int64_t tok = tok64 ? ((const int64_t*)tokens)[row] : ((const int32_t*)tokens)[row];
  if (tok >= vocab) tok = -1;
  const float g = g_lp && tok >= 0 && !empty ? g_lp[row] : 0.f;
  float all = g;
  if (g_top && !empty)
    for (int i = 0; i < top; ++i) all += g_top[row * top + i];
  const float ge = g_ent && !empty ? g_ent[row] : 0.f;
  // -p (g_H (lp + H) + all), y = lp in base 2
  const float slope = -ge * kLn2, base = -(all + (ge != 0.f ? ge * ent[row] : 0.f));
  const auto dense = [&](float xv) {
    const float y = (xv - ls) * kLog2e;
    return __builtin_amdgcn_exp2f(y) * fmaf(slope, y, base);
  };
  // The exponential's results end at 2^-126, but a large gradient may lift smaller
  // probabilities: these are computed 2^64 larger, down to 2^-190.  (For all entries
  // the 64 in the argument would cost their last bits.)  Chunks without such an entry
  // do without the distinction.
  const float tiny = ls - 120.f * kLn2;  // well before 2^-126, as its own rounding goes
  const auto dense_far = [&](float xv) {
    const float y = (xv - ls) * kLog2e;
    const bool small = y < -126.f;
    const float p = __builtin_amdgcn_exp2f(small ? y + 64.f : y);
    return p * fmaf(slope, fmaxf(y, -300.f), base) * (small ? 0x1p-64f : 1.f);
  };
  for (int c0 = beg; c0 < end; c0 += L * VE * V) {
    if (c0 > beg) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + (i * L + tid) * VE;
        v[i] = load16_part(xr + c, end - c, (T)0.f);
      }
    }
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) least = fminf(least, (float)v[i].v[e]);
    const auto put = [&](const auto& f) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + (i * L + tid) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i].v[e] = (T)f((float)v[i].v[e]);
        store16_part(dr + c, v[i], end - c);
      }
    };
    if (__any(least < tiny))
      put(dense_far);
    else
      put(dense);
    if constexpr (L < 256) break;
  }
  // The named tokens' entries, written again by the lane that wrote them
  // above (one thread's stores to one address stay in order), from the
  // unrounded sum.
  const auto named = [&](int64_t j) {
    if (j < beg || j >= end || (int)(((j - beg) / VE) % L) != tid) return;
    float d = dense_far((float)xr[j]);
    if (tok == j) d += g;
    if (g_top)
      for (int i = 0; i < top; ++i)
        if (top_ids[row * top + i] == j) d += g_top[row * top + i];
    dr[j] = (T)d;
  };
  if (empty) return;
  if (tok >= 0) named(tok);
  if (g_top)
    for (int i = 0; i < top; ++i) named(top_ids[row * top + i]);
}

#define FM_SCORE_SHAPES(X) X(16, 1) X(16, 2) X(16, 4) X(64, 2) X(64, 4)
#define FM_SCORE_TOP_SHAPES(X) X(64, 1) X(64, 2) X(64, 4)

// The part of a call from row `at` on.
inline const void* score_tokens(const void* tokens, int tok64, int64_t at) {
  return (const char*)tokens + at * (tok64 ? 8 : 4);
}
template <class P>
P* score_rows(P* p, int64_t at) {
  return p ? p + at : nullptr;
}

template <class T>
int score_forward_t(const ScoreForward& a) {
  const ScoreSplit p = score_split(a.rows, a.vocab, Vec16<T>::n, a.top);
  const auto out_at = [&](int64_t at) {
    return ScoreOut{score_rows(a.lp, at), score_rows(a.ent, at), score_rows(a.lse, at),
                    score_rows(a.top_ids, at * a.top), score_rows(a.top_lp, at * a.top)};
  };
#define FM_SCORE_ROW(L, V, TOP)                                                                    \
  if (p.lanes == L && p.vecs == V)                                                                \
    return by_rows(a.rows, kGridThreads / L, [&](int64_t at, int64_t rows) {                      \
      return launch("token log probabilities", score_row_kernel<T, L, V, TOP>,                    \
                    dim3((unsigned)((rows + 256 / L - 1) / (256 / L))), dim3(256), 0, a.stream,   \
                    score_in<T>(a, at),                                  \
                    score_tokens(a.tokens, a.tok64, at), a.tok64, out_at(at), rows, a.vocab,      \
                    a.top);                                                                       \
    });
#define FM_SCORE_PLAIN_ROW(L, V) FM_SCORE_ROW(L, V, false)
#define FM_SCORE_TOP_ROW(L, V) FM_SCORE_ROW(L, V, true)
  if (a.top == 0) {
    FM_SCORE_SHAPES(FM_SCORE_PLAIN_ROW)
  } else {
    FM_SCORE_TOP_SHAPES(FM_SCORE_TOP_ROW)
  }
#undef FM_SCORE_PLAIN_ROW
#undef FM_SCORE_TOP_ROW
#undef FM_SCORE_ROW
  float* part = (float*)a.workspace;
  key_t* keys = (key_t*)((char*)a.workspace + score_part_bytes(a.rows, p.segs));
  const auto go = [&](auto kernel) {
    return by_rows(a.rows, kGridThreads / 256 / p.segs, [&](int64_t at, int64_t rows) {
      return launch("token log probabilities", kernel, dim3((unsigned)(rows * p.segs)), dim3(256), 0,
                    a.stream, score_in<T>(a, at),
                    score_tokens(a.tokens, a.tok64, at), a.tok64, out_at(at), part + at * p.segs * 3,
                    keys + at * p.segs * a.top, a.vocab, a.top, p.seg_len, p.segs);
    });
  };
  const int st = p.vecs == 1 ? (a.top ? go(score_forward_kernel<T, 1, true>)
                                      : go(score_forward_kernel<T, 1, false>))
                             : (a.top ? go(score_forward_kernel<T, 4, true>)
                                      : go(score_forward_kernel<T, 4, false>));
  if (st != FM_OK || p.segs == 1) return st;
  // few rows: more than one segment each
  return launch("token log probabilities (join)", score_join_kernel<T>, dim3((unsigned)a.rows),
                dim3(64), 0, a.stream, score_in<T>(a, 0), a.tokens, a.tok64, out_at(0), part, keys,
                a.vocab, a.top, p.segs);
}

template <class T>
int score_backward_t(const ScoreBackward& a) {
  const ScoreSplit p = score_split(a.rows, a.vocab, Vec16<T>::n, 0);
#define FM_SCORE_BWD(L, V)                                                                        \
  if (p.lanes == L && (L < 256 ? p.vecs == V : true))                                             \
    return by_rows(a.rows, kGridThreads / L / p.segs, [&](int64_t at, int64_t rows) {             \
      return launch("token log probabilities backward", score_backward_kernel<T, L, V>,           \
                    dim3((unsigned)((rows * p.segs + 256 / L - 1) / (256 / L))), dim3(256), 0,    \
                    a.stream, score_in<T>(a, at),                        \
                    score_tokens(a.tokens, a.tok64, at), a.tok64, a.lse + at,                     \
                    score_rows(a.ent, at), score_rows(a.g_lp, at), score_rows(a.g_ent, at),       \
                    score_rows(a.top_ids, at * a.top), score_rows(a.g_top, at * a.top),           \
                    (T*)a.dx + at * a.vocab, rows, a.vocab, a.top, p.seg_len, p.segs);            \
    });
  FM_SCORE_SHAPES(FM_SCORE_BWD)
  FM_SCORE_BWD(256, 4)
#undef FM_SCORE_BWD
  return set_error(FM_E_UNSUPPORTED, "token log probabilities: no kernel for this shape");
}

}  // namespace fm
