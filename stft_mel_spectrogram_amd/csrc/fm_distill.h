// Distillation from a teacher's top log probabilities: the loss of every row and
// the logits' gradient.
//
//   z = x / T, p = softmax(z), lp = log p
//   loss = T^2 sum_k q_k (log q_k - lp_k),  q = softmax(t / T) over the row's entries
//   dx_j = T g (p_j - [sum of q over the entries equal to j])
// with the rest (T = 1): q = exp(t), r = max(0, 1 - sum q), R the probability of the
// tokens that are not named: loss += r (log r - log R),
//   dx_j = g (S p_j - sum of q) for named ones, g p_j / R (S R - r) for others,
// S = sum q + r.  R is a sum over the tokens that are not named, never 1 minus a
// sum, and r is taken in 64 bits: both may be small.
//
// One pass over the logits with a running maximum and sum, the row layouts of the
// token log probabilities; few long rows are cut into segments that a second
// launch joins.  With the rest the pass leaves out the named tokens: in short rows
// by a bit per token in LDS, in long ones by asking, for every 64 groups of a wave,
// whether one of the entries (one per lane) lies there.  The backward writes the
// others' formula everywhere and then the named tokens again, after a barrier.
// 4096 x 32000 bf16, the best 20 and the rest: forward 78 us (3.4 TB/s, vector units
// busy 67% of the time: twelve instructions per logit, one an exponential), backward 124
// (4.2 TB/s); 24008 x 129 f32, the best 8: 6.7 and 9.6.
#pragma once

#include "fm_logit.h"
#include "fm_score.h"

namespace fm {

// A row's entries in groups of L lanes, E of a lane: entry e * L + lane.  id -1: none.
template <int L, int E>
struct Teacher {
  int id[E];
  float t[E];
  bool lost = false;  // an id past the vocabulary
  __device__ __forceinline__ Teacher(const int64_t* ids, const float* lps, int64_t row, int top, int vocab, int lane,
                                     bool real) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = e * L + lane;
      id[e] = -1;
      t[e] = -INFINITY;
      if (real && k < top) {
        const int64_t j = ids[row * top + k];
        if (j >= vocab) lost = true;
        if (j >= 0 && j < vocab) {
          id[e] = (int)j;
          t[e] = lps[row * top + k];
        }
      }
    }
  }
  // f(k, entry k's id, value v[e] of entry k) for all entries in order.
  template <class F>
  __device__ __forceinline__ void each(int top, const float (&v)[E], F f) const {
#pragma unroll
    for (int e = 0; e < E; ++e)
      for (int l = 0; l < L && e * L + l < top; ++l) f(e * L + l, __shfl(id[e], l, L), __shfl(v[e], l, L));
  }
};
template <int L>
__device__ __forceinline__ bool lanes_any(bool b) {
  return lanes_max<L>(b ? 1.f : 0.f) > 0.f;
}
// A NaN is larger than any number.
template <int L>
__device__ __forceinline__ float lanes_max_nan(float v) {
  return lanes_any<L>(v != v) ? NAN : lanes_max<L>(v);
}

// q of the lane's entries, r, whether the row has a target at all.
template <int L, int E>
struct Target {
  float q[E], logq[E];
  float r = 0.f, sum = 1.f;
  bool none;
};
template <int L, int E, bool REST>
__device__ __forceinline__ Target<L, E> distill_target(const Teacher<L, E>& t, float inv_t) {
  Target<L, E> o;
  bool any = false;
#pragma unroll
  for (int e = 0; e < E; ++e) any |= t.id[e] >= 0;
  o.none = !lanes_any<L>(any);
  if constexpr (REST) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o.logq[e] = t.t[e];
      o.q[e] = t.id[e] >= 0 ? expf(t.t[e]) : 0.f;
      s += t.id[e] >= 0 ? exp((double)t.t[e]) : 0.0;
    }
#pragma unroll
    for (int d = 1; d < L; d *= 2) s += __shfl_xor(s, d, L);
    o.sum = (float)s;
    o.r = s < 1.0 ? (float)(1.0 - s) : 0.f;
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      // a NaN wins
      const float z = t.t[e] * inv_t;
      m = z != z || m != m ? NAN : fmaxf(m, z);
    }
    m = lanes_max_nan<L>(m);
    if (m == -INFINITY) o.none = true;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o.logq[e] = o.none ? -INFINITY : t.t[e] * inv_t - m;
      o.q[e] = t.id[e] >= 0 && !o.none ? expf(o.logq[e]) : 0.f;
      s += o.q[e];
    }
    s = lanes_sum<L>(s);
    const float log_s = logf(s);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o.q[e] /= s;
      o.logq[e] -= log_s;
    }
  }
  return o;
}

// exp((x - m) / T) added up around a maximum m of x itself; m finite or everything is -inf.
struct DistillSum {
  float m, s;
};
// exp((from - to) / T), scale as below: a difference of the maxima as they are, since
// maxima over T would be off by a rounding of their size, not of their distance's.
__device__ __forceinline__ float distill_shift(float from, float to, float2 scale) {
  const float d = from - to;
  // a set of -inf has s = 0
  return from == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(fmaf(d, scale.x, d * scale.y));
}
__device__ __forceinline__ DistillSum distill_join(DistillSum a, DistillSum b, float2 scale) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * distill_shift(a.m, m, scale) + b.s * distill_shift(b.m, m, scale)};
}
template <int L>
__device__ __forceinline__ DistillSum distill_join_lanes(DistillSum a, float2 scale) {
  const float m = lanes_max<L>(a.m);
  return {m, lanes_sum<L>(a.s * distill_shift(a.m, m, scale))};
}
// scale: log2 e / T in two parts (what one alone is off by goes the same way in
// every term, and a loss is a small difference).
template <class T, int V>
__device__ __forceinline__ float distill_add(const Vec16<T> (&v)[V], float m, float2 scale) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < Vec16<T>::n; ++e) {
      const float d = (float)v[i].v[e] - m;
      s += __builtin_amdgcn_exp2f(fmaf(d, scale.x, d * scale.y));
    }
  return s;
}
__device__ __forceinline__ float2 distill_scale(float temperature) {
  const double c = 1.4426950408889634 / (double)temperature;
  float hi = (float)c;
  // the low part above 0: entries of -inf times it are -inf too
  if ((double)hi >= c) hi = __uint_as_float(__float_as_uint(hi) - 1);
  return make_float2(hi, (float)(c - (double)hi));
}

// The row's loss and statistics from `all`, the sum over its tokens (REST: those
// that are not named); m in units of x.
template <class T, int L, int E, bool REST>
__device__ __forceinline__ void distill_finish(DistillSum all, const Teacher<L, E>& t, const T* xr, int64_t row, int top,
                                               float temperature, float inv_t, float* loss, float* stats, int lane) {
  const Target<L, E> q = distill_target<L, E, REST>(t, inv_t);
  float xk[E];
#pragma unroll
  for (int e = 0; e < E; ++e) xk[e] = t.id[e] >= 0 ? (float)xr[t.id[e]] : -INFINITY;
  const float m_rest = all.m, s_rest = all.s;
  if constexpr (REST) {
    // named tokens, each once
    bool again[E];
#pragma unroll
    for (int e = 0; e < E; ++e) again[e] = false;
    t.each(top, xk, [&](int k, int id, float) {
#pragma unroll
      for (int e = 0; e < E; ++e) again[e] |= k < e * L + lane && id == t.id[e];
    });
    float most = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) most = fmaxf(most, xk[e]);
    const float m = fmaxf(all.m, lanes_max<L>(most));
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (t.id[e] >= 0 && !again[e]) s += expf(m == -INFINITY ? -INFINITY : xk[e] - m);
    all.s = all.s * __builtin_amdgcn_exp2f(score_shift(all.m, m)) + lanes_sum<L>(s);
    all.m = m;
  }
  const bool empty = all.m == -INFINITY && all.s == 0.f;
  const float log_s = logf(all.s);
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (t.id[e] >= 0 && q.q[e] != 0.f) sum += q.q[e] * (q.logq[e] - (empty ? -INFINITY : (xk[e] - all.m) * inv_t - log_s));
  sum = lanes_sum<L>(sum);
  if constexpr (REST) {
    if (q.r > 0.f && s_rest != 0.f) {
      // one logarithm of r / R, which may be near 1; two where R is too small for that
      const float share = s_rest * __builtin_amdgcn_exp2f(score_shift(m_rest, all.m)) / all.s;
      sum += q.r * (share > 0x1p-60f ? logf(q.r / share) : logf(q.r) - ((m_rest - all.m) + logf(s_rest) - log_s));
    }
  }
  const bool lost = lanes_any<L>(t.lost);
  if (lane != 0) return;
  loss[row] = lost ? NAN : q.none ? 0.f : sum * temperature * temperature;
  if (stats) {
    // maximum and log sum apart: their sum would lose the latter beside the lowest numbers
    const bool others = REST && s_rest != 0.f;
    stats[4 * row + 0] = empty ? -INFINITY : all.m == -INFINITY ? NAN : all.m;
    stats[4 * row + 1] = empty ? 0.f : log_s;
    stats[4 * row + 2] = !others ? -INFINITY : m_rest == -INFINITY ? NAN : m_rest;
    stats[4 * row + 3] = !others ? 0.f : logf(s_rest);
  }
}

// Rows that L lanes hold, V groups each.
template <class T, int L, int V, int E, bool REST>
__global__ __launch_bounds__(256) void distill_row_kernel(const ScoreIn<T> x, const int64_t* __restrict__ ids,
                                                          const float* __restrict__ lps, float* __restrict__ loss,
                                                          float* __restrict__ stats, int64_t rows, int vocab, int top,
                                                          float temperature, float inv_t) {
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
  const Teacher<L, E> t(ids, lps, row, top, vocab, lane, row < rows);
  if constexpr (REST) {
    // a byte per group of the row, a bit per token
    __shared__ uint32_t named[64 * V];
    uint32_t* mine = named + threadIdx.x / L * (L * V / 4);
#pragma unroll
    for (int i = 0; i < V; ++i) ((uint8_t*)mine)[i * L + lane] = 0;
    wave_lds_fence();
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (t.id[e] >= 0) {
        const int group = t.id[e] / VE;
        atomicOr(mine + group / 4, 1u << (group % 4 * 8 + t.id[e] % VE));
      }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t b = ((uint8_t*)mine)[i * L + lane];
#pragma unroll
      for (int e = 0; e < VE; ++e) v[i].v[e] = b >> e & 1u ? (T)-INFINITY : v[i].v[e];
    }
  }
  DistillSum r;
  r.m = lanes_max<L>(score_max(v));
  r.s = lanes_sum<L>(distill_add(v, r.m == -INFINITY ? 0.f : r.m, distill_scale(temperature)));
  if (row < rows)
    distill_finish<T, L, E, REST>(r, t, xr, row, top, temperature, inv_t, loss, stats, lane);
}

// 4 waves per row segment; with several segments `part` gets (m, s) of each.
template <class T, int V, bool REST>
__global__ __launch_bounds__(256) void distill_forward_kernel(
    const ScoreIn<T> x, const int64_t* __restrict__ ids, const float* __restrict__ lps, float* __restrict__ loss,
    float* __restrict__ stats, float* __restrict__ part, int vocab, int top, float temperature, float inv_t,
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
  const Teacher<64, 1> t(ids, lps, row, top, vocab, lane, REST || wave == 0);
  const float2 scale = distill_scale(temperature);
  DistillSum acc = {-INFINITY, 0.f};
  for (int c0 = beg; c0 < end; c0 += CH) {
    Vec16<T> v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + (i * NT + tid) * VE;
      v[i] = load16_part(xr + c, end - c, (T)-INFINITY);
    }
    if constexpr (REST) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int first = c0 + (i * NT + wave * 64) * VE;
        for (uint64_t who = __ballot((uint32_t)(t.id[0] - first) < 64u * VE && t.id[0] >= 0); who; who &= who - 1) {
          const int at = __builtin_amdgcn_readlane(t.id[0], __builtin_ctzll(who)) - first;
#pragma unroll
          for (int e = 0; e < VE; ++e) v[i].v[e] = at == lane * VE + e ? (T)-INFINITY : v[i].v[e];
        }
      }
    }
    const float m = fmaxf(acc.m, score_max(v));
    acc.s = acc.s * distill_shift(acc.m, m, scale) + distill_add(v, m == -INFINITY ? 0.f : m, scale);
    acc.m = m;
  }
  acc = distill_join_lanes<64>(acc, scale);
  __shared__ DistillSum sums[4];
  if (lane == 0) sums[wave] = acc;
  __syncthreads();
  if (wave != 0) return;
  acc = sums[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) acc = distill_join(acc, sums[w], scale);
  if (segs == 1) {
    distill_finish<T, 64, 1, REST>(acc, t, xr, row, top, temperature, inv_t, loss, stats, lane);
  } else if (lane == 0) {
    part[unit * 2 + 0] = acc.m;
    part[unit * 2 + 1] = acc.s;
  }
}

// One wave per row: joins the segments in order.
template <class T, bool REST>
__global__ __launch_bounds__(64) void distill_join_kernel(
    const ScoreIn<T> x, const int64_t* __restrict__ ids, const float* __restrict__ lps, float* __restrict__ loss,
    float* __restrict__ stats, const float* __restrict__ part, int vocab, int top, float temperature, float inv_t,
    int segs) {
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const Teacher<64, 1> t(ids, lps, row, top, vocab, lane, true);
  const float2 scale = distill_scale(temperature);
  DistillSum acc = {-INFINITY, 0.f};
  for (int s = lane; s < segs; s += 64) {
    const float* p = part + (row * segs + s) * 2;
    acc = distill_join(acc, DistillSum{p[0], p[1]}, scale);
  }
  acc = distill_join_lanes<64>(acc, scale);
  distill_finish<T, 64, 1, REST>(acc, t, x.row(row), row, top, temperature, inv_t, loss, stats, lane);
}

// dx of one row segment (L = 256), or of whole rows that L < 256 lanes hold with V
// groups each.
template <class T, int L, int V, int E, bool REST>
__global__ __launch_bounds__(256) void distill_backward_kernel(
    const ScoreIn<T> x, const int64_t* __restrict__ ids, const float* __restrict__ lps,
    const float* __restrict__ stats, const float* __restrict__ grad, T* __restrict__ dx, int64_t rows, int vocab,
    int top, float temperature, float inv_t, int seg_len, int segs) {
  constexpr int VE = Vec16<T>::n;
  constexpr int LT = L < 64 ? L : 64;  // lanes that hold the teacher's entries
  const int tid = threadIdx.x % L, lane = threadIdx.x % LT;
  const int64_t unit = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int64_t row = L == 256 ? unit / segs : unit;
  const int seg = L == 256 ? (int)(unit - row * segs) : 0;
  const bool real = row < rows;  // a workgroup of one row has one
  const T* __restrict__ xr = x.row(row);
  T* dr = dx + row * vocab;
  const int beg = seg * seg_len;
  const int end = real ? score_segment_end(beg, seg_len, vocab) : 0;
  Vec16<T> v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = beg + (i * L + tid) * VE;
    v[i] = load16_part(xr + c, end - c, (T)0.f);
  }
  const Teacher<LT, E> t(ids, lps, row, top, vocab, lane, real);
  const Target<LT, E> q = distill_target<LT, E, REST>(t, inv_t);
  const float m = real ? stats[4 * row] : 0.f, log_s = real ? stats[4 * row + 1] : 0.f;
  const float g = real ? grad[row] * temperature : 0.f;
  const bool zero = q.none || m == -INFINITY;
  float total = 1.f, most = m, less = log_s, coef = g;
  if constexpr (REST) {
    most = real ? stats[4 * row + 2] : 0.f;
    less = real ? stats[4 * row + 3] : 0.f;
    const bool others = most != -INFINITY;
    total = q.sum + (others ? q.r : 0.f);
    coef = others ? g * (total * expf((most - m) + (less - log_s)) - q.r) : 0.f;
    if (!others) most = 0.f;  // all of them are -inf
  }
  if (zero) coef = most = less = 0.f;
  const float scale = inv_t * kLog2e, shift = -less * kLog2e;
  const auto dense = [&](float xv) {
    return zero ? 0.f : coef * __builtin_amdgcn_exp2f(fmaf(xv - most, scale, shift));
  };
  for (int c0 = beg; c0 < end; c0 += L * VE * V) {
    if (c0 > beg) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + (i * L + tid) * VE;
        v[i] = load16_part(xr + c, end - c, (T)0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + (i * L + tid) * VE;
#pragma unroll
      for (int e = 0; e < VE; ++e) v[i].v[e] = (T)dense((float)v[i].v[e]);
      if (end - c > 0) store16_part(dr + c, v[i], end - c);
    }
    if constexpr (L < 256) break;
  }
  // the named tokens, each by its first entry, after their lanes' own stores
  float mass[E];
  bool again[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    mass[e] = 0.f;
    again[e] = false;
  }
  t.each(top, q.q, [&](int k, int id, float qk) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (id == t.id[e]) {
        mass[e] += qk;
        again[e] |= k < e * LT + lane;
      }
  });
  if constexpr (L == 256)
    __syncthreads();
  else
    wave_lds_fence();
  if (zero || tid >= LT) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (t.id[e] >= beg && t.id[e] < end && !again[e]) {
      const float p = expf(fmaf((float)xr[t.id[e]] - m, inv_t, -log_s));
      dr[t.id[e]] = (T)(g * (total * p - mass[e]));
    }
}

template <class T>
int distill_forward_t(const DistillArgs& a) {
  const ScoreSplit p = score_split(a.rows, a.vocab, Vec16<T>::n, 0);
  const float inv_t = 1.f / a.temperature;
  const auto stats_at = [&](int64_t at) { return a.stats ? a.stats + 4 * at : nullptr; };
#define FM_DISTILL_ROW_E(L, V, E)                                                               \
  if (p.lanes == L && p.vecs == V && a.top <= L * E)                                            \
    return by_rows(a.rows, kGridThreads / L, [&](int64_t at, int64_t rows) {                    \
      return launch("distillation",                                                             \
                    a.rest ? distill_row_kernel<T, L, V, E, true> : distill_row_kernel<T, L, V, E, false>, \
                    dim3((unsigned)((rows + 256 / L - 1) / (256 / L))), dim3(256), 0, a.stream, \
                    score_in<T>(a, at), a.ids + at * a.top, a.lps + at * a.top, a.loss + at,    \
                    stats_at(at), rows, a.vocab, a.top, a.temperature, inv_t);                  \
    });
// one entry of a lane where that holds them (24008 x 129 f32, the best 8: 6.7 us, with
// room for 64 of them 8.1; backward 9.6 and 12.6)
#define FM_DISTILL_ROW(L, V)                                                                    \
  FM_DISTILL_ROW_E(L, V, 1)                                                                     \
  if constexpr (L < 64) {                                                                       \
    FM_DISTILL_ROW_E(L, V, 64 / L)                                                              \
  }
  FM_SCORE_SHAPES(FM_DISTILL_ROW)
#undef FM_DISTILL_ROW
#undef FM_DISTILL_ROW_E
  float* part = (float*)a.workspace;
  const auto go = [&](auto kernel) {
    return by_rows(a.rows, kGridThreads / 256 / p.segs, [&](int64_t at, int64_t rows) {
      return launch("distillation", kernel, dim3((unsigned)(rows * p.segs)), dim3(256), 0, a.stream,
                    score_in<T>(a, at), a.ids + at * a.top, a.lps + at * a.top, a.loss + at, stats_at(at),
                    part + at * p.segs * 2, a.vocab, a.top, a.temperature, inv_t, p.seg_len, p.segs);
    });
  };
  const int st = p.vecs == 1
                     ? (a.rest ? go(distill_forward_kernel<T, 1, true>) : go(distill_forward_kernel<T, 1, false>))
                     : (a.rest ? go(distill_forward_kernel<T, 4, true>) : go(distill_forward_kernel<T, 4, false>));
  if (st != FM_OK || p.segs == 1) return st;
  return launch("distillation (join)", a.rest ? distill_join_kernel<T, true> : distill_join_kernel<T, false>,
                dim3((unsigned)a.rows), dim3(64), 0, a.stream, score_in<T>(a, 0), a.ids, a.lps, a.loss, a.stats, part,
                a.vocab, a.top, a.temperature, inv_t, p.segs);
}

template <class T>
int distill_backward_t(const DistillArgs& a) {
  const ScoreSplit p = score_split(a.rows, a.vocab, Vec16<T>::n, 0);
  const float inv_t = 1.f / a.temperature;
#define FM_DISTILL_BWD_E(L, V, E)                                                                \
  if (p.lanes == L && (L < 256 ? p.vecs == V : true) && a.top <= (L < 64 ? L : 64) * E)          \
    return by_rows(a.rows, kGridThreads / L / p.segs, [&](int64_t at, int64_t rows) {            \
      return launch("distillation backward",                                                     \
                    a.rest ? distill_backward_kernel<T, L, V, E, true>                            \
                           : distill_backward_kernel<T, L, V, E, false>,                            \
                    dim3((unsigned)((rows * p.segs + 256 / L - 1) / (256 / L))), dim3(256), 0,   \
                    a.stream, score_in<T>(a, at), a.ids + at * a.top, a.lps + at * a.top,        \
                    a.stats + 4 * at, a.grad + at, (T*)a.dx + at * a.vocab, rows, a.vocab, a.top, \
                    a.temperature, inv_t, p.seg_len, p.segs);                                    \
    });
#define FM_DISTILL_BWD(L, V)                                                                     \
  FM_DISTILL_BWD_E(L, V, 1)                                                                      \
  if constexpr (L < 64) {                                                                        \
    FM_DISTILL_BWD_E(L, V, 64 / L)                                                               \
  }
  FM_SCORE_SHAPES(FM_DISTILL_BWD)
  FM_DISTILL_BWD_E(256, 4, 1)
#undef FM_DISTILL_BWD
#undef FM_DISTILL_BWD_E
  return set_error(FM_E_UNSUPPORTED, "distillation: no kernel for this shape");
}

}  // namespace fm
