// Attention forward: the kernel for many queries (a wave's 32 queries in its
// registers, key tiles in LDS shared by 4 waves), the one for few queries
// (the waves divide the keys), and the join of key ranges.
#pragma once

#include "fm_attn.h"

namespace fm {

constexpr int kAttnThreads = 256;
// Keys per LDS tile.  32 and 64 take the same time (8 x 16 heads x 1501, 64
// columns: 87 us); 32 leave the registers and the LDS for four waves per SIMD.
constexpr int kAttnKeys = 32;

// Probabilities are rounded to the element type for their product, and the sum
// that divides them is not: in float16, 2^shift p is a normal number, rounded by
// half a step of itself, for probabilities down to 2^(-14 - shift) of the row's
// largest (a sink key of value 0 leaves the result to those). With a maximum that
// is raised only by 2^slack, 2^(shift + slack) p has to stay below 2^16: beside a
// slack of 2^4 shift 11, normal down to 17 nats (8 x 16 x 1501, 64 columns: 109.5 us;
// slack 2^8, which leaves 7 and 14 nats, 108). The kernel for few queries raises at
// once and takes 15.
template <class T>
constexpr float kSlack = 8.f;
template <>
inline constexpr float kSlack<f16_t> = 4.f;
template <class T>
constexpr float kShift = 0.f;
template <>
inline constexpr float kShift<f16_t> = 11.f;
template <class T>
constexpr float kTokenShift = 0.f;
template <>
inline constexpr float kTokenShift<f16_t> = 15.f;

template <class T, int DP>
constexpr size_t attn_forward_lds(int far) {
  return 4 * Tile<T, DP>::size(kAttnKeys) * sizeof(Lds<T>) + (bias_window(far) + 8) * sizeof(float);
}

// The transposed scores s' = K q' have queries as columns, so that a lane
// keeps one query's running maximum and sum, and the probabilities are the
// next product's right operand as they stand: o' = V' p'.  8 x 16 heads x 1501, 64
// columns, bf16: 88 us, 655 TFLOP/s; bound by the vector units, busy 69% of the time
// with about 100 instructions per tile and wave, 16 of them exponentials (without
// those 60 us, without fetches and barriers 74), the matrix units 35%.
template <class T, int DP, bool SPLIT, bool VEC>
__global__ __launch_bounds__(kAttnThreads, (sizeof(T) == 2 && DP == 64 && VEC ? 4 : attn_waves<T, DP>())) void attn_forward_kernel(const AttnArgs a) {
  constexpr int BK = kAttnKeys, NS = BK / 32, TS = Tile<T, DP>::size(BK), KS = DP / 16, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Lds<T>* kt = (Lds<T>*)smem;  // [2][TS]
  Lds<T>* vt = kt + 2 * TS;    // [2][TS]
  float* ends = (float*)(vt + 2 * TS);  // [4][2]
  float* bias = ends + 8;

  const int tid = threadIdx.x, wave = wave_index(), lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries;
  const int group = a.heads / a.kv_heads;
  const Place at = place_of(a.batch * a.kv_heads, blocks * group, blockIdx.x);
  if (at.none) return;
  const int b = at.unit / a.kv_heads, kvh = at.unit % a.kv_heads, head = kvh * group + at.block % group;
  // the last queries see the most keys when causal: they start first
  const int qb = a.causal ? blocks - 1 - at.block / group : at.block / group;
  const int q0 = qb * kAttnQueries + wave * 32;
  const int i = q0 + n;
  const int len = key_count(a, b), first = position_of_first(a, b);
  const int q_end = min((qb + 1) * kAttnQueries, a.q_len);  // of the workgroup
  int k_beg = 0, k_end = a.causal ? clamp_int(first + q_end, 0, len) : len;
  if constexpr (SPLIT) {
    const int per = ((len + a.splits - 1) / a.splits + BK - 1) / BK * BK;
    k_beg = min((int)blockIdx.y * per, k_end);
    k_end = min(k_beg + per, k_end);
  }

  const T* kp = (const T*)a.k + b * a.ks[0] + kvh * a.ks[1];
  const T* vp = (const T*)a.v + b * a.vs[0] + kvh * a.vs[1];
  TileLoad<T, DP, BK, kAttnThreads, VEC> kl, vl;
  kl.init(a.ks[2], a.dim, tid);
  vl.init(a.vs[2], a.dim, tid);
  kl.load(kp + k_beg * a.ks[2], a.ks[2], k_end - k_beg, a.dim, tid);
  vl.load(vp + k_beg * a.vs[2], a.vs[2], k_end - k_beg, a.dim, tid);
  Frag<T> qf[KS];
  const int qw = qb * kAttnQueries;  // the workgroup's first query
  const Rows<T, VEC> qr = {(const T*)a.q + b * a.qs[0] + head * a.qs[1] + qw * a.qs[2], a.qs[2],
                           a.q_len - qw, a.dim};
#pragma unroll
  for (int s = 0; s < KS; ++s) qf[s] = to_frag(qr.at(i - qw, 16 * s + 8 * h));
  fill_bias<T>(a, head, bias, ends, tid, kAttnThreads);
  const float c = a.scale * kLog2e;
  kl.store(kt, tid);
  vl.store(vt, tid);
  __syncthreads();
  const float lo = as_scalar(bias[0] * c), hi = as_scalar(bias[bias_window(a.far) - 1] * c);
  const Reach reach = reach_of(ends);

  acc16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
  // running maximum of the scores in base 2, its finite negative (with the shift),
  // and the sum
  float m = -INFINITY, neg = 0.f, l = 0.f;
  const int mine = a.causal ? min(len, first + i + 1) : len;   // keys this lane's query sees
  const int least = a.causal ? min(len, first + q0 + 1) : len; // of the wave's first query
  const int wave_end = a.causal ? min(k_end, first + q0 + 32) : k_end;
  const bool idle = q0 >= a.q_len;

  int buf = 0;
  for (int j0 = k_beg; j0 < k_end; j0 += BK, buf ^= 1) {
    const bool more = j0 + BK < k_end;
    if (more) {
      kl.load(kp + (int64_t)(j0 + BK) * a.ks[2], a.ks[2], k_end - j0 - BK, a.dim, tid);
      vl.load(vp + (int64_t)(j0 + BK) * a.vs[2], a.vs[2], k_end - j0 - BK, a.dim, tid);
    }
    if (!idle && j0 < wave_end) {
      const Lds<T>* ktb = kt + buf * TS;
      const Lds<T>* vtb = vt + buf * TS;
      acc16 s[NS];
      float far_bias[NS];  // of a tile that lies outside the window, in base 2
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int dist = j0 + 32 * u - first - q0;
        const Frag<T> k0 = tile_rows<T, DP>(ktb, 32 * u + n, 0, h);
        const bool is_before = tile_before(dist, reach);
        if (is_before || tile_behind(dist, reach)) {
          s[u] = mma32(k0, qf[0], acc_zero());
          far_bias[u] = is_before ? lo : hi;
        } else {
          s[u] = mma32(k0, qf[0], bias_start_keys(bias, a.far, dist, h, n));
          far_bias[u] = 0.f;
        }
        steps<T, KS - 1>([&](int t) { return tile_rows<T, DP>(ktb, 32 * u + n, 1 + t, h); },
                         [&](int t, const Frag<T>& f) { s[u] = mma32(f, qf[1 + t], s[u]); });
      }
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        if (j0 + 32 * u + 32 > least) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[u][r] = j0 + 32 * u + 8 * (r / 4) + 4 * h + r % 4 < mine ? s[u][r] : -INFINITY;
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        float mu = s[u][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mu = fmaxf(mu, s[u][r]);
        mx = fmaxf(mx, fmaf(mu, c, far_bias[u]));
      }
      mx = halves_max(mx);
      // a maximum raised by less than 2^kSlack leaves m as it is: every later
      // product with o and l waits for it
      const bool raise = mx > m + kSlack<T>;
      if (__any(raise)) {
        const float m2 = raise ? mx : m;
        // nothing seen yet: o and l are 0
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - m2);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] *= f;
        l *= f;
        m = m2;
        neg = m == -INFINITY ? 0.f : kShift<T> - m;
      }
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const float t = far_bias[u] + neg;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], c, t));
          sum += s[u][r];
        }
      }
      l += sum;
#pragma unroll
      for (int t = 0; t < 2 * NS; ++t) {
        // rounded to the element type for the product: half a step of each
        // probability (in float16 while 2^kShift p is normal), as the result's own
        // rounding; the sum l is not
        const Frag<T> p = acc_frag<T>(s[t / 2], t & 1);
        steps<T, DT>([&](int d) { return tile_cols<T, DP>(vtb, 16 * t, 32 * d, lane); },
                     [&](int d, const Frag<T>& f) { o[d] = mma32(f, p, o[d]); });
      }
    }
    if (more) {
      kl.store(kt + (buf ^ 1) * TS, tid);
      vl.store(vt + (buf ^ 1) * TS, tid);
    }
    __syncthreads();
  }

  l = halves_sum(l);
  const int ie = afresh(q0 + n), he = afresh(lane >> 5);
  if (ie >= a.q_len) return;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const int64_t row = (int64_t)(b * a.heads + head) * a.q_len + ie;
  const float lse = l != l ? l : m == -INFINITY ? -INFINITY : fmaf(m - kShift<T>, kLn2, logf(l));
  if constexpr (SPLIT) {
    const int64_t rows = (int64_t)a.batch * a.heads * a.q_len;
    if (he == 0) a.part_lse[blockIdx.y * rows + row] = lse;
    float* po = a.part_o + (blockIdx.y * rows + row) * a.dim;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at_d = 32 * d + 8 * y + 4 * he;
        if (at_d < a.dim)
          store4<float, VEC>(po + at_d, o[d][4 * y] * inv, o[d][4 * y + 1] * inv, o[d][4 * y + 2] * inv,
                 o[d][4 * y + 3] * inv, a.dim - at_d);
      }
  } else {
    if (a.lse && he == 0) a.lse[row] = lse;
    const int64_t off = b * a.os[0] + head * a.os[1] + ie * a.os[2];
    T* op = (T*)a.o + off;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at_d = 32 * d + 8 * y + 4 * he;
        if (at_d < a.dim)
          store4<T, VEC>(op + at_d, o[d][4 * y] * inv, o[d][4 * y + 1] * inv, o[d][4 * y + 2] * inv,
                 o[d][4 * y + 3] * inv, a.dim - at_d);
      }
  }
}

// Few queries: the rows of a key head (heads of the group x queries) go into
// 16-column fragments, one per workgroup; its waves take 32 keys each in turn,
// straight from memory, and join at the end.  Memory bound: keys are the left
// operand as they lie in memory, values pass through a wave's own LDS tile to be
// read by columns.  The fragments of a key range follow each other on one XCD, so
// that the second one finds the keys in its L2.  2 x 32 heads on 8, 100003 keys of
// 128 columns, f16: 130 us (5.5 TB/s); 8 x 16 heads, 1501 keys of 64, bf16: 13.5 us,
// three tiles per wave behind a prologue and the waves' join.
constexpr int kTokenKeys = 32;
// The group's bias windows are kept in LDS where they take at most this much;
// larger ones are looked up in memory by the few tiles that need them.
constexpr int kTokenBias = 16384;
inline int attn_token_bias(const AttnArgs& a) {
  const int64_t n = 4 * (int64_t)(2 * a.far + 1) * (a.heads / a.kv_heads);
  return n <= kTokenBias ? (int)n : 0;
}
template <class T, int DP>
constexpr size_t attn_token_lds(int bias) {
  constexpr int nw = attn_token_waves(sizeof(T), DP);
  constexpr size_t tiles = nw * Tile<T, DP>::size(kTokenKeys) * sizeof(Lds<T>);
  constexpr size_t join = nw * 16 * (DP + 2) * sizeof(float);
  return (tiles > join ? tiles : join) + bias;
}

template <class T, int DP, bool SPLIT, bool VEC>
__global__ __launch_bounds__((attn_token_waves(sizeof(T), DP) * 64)) void attn_token_kernel(const AttnArgs a) {
  constexpr int NW = attn_token_waves(sizeof(T), DP), NT = NW * 64;
  constexpr int LD = Tile<T, DP>::ld, KS = DP / 32, DT = DP / 16;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, wave = wave_index(), lane = tid & 63, n = lane & 15, g = lane >> 4;
  Lds<T>* vt = (Lds<T>*)smem + wave * Tile<T, DP>::size(kTokenKeys);
  const int group = a.heads / a.kv_heads, rows = group * a.q_len;
  const int units = a.batch * a.kv_heads;
  const Place at = place_of(units * a.splits, (rows + 15) / 16, blockIdx.x);
  if (at.none) return;
  const int range = at.unit / units, unit = at.unit - range * units;
  const int b = unit / a.kv_heads, kvh = unit - b * a.kv_heads;
  // this lane's column: a head of the group and a query
  const int row0 = 16 * at.block, mine_at = row0 + n;
  const bool real = mine_at < rows;
  const int member = real ? mine_at / a.q_len : 0, i = real ? mine_at - member * a.q_len : 0;
  const int head = kvh * group + member;
  const int len = key_count(a, b), first = position_of_first(a, b);
  int k_beg = 0, k_end = a.causal ? clamp_int(first + a.q_len, 0, len) : len;
  if constexpr (SPLIT) {
    const int per = ((k_end + a.splits - 1) / a.splits + kTokenKeys - 1) / kTokenKeys * kTokenKeys;
    k_beg = min(range * per, k_end);
    k_end = min(k_beg + per, k_end);
  }
  const T* kp = (const T*)a.k + b * a.ks[0] + kvh * a.ks[1];
  const T* vp = (const T*)a.v + b * a.vs[0] + kvh * a.vs[1];

  const float c = a.scale * kLog2e;
  Raw<T> kf[2][KS];
  TileLoad<T, DP, kTokenKeys, 64, VEC> vl;
  vl.init(a.vs[2], a.dim, lane);
  const auto fetch = [&](int j) __attribute__((always_inline)) {
    const Rows<T, VEC> kr = {kp + (int64_t)j * a.ks[2], a.ks[2], k_end - j, a.dim};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < KS; ++s) kf[u][s] = kr.at(16 * u + n, 32 * s + 8 * g);
    vl.load(vp + (int64_t)j * a.vs[2], a.vs[2], k_end - j, a.dim, lane);
  };
  int j0 = k_beg + wave * kTokenKeys;
  if (j0 < k_end) fetch(j0);
  Frag<T> qf[KS];
  const T* qp = (const T*)a.q + b * a.qs[0] + head * a.qs[1] + i * a.qs[2];
#pragma unroll
  for (int s = 0; s < KS; ++s) qf[s] = to_frag(load_raw(qp + 32 * s + 8 * g, real ? a.dim - 32 * s - 8 * g : 0));
  // the bias in units of the product: [group][2 far + 1]
  const int dists = 2 * a.far + 1;
  const bool table = (int64_t)dists * group * 4 <= kTokenBias;
  float* bias = (float*)(smem + attn_token_lds<T, DP>(0));
  const float inv_scale = 1.f / a.scale;
  if (table) {
    for (int t = tid; t < dists * group; t += NT) {
      const int x = t / dists;
      bias[t] = bias_of<T>(a, kvh * group + x, t - x * dists - a.far) * inv_scale;
    }
    __syncthreads();
  }
  const auto bias_at = [&](int d) {
    return table ? bias[member * dists + clamp_int(d + a.far, 0, dists - 1)]
                 : bias_of<T>(a, head, d) * inv_scale;
  };
  const float lo = real ? bias_at(-a.far) : 0.f, hi = real ? bias_at(a.far) : 0.f;
  const int pos = first + i;
  const int mine = real ? (a.causal ? min(len, pos + 1) : len) : 0;
  const int least = a.causal ? min(len, first + 1) : len;

  acc4 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = acc4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  for (; j0 < k_end; j0 += NW * kTokenKeys) {
    // the wave's own tile, written by lanes for other lanes
    wave_lds_fence();
    vl.store(vt, lane);
    wave_lds_fence();
    acc4 s[2];
    const int dist = j0 - first;  // of key j0 to the first query
    const bool left = dist + kTokenKeys - 1 <= -a.far, right = dist - (a.q_len - 1) >= a.far;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (left || right) {
        const float v = left ? lo : hi;
        s[u] = acc4{v, v, v, v};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[u][r] = real ? bias_at(j0 + 16 * u + 4 * g + r - pos) : 0.f;
      }
#pragma unroll
      for (int x = 0; x < KS; ++x) s[u] = mma16(to_frag(kf[u][x]), qf[x], s[u]);
    }
    const int j = j0;
    if (j0 + NW * kTokenKeys < k_end) fetch(j0 + NW * kTokenKeys);
    if (j + kTokenKeys > least || rows < row0 + 16) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[u][r] = j + 16 * u + 4 * g + r < mine ? s[u][r] : -INFINITY;
    }
    float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                     fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = halves_max(mx);
    if (__any(mx > m)) {
      const float m2 = fmaxf(m, mx);
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - m2) * c);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
      l *= f;
      m = m2;
    }
    const float mc = m == -INFINITY ? 0.f : fmaf(m, c, -kTokenShift<T>);
    Frag<T> p;
    {
      Raw<float> e;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[4 * u + r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], c, -mc));
          l += e[4 * u + r];
        }
      p = round_frag<T>(e);
    }
    // contraction over rows 4 g + 0..3 and 16 + 4 g + 0..3 of the tile
#pragma unroll
    for (int d = 0; d < DT; ++d)
      o[d] = mma16(lds_columns_of<T>(vt + (4 * g + (n >> 2)) * LD + 16 * d + 4 * (n & 3), 16 * LD,
                                     Tile<T, DP>::plane),
                   p, o[d]);
  }
  l += __shfl_xor(l, 16, 64);
  l = halves_sum(l);

  // the waves' shares: o[row][d], m and l per row
  __syncthreads();
  float* join = (float*)smem;
  constexpr int JL = DP + 2;
  float* jw = join + (wave * 16 + n) * JL;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) jw[16 * d + 4 * g + r] = o[d][r];
  if (g == 0) {
    jw[DP] = m;
    jw[DP + 1] = l;
  }
  __syncthreads();
  for (int t = tid; t < min(rows - row0, 16) * DP; t += NT) {
    const int r = t / DP, d = t - r * DP;
    if (d >= a.dim) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) mm = fmaxf(mm, join[(w * 16 + r) * JL + DP]);
    float sum = 0.f, val = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* p = join + (w * 16 + r) * JL;
      const float f = p[DP] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((p[DP] - mm) * c);
      // a NaN sum has to survive a maximum that never was one
      sum += p[DP + 1] != p[DP + 1] ? p[DP + 1] : f * p[DP + 1];
      val = fmaf(f, p[d], val);
    }
    const float out = sum == 0.f ? 0.f : val / sum;
    const float lse = sum != sum ? sum : mm == -INFINITY ? -INFINITY : fmaf(mm, a.scale, logf(sum) - kTokenShift<T> * kLn2);
    const int hd = kvh * group + (row0 + r) / a.q_len, qi = (row0 + r) % a.q_len;
    const int64_t row = (int64_t)(b * a.heads + hd) * a.q_len + qi;
    if constexpr (SPLIT) {
      const int64_t all = (int64_t)a.batch * a.heads * a.q_len;
      a.part_o[(range * all + row) * a.dim + d] = out;
      if (d == 0) a.part_lse[range * all + row] = lse;
    } else {
      const int64_t off = b * a.os[0] + hd * a.os[1] + qi * a.os[2] + d;
      ((T*)a.o)[off] = (T)out;
      if (a.lse && d == 0) a.lse[row] = lse;
    }
  }
}

// Joins the key ranges of a row: one workgroup per row, groups of threads over
// shares of the ranges.
template <class T>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(const AttnArgs a) {
  __shared__ float weight[kAttnMaxSplits];
  __shared__ float red[8];
  __shared__ float acc[kAttnThreads];
  const int64_t rows = (int64_t)a.batch * a.heads * a.q_len, row = blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6;
  // thread (share, column)
  const int cols = a.dim <= 64 ? 64 : 128, shares = kAttnThreads / cols;
  const int d = tid & (cols - 1), share = tid / cols;
  float v = tid < a.splits ? a.part_lse[tid * rows + row] : -INFINITY;
  float v2 = tid + kAttnThreads < a.splits ? a.part_lse[(tid + kAttnThreads) * rows + row] : -INFINITY;
  const bool bad = v != v || v2 != v2;
  float m = lanes_max<64>(fmaxf(v, v2));
  if ((tid & 63) == 0) red[wave] = m;
  if (tid < 4) red[4 + tid] = 0.f;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ms = m == -INFINITY ? 0.f : m;
  v = __builtin_amdgcn_exp2f((v - ms) * kLog2e);
  v2 = __builtin_amdgcn_exp2f((v2 - ms) * kLog2e);
  if (tid < a.splits) weight[tid] = v;
  if (tid + kAttnThreads < a.splits) weight[tid + kAttnThreads] = v2;
  // a NaN weight makes the sum NaN, and with it the row
  const float part = lanes_sum<64>(bad ? NAN : v + v2);
  if ((tid & 63) == 0) red[4 + wave] = part;
  __syncthreads();
  const float sum = (red[4] + red[5]) + (red[6] + red[7]);
  float o = 0.f;
  if (d < a.dim) {
    const float* p = a.part_o + row * a.dim + d;
    const int64_t step = rows * a.dim;
#pragma unroll 8
    for (int s = share; s < a.splits; s += shares) o = fmaf(weight[s], p[s * step], o);
  }
  acc[tid] = o;
  __syncthreads();
  if (share == 0 && d < a.dim) {
    for (int x = 1; x < shares; ++x) o += acc[x * cols + d];
    const int64_t bh = row / a.q_len, i = row - bh * a.q_len;
    const int64_t off = bh / a.heads * a.os[0] + bh % a.heads * a.os[1] + i * a.os[2];
    ((T*)a.o)[off + d] = (T)(sum == 0.f ? 0.f : o / sum);
    if (a.lse && d == 0) a.lse[row] = sum == 0.f ? -INFINITY : ms + logf(sum);
  }
}

// Few ranges: a row per wave, its weights in the lanes, a lane per column (2 x 4
// heads, 1777 queries, 4 ranges: 4 us, by whole workgroups 16).  One wave is slow
// over many of them (whole call, 1 x 2 key heads, one token, 20000 keys, 39 ranges:
// 12.4 us by workgroups, 15.5 by waves; 32 ranges of 131072 keys: 46 and 49).
constexpr int kAttnFewRanges = 16;
template <class T>
__global__ __launch_bounds__(kAttnThreads) void attn_join_rows_kernel(const AttnArgs a) {
  const int64_t rows = (int64_t)a.batch * a.heads * a.q_len;
  const int64_t row = (int64_t)blockIdx.x * (kAttnThreads / 64) + wave_index();
  if (row >= rows) return;
  const int lane = threadIdx.x & 63;
  const float* p = a.part_o + row * a.dim + lane;
  const int64_t step = rows * a.dim;
  const bool one = lane < a.dim, two = lane + 64 < a.dim;
  const float v = lane < a.splits ? a.part_lse[lane * rows + row] : -INFINITY;
  const float m = lanes_max<64>(v);
  const float ms = m == -INFINITY ? 0.f : m;
  // a NaN weight makes the sum NaN, and with it the row
  const float w = __builtin_amdgcn_exp2f((v - ms) * kLog2e), sum = lanes_sum<64>(w);
  float o = 0.f, o2 = 0.f;
  for (int s = 0; s < a.splits; s += 4) {
    float x[4], y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = s + k < a.splits;
      x[k] = in && one ? p[(s + k) * step] : 0.f;
      y[k] = in && two ? p[(s + k) * step + 64] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), s + k));
      o = fmaf(f, x[k], o);
      o2 = fmaf(f, y[k], o2);
    }
  }
  const int64_t bh = row / a.q_len, i = row - bh * a.q_len;
  T* to = (T*)a.o + bh / a.heads * a.os[0] + bh % a.heads * a.os[1] + i * a.os[2] + lane;
  if (one) to[0] = (T)(sum == 0.f ? 0.f : o / sum);
  if (two) to[64] = (T)(sum == 0.f ? 0.f : o2 / sum);
  if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : ms + logf(sum);
}

template <class T, int DP, bool VEC>
int attn_forward_dim(const AttnArgs& a, void* stream) {
  if (attn_token_kernel(a)) {
    static DeviceOnce once;
    const int opted = opted_in(once, [] {
      return lds_opt_in(attn_token_kernel<T, DP, false, VEC>, attn_token_lds<T, DP>(kTokenBias)) |
             lds_opt_in(attn_token_kernel<T, DP, true, VEC>, attn_token_lds<T, DP>(kTokenBias));
    });
    if (opted != FM_OK) return opted;
    return launch("attention of few queries",
                  a.splits > 1 ? attn_token_kernel<T, DP, true, VEC>
                               : attn_token_kernel<T, DP, false, VEC>,
                  dim3(place_grid((int64_t)a.batch * a.kv_heads * a.splits, attn_token_blocks(a))),
                  dim3(64 * attn_token_waves(sizeof(T), DP)),
                  attn_token_lds<T, DP>(attn_token_bias(a)), stream, a);
  }
  static DeviceOnce once;
  const int opted = opted_in(once, [] {
    return lds_opt_in(attn_forward_kernel<T, DP, false, VEC>, attn_forward_lds<T, DP>(kAttnMaxFar)) |
           lds_opt_in(attn_forward_kernel<T, DP, true, VEC>, attn_forward_lds<T, DP>(kAttnMaxFar));
  });
  if (opted != FM_OK) return opted;
  return launch("attention",
                a.splits > 1 ? attn_forward_kernel<T, DP, true, VEC>
                             : attn_forward_kernel<T, DP, false, VEC>,
                dim3(place_grid((int64_t)a.batch * a.kv_heads,
                                (int64_t)attn_query_blocks(a) * (a.heads / a.kv_heads)),
                     (unsigned)a.splits),
                dim3(kAttnThreads), attn_forward_lds<T, DP>(a.far), stream, a);
}

template <class T>
int attn_forward_t(const AttnArgs& a, void* stream) {
  const bool vec = attn_groups(a.q, a.qs, a.dim, sizeof(T)) && attn_groups(a.k, a.ks, a.dim, sizeof(T)) &&
                   attn_groups(a.v, a.vs, a.dim, sizeof(T));
  const auto go = [&](auto narrow, auto wide, auto widest) {
    return a.dim <= 64 ? narrow(a, stream) : a.dim <= 96 ? wide(a, stream) : widest(a, stream);
  };
  const int st = vec ? go(attn_forward_dim<T, 64, true>, attn_forward_dim<T, 96, true>,
                          attn_forward_dim<T, 128, true>)
                     : go(attn_forward_dim<T, 64, false>, attn_forward_dim<T, 96, false>,
                          attn_forward_dim<T, 128, false>);
  if (st != FM_OK || a.splits == 1) return st;
  if (a.splits <= kAttnFewRanges)
    return launch("attention (join)", attn_join_rows_kernel<T>, dim3((unsigned)((attn_rows(a) + 3) / 4)),
                  dim3(kAttnThreads), 0, stream, a);
  return launch("attention (join)", attn_join_kernel<T>, dim3((unsigned)attn_rows(a)), dim3(kAttnThreads),
                0, stream, a);
}

}  // namespace fm
