// Attention backward: one kernel for dq and the bias table (a wave's 32
// queries in its registers, key tiles in LDS), one for dk and dv (a wave's 32
// keys in its registers, query tiles in LDS), and the table's sums.  Scores
// are computed again in both: seven matrix products instead of five, but no
// gradient is added up by atomics in memory, so results do not depend on the
// order in which workgroups run.
// 8 x 16 heads x 1501, 64 columns, bf16, us: dq 140 (620 TFLOP/s over its three
// products), dk and dv 185 (620 over four), the table's sums 10.  Matrix units are
// busy 35% of the time in both, vector units 62% and 34%; dk and dv hold keys,
// values and both sums in registers (two waves per SIMD) and read queries and
// gradients from LDS in both orders, dq adds up the table's diagonals beside its
// products.
#pragma once

#include "fm_attn.h"

namespace fm {

constexpr int kAttnThreads = 256;
template <class T>
constexpr bool kIsF16 = false;
template <>
inline constexpr bool kIsF16<f16_t> = true;
// Rows of an LDS tile: two 32-row steps for bfloat16 in the dk, dv kernel (211
// us with one, 197 with two), one where the registers do not hold two (float16
// needs some for its scales) and in the dq kernel (at 64 columns three waves per
// SIMD then fit, by registers and by LDS: 157 us against 166 with 64 rows).
template <class T>
constexpr int attn_step() { return sizeof(T) == 2 && !kIsF16<T> ? 64 : 32; }
constexpr int kDqStep = 32;

// float16 has no room for gradients of any size: ds is scaled by powers of two,
// which are taken out at the end.  The other types have float32's exponents.
//
// dk, dv: one scale per key j (a lane's column), from |ds| <= |do_i| |v_j| +
// |delta_i| with the largest norm and delta of the group's queries: below 2^15
// whatever the values are, and with random ones (a bound 10 times too wide at 128
// columns) normal numbers down to probabilities of 2^-25.  The largest |do| alone
// does not bound ds, which holds a sum over the columns.
// dq: a scale per query (a lane's column again), lowered with the sums so far when
// a tile's largest |ds| leaves 2^15 behind; it then has room for 2^3 more.
__device__ __forceinline__ float scale_to(float size, int top) {
  // the power of two that brings size into [2^top, 2^(top + 1))
  const int e = clamp_int((int)(__float_as_uint(size) >> 23) & 255, top, 255);
  return __uint_as_float((uint32_t)(254 + top - e) << 23);
}
constexpr float kDqUnit = 0x1p100f;  // of a row without any ds yet
// float16 probabilities are scaled too: at most 1, so that 2^15 p is in range, and a
// normal number from p = 1.9e-9 on (dv of the keys beside one that takes nearly
// all the probability).
template <class T>
constexpr float kProbShift = 0.f;
template <>
inline constexpr float kProbShift<f16_t> = 15.f;
// Sums of ds by distance inside the window.  A 32x32 tile's 63 diagonals come
// from a wave's scratch in LDS: 16 queries at a time are stored as rows of 32
// keys with zeros between them, and lane t adds up diagonal t (key - query = t -
// 31) over the 16 rows, consecutive lanes at consecutive addresses.  The sums
// are added to the wave's own window without atomics: 16 atomic additions per
// tile and wave instead cost 170 cycles each (dq at 64 columns, 8 x 16 heads x
// 1501: 510 us, most of it there).
constexpr int kDiagRow = 68;  // 32 keys, 36 zeros (at least 31 on either side)
constexpr int kDiagScratch = 32 + 16 * kDiagRow;

// float16's scale takes the registers that a third wave would need, and so do the
// ranges of the keys, whose workgroups have a compute unit to themselves.
template <class T, int DP, bool VEC, bool RANGES>
constexpr int kDqWaves =
    sizeof(T) == 2 && DP == 64 && VEC && !RANGES && !kIsF16<T> ? 3 : attn_waves<T, DP>();

// Tiles of keys and of values in LDS: one computed on and one arriving, but a
// single one where two would leave no room for the widest bias window.
template <class T, int DP>
constexpr int kDqTiles = sizeof(T) == 4 && DP == 128 ? 1 : 2;

template <class T, int DP>
constexpr size_t attn_dq_lds(int far, bool table) {
  return 2 * kDqTiles<T, DP> * Tile<T, DP>::size(kDqStep) * sizeof(Lds<T>) +
         (table ? (4 * kDiagScratch + 2 * kAttnThreads) * sizeof(float) : 0) +
         bias_window(far) * sizeof(float) * (table ? 5 : 1) + 8 * sizeof(float);
}

__device__ __forceinline__ float tile_diagonals(float* scratch, const acc16& s, int h, int n, int lane) {
  float sum = 0.f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if ((n >> 4) == half) {
#pragma unroll
      for (int y = 0; y < 4; ++y)
        *(float4*)(scratch + 32 + (n & 15) * kDiagRow + 8 * y + 4 * h) =
            make_float4(s[4 * y], s[4 * y + 1], s[4 * y + 2], s[4 * y + 3]);
    }
    wave_lds_fence();
    const float* p = scratch + 1 + 16 * half + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += p[(kDiagRow + 1) * i];
    wave_lds_fence();
  }
  return sum;
}

template <class T, int DP, bool TABLE, bool VEC, bool RANGES>
__global__ __launch_bounds__(kAttnThreads, (kDqWaves<T, DP, VEC, RANGES>)) void attn_dq_kernel(const AttnArgs a) {
  constexpr int BK = kDqStep, NS = BK / 32, TS = Tile<T, DP>::size(BK), KS = DP / 16, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Lds<T>* kt = (Lds<T>*)smem;
  constexpr int TILES = kDqTiles<T, DP>;
  Lds<T>* vt = kt + TILES * TS;
  float* diag = (float*)(vt + TILES * TS);  // [4][kDiagScratch]
  float* bias = diag + (TABLE ? 4 * kDiagScratch : 0);
  const int win = bias_window(a.far);
  float* ends = bias + win;      // [4][2]
  float* before = ends + 8;      // [2][256]
  float* sums = before + 2 * kAttnThreads;  // [4][win]

  const int tid = threadIdx.x, wave = wave_index(), lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries;
  const int group = a.heads / a.kv_heads;
  const Place at = place_of(a.batch * a.kv_heads, blocks * group, blockIdx.x);
  if (at.none) return;
  const int b = at.unit / a.kv_heads, kvh = at.unit % a.kv_heads, head = kvh * group + at.block % group;
  const int qb = a.causal ? blocks - 1 - at.block / group : at.block / group;
  const int q0 = qb * kAttnQueries + wave * 32;
  const int i = q0 + n;
  const bool real = i < a.q_len;
  const int len = key_count(a, b), first = position_of_first(a, b);
  const int q_end = min((qb + 1) * kAttnQueries, a.q_len);
  // this workgroup's range of the keys
  const int all_end = a.causal ? clamp_int(first + q_end, 0, len) : len, range = RANGES ? blockIdx.y : 0;
  int k_beg = 0, k_end = all_end;
  if constexpr (RANGES) {
    const int per = ((len + a.dq_splits - 1) / a.dq_splits + BK - 1) / BK * BK;
    k_beg = min(range * per, all_end);
    k_end = min(k_beg + per, all_end);
  }

  const T* kp = (const T*)a.k + b * a.ks[0] + kvh * a.ks[1];
  const T* vp = (const T*)a.v + b * a.vs[0] + kvh * a.vs[1];
  TileLoad<T, DP, BK, kAttnThreads, VEC> kl, vl;
  kl.init(a.ks[2], a.dim, tid);
  vl.init(a.vs[2], a.dim, tid);
  kl.load(kp + k_beg * a.ks[2], a.ks[2], k_end - k_beg, a.dim, tid);
  vl.load(vp + k_beg * a.vs[2], a.vs[2], k_end - k_beg, a.dim, tid);
  const int64_t row = (int64_t)(b * a.heads + head) * a.q_len + i;
  Frag<T> qf[KS], gf[KS];
  float delta = 0.f, size = 0.f;
  {
    const int qw = qb * kAttnQueries, count = a.q_len - qw;  // the workgroup's first query
    const Rows<T, VEC> qr = {(const T*)a.q + b * a.qs[0] + head * a.qs[1] + qw * a.qs[2], a.qs[2], count, a.dim};
    const Rows<T, VEC> dr = {(const T*)a.d_o + b * a.dos[0] + head * a.dos[1] + qw * a.dos[2], a.dos[2], count,
                             a.dim};
    const Rows<T, VEC> rr = {(const T*)a.o + b * a.os[0] + head * a.os[1] + qw * a.os[2], a.os[2], count, a.dim};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * h;
      qf[s] = to_frag(qr.at(i - qw, d));
      const Raw<T> gr = dr.at(i - qw, d), of = rr.at(i - qw, d);
      gf[s] = to_frag(gr);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        delta = fmaf((float)gr[e], (float)of[e], delta);
        if constexpr (kIsF16<T>) size = fmaf((float)gr[e], (float)gr[e], size);
      }
    }
    delta = halves_sum(delta);
    if constexpr (kIsF16<T>) size = halves_sum(size);
  }
  // empty rows and rows past the end: every probability is 0
  float lse2 = INFINITY;
  if (real) {
    const float v = a.lse[row];
    if (v != -INFINITY) lse2 = v * kLog2e;
    if (kIsF16<T> && h == 0 && range == 0) a.amax[row] = sqrtf(size);
  }
  float unit = kIsF16<T> ? kDqUnit : 1.f;
  fill_bias<T>(a, head, bias, ends, tid, kAttnThreads);
  if constexpr (TABLE) {
    for (int t = tid; t < 4 * win; t += kAttnThreads) sums[t] = 0.f;
    for (int t = tid; t < 4 * kDiagScratch; t += kAttnThreads) diag[t] = 0.f;
  }
  kl.store(kt, tid);
  vl.store(vt, tid);
  __syncthreads();

  const float c = a.scale * kLog2e;
  const float lo = as_scalar(bias[0] * c), hi = as_scalar(bias[win - 1] * c);
  const Reach reach = reach_of(ends);
  const int mine = a.causal ? min(len, first + i + 1) : len;
  const int least = a.causal ? min(len, first + q0 + 1) : len;
  const int wave_end = a.causal ? min(k_end, first + q0 + 32) : k_end;
  const bool idle = q0 >= a.q_len;
  if (!idle && range == 0 && (a.causal ? min(all_end, first + q0 + 32) : all_end) <= 32) {
    // All keys of these queries lie in the first tile: delta from p and dp
    // themselves.  Their few probabilities are large, and so would be the error
    // that the rounding of o leaves in delta.
    const int dist = -first - q0;
    const bool is_before = tile_before(dist, reach), far = is_before || tile_behind(dist, reach);
    acc16 s = far ? acc_zero() : bias_start_keys(bias, a.far, dist, h, n), dp = acc_zero();
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      s = mma32(tile_rows<T, DP>(kt, n, x, h), qf[x], s);
      dp = mma32(tile_rows<T, DP>(vt, n, x, h), gf[x], dp);
    }
    const float t = (far ? (is_before ? lo : hi) : 0.f) - lse2;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (8 * (r / 4) + 4 * h + r % 4 < mine)
        sum = fmaf(__builtin_amdgcn_exp2f(fmaf(s[r], c, t)), dp[r], sum);
    delta = halves_sum(sum);
  }

  acc16 dq[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[d][r] = 0.f;
  // per query: ds and p over the tiles on one side of the window (keys come in
  // order: those before it are put away when the first other tile comes), and
  // ds over all tiles
  float far_ds = 0.f, far_p = 0.f, all = 0.f;
  bool put_away = false;
  float* mysums = sums + wave * win;
  float* mydiag = diag + wave * kDiagScratch;
  int buf = 0;
  for (int j0 = k_beg; j0 < k_end; j0 += BK, buf ^= TILES - 1) {
    const bool more = j0 + BK < k_end;
    if (more) {
      kl.load(kp + (int64_t)(j0 + BK) * a.ks[2], a.ks[2], k_end - j0 - BK, a.dim, tid);
      vl.load(vp + (int64_t)(j0 + BK) * a.vs[2], a.vs[2], k_end - j0 - BK, a.dim, tid);
    }
    if (!idle && j0 < wave_end) {
      const Lds<T>* ktb = kt + buf * TS;
      const Lds<T>* vtb = vt + buf * TS;
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int dist = j0 + 32 * u - first - q0;
        const bool is_before = tile_before(dist, reach), is_behind = tile_behind(dist, reach);
        const Frag<T> k0 = tile_rows<T, DP>(ktb, 32 * u + n, 0, h);
        acc16 s;
        float far_bias;
        if (is_before || is_behind) {
          s = mma32(k0, qf[0], acc_zero());
          far_bias = is_before ? lo : hi;
        } else {
          s = mma32(k0, qf[0], bias_start_keys(bias, a.far, dist, h, n));
          far_bias = 0.f;
        }
        acc16 dp = acc_zero();
        steps<T, 2 * KS - 1>(
            [&](int t) { return tile_rows<T, DP>(t < KS - 1 ? ktb : vtb, 32 * u + n, (t + 1) % KS, h); },
            [&](int t, const Frag<T>& f) {
              if (t < KS - 1)
                s = mma32(f, qf[t + 1], s);
              else
                dp = mma32(f, gf[(t + 1) % KS], dp);
            });
        if (j0 + 32 * u + 32 > least) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[r] = j0 + 32 * u + 8 * (r / 4) + 4 * h + r % 4 < mine ? s[r] : -INFINITY;
        }
        const float t = far_bias - lse2;
        if (TABLE && !is_before && !put_away) {
          before[tid] = far_ds;
          before[kAttnThreads + tid] = far_p;
          far_ds = far_p = 0.f;
          put_away = true;
        }
        if (TABLE && (is_before || is_behind)) {
          float ds_sum = 0.f;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, t));
            far_p += p;
            s[r] = p * (dp[r] - delta);
            ds_sum += s[r];
          }
          far_ds += ds_sum;
          all += ds_sum;
        } else {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, t)) * (dp[r] - delta);
          if constexpr (TABLE) {
#pragma unroll
            for (int r = 0; r < 16; ++r) all += s[r];
            mysums[dist - 31 + a.far + kBiasPad + lane] += tile_diagonals(mydiag, s, h, n, lane);
          }
        }
        if constexpr (kIsF16<T>) {
          float most = 0.f;
#pragma unroll
          for (int r = 0; r < 16; ++r) most = fmaxf(most, fabsf(s[r]));
          most = halves_max(most);
          const bool lower = most * unit > 0x1p15f;
          if (__any(lower)) {
            const float to = lower ? scale_to(most, 11) : unit, f = to / unit;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int r = 0; r < 16; ++r) dq[d][r] *= f;
            unit = to;
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] *= unit;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Frag<T> ds = acc_frag<T>(s, x);
          steps<T, DT>([&](int d) { return tile_cols<T, DP>(ktb, 32 * u + 16 * x, 32 * d, lane); },
                       [&](int d, const Frag<T>& f) { dq[d] = mma32(f, ds, dq[d]); });
        }
      }
    }
    if (TILES == 1) __syncthreads();
    if (more) {
      kl.store(kt + (buf ^ (TILES - 1)) * TS, tid);
      vl.store(vt + (buf ^ (TILES - 1)) * TS, tid);
    }
    __syncthreads();
  }

  const int ie = afresh(q0 + n), he = afresh(lane >> 5);
  if (ie < a.q_len) {
    const int64_t at_row = (int64_t)(b * a.heads + head) * a.q_len + ie;
    if (he == 0 && range == 0) a.delta[at_row] = delta;
    const float f = a.scale / unit;
    float* part = a.part_dq + (range * attn_row_count(a) + at_row) * a.dim;
    T* out = (T*)a.dq + b * a.dqs[0] + head * a.dqs[1] + ie * a.dqs[2];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at_d = 32 * d + 8 * y + 4 * he;
        if (at_d >= a.dim) continue;
        if constexpr (RANGES)
          store4<float, VEC>(part + at_d, dq[d][4 * y] * f, dq[d][4 * y + 1] * f, dq[d][4 * y + 2] * f,
                             dq[d][4 * y + 3] * f, a.dim - at_d);
        else
          store4<T, VEC>(out + at_d, dq[d][4 * y] * f, dq[d][4 * y + 1] * f, dq[d][4 * y + 2] * f,
                 dq[d][4 * y + 3] * f, a.dim - at_d);
      }
  }
  if constexpr (TABLE) {
    // A query's ds add up to 0.  What they add up to here is the error of
    // delta, whose o was rounded (its probabilities before, itself after): as
    // much times a pair's p is in each ds.  The far sides hold most of a long
    // row's probability in one bucket each, where these errors would add up;
    // there they are taken out.
    float off = halves_sum(all);
    float left = far_ds, left_p = far_p, right = 0.f, right_p = 0.f;
    if (put_away) {
      right = far_ds;
      right_p = far_p;
      left = before[tid];
      left_p = before[kAttnThreads + tid];
    }
    if constexpr (RANGES) {
      // the whole row's is known to the join only
      const float lp = halves_sum(left_p), rp = halves_sum(right_p);
      if (ie < a.q_len && he == 0) {
        float* r = a.part_row + (range * attn_row_count(a) + (int64_t)(b * a.heads + head) * a.q_len + ie) * 3;
        r[0] = off;
        r[1] = lp;
        r[2] = rp;
      }
      off = 0.f;
    }
    left = lanes_sum<64>(fmaf(-off, left_p, left));
    right = lanes_sum<64>(fmaf(-off, right_p, right));
    // without any tile, other waves may still be reading the map's reach there
    __syncthreads();
    if (lane == 0) {
      ends[2 * wave] = left;
      ends[2 * wave + 1] = right;
    }
    __syncthreads();
    // the window's first and last distances have the buckets of the far tiles
    float* out = a.table_part + (((int64_t)(b * a.heads + head) * blocks + qb) * (RANGES ? a.dq_splits : 1) + range) * win;
    for (int t = tid; t < win; t += kAttnThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += sums[w * win + t];
      if (t == 0) v += (ends[0] + ends[2]) + (ends[4] + ends[6]);
      if (t == win - 1) v += (ends[1] + ends[3]) + (ends[5] + ends[7]);
      out[t] = v;
    }
  }
}

constexpr int kDqJoinRows = 8;  // of a workgroup
// Joins the key ranges of a query block: dq, and the correction of the bias
// table's end buckets (see above) with the rows' whole sums.
template <class T>
__global__ __launch_bounds__(kAttnThreads) void attn_dq_join_kernel(const AttnArgs a) {
  __shared__ float red[4][2];
  const int blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries, tid = threadIdx.x;
  const int64_t bh = blockIdx.x / blocks, rows = attn_row_count(a);
  const int qb = blockIdx.x - (int)bh * blocks, i0 = qb * kAttnQueries, have = min(kAttnQueries, a.q_len - i0);
  const int64_t b = bh / a.heads, head = bh - b * a.heads, row0 = bh * a.q_len + i0, step = rows * a.dim;
  const float* p = a.part_dq + row0 * a.dim;
  T* out = (T*)a.dq + b * a.dqs[0] + head * a.dqs[1];
  const int t_end = min((int)(blockIdx.y + 1) * kDqJoinRows, have) * a.dim;
  for (int t = blockIdx.y * kDqJoinRows * a.dim + tid; t < t_end; t += kAttnThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int r = 0; r < a.dq_splits; ++r) s += p[r * step + t];
    const int i = t / a.dim;
    out[(i0 + i) * a.dqs[2] + t - i * a.dim] = (T)s;
  }
  if (!a.d_table || blockIdx.y > 0) return;
  float left = 0.f, right = 0.f;
  if (tid < have) {
    float off = 0.f, lp = 0.f, rp = 0.f;
    for (int r = 0; r < a.dq_splits; ++r) {
      const float* x = a.part_row + (r * rows + row0 + tid) * 3;
      off += x[0];
      lp += x[1];
      rp += x[2];
    }
    left = -off * lp;
    right = -off * rp;
  }
  left = lanes_sum<64>(left);
  right = lanes_sum<64>(right);
  if ((tid & 63) == 0) {
    red[tid >> 6][0] = left;
    red[tid >> 6][1] = right;
  }
  __syncthreads();
  if (tid < 2) {
    const int win = bias_window(a.far);
    float* at = a.table_part + (bh * blocks + qb) * a.dq_splits * win + (tid ? win - 1 : 0);
    *at += (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
  }
}

// Sums over entries and query blocks: by distance, 64 distances of a head per
// workgroup, 16 interleaved sets of partials.
template <class T>
__global__ __launch_bounds__(1024) void attn_table_distances_kernel(const AttnArgs a) {
  __shared__ float red[16][64];
  const int win = bias_window(a.far), blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries * a.dq_splits;
  const int lane = threadIdx.x & 63, set = threadIdx.x >> 6, head = blockIdx.y;
  const int t = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (t < win)
#pragma unroll 4
    for (int p = set; p < a.batch * blocks; p += 16) {
      const int b = p / blocks, qb = p - b * blocks;
      s += a.table_part[((int64_t)(b * a.heads + head) * blocks + qb) * win + t];
    }
  red[set][lane] = s;
  __syncthreads();
  if (set == 0 && t < win) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += red[k][lane];
    a.table_dist[(int64_t)head * win + t] = v;
  }
}

// ... and by bucket, one head per workgroup: the threads beyond one per bucket
// take further shares of the distances.  Up to kTableRows partials (entries
// times query blocks) the sums by distance are formed here too, which saves a
// launch (whole backward, us: 1 partial 41.1, with both launches 43.0; 12: 88.0
// and 88.4; 32: 74.0 and 72.4; 64: 101 and 95).
constexpr int kTableRows = 16;
template <class W>
__global__ __launch_bounds__(1024) void attn_table_buckets_kernel(const AttnArgs a) {
  constexpr int AHEAD = 8;  // LDS reads on their way at a time
  __shared__ float2 dist[bias_window(kAttnMaxFar) + AHEAD];  // sum, bucket
  __shared__ float red[1024];
  const int win = bias_window(a.far), head = blockIdx.x, tid = threadIdx.x;
  const int blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries * a.dq_splits, rows = a.batch * blocks;
  for (int t = tid; t < win; t += 1024) {
    const int bucket = a.map[clamp_int(t - kBiasPad, 0, 2 * a.far)];
    float s = 0.f;
    if (rows > kTableRows) {
      s = a.table_dist[(int64_t)head * win + t];
    } else {
#pragma unroll 8
      for (int p = 0; p < rows; ++p) {
        const int b = p / blocks, qb = p - b * blocks;
        s += a.table_part[((int64_t)(b * a.heads + head) * blocks + qb) * win + t];
      }
    }
    dist[t] = make_float2(s, __int_as_float(bucket));
  }
  __syncthreads();
  const int shares = 1024 / a.num_buckets, k = tid % a.num_buckets, share = tid / a.num_buckets;
  const int per = (win + shares - 1) / shares;
  float s = 0.f;
  if (share < shares)
    for (int t = share * per; t < min((share + 1) * per, win); t += AHEAD) {
      float2 x[AHEAD];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) x[e] = dist[t + e];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
        s += t + e < min((share + 1) * per, win) && __float_as_int(x[e].y) == k ? x[e].x : 0.f;
    }
  red[tid] = s;
  __syncthreads();
  if (tid < a.num_buckets) {
    float v = 0.f;
#pragma unroll 8
    for (int x = 0; x < shares; ++x) v += red[x * a.num_buckets + tid];
    ((W*)a.d_table)[(int64_t)tid * a.heads + head] = (W)v;
  }
}

template <class T, int DP>
constexpr size_t attn_dkv_lds(int far) {
  return 4 * Tile<T, DP>::size(attn_step<T>()) * sizeof(Lds<T>) +
         (4 * attn_step<T>() + 8 + bias_window(far)) * sizeof(float);
}

template <class T, int DP, bool VEC>
__global__ __launch_bounds__(kAttnThreads, (sizeof(T) == 2 && DP == 64 && VEC ? 2 : 1)) void attn_dkv_kernel(const AttnArgs a) {
  constexpr int BQ = attn_step<T>(), NS = BQ / 32, TS = Tile<T, DP>::size(BQ), KS = DP / 16, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  // float32 fragments of 128 columns leave no registers for the next tile, and
  // neither do loads of odd rows
  constexpr bool AHEAD = VEC && !(sizeof(T) == 4 && DP == 128);
  // float32's three-part fragments leave none for operands read ahead
  constexpr bool STAGED = sizeof(T) == 2;
  // nor for the map's reach, which is +-far at least
  constexpr bool REACH = sizeof(T) == 2;
  Lds<T>* qt = (Lds<T>*)smem;
  Lds<T>* gt = qt + 2 * TS;
  // -lse in units of the product and -delta start the accumulators: exp2 of the
  // scaled scores then is p, and dp comes out less delta.  In float32 the sums
  // would be rounded at lse's size instead of the scores': there it is -lse in
  // base 2, added after.
  constexpr bool LSE_LATE = sizeof(T) == 4;
  float* neg_lse = (float*)(gt + 2 * TS);  // [2][BQ]
  float* neg_delta = neg_lse + 2 * BQ;     // [2][BQ]
  float* ends = neg_delta + 2 * BQ;  // [4][2]
  float* bias = ends + 8;

  const int tid = threadIdx.x, wave = wave_index(), lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int blocks = (a.k_len + kAttnBlockKeys - 1) / kAttnBlockKeys;
  const Place at = place_of(a.batch * a.kv_heads, blocks, blockIdx.x);
  if (at.none) return;
  const int b = at.unit / a.kv_heads, kvh = at.unit % a.kv_heads, group = a.heads / a.kv_heads;
  const int j_wg = at.block * kAttnBlockKeys, jw = j_wg + wave * 32, j = jw + n;
  const int len = key_count(a, b), first = position_of_first(a, b);

  Frag<T> kf[KS], vf[KS];
  {
    const Rows<T, VEC> kr = {(const T*)a.k + b * a.ks[0] + kvh * a.ks[1] + j_wg * a.ks[2], a.ks[2], len - j_wg,
                             a.dim};
    const Rows<T, VEC> vr = {(const T*)a.v + b * a.vs[0] + kvh * a.vs[1] + j_wg * a.vs[2], a.vs[2], len - j_wg,
                             a.dim};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kf[s] = to_frag(kr.at(j - j_wg, 16 * s + 8 * h));
      vf[s] = to_frag(vr.at(j - j_wg, 16 * s + 8 * h));
    }
  }
  acc16 dk[DT], dv[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[d][r] = dv[d][r] = 0.f;

  // queries that may see the first key of the workgroup
  const int i_beg = a.causal ? clamp_int(j_wg - first, 0, a.q_len) / BQ * BQ : 0;
  const int i_end = j_wg < len ? a.q_len : 0;
  float unit = 1.f;
  if constexpr (kIsF16<T>) {
    float g = 0.f, t_most = 0.f, v = 0.f;
    const int64_t row0 = (int64_t)(b * a.heads + kvh * group) * a.q_len;
    for (int64_t t = tid; t < (int64_t)group * a.q_len; t += kAttnThreads) {
      g = fmaxf(g, a.amax[row0 + t]);
      t_most = fmaxf(t_most, fabsf(a.delta[row0 + t]));
    }
    g = lanes_max<64>(g);
    t_most = lanes_max<64>(t_most);
    if (lane == 0) {
      neg_lse[wave] = g;
      neg_delta[wave] = t_most;
    }
    __syncthreads();
    g = fmaxf(fmaxf(neg_lse[0], neg_lse[1]), fmaxf(neg_lse[2], neg_lse[3]));
    t_most = fmaxf(fmaxf(neg_delta[0], neg_delta[1]), fmaxf(neg_delta[2], neg_delta[3]));
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) v = fmaf((float)vf[s][e], (float)vf[s][e], v);
    unit = scale_to(fmaf(g, sqrtf(halves_sum(v)), t_most), 14);
    __syncthreads();
  }
  const float c = a.scale * kLog2e, inv_c = 1.f / c;
  const float back = kIsF16<T> ? unit * __builtin_amdgcn_exp2f(-kProbShift<T>) : 1.f;
  // row i of the tile at i0 sees this lane's key if i >= need
  const int need = j >= len ? a.q_len : a.causal ? max(j - first, 0) : 0;

  // this workgroup's share of the query tiles, head after head
  const int tiles = max(i_end - i_beg + BQ - 1, 0) / BQ, per = (group * tiles + a.dkv_splits - 1) / a.dkv_splits;
  const int t_end = min(((int)blockIdx.y + 1) * per, group * tiles);
  for (int t_head = blockIdx.y * per; t_head < t_end;) {
    const int gi = t_head / tiles, head = kvh * group + gi;
    const int i_first = i_beg + (t_head - gi * tiles) * BQ;
    t_head = min(t_end, (gi + 1) * tiles);
    const int i_last = min(i_end, i_beg + (t_head - gi * tiles) * BQ);
    const T* qp = (const T*)a.q + b * a.qs[0] + head * a.qs[1];
    const T* gp = (const T*)a.d_o + b * a.dos[0] + head * a.dos[1];
    const int64_t row0 = (int64_t)(b * a.heads + head) * a.q_len;
    TileLoad<T, DP, BQ, kAttnThreads, VEC> ql, gl;
    ql.init(a.qs[2], a.dim, tid);
    gl.init(a.dos[2], a.dim, tid);
    float l_next = 0.f, d_next = 0.f;
    const auto fetch = [&](int i0) __attribute__((always_inline)) {
      ql.load(qp + (int64_t)i0 * a.qs[2], a.qs[2], i_end - i0, a.dim, tid);
      gl.load(gp + (int64_t)i0 * a.dos[2], a.dos[2], i_end - i0, a.dim, tid);
      if (tid < BQ) {
        const bool in = i0 + tid < i_end;
        const float v = in ? a.lse[row0 + i0 + tid] : -INFINITY;
        l_next = v == -INFINITY ? v : fmaf(v, -kLog2e, kProbShift<T>) * (LSE_LATE ? 1.f : inv_c);
        d_next = in ? -a.delta[row0 + i0 + tid] : 0.f;
      }
    };
    const auto put = [&](int buf) __attribute__((always_inline)) {
      ql.store(qt + buf * TS, tid);
      gl.store(gt + buf * TS, tid);
      if (tid < BQ) {
        neg_lse[buf * BQ + tid] = l_next;
        neg_delta[buf * BQ + tid] = d_next;
      }
    };
    fetch(i_first);
    fill_bias<T, REACH>(a, head, bias, ends, tid, kAttnThreads);
    put(0);
    __syncthreads();
    const float lo = as_scalar(bias[0] * c), hi = as_scalar(bias[bias_window(a.far) - 1] * c);
    const Reach reach = REACH ? reach_of(ends) : Reach{-a.far, a.far};
    int buf = 0;
    for (int i0 = i_first; i0 < i_last; i0 += BQ, buf ^= 1) {
      const bool more = i0 + BQ < i_last;
      if (AHEAD && more) fetch(i0 + BQ);
      if (jw < len && !(a.causal && i0 + BQ - 1 + first < jw)) {
        const Lds<T>* qtb = qt + buf * TS;
        const Lds<T>* gtb = gt + buf * TS;
        acc16 s[NS], ds[NS];
        float far_bias[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          const int dist = jw - first - i0 - 32 * u;
          s[u] = LSE_LATE ? acc_zero() : acc_rows(neg_lse + buf * BQ + 32 * u, h);
          const bool is_before = tile_before(dist, reach);
          if (is_before || tile_behind(dist, reach)) {
            far_bias[u] = is_before ? lo : hi;
          } else {
            s[u] += bias_start_queries(bias, a.far, dist, h, n);
            far_bias[u] = 0.f;
          }
        }
        // Products in stages, each reading the next one's operands: queries and
        // gradients by rows, then by columns.
        if constexpr (STAGED) {
          Frag<T> rows[2][KS];
          const auto read_rows = [&](const Lds<T>* tile, int u, Frag<T>(&f)[KS]) __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < KS; ++x) f[x] = tile_rows<T, DP>(tile, 32 * u + n, x, h);
          };
          read_rows(qtb, 0, rows[0]);
          ds[0] = acc_rows(neg_delta + buf * BQ, h);
          stage();
#pragma unroll
          for (int u = 0; u < NS; ++u) {
            read_rows(gtb, u, rows[1]);
            stage();
#pragma unroll
            for (int x = 0; x < KS; ++x) s[u] = mma32(rows[0][x], kf[x], s[u]);
            stage();
            if (u + 1 < NS) {
              read_rows(qtb, u + 1, rows[0]);
              ds[u + 1] = acc_rows(neg_delta + buf * BQ + 32 * (u + 1), h);
            }
            stage();
#pragma unroll
            for (int x = 0; x < KS; ++x) ds[u] = mma32(rows[1][x], vf[x], ds[u]);
            stage();
          }
        } else {
#pragma unroll
          for (int u = 0; u < NS; ++u) {
            ds[u] = acc_rows(neg_delta + buf * BQ + 32 * u, h);
            steps<T, 2 * KS>(
                [&](int t) { return tile_rows<T, DP>(t & 1 ? gtb : qtb, 32 * u + n, t >> 1, h); },
                [&](int t, const Frag<T>& f) {
                  if (t & 1)
                    ds[u] = mma32(f, vf[t >> 1], ds[u]);
                  else
                    s[u] = mma32(f, kf[t >> 1], s[u]);
                });
          }
        }
        if (jw + 32 > len || (a.causal && jw + 31 - first > i0)) {
#pragma unroll
          for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              s[u][r] = i0 + 32 * u + 8 * (r / 4) + 4 * h + r % 4 >= need ? s[u][r] : -INFINITY;
        }
        // step t: rows 16 t .. 16 t + 15 of the tile
        Frag<T> p[2], f[2];
        const auto scores = [&](int t) __attribute__((always_inline)) {
          const int u = t >> 1, x = t & 1;
          acc16 late;
          if constexpr (LSE_LATE) late = acc_rows(neg_lse + buf * BQ + 32 * u, h);
#pragma unroll
          for (int r = 8 * x; r < 8 * x + 8; ++r) {
            s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], c, LSE_LATE ? far_bias[u] + late[r] : far_bias[u]));
            if constexpr (kIsF16<T>)
              ds[u][r] *= s[u][r] * back;
            else
              ds[u][r] *= s[u][r];
          }
          p[t & 1] = acc_frag<T>(s[u], x);
          f[t & 1] = acc_frag<T>(ds[u], x);
        };
        if constexpr (STAGED) {
          Frag<T> cols[2][2 * DT];
          const auto read_cols = [&](int t, Frag<T>(&c)[2 * DT]) __attribute__((always_inline)) {
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              c[d] = tile_cols<T, DP>(gtb, 16 * t, 32 * d, lane);
              c[DT + d] = tile_cols<T, DP>(qtb, 16 * t, 32 * d, lane);
            }
          };
          read_cols(0, cols[0]);
          stage();
          scores(0);
          stage();
#pragma unroll
          for (int t = 0; t < 2 * NS; ++t) {
            if (t + 1 < 2 * NS) read_cols(t + 1, cols[(t + 1) & 1]);
            stage();
            if (t + 1 < 2 * NS) scores(t + 1);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              dv[d] = mma32(cols[t & 1][d], p[t & 1], dv[d]);
              dk[d] = mma32(cols[t & 1][DT + d], f[t & 1], dk[d]);
            }
            if constexpr (sizeof(T) == 2) alternate<2 * DT, 32 / (2 * DT)>();
            stage();
          }
        } else {
#pragma unroll
          for (int t = 0; t < 2 * NS; ++t) {
            scores(t);
            steps<T, 2 * DT>(
                [&](int i) { return tile_cols<T, DP>(i & 1 ? qtb : gtb, 16 * t, 32 * (i >> 1), lane); },
                [&](int i, const Frag<T>& c) {
                  if (i & 1)
                    dk[i >> 1] = mma32(c, f[t & 1], dk[i >> 1]);
                  else
                    dv[i >> 1] = mma32(c, p[t & 1], dv[i >> 1]);
                });
          }
        }
      }
      if (!AHEAD && more) fetch(i0 + BQ);
      if (more) put(buf ^ 1);
      __syncthreads();
    }
  }
  if (j >= a.k_len) return;
  const float fk = a.scale / unit, fv = __builtin_amdgcn_exp2f(-kProbShift<T>);
  if (a.dkv_splits > 1) {
    const int64_t unit_of = (int64_t)blockIdx.y * a.batch * a.kv_heads + at.unit;
    float* pk = a.part_dkv + (unit_of * a.k_len + j) * 2 * a.dim;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at_d = 32 * d + 8 * y + 4 * h;
        if (at_d < a.dim) {
          store4<float, VEC>(pk + at_d, dk[d][4 * y] * fk, dk[d][4 * y + 1] * fk, dk[d][4 * y + 2] * fk,
                             dk[d][4 * y + 3] * fk, a.dim - at_d);
          store4<float, VEC>(pk + a.dim + at_d, dv[d][4 * y] * fv, dv[d][4 * y + 1] * fv, dv[d][4 * y + 2] * fv,
                             dv[d][4 * y + 3] * fv, a.dim - at_d);
        }
      }
    return;
  }
  T* ok = (T*)a.dk + b * a.dks[0] + kvh * a.dks[1] + j * a.dks[2];
  T* ov = (T*)a.dv + b * a.dvs[0] + kvh * a.dvs[1] + j * a.dvs[2];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int at_d = 32 * d + 8 * y + 4 * h;
      if (at_d < a.dim) {
        store4<T, VEC>(ok + at_d, dk[d][4 * y] * fk, dk[d][4 * y + 1] * fk, dk[d][4 * y + 2] * fk,
               dk[d][4 * y + 3] * fk, a.dim - at_d);
        store4<T, VEC>(ov + at_d, dv[d][4 * y] * fv, dv[d][4 * y + 1] * fv, dv[d][4 * y + 2] * fv,
               dv[d][4 * y + 3] * fv, a.dim - at_d);
      }
    }
}

// Adds up the shares in order: a thread per column of [dk | dv], 256 / cols rows
// of keys per workgroup.
template <class T>
__global__ __launch_bounds__(kAttnThreads) void attn_dkv_join_kernel(const AttnArgs a) {
  const int cols = a.dim <= 32 ? 64 : a.dim <= 64 ? 128 : 256;
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.k_len;
  const int64_t row = (int64_t)blockIdx.x * (kAttnThreads / cols) + threadIdx.x / cols;
  const int c = threadIdx.x & (cols - 1);
  if (row >= rows || c >= 2 * a.dim) return;
  const float* p = a.part_dkv + row * 2 * a.dim + c;
  const int64_t step = rows * 2 * a.dim;
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < a.dkv_splits; ++i) s += p[i * step];
  const int64_t unit = row / a.k_len, b = unit / a.kv_heads, kvh = unit - b * a.kv_heads, j = row - unit * a.k_len;
  if (c < a.dim)
    ((T*)a.dk)[b * a.dks[0] + kvh * a.dks[1] + j * a.dks[2] + c] = (T)s;
  else
    ((T*)a.dv)[b * a.dvs[0] + kvh * a.dvs[1] + j * a.dvs[2] + c - a.dim] = (T)s;
}

template <class T, int DP, bool VEC>
int attn_backward_dim(const AttnArgs& a, void* stream) {
  static DeviceOnce once;
  const int opted = opted_in(once, [] {
    return lds_opt_in(attn_dq_kernel<T, DP, false, VEC, false>, attn_dq_lds<T, DP>(kAttnMaxFar, false)) |
           lds_opt_in(attn_dq_kernel<T, DP, true, VEC, false>, attn_dq_lds<T, DP>(kAttnMaxFar, true)) |
           lds_opt_in(attn_dq_kernel<T, DP, false, VEC, true>, attn_dq_lds<T, DP>(kAttnMaxFar, false)) |
           lds_opt_in(attn_dq_kernel<T, DP, true, VEC, true>, attn_dq_lds<T, DP>(kAttnMaxFar, true)) |
           lds_opt_in(attn_dkv_kernel<T, DP, VEC>, attn_dkv_lds<T, DP>(kAttnMaxFar));
  });
  if (opted != FM_OK) return opted;
  const bool table = a.d_table != nullptr;
  if (a.q_len > 0) {
    const int st = launch("attention backward (dq)",
                          a.dq_splits > 1 ? (table ? attn_dq_kernel<T, DP, true, VEC, true>
                                                   : attn_dq_kernel<T, DP, false, VEC, true>)
                                          : (table ? attn_dq_kernel<T, DP, true, VEC, false>
                                                   : attn_dq_kernel<T, DP, false, VEC, false>),
                          dim3(place_grid((int64_t)a.batch * a.kv_heads,
                                          (int64_t)attn_query_blocks(a) * (a.heads / a.kv_heads)),
                               (unsigned)a.dq_splits),
                          dim3(kAttnThreads), attn_dq_lds<T, DP>(a.far, table), stream, a);
    if (st != FM_OK) return st;
    if (a.dq_splits > 1) {
      const int st2 = launch("attention backward (dq join)", attn_dq_join_kernel<T>,
                             dim3((unsigned)(a.batch * a.heads * attn_query_blocks(a)), kAttnQueries / kDqJoinRows),
                             dim3(kAttnThreads), 0, stream, a);
      if (st2 != FM_OK) return st2;
    }
  }
  if (a.k_len > 0) {
    const int st = launch("attention backward (dk, dv)", attn_dkv_kernel<T, DP, VEC>,
                          dim3(place_grid((int64_t)a.batch * a.kv_heads,
                                          (a.k_len + kAttnBlockKeys - 1) / kAttnBlockKeys),
                               (unsigned)a.dkv_splits),
                          dim3(kAttnThreads), attn_dkv_lds<T, DP>(a.far), stream, a);
    if (st != FM_OK || a.dkv_splits == 1) return st;
    const int per = kAttnThreads / (a.dim <= 32 ? 64 : a.dim <= 64 ? 128 : 256);
    return launch("attention backward (join)", attn_dkv_join_kernel<T>,
                  dim3((unsigned)(((int64_t)a.batch * a.kv_heads * a.k_len + per - 1) / per)),
                  dim3(kAttnThreads), 0, stream, a);
  }
  return FM_OK;
}

template <class T>
int attn_backward_t(const AttnArgs& a, void* stream) {
  int st = FM_OK;
  if (a.batch > 0) {
    const bool vec = attn_groups(a.q, a.qs, a.dim, sizeof(T)) && attn_groups(a.k, a.ks, a.dim, sizeof(T)) &&
                     attn_groups(a.v, a.vs, a.dim, sizeof(T)) && attn_groups(a.d_o, a.dos, a.dim, sizeof(T)) && attn_groups(a.o, a.os, a.dim, sizeof(T));
    const auto go = [&](auto narrow, auto wide, auto widest) {
      return a.dim <= 64 ? narrow(a, stream) : a.dim <= 96 ? wide(a, stream) : widest(a, stream);
    };
    st = vec ? go(attn_backward_dim<T, 64, true>, attn_backward_dim<T, 96, true>,
                  attn_backward_dim<T, 128, true>)
             : go(attn_backward_dim<T, 64, false>, attn_backward_dim<T, 96, false>,
                  attn_backward_dim<T, 128, false>);
  }
  if (st != FM_OK || !a.d_table) return st;
  if ((int64_t)a.batch * attn_query_blocks(a) * a.dq_splits > kTableRows) {
    st = launch("attention backward (distances)", attn_table_distances_kernel<T>,
                dim3((unsigned)(bias_window(a.far) + 63) / 64, (unsigned)a.heads), dim3(1024), 0, stream, a);
    if (st != FM_OK) return st;
  }
  return launch("attention backward (buckets)",
                a.table32 ? attn_table_buckets_kernel<float> : attn_table_buckets_kernel<T>,
                dim3((unsigned)a.heads), dim3(1024), 0, stream, a);
}

}  // namespace fm
