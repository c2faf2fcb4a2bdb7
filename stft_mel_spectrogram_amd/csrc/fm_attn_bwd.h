// Attention backward: one kernel for dq and the bias table (a wave's 32
// queries in its registers, key tiles in LDS), one for dk and dv (a wave's 32
// keys in its registers, query tiles in LDS), and the table's sums.  Scores
// are computed again in both: seven matrix products instead of five, but no
// gradient is added up by atomics in memory, so results do not depend on the
// order in which workgroups run.
#pragma once

#include "fm_attn.h"

namespace fm {

constexpr int kAttnThreads = 256;
constexpr int kAttnBlockKeys = 128;  // keys of a dk, dv workgroup
template <class T>
constexpr int attn_step() { return sizeof(T) == 2 ? 64 : 32; }

// float16 has no room for small gradients: ds is scaled by the power of two
// that brings the largest |do| into [1, 2), so that ds stays within a few
// powers of two of v's size, and the scale is taken out at the end.  The
// other types have float32's exponents.
__device__ __forceinline__ float unit_scale(float amax) {
  const int e = clamp_int((int)(__float_as_uint(amax) >> 23) & 255, 1, 253);
  return amax == 0.f ? 1.f : __uint_as_float((uint32_t)(254 - e) << 23);
}
// float16 probabilities are scaled too: 2^8 p is a normal number from p =
// 2.4e-7 on.
template <class T>
constexpr float kProbShift = 0.f;
template <>
inline constexpr float kProbShift<f16_t> = 8.f;
template <class T>
constexpr bool kIsF16 = false;
template <>
inline constexpr bool kIsF16<f16_t> = true;

// Sums of ds by distance: one array per half wave, so that no two lanes of an
// instruction add to one address and the order of additions is the program's.
constexpr int kTableArrays = 8;

template <class T, int DP>
constexpr size_t attn_dq_lds(int far, bool table) {
  return 4 * attn_step<T>() * Tile<T, DP>::ld * sizeof(T) +
         bias_window(far) * sizeof(float) * (table ? 1 + kTableArrays : 1) + 8 * sizeof(float);
}

template <class T, int DP, bool TABLE>
__global__ __launch_bounds__(kAttnThreads) void attn_dq_kernel(const AttnArgs a) {
  constexpr int BK = attn_step<T>(), NS = BK / 32, LD = Tile<T, DP>::ld, KS = DP / 16, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  T* kt = (T*)smem;
  T* vt = kt + 2 * BK * LD;
  float* bias = (float*)(vt + 2 * BK * LD);
  const int win = bias_window(a.far);
  float* ends = bias + win;  // [4][2]
  float* sums = ends + 8;    // [kTableArrays][win]

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries;
  const Place at = place_of(a.batch * a.heads, blocks, blockIdx.x);
  if (at.none) return;
  const int b = at.unit / a.heads, head = at.unit % a.heads, kvh = head / (a.heads / a.kv_heads);
  const int qb = a.causal ? blocks - 1 - at.block : at.block;
  const int q0 = qb * kAttnQueries + wave * 32;
  const int i = q0 + n;
  const bool real = i < a.q_len;
  const int len = key_count(a, b), first = position_of_first(a, b);
  const int q_end = min((qb + 1) * kAttnQueries, a.q_len);
  const int k_end = a.causal ? clamp_int(first + q_end, 0, len) : len;

  const T* kp = (const T*)a.k + b * a.ks[0] + kvh * a.ks[1];
  const T* vp = (const T*)a.v + b * a.vs[0] + kvh * a.vs[1];
  TileLoad<T, DP, BK, kAttnThreads> kl, vl;
  kl.load(kp, a.ks[2], k_end, a.dim, tid);
  vl.load(vp, a.vs[2], k_end, a.dim, tid);
  const int64_t row = (int64_t)(b * a.heads + head) * a.q_len + i;
  Frag<T> qf[KS], gf[KS];
  float delta = 0.f, amax = 0.f;
  {
    const T* qp = (const T*)a.q + b * a.qs[0] + head * a.qs[1] + i * a.qs[2];
    const T* gp = (const T*)a.d_o + b * a.dos[0] + head * a.dos[1] + i * a.dos[2];
    const int64_t off = b * a.os[0] + head * a.os[1] + i * a.os[2];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * h, have = real ? a.dim - d : 0;
      qf[s] = load_frag(qp + d, have);
      gf[s] = load_frag(gp + d, have);
      const Frag<T> of = load_frag((const T*)a.o + off + d, have);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        delta = fmaf((float)gf[s][e], (float)of[e], delta);
        amax = fmaxf(amax, fabsf((float)gf[s][e]));
      }
      if (a.o_rest) {
        const Frag<T> rf = load_frag((const T*)a.o_rest + off + d, have);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf((float)gf[s][e], (float)rf[e], delta);
      }
    }
    delta += __shfl_xor(delta, 32, 64);
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
  }
  // empty rows and rows past the end: every probability is 0
  float lse2 = INFINITY;
  if (real) {
    const float v = a.lse[row];
    if (v != -INFINITY) lse2 = v * kLog2e;
    if (h == 0) {
      a.delta[row] = delta;
      if (kIsF16<T>) a.amax[row] = amax;
    }
  }
  const float unit = kIsF16<T> ? unit_scale(amax) : 1.f;
  fill_bias<T>(a, head, bias, tid, kAttnThreads);
  const float lo = bias_of<T>(a, head, -a.far) / a.scale, hi = bias_of<T>(a, head, a.far) / a.scale;
  if constexpr (TABLE)
    for (int t = tid; t < kTableArrays * win; t += kAttnThreads) sums[t] = 0.f;
  kl.store(kt, tid);
  vl.store(vt, tid);
  __syncthreads();

  acc16 dq[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[d][r] = 0.f;
  float before = 0.f, behind = 0.f;  // ds of the far tiles on either side
  float* mysums = sums + (wave * 2 + h) * win;
  const float c = a.scale * kLog2e;
  const int mine = a.causal ? min(len, first + i + 1) : len;
  const int least = a.causal ? min(len, first + q0 + 1) : len;
  const int wave_end = a.causal ? min(k_end, first + q0 + 32) : k_end;
  const bool idle = q0 >= a.q_len;

  int buf = 0;
  for (int j0 = 0; j0 < k_end; j0 += BK, buf ^= 1) {
    const bool more = j0 + BK < k_end;
    if (more) {
      kl.load(kp + (int64_t)(j0 + BK) * a.ks[2], a.ks[2], k_end - j0 - BK, a.dim, tid);
      vl.load(vp + (int64_t)(j0 + BK) * a.vs[2], a.vs[2], k_end - j0 - BK, a.dim, tid);
    }
    if (!idle && j0 < wave_end) {
      const T* ktb = kt + buf * BK * LD;
      const T* vtb = vt + buf * BK * LD;
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int dist = j0 + 32 * u - first - q0;
        acc16 s = bias_start_keys(bias, a.far, dist, lo, hi, h, n);
        acc16 dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) s = mma32(tile_rows<T, DP>(ktb, 32 * u + n, x, h), qf[x], s);
#pragma unroll
        for (int x = 0; x < KS; ++x) dp = mma32(tile_rows<T, DP>(vtb, 32 * u + n, x, h), gf[x], dp);
        if (j0 + 32 * u + 32 > least) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[r] = j0 + 32 * u + 8 * (r / 4) + 4 * h + r % 4 < mine ? s[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
        if constexpr (TABLE) {
          if (dist + 31 <= -a.far) {
#pragma unroll
            for (int r = 0; r < 16; ++r) before += s[r];
          } else if (dist - 31 >= a.far) {
#pragma unroll
            for (int r = 0; r < 16; ++r) behind += s[r];
          } else {
            float* p = mysums + dist + a.far + kBiasPad + 4 * h - n;
#pragma unroll
            for (int r = 0; r < 16; ++r)
              __hip_atomic_fetch_add(p + 8 * (r / 4) + r % 4, s[r], __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_WORKGROUP);
          }
        }
        if constexpr (kIsF16<T>) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] *= unit;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Frag<T> f = acc_frag<T>(s, x);
#pragma unroll
          for (int d = 0; d < DT; ++d)
            dq[d] = mma32(tile_cols<T, DP>(ktb, 32 * u + 16 * x, 32 * d, lane), f, dq[d]);
        }
      }
    }
    if (more) {
      kl.store(kt + (buf ^ 1) * BK * LD, tid);
      vl.store(vt + (buf ^ 1) * BK * LD, tid);
    }
    __syncthreads();
  }

  if (real) {
    const float f = a.scale / unit;
    T* out = (T*)a.dq + b * a.dqs[0] + head * a.dqs[1] + i * a.dqs[2];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at_d = 32 * d + 8 * y + 4 * h;
        if (at_d < a.dim)
          store4(out + at_d, dq[d][4 * y] * f, dq[d][4 * y + 1] * f, dq[d][4 * y + 2] * f,
                 dq[d][4 * y + 3] * f, a.dim - at_d);
      }
  }
  if constexpr (TABLE) {
    before = lanes_sum<64>(before);
    behind = lanes_sum<64>(behind);
    if (lane == 0) {
      ends[2 * wave] = before;
      ends[2 * wave + 1] = behind;
    }
    __syncthreads();
    // the window's first and last distances lie beyond +-far like the far tiles
    float* out = a.table_part + ((int64_t)at.unit * blocks + qb) * win;
    for (int t = tid; t < win; t += kAttnThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kTableArrays; ++w) v += sums[w * win + t];
      if (t == 0) v += (ends[0] + ends[2]) + (ends[4] + ends[6]);
      if (t == win - 1) v += (ends[1] + ends[3]) + (ends[5] + ends[7]);
      out[t] = v;
    }
  }
}

// Sums over entries and query blocks: by distance, 64 distances of a head per
// workgroup, 16 interleaved sets of partials.
template <class T>
__global__ __launch_bounds__(1024) void attn_table_distances_kernel(const AttnArgs a) {
  __shared__ float red[16][64];
  const int win = bias_window(a.far), blocks = (a.q_len + kAttnQueries - 1) / kAttnQueries;
  const int lane = threadIdx.x & 63, set = threadIdx.x >> 6, head = blockIdx.y;
  const int t = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (t < win)
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

// ... and by bucket, one head per workgroup, one thread per bucket.
template <class W>
__global__ __launch_bounds__(kAttnThreads) void attn_table_buckets_kernel(const AttnArgs a) {
  __shared__ float dist[bias_window(kAttnMaxFar)];
  __shared__ int16_t bucket[bias_window(kAttnMaxFar)];
  const int win = bias_window(a.far), head = blockIdx.x;
  for (int t = threadIdx.x; t < win; t += kAttnThreads) {
    dist[t] = a.table_dist[(int64_t)head * win + t];
    const int b = a.map[clamp_int(t - kBiasPad, 0, 2 * a.far)];
    bucket[t] = (int16_t)(b < 0 || b >= a.num_buckets ? -1 : b);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < a.num_buckets; k += kAttnThreads) {
    float s = 0.f;
    for (int t = 0; t < win; ++t) s += bucket[t] == k ? dist[t] : 0.f;
    ((W*)a.d_table)[(int64_t)k * a.heads + head] = (W)s;
  }
}

template <class T, int DP>
constexpr size_t attn_dkv_lds(int far) {
  return 4 * attn_step<T>() * Tile<T, DP>::ld * sizeof(T) + 4 * attn_step<T>() * sizeof(float) +
         bias_window(far) * sizeof(float);
}

template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_dkv_kernel(const AttnArgs a) {
  constexpr int BQ = attn_step<T>(), NS = BQ / 32, LD = Tile<T, DP>::ld, KS = DP / 16, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  // float32 fragments of 128 columns leave no registers for the next tile
  constexpr bool AHEAD = !(sizeof(T) == 4 && DP == 128);
  T* qt = (T*)smem;
  T* gt = qt + 2 * BQ * LD;
  float* lse2 = (float*)(gt + 2 * BQ * LD);  // [2][BQ]
  float* delta = lse2 + 2 * BQ;              // [2][BQ]
  float* bias = delta + 2 * BQ;

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int blocks = (a.k_len + kAttnBlockKeys - 1) / kAttnBlockKeys;
  const Place at = place_of(a.batch * a.kv_heads, blocks, blockIdx.x);
  if (at.none) return;
  const int b = at.unit / a.kv_heads, kvh = at.unit % a.kv_heads, group = a.heads / a.kv_heads;
  const int j_wg = at.block * kAttnBlockKeys, jw = j_wg + wave * 32, j = jw + n;
  const int len = key_count(a, b), first = position_of_first(a, b);

  Frag<T> kf[KS], vf[KS];
  {
    const T* kp = (const T*)a.k + b * a.ks[0] + kvh * a.ks[1] + j * a.ks[2];
    const T* vp = (const T*)a.v + b * a.vs[0] + kvh * a.vs[1] + j * a.vs[2];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * h, have = j < len ? a.dim - d : 0;
      kf[s] = load_frag(kp + d, have);
      vf[s] = load_frag(vp + d, have);
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
    // one scale for every query of the sums: the group's largest |do|
    float m = 0.f;
    const float* am = a.amax + (int64_t)(b * a.heads + kvh * group) * a.q_len;
    for (int64_t t = tid; t < (int64_t)group * a.q_len; t += kAttnThreads) m = fmaxf(m, am[t]);
    m = lanes_max<64>(m);
    if (lane == 0) lse2[wave] = m;
    __syncthreads();
    unit = unit_scale(fmaxf(fmaxf(lse2[0], lse2[1]), fmaxf(lse2[2], lse2[3])));
    __syncthreads();
  }
  const float c = a.scale * kLog2e;
  const float back = kIsF16<T> ? unit * __builtin_amdgcn_exp2f(-kProbShift<T>) : 1.f;
  // row i of the tile at i0 sees this lane's key if i >= need
  const int need = j >= len ? a.q_len : a.causal ? max(j - first, 0) : 0;

  for (int gi = 0; gi < group; ++gi) {
    const int head = kvh * group + gi;
    const T* qp = (const T*)a.q + b * a.qs[0] + head * a.qs[1];
    const T* gp = (const T*)a.d_o + b * a.dos[0] + head * a.dos[1];
    const int64_t row0 = (int64_t)(b * a.heads + head) * a.q_len;
    TileLoad<T, DP, BQ, kAttnThreads> ql, gl;
    float l_next = 0.f, d_next = 0.f;
    const auto fetch = [&](int i0) {
      ql.load(qp + (int64_t)i0 * a.qs[2], a.qs[2], i_end - i0, a.dim, tid);
      gl.load(gp + (int64_t)i0 * a.dos[2], a.dos[2], i_end - i0, a.dim, tid);
      if (tid < BQ) {
        const bool in = i0 + tid < i_end;
        const float v = in ? a.lse[row0 + i0 + tid] : -INFINITY;
        l_next = v == -INFINITY ? INFINITY : fmaf(v, kLog2e, -kProbShift<T>);
        d_next = in ? a.delta[row0 + i0 + tid] : 0.f;
      }
    };
    const auto put = [&](int buf) {
      ql.store(qt + buf * BQ * LD, tid);
      gl.store(gt + buf * BQ * LD, tid);
      if (tid < BQ) {
        lse2[buf * BQ + tid] = l_next;
        delta[buf * BQ + tid] = d_next;
      }
    };
    fetch(i_beg);
    fill_bias<T>(a, head, bias, tid, kAttnThreads);
    const float lo = bias_of<T>(a, head, -a.far) / a.scale, hi = bias_of<T>(a, head, a.far) / a.scale;
    put(0);
    __syncthreads();
    int buf = 0;
    for (int i0 = i_beg; i0 < i_end; i0 += BQ, buf ^= 1) {
      const bool more = i0 + BQ < i_end;
      if (AHEAD && more) fetch(i0 + BQ);
      if (jw < len && !(a.causal && i0 + BQ - 1 + first < jw)) {
        const T* qtb = qt + buf * BQ * LD;
        const T* gtb = gt + buf * BQ * LD;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          const int iu = i0 + 32 * u;
          acc16 s = bias_start_queries(bias, a.far, jw - first - iu, lo, hi, h, n);
          acc16 dp;
#pragma unroll
          for (int r = 0; r < 16; ++r) dp[r] = 0.f;
#pragma unroll
          for (int x = 0; x < KS; ++x) {
            s = mma32(tile_rows<T, DP>(qtb, 32 * u + n, x, h), kf[x], s);
            dp = mma32(tile_rows<T, DP>(gtb, 32 * u + n, x, h), vf[x], dp);
          }
          if (jw + 32 > len || (a.causal && jw + 31 - first > iu)) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
              s[r] = iu + 8 * (r / 4) + 4 * h + r % 4 >= need ? s[r] : -INFINITY;
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 l4 = *(const float4*)(lse2 + buf * BQ + 32 * u + 8 * y + 4 * h);
            const float4 d4 = *(const float4*)(delta + buf * BQ + 32 * u + 8 * y + 4 * h);
            const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 4 * y + e;
              s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -ls[e]));
              if constexpr (kIsF16<T>)
                dp[r] = s[r] * ((dp[r] - ds[e]) * back);
              else
                dp[r] = s[r] * (dp[r] - ds[e]);
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const Frag<T> p = acc_frag<T>(s, x), f = acc_frag<T>(dp, x);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              dv[d] = mma32(tile_cols<T, DP>(gtb, 32 * u + 16 * x, 32 * d, lane), p, dv[d]);
              dk[d] = mma32(tile_cols<T, DP>(qtb, 32 * u + 16 * x, 32 * d, lane), f, dk[d]);
            }
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
  T* ok = (T*)a.dk + b * a.dks[0] + kvh * a.dks[1] + j * a.dks[2];
  T* ov = (T*)a.dv + b * a.dvs[0] + kvh * a.dvs[1] + j * a.dvs[2];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int at_d = 32 * d + 8 * y + 4 * h;
      if (at_d < a.dim) {
        store4(ok + at_d, dk[d][4 * y] * fk, dk[d][4 * y + 1] * fk, dk[d][4 * y + 2] * fk,
               dk[d][4 * y + 3] * fk, a.dim - at_d);
        store4(ov + at_d, dv[d][4 * y] * fv, dv[d][4 * y + 1] * fv, dv[d][4 * y + 2] * fv,
               dv[d][4 * y + 3] * fv, a.dim - at_d);
      }
    }
}

template <class T, int DP>
int attn_backward_dim(const AttnArgs& a, void* stream) {
  static const int opted = lds_opt_in(attn_dq_kernel<T, DP, false>, attn_dq_lds<T, DP>(kAttnMaxFar, false)) |
                           lds_opt_in(attn_dq_kernel<T, DP, true>, attn_dq_lds<T, DP>(kAttnMaxFar, true)) |
                           lds_opt_in(attn_dkv_kernel<T, DP>, attn_dkv_lds<T, DP>(kAttnMaxFar));
  if (opted != FM_OK) return set_error(FM_E_HIP, "attention backward: LDS size refused");
  const bool table = a.d_table != nullptr;
  if (a.q_len > 0) {
    const int st = launch("attention backward (dq)",
                          table ? attn_dq_kernel<T, DP, true> : attn_dq_kernel<T, DP, false>,
                          dim3(place_grid((int64_t)a.batch * a.heads, attn_query_blocks(a))),
                          dim3(kAttnThreads), attn_dq_lds<T, DP>(a.far, table), stream, a);
    if (st != FM_OK) return st;
  }
  if (a.k_len > 0)
    return launch("attention backward (dk, dv)", attn_dkv_kernel<T, DP>,
                  dim3(place_grid((int64_t)a.batch * a.kv_heads,
                                  (a.k_len + kAttnBlockKeys - 1) / kAttnBlockKeys)),
                  dim3(kAttnThreads), attn_dkv_lds<T, DP>(a.far), stream, a);
  return FM_OK;
}

template <class T>
int attn_backward_t(const AttnArgs& a, void* stream) {
  int st = FM_OK;
  if (a.batch > 0)
    st = a.dim <= 64   ? attn_backward_dim<T, 64>(a, stream)
         : a.dim <= 96 ? attn_backward_dim<T, 96>(a, stream)
                       : attn_backward_dim<T, 128>(a, stream);
  if (st != FM_OK || !a.d_table) return st;
  st = launch("attention backward (distances)", attn_table_distances_kernel<T>,
              dim3((unsigned)(bias_window(a.far) + 63) / 64, (unsigned)a.heads), dim3(1024), 0, stream, a);
  if (st != FM_OK) return st;
  return launch("attention backward (buckets)",
                a.table32 ? attn_table_buckets_kernel<float> : attn_table_buckets_kernel<T>,
                dim3((unsigned)a.heads), dim3(kAttnThreads), 0, stream, a);
}

}  // namespace fm
