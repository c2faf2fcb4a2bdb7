// Logits before a token is chosen: penalties for tokens of the history, biases,
// and a mask of allowed tokens.
//
//   x = x > 0 ? x / rep : x rep (tokens seen), x -= freq count + pres [count > 0],
//   x += sum of the token's biases, x = -inf where its bit is 0
//
// A workgroup takes a segment of a row: its logits go to registers while the
// history is counted into LDS (whole numbers, so that the order of the atomics is
// of no account: bit 0 says seen, the rest counts), then each lane works on its
// own elements: one read and one write, in place too.  The segment's biases are
// listed in order by one wave, and the first entry of each token writes their sum
// into the slots that the counts have left.  Memory bound where the history is
// short against the vocabulary; every segment reads the row's history again, from
// the cache.
#pragma once

#include "fm_logit.h"
#include "fm_op.h"

namespace fm {

template <class T, int V>
__global__ __launch_bounds__(256) void adjust_kernel(const AdjustArgs a) {
  constexpr int VE = Vec16<T>::n, SEG = 256 * VE * V;
  __shared__ __attribute__((aligned(16))) uint32_t count[SEG];
  __shared__ int bias_id[kAdjustMaxBiases];
  __shared__ float bias_val[kAdjustMaxBiases];
  __shared__ int bias_n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t row = blockIdx.x / a.segs;
  const int beg = (int)(blockIdx.x - row * a.segs) * SEG;
  const int n = a.vocab - beg < SEG ? a.vocab - beg : SEG;
  const T* x = (const T*)a.x + row * a.x_stride + beg;
  T* out = (T*)a.out + row * a.vocab + beg;
  Vec16<T> raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * 256 + tid) * VE;
    raw[i] = load16_part(x + c, n - c, (T)0.f);
  }
  uint32_t bits[V];
  if (a.allowed) {
    const uint8_t* p = a.allowed + row * a.allowed_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * 256 + tid) * VE;
      bits[i] = c < n ? (uint32_t)p[(beg + c) >> 3] >> (VE == 4 ? c & 4 : 0) : 0u;
    }
  }
  float v[V][VE];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < VE; ++e) v[i][e] = (float)raw[i].v[e];

  int len = a.history_len;
  if (a.history_lengths && len > 0) {
    const int l = a.history_lengths[row];
    len = l < 0 ? 0 : l < len ? l : len;
  }
  uint4* mine = (uint4*)count;  // group (i * 256 + tid): VE / 4 of these
  const auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VE / 4; ++j) mine[(i * 256 + tid) * (VE / 4) + j] = make_uint4(0, 0, 0, 0);
  };
  // the segment's biases, in their order, by the last wave
  if (a.biases > 0 && tid >= 192) {
    int m = 0;
    for (int i = 0; i < a.biases; i += 64) {
      const int k = i + lane;
      int64_t id = -1;
      float b = 0.f;
      if (k < a.biases) {
        id = a.bias_ids[row * a.biases + k];
        b = a.bias[row * a.biases + k];
      }
      const bool in = id >= beg && id < (int64_t)beg + n;
      const uint64_t who = __ballot(in);
      const int at = m + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
      if (in) {
        bias_id[at] = (int)(id - beg);
        bias_val[at] = b;
      }
      m += __popcll(who);
    }
    if (lane == 0) bias_n = m;
  }
  if (len > 0) {
    clear();
    __syncthreads();
    int prompt = 0;
    if (a.prompt_lengths) prompt = a.prompt_lengths[row];
    const auto add = [&](int i, int64_t token) {
      const int64_t c = token - beg;
      if (c < 0 || c >= n) return;
      if (i < prompt)
        atomicOr(count + c, 1u);
      else
        atomicAdd(count + c, 2u);
    };
    const char* h = (const char*)a.history + row * a.history_stride * (a.history64 ? 8 : 4);
    for (int i = tid; i < len; i += 1024) {
      int64_t tok[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = i + 256 * j;
        tok[j] = k >= len ? -1 : a.history64 ? ((const int64_t*)h)[k] : ((const int32_t*)h)[k];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) add(i + 256 * j, tok[j]);
    }
    __syncthreads();
    const float rep = a.repetition ? a.repetition[row] : a.repetition_value;
    const float freq = a.frequency ? a.frequency[row] : a.frequency_value;
    const float pres = a.presence ? a.presence[row] : a.presence_value;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t k[VE];
      uint32_t any = 0;
      __builtin_memcpy(k, mine + (i * 256 + tid) * (VE / 4), sizeof(k));
#pragma unroll
      for (int e = 0; e < VE; ++e) any |= k[e];
      if (any) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (k[e]) {
            const float s = v[i][e] > 0.f ? v[i][e] / rep : v[i][e] * rep;
            v[i][e] = k[e] > 1u ? s - freq * (float)(k[e] >> 1) - pres : s;
          }
      }
    }
  }
  if (a.biases > 0) {
    clear();
    __syncthreads();
    const int m = bias_n;
    if (m > 0) {
      for (int k = tid; k < m; k += 256) {
        const int id = bias_id[k];
        float s = 0.f;
        bool first = true;
        for (int j = 0; j < m; ++j)
          if (bias_id[j] == id) {
            s += bias_val[j];
            first &= j >= k;
          }
        if (first) count[id] = __float_as_uint(s);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float b[VE];
        __builtin_memcpy(b, mine + (i * 256 + tid) * (VE / 4), sizeof(b));
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] += b[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * 256 + tid) * VE;
    if (c < n) {
      Vec16<T> o;
#pragma unroll
      for (int e = 0; e < VE; ++e) o.v[e] = (T)(a.allowed && !(bits[i] >> e & 1u) ? -INFINITY : v[i][e]);
      store16_part(out + c, o, n - c);
    }
  }
}

template <class T>
int adjust_t(AdjustArgs a, void* stream) {
  constexpr int VE = Vec16<T>::n;
  a.segs = adjust_segments(a.rows, a.vocab, VE);
  const int vecs = adjust_vecs(a.rows, a.vocab, VE);
  return launch("adjusted logits",
                vecs == 1 ? adjust_kernel<T, 1> : vecs == 2 ? adjust_kernel<T, 2> : adjust_kernel<T, 4>,
                dim3((unsigned)(a.rows * a.segs)), dim3(256), 0, stream, a);
}

}  // namespace fm
