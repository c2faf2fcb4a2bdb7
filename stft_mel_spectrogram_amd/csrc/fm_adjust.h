// Logits before a token is chosen: penalties for tokens of the history, biases,
// and a mask of allowed tokens.
//
//   x = x > 0 ? x (1 / rep) : x rep (tokens seen), x -= freq count + pres [count > 0],
//   x += sum of the token's biases, x = -inf where its bit is 0
//
// A workgroup of 512 lanes takes a segment of a row.  Its logits, the history and
// the biases are asked for at once; the history is counted into a slot per token in
// LDS while the logits are on their way (whole numbers, so that the order of the
// atomics is of no account).  Before that the biases have left the number of their
// token's first entry in its slot; where a token has several, that entry adds them up
// in order.  Then each lane works on its own elements: one read, one write, in place
// too.  Every segment reads the row's history and biases again, from the cache.
// Without a history bound by memory; with a long one by the vector units, 34 instructions
// per token (256 x 131072 f16, a history of 4000, 300 biases: 52 us from memory, 46 where
// the last-level cache still holds the operands, the units then busy 79% of the time;
// there without biases 38; with a mask alone 29 from memory, 4.7 TB/s).  8 x 50001 bf16: 5.
#pragma once

#include "fm_logit.h"
#include "fm_op.h"

namespace fm {

// A slot: bit 0 the token is in the history, 20 bits how often it counts, 11 bits
// kAdjustMaxBiases less the number of its first bias entry.
constexpr uint32_t kSlotOnce = 2, kSlotBias = 1u << 21;

template <class T, int V>
__global__ __launch_bounds__(kAdjustThreads) void adjust_kernel(const AdjustArgs a) {
  constexpr int VE = Vec16<T>::n, NT = kAdjustThreads, SEG = NT * VE * V;
  constexpr int HIST = V > 2 ? 4 : 8;                         // tokens of a lane at a time
  constexpr int BIAS = kAdjustMaxBiases / NT;      // bias entries of a lane
  extern __shared__ __attribute__((aligned(16))) uint32_t slots[];  // [SEG], ids and values of the biases
  int* bias_id = (int*)slots + SEG;
  float* bias_val = (float*)bias_id + a.biases;
  __shared__ int again;  // a token has several biases
  const int tid = threadIdx.x;
  // the segments of a row on one XCD, whose L2 then holds its history: workgroups 8
  // apart, for as many rows as are a multiple of 8
  const unsigned b = blockIdx.x;
  const bool spread = b >= (unsigned)(a.rows & ~(int64_t)7) * a.segs;
  const unsigned at = spread ? b : b / 8;
  const int64_t row = spread ? at / a.segs : at / a.segs * 8 + b % 8;
  const int beg = (int)(at % a.segs) * SEG;
  const int n = a.vocab - beg < SEG ? a.vocab - beg : SEG;
  const T* x = (const T*)a.x + row * a.x_stride + beg;
  T* out = (T*)a.out + row * a.vocab + beg;
  int len = a.history_len;
  if (a.history_lengths && len > 0) {
    const int l = a.history_lengths[row];
    len = l < 0 ? 0 : l < len ? l : len;
  }
  const int prompt = a.prompt_lengths && len > 0 ? a.prompt_lengths[row] : 0;
  const float rep = a.repetition ? a.repetition[row] : a.repetition_value;
  const float over = 1.f / rep;  // one rounding of 2^-24 more than a division, for a tenth of its instructions
  const float freq = a.frequency ? a.frequency[row] : a.frequency_value;
  const float pres = a.presence ? a.presence[row] : a.presence_value;
  // tokens as slots of this segment, or -1
  const auto slot = [&](uint32_t lo, uint32_t hi) {
    const uint32_t c = lo - (uint32_t)beg;
    const bool in = (int)(hi == 0) & (int)(c < (uint32_t)n);
    return in ? (int)c : -1;
  };
  const char* h = (const char*)a.history + row * a.history_stride * (a.history64 ? 8 : 4);
  int tok[HIST];
  // all of them, so that no load waits for the row's length, and without branches
  const auto history = [&](int first) {
    uint64_t id[HIST];
    const auto at = [&](int j) {
      const int k = first + j * NT + tid;
      return k < a.history_len ? k : a.history_len - 1;
    };
    if (a.history64) {
#pragma unroll
      for (int j = 0; j < HIST; ++j) id[j] = ((const uint64_t*)h)[at(j)];
    } else {
      // (a negative one is past every vocabulary)
#pragma unroll
      for (int j = 0; j < HIST; ++j) id[j] = ((const uint32_t*)h)[at(j)];
    }
#pragma unroll
    for (int j = 0; j < HIST; ++j) tok[j] = slot((uint32_t)id[j], (uint32_t)(id[j] >> 32));
  };
  const bool any = a.history_len > 0 || a.biases > 0;
  uint4* mine = (uint4*)slots;  // of group i * NT + tid: VE / 4 of these
  Vec16<T> raw[V];
  uint32_t bits[V];
  const auto logits = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * NT + tid) * VE;
      raw[i] = load16_part(x + c, n - c, (T)0.f);
    }
    if (a.allowed) {
      const uint8_t* p = a.allowed + row * a.allowed_stride;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * NT + tid) * VE;
        bits[i] = c < n ? (uint32_t)p[(beg + c) >> 3] >> (VE == 4 ? c & 4 : 0) : 0u;
      }
    }
  };
  if (any) {
    if (a.history_len > 0) history(0);
    int id[BIAS];
    float val[BIAS];
    if (a.biases > 0) {
      uint64_t t[BIAS];
#pragma unroll
      for (int j = 0; j < BIAS; ++j) {
        const int k = j * NT + tid < a.biases ? j * NT + tid : a.biases - 1;
        t[j] = ((const uint64_t*)a.bias_ids)[row * a.biases + k];
        val[j] = a.bias[row * a.biases + k];
      }
#pragma unroll
      for (int j = 0; j < BIAS; ++j)
        id[j] = j * NT + tid < a.biases ? slot((uint32_t)t[j], (uint32_t)(t[j] >> 32)) : -1;
    }
    logits();
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VE / 4; ++j) mine[(i * NT + tid) * (VE / 4) + j] = make_uint4(0, 0, 0, 0);
    if (tid == 0) again = 0;
    if (a.biases > 0) {
#pragma unroll
      for (int j = 0; j < BIAS; ++j)
        if (j * NT + tid < a.biases) {
          bias_id[j * NT + tid] = id[j];
          bias_val[j * NT + tid] = val[j];
        }
    }
    __syncthreads();
    if (a.biases > 0) {
#pragma unroll
      for (int j = 0; j < BIAS; ++j)
        if (id[j] >= 0) atomicMax(slots + id[j], (uint32_t)(kAdjustMaxBiases - (j * NT + tid)) * kSlotBias);
      __syncthreads();
    }
    if (a.history_len > 0) {
      for (int k = 0; k < len; k += HIST * NT) {
#pragma unroll
        for (int j = 0; j < HIST; ++j) {
          const int at = k + j * NT + tid;
          if (tok[j] >= 0 && at < len) {
            if (at < prompt)
              atomicOr(slots + tok[j], 1u);
            else
              atomicAdd(slots + tok[j], kSlotOnce);
          }
        }
        if (k + HIST * NT < len) history(k + HIST * NT);
      }
    }
    if (a.biases > 0) {
      // the others add to the slots' lower bits alone
#pragma unroll
      for (int j = 0; j < BIAS; ++j)
        if (id[j] >= 0 && slots[id[j]] / kSlotBias != (uint32_t)(kAdjustMaxBiases - (j * NT + tid))) again = 1;
    }
    __syncthreads();
    if (a.biases > 0 && again) {
      // a wave at a time looks for the entries of its lanes' tokens, 64 at a time
      float s[BIAS];
      bool first[BIAS];
#pragma unroll
      for (int j = 0; j < BIAS; ++j) {
        const int k = j * NT + tid;
        first[j] = id[j] >= 0 && slots[id[j]] / kSlotBias == (uint32_t)(kAdjustMaxBiases - k);
        s[j] = 0.f;
        for (uint64_t who = __ballot(first[j]); who; who &= who - 1) {
          const int lead = __builtin_ctzll(who);
          const int token = __builtin_amdgcn_readlane(id[j], lead);
          float sum = 0.f;
          for (int i = 0; i < a.biases; i += 64) {
            const int at = i + (tid & 63);
            const bool same = at < a.biases && bias_id[at] == token;
            const float v = same ? bias_val[at] : 0.f;
            for (uint64_t more = __ballot(same); more; more &= more - 1)
              sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), __builtin_ctzll(more)));
          }
          if ((tid & 63) == lead) s[j] = sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < BIAS; ++j)
        if (first[j]) bias_val[j * NT + tid] = s[j];
      __syncthreads();
    }
  } else {
    logits();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * NT + tid) * VE;
    if (any) {
      uint32_t k[VE], seen = 0;
      __builtin_memcpy(k, mine + (i * NT + tid) * (VE / 4), sizeof(k));
#pragma unroll
      for (int e = 0; e < VE; ++e) seen |= k[e];
      if (seen) {
        // without a branch per token: some lane of a wave takes nearly every one of them
        float v[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float r = (float)raw[i].v[e];
          const uint32_t once = k[e] % kSlotBias, count = once / kSlotOnce;
          const float w = once ? r * (r > 0.f ? over : rep) : r;
          v[e] = count ? fmaf(-freq, (float)count, w) - pres : w;
        }
        if (seen >= kSlotBias) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (k[e] >= kSlotBias) v[e] += bias_val[kAdjustMaxBiases - k[e] / kSlotBias];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) raw[i].v[e] = k[e] ? (T)v[e] : raw[i].v[e];
      }
    }
    if (c < n) {
      if (a.allowed) {
#pragma unroll
        for (int e = 0; e < VE; ++e) raw[i].v[e] = bits[i] >> e & 1u ? raw[i].v[e] : (T)-INFINITY;
      }
      store16_part(out + c, raw[i], n - c);
    }
  }
}

template <class T>
int adjust_t(AdjustArgs a, void* stream) {
  constexpr int VE = Vec16<T>::n;
  a.segs = adjust_segments(a.rows, a.vocab, VE);
  const int vecs = adjust_vecs(a.rows, a.vocab, VE);
  const bool any = a.history_len > 0 || a.biases > 0;
  const size_t lds = any ? 4 * (size_t)kAdjustThreads * VE * vecs + 8 * (size_t)a.biases : 0;
  const auto go = [&](auto kernel) {
    return launch("adjusted logits", kernel, dim3((unsigned)(a.rows * a.segs)), dim3(kAdjustThreads), lds, stream, a);
  };
  if constexpr (sizeof(T) == 4) {
    if (vecs == 4) return go(adjust_kernel<T, 4>);
  }
  return vecs == 1 ? go(adjust_kernel<T, 1>) : go(adjust_kernel<T, 2>);
}

}  // namespace fm
