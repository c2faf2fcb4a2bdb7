// Internal declarations of the speech-model operators: the arguments that
// the C ABI (fm_ops.cpp) has checked, and the launches per element type
// (fm_op_*.hip).  No HIP types, so that host-only builds can include it.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "fm_internal.h"

namespace fm {

// Work that each device needs once, such as a kernel's attributes.  What fails is
// tried again by the next call; devices from 64 on do it every time.
class DeviceOnce {
 public:
  template <class F>
  int operator()(int device, F work) {
    const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return FM_OK;
    const int st = work();
    if (st == FM_OK) done_.fetch_or(bit, std::memory_order_release);
    return st;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// A grid may have fewer than 2^32 threads in a dimension.  Calls launch(first, count)
// for consecutive ranges of at most `most` rows; kGridThreads over a row's threads is
// such a number of rows.
constexpr int64_t kGridThreads = int64_t(1) << 31;
template <class F>
int by_rows(int64_t rows, int64_t most, F launch) {
  for (int64_t at = 0; at < rows; at += most) {
    const int st = launch(at, rows - at < most ? rows - at : most);
    if (st != FM_OK) return st;
  }
  return FM_OK;
}

struct NormForward {
  const void* x;
  int64_t x_stride;  // elements between rows
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows;
  int width;
  float eps;
  void* stream;
};

struct NormBackward {
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dw;
  void* db;
  void* workspace;
  int64_t rows;
  int width;
  void* stream;
};

constexpr int kNormMaxWidth = 1 << 20;
constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 2048;  // workgroups that walk over rows: 8 per CU

// Lane layout of a width: lanes per row and 16-byte groups per lane.  At most 16
// elements per lane, and at most 8 in workgroups of 512 and 1024 threads, so that
// the backward's two sums per column fit beside the row with four waves per SIMD.
// Few lanes with more groups suit short rows (us, backward: 24008 x 128 f32, 16
// lanes of 2 groups 12.3, 64 lanes of 1 14.3; 96064 x 1024 bf16, 64 lanes of 2
// groups 130, 256 lanes of 1 197), more lanes long ones (24016 x 4096 bf16: 512
// lanes of 1 group 136, 256 lanes of 2 150; 12008 x 8192: 1024 of 1 130, 256 of 4
// 200).  Rows beyond 1024 lanes do not stay in registers: {1024, 0}, sweeps that
// read the row again from the cache.
struct NormShape {
  int lpr, vpl;
};
inline NormShape norm_shape(int width, int ve) {
  const int nvec = (width + ve - 1) / ve;
  if (nvec <= 16) return {16, 1};
  if (nvec <= 32) return {16, 2};
  if (nvec <= 64) return {64, 1};
  if (nvec <= 128) return {64, 2};
  if (nvec <= 256) return {256, 1};
  if (nvec <= 512) return {512, 1};
  if (nvec <= 1024) return {1024, 1};
  if (nvec <= 2048 && ve == 4) return {1024, 2};
  return {1024, 0};
}
#define FM_NORM_SHAPES(X) X(16, 1) X(16, 2) X(64, 1) X(64, 2) X(256, 1) X(512, 1) X(1024, 1) X(1024, 2)
// Threads of a workgroup and the rows it holds at a time.
constexpr int norm_threads(int lpr) { return lpr > kNormThreads ? lpr : kNormThreads; }
constexpr int norm_most(int lpr) { return lpr > 256 ? 8 : 16; }  // elements of a lane
constexpr int norm_rows(int lpr) { return norm_threads(lpr) / lpr; }

// Whether one workgroup of the backward takes all rows: four passes over its
// rows take about as long on the GPU as two launches (us: 16 x 122 f32 3.5
// against 5.2, 64 x 122 5.9 against 5.5, 16 x 1024 bf16 9.1 against 7.2), and a
// call 5 us less on the host (14.5 against 19.3).
inline bool norm_single(int64_t rows, int width, int ve) {
  const NormShape s = norm_shape(width, ve);
  return s.vpl > 0 && rows > 0 && rows <= 4 * norm_rows(s.lpr);
}
// Partial rows (workgroups of the backward, which walk over the rows): as many
// as the chip holds at once, 1024 threads per compute unit (24016 x 4096 bf16:
// 136 us, 150 with twice as many; 48032 x 2048: 135, 198 with half).  Fewer for few
// rows, 8 per partial row while that leaves one workgroup per unit, since a
// partial row's sums cost as much traffic as three rows (1000 x 2048: 12 us, 25
// with a partial row per row).
inline int norm_parts(int64_t rows, int width, int ve) {
  const NormShape s = norm_shape(width, ve);
  if (norm_single(rows, width, ve)) return 1;
  const int rpb = s.vpl > 0 ? norm_rows(s.lpr) : 1;
  const int64_t need = (rows + rpb - 1) / rpb;
  int64_t most = s.vpl == 0 ? 64 : 1024 * kNormThreads / norm_threads(s.lpr);
  if (s.vpl > 0 && rows / 8 < most) most = rows / 8 < 256 ? 256 : rows / 8;
  return (int)(need < most ? need : most);
}

// One translation unit per element type; w32: float32 parameters.
int norm_forward_f32(const NormForward& a);
int norm_forward_f16(const NormForward& a, bool w32);
int norm_forward_bf16(const NormForward& a, bool w32);
int norm_backward_f32(const NormBackward& a);
int norm_backward_f16(const NormBackward& a, bool w32);
int norm_backward_bf16(const NormBackward& a, bool w32);

struct ScoreForward {
  const void* x;
  int64_t x_stride;  // elements between rows
  int64_t x_inner;   // 0, or rows of a group at that stride and
  int64_t x_outer;   // the elements between groups
  const void* tokens;
  int tok64;
  float* lp;
  float* ent;
  float* lse;
  int64_t* top_ids;
  float* top_lp;
  void* workspace;
  int64_t rows;
  int vocab;
  int top;
  void* stream;
};

struct ScoreBackward {
  const void* x;
  int64_t x_stride;
  int64_t x_inner;
  int64_t x_outer;
  const void* tokens;
  int tok64;
  const float* lse;
  const float* ent;
  const float* g_lp;
  const float* g_ent;
  const int64_t* top_ids;
  const float* g_top;
  void* dx;
  int64_t rows;
  int vocab;
  int top;
  void* stream;
};

constexpr int kScoreMaxTop = 64;  // one kept entry per lane of a wave

// Work split of a call: lanes of a row (256: a workgroup per row segment), 16-
// byte groups of a lane, segments and their length.  Short rows lie in 16 lanes
// (24008 x 129 f32: 4.5 us, in a whole wave 8.3), with top alternatives in a wave.
// Long rows take segments while their workgroups fit on the chip at once, 5 per
// compute unit: of one chunk of 4 groups per lane below 256 rows (128 x 32000, 5
// alternatives: 13 us, unsegmented 30; 64 x 32000 without: 5.9 and 7.2), of 4
// chunks for more rows (300 x 131072, 20 alternatives: 43 us, unsegmented 58; 512 x
// 32000 of one chunk 11.8, unsegmented 10.9).  Chunks of one group per lane where
// the others leave units idle (8 x 50001, 5 alternatives: 10 us, of 4 groups 16,
// unsegmented 38; without: 5.0, 5.9 and 10.9).
struct ScoreSplit {
  int lanes, vecs, segs, seg_len;
};
inline ScoreSplit score_split(int64_t rows, int vocab, int ve, int top) {
  const int groups = (vocab + ve - 1) / ve;
  if (groups <= 256) {
    if (top > 0) return {64, groups <= 64 ? 1 : groups <= 128 ? 2 : 4, 1, vocab};
    if (groups <= 64) return {16, groups <= 16 ? 1 : groups <= 32 ? 2 : 4, 1, vocab};
    return {64, groups <= 128 ? 2 : 4, 1, vocab};
  }
  int vecs = 4, chunk = 256 * ve * 4, chunks = (vocab + chunk - 1) / chunk;
  if (rows * chunks < 256) {
    vecs = 1;
    chunk = 256 * ve;
    chunks = (vocab + chunk - 1) / chunk;
  }
  int64_t segs = rows > 0 ? 1280 / rows : 1;
  const int most = rows < 256 ? chunks : chunks / 4;
  if (segs > most) segs = most;
  if (segs < 1) segs = 1;
  const int per = (chunks + (int)segs - 1) / (int)segs;
  return {256, vecs, (chunks + per - 1) / per, per * chunk};
}
// Where a segment ends.  The last ones may reach past the row by up to segs - 1
// chunks: beg + seg_len alone would leave int near the longest vocabularies.
constexpr int score_segment_end(int beg, int seg_len, int vocab) {
  return vocab - beg < seg_len ? vocab : beg + seg_len;
}
inline int64_t score_part_bytes(int64_t rows, int segs) {
  return (rows * segs * 3 * (int64_t)sizeof(float) + 15) / 16 * 16;
}
inline int64_t score_workspace(int64_t rows, int vocab, int top, int ve) {
  const ScoreSplit p = score_split(rows, vocab, ve, top);
  return p.segs == 1 ? 0 : score_part_bytes(rows, p.segs) + rows * p.segs * (int64_t)top * 8;
}

// Attention with a relative position bias; strides in elements (entry, head,
// time), the last axis contiguous.  Also the kernels' argument.
struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* table;         // [num_buckets, heads]
  const int32_t* map;        // [2 far + 1]
  const int32_t* key_lengths;   // [batch] or NULL
  const int32_t* query_offset;  // [batch] or NULL: query_offset_value
  int query_offset_value;
  int far, num_buckets, table32, causal;
  int batch, heads, kv_heads, q_len, k_len, dim;
  int size;  // bytes of an element
  float scale;
  int64_t qs[3], ks[3], vs[3], os[3];
  void* o;
  float* lse;    // [batch, heads, q_len] or NULL
  // backward
  const void* d_o;
  int64_t dos[3], dqs[3], dks[3], dvs[3];
  void* dq;
  void* dk;
  void* dv;
  void* d_table;
  float* delta;       // [batch, heads, q_len]
  float* amax;        // [batch, heads, q_len] norm of a row of do, float16 only
  float* table_part;  // [batch * heads * query blocks * dq_splits, distances of the window]
  float* table_dist;  // [heads, distances of the window]
  float* part_dkv;    // [dkv_splits, batch, kv_heads, k_len, 2, dim]
  float* part_dq;     // [dq_splits, batch, heads, q_len, dim]
  float* part_row;    // [dq_splits, batch, heads, q_len, 3]
  int dkv_splits, dq_splits;
  // forward over key ranges
  float* part_o;    // [splits, batch, heads, q_len, dim]
  float* part_lse;  // [splits, batch, heads, q_len]
  int splits;
};

constexpr int kAttnMaxDim = 128;
constexpr int kAttnMaxFar = 1024;
constexpr int kAttnMaxBuckets = 1024;
constexpr int kAttnMaxSplits = 512; // key ranges of a forward call
constexpr int kAttnQueries = 128;   // queries of a workgroup

// Few queries against a cache take a kernel of their own, whose waves divide the
// keys instead of the queries (bf16 at 64 columns, us: 8 x 16 heads, 1501 keys, 1
// query 13, the other kernel 19; 32 queries 14.3 and 18.3, 48 queries 25.9 and
// 20.3; 6 x 4 heads on 1, 7 queries, 68001 keys 30 and 102).  Short rows do not
// make up for its join of the waves (8 x 16, 32 queries, 128 keys: 9.6 and 6.0; 300
// keys, 1 query: 7.1 and 8.7).
inline bool attn_token_kernel(const AttnArgs& a) { return a.q_len <= 32 && a.k_len > 256; }
inline int64_t attn_token_blocks(const AttnArgs& a) {
  return ((int64_t)a.q_len * (a.heads / a.kv_heads) + 15) / 16;
}
// Waves of its workgroups: as many as its registers and LDS let one compute unit
// hold, since they join without a second launch.
constexpr int attn_token_waves(int size, int dp) {
  return size == 2 ? (dp == 64 ? 16 : 8) : (dp == 64 ? 8 : 4);
}
// Key ranges a forward call is cut into while its workgroups alone do not fill
// the chip (256 compute units), us in bf16 at 64 columns, a call's GPU time:
// Few queries: one of their large workgroups per unit (2 x 8 key heads, 20000
// keys: 20.8, with two 23.8), of 512 keys, one round of 16 waves (1 x 8, 8000: 12.3;
// ranges of 2048 keys 17.2, none 39.4).  Where the workgroups reach a third of the
// units they draw the whole memory rate without a join (8 x 16, 8000: 40.3, two
// ranges 44.5), and a short call's join costs more on the host than it gains
// (8 x 16, 1501: 12.7; 1 x 1, 1501: 11.6 and 14.6 with the host's part, 11.5 and
// 19.5 with ranges).
// Others: two workgroups per unit, of 256 keys (1 x 8 heads, 101 queries, 4000
// keys: 15.0; ranges of 512 17.3, none 70.2), from 1024 keys on (1 x 8, 600
// queries, 600 keys: 15.3, with ranges 17.7; 1 x 16, 400, 1000: 21.9 and 21.3).
inline int attn_splits(const AttnArgs& a) {
  const bool token = attn_token_kernel(a);
  const int64_t wgs = token ? (int64_t)a.batch * a.kv_heads * attn_token_blocks(a)
                            : (int64_t)a.batch * a.heads * ((a.q_len + kAttnQueries - 1) / kAttnQueries);
  if (wgs == 0 || wgs > (token ? 85 : 256) || a.k_len < (token ? 2048 : 1024)) return 1;
  const int64_t fill = (token ? 256 : 512) / wgs, most = a.k_len / (token ? 512 : 256);
  return (int)(fill < most ? fill : most);
}
inline int64_t attn_round16(int64_t n) { return (n + 15) / 16 * 16; }
inline int64_t attn_rows(const AttnArgs& a) { return (int64_t)a.batch * a.heads * a.q_len; }
inline int attn_query_blocks(const AttnArgs& a) {
  return (a.q_len + kAttnQueries - 1) / kAttnQueries;
}
inline int64_t attn_forward_workspace(const AttnArgs& a) {
  const int s = attn_splits(a);
  return s == 1 ? 0 : attn_round16(4 * s * attn_rows(a) * a.dim) + 4 * s * attn_rows(a);
}
// Distances of the bias window: +-(far + 63), see fm_attn.h.
constexpr int kBiasPad = 63;
constexpr int bias_window(int far) { return 2 * (far + kBiasPad) + 1; }
constexpr int kAttnBlockKeys = 128;  // keys of a dk, dv workgroup
// Shares of the queries (of all heads of a group, in order) that workgroups of the
// dk, dv kernel take of a key block, while the blocks alone leave compute units
// idle; a second launch adds them up.  Shares of at least 4 tiles of 64 queries,
// 16 where there are blocks for a quarter of the units, since the sums are as much
// traffic per block then as they save.  Whole backward with dq in one range, us: 2
// x 4 heads on 1, 1777 queries, 28 blocks, 18 shares 109, unshared 268; 3 x 8 on 4,
// 1098, 128 columns, 108 blocks, 2 shares 130 and 165; 2 x 8 on 8, 1000, 128 blocks,
// unshared 68, 4 shares 74.  float32, whose tiles of 32 queries take as long as two
// of those and whose workgroups have a compute unit to themselves: single tiles
// below 48 blocks (1 x 8, 101 queries, 96 columns: 4 shares 46, unshared 55; 5 x 16
// on 4, 202, 40 blocks, 6 shares 62, unshared 131; 1 x 8, 500: 8 shares 77, 2 shares
// 87, 16 shares 89), else 8 (8 x 8, 101, 64 blocks: unshared 44, 4 shares 46).
inline int attn_dkv_splits(const AttnArgs& a) {
  const int64_t wgs = (int64_t)a.batch * a.kv_heads * ((a.k_len + kAttnBlockKeys - 1) / kAttnBlockKeys);
  if (wgs == 0 || wgs > 256) return 1;
  const bool f32 = a.size == 4;
  const int rows = f32 ? 32 : 64;
  const int64_t tiles = (int64_t)(a.heads / a.kv_heads) * ((a.q_len + rows - 1) / rows);
  const int64_t least = f32 ? (wgs <= 48 ? 1 : 8) : wgs <= 64 ? 4 : 16;
  const int64_t fill = (f32 ? 256 : 512) / wgs, most = tiles / least;
  const int64_t s = fill < most ? fill : most;
  return s < 1 ? 1 : (int)s;
}
// Ranges of the keys that workgroups of the dq kernel take while the query blocks
// alone leave compute units idle, of at least 8 tiles of 32 keys (float32, whose
// tiles take longer: 4); a second launch joins them.  Whole backward, us, against
// one range: 1 x 1 head, 2295, 80 columns, f32 causal 98 and 289; 1 x 2, 825, 128, f32
// 93 and 177 (with 8 tiles 109); 1 x 1, 2139, 128, f16 75 and 129 (with 4 tiles 83);
// 1 x 8, 1501, 64, bf16, 96 blocks 80 and 87; 2 x 8, 1000, 128 blocks 69 and 67.
inline int attn_dq_splits(const AttnArgs& a) {
  const int64_t wgs = (int64_t)a.batch * a.heads * attn_query_blocks(a);
  if (wgs == 0 || wgs > 128) return 1;
  const int64_t fill = 256 / wgs, most = a.k_len / (a.size == 4 ? 128 : 256);
  const int64_t s = fill < most ? fill : most;
  return s < 1 ? 1 : (int)s;
}
struct AttnBackwardSpace {
  int64_t amax, part, dist, dkv, dq, row, total;  // byte offsets; delta at 0
};
inline AttnBackwardSpace attn_backward_space(const AttnArgs& a, bool f16) {
  const int64_t rows = attn_round16(4 * attn_rows(a));
  AttnBackwardSpace s;
  s.amax = rows;
  s.part = rows * (f16 ? 2 : 1);
  const int splits = attn_dkv_splits(a), ranges = attn_dq_splits(a);
  s.dist = s.part +
           attn_round16(4 * (int64_t)a.batch * a.heads * attn_query_blocks(a) * ranges * bias_window(a.far));
  s.dkv = s.dist + attn_round16(4 * (int64_t)a.heads * bias_window(a.far));
  s.dq = s.dkv +
         (splits == 1 ? 0 : attn_round16(8 * (int64_t)splits * a.batch * a.kv_heads * a.k_len * a.dim));
  s.row = s.dq + (ranges == 1 ? 0 : attn_round16(4 * ranges * attn_rows(a) * a.dim));
  s.total = s.row + (ranges == 1 ? 0 : 12 * ranges * attn_rows(a));
  return s;
}

// Whether a call's grids stay below 2^32 threads (units rounded up to the 8 XCDs).
inline bool attn_fits_grids(const AttnArgs& a) {
  const auto fits = [](int64_t units, int64_t blocks, int threads) {
    const int64_t most = (int64_t(1) << 32) / threads;
    return units < most && blocks < most && units * blocks < most;
  };
  const int64_t units = (int64_t)a.batch * a.kv_heads + 7, group = a.heads / a.kv_heads;
  const int64_t queries = (a.q_len + (int64_t)kAttnQueries - 1) / kAttnQueries;
  const int64_t keys = (a.k_len + (int64_t)kAttnBlockKeys - 1) / kAttnBlockKeys;
  const int dp = a.dim <= 64 ? 64 : a.dim <= 96 ? 96 : 128;
  return fits(units, queries * group, 256) && fits(units, keys, 256) &&
         (!attn_token_kernel(a) || fits(units, attn_token_blocks(a), 64 * attn_token_waves(a.size, dp)));
}

// Whether rows are whole, aligned 16-byte groups and a block of them lies
// within a buffer load's reach (128 rows, 31-bit byte offsets).
inline bool attn_groups(const void* p, const int64_t* stride, int dim, int size) {
  const int n = 16 / size;
  return dim % n == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride[0] % n == 0 &&
         stride[1] % n == 0 && stride[2] % n == 0 &&
         (127 * stride[2] + dim) * size < 0x7fff0000;
}

int attn_forward_f32(const AttnArgs& a, void* stream);
int attn_forward_f16(const AttnArgs& a, void* stream);
int attn_forward_bf16(const AttnArgs& a, void* stream);
int attn_backward_f32(const AttnArgs& a, void* stream);
int attn_backward_f16(const AttnArgs& a, void* stream);
int attn_backward_bf16(const AttnArgs& a, void* stream);

int score_forward_f32(const ScoreForward& a);
int score_forward_f16(const ScoreForward& a);
int score_forward_bf16(const ScoreForward& a);
int score_backward_f32(const ScoreBackward& a);
int score_backward_f16(const ScoreBackward& a);
int score_backward_bf16(const ScoreBackward& a);

}  // namespace fm
