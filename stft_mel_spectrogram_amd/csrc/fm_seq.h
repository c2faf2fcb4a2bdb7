// Internal declarations of the gated recurrence and the root-mean-square norm:
// the arguments that the C ABI (fm_seq.cpp) has checked, the rules that split
// work, and the launches per element type (fm_op_scan_*.hip, fm_op_rms_*.hip).
// No HIP types, so that host-only builds can include it.
#pragma once

#include "fm_ops.h"

namespace fm {

// Gated linear recurrence; strides in elements of (entry, time), the last axis
// contiguous.  Also the kernels' argument.
struct ScanArgs {
  const void* x;
  const void* f;
  const void* g;  // or NULL
  int64_t xs[2], fs[2], gs[2];
  const float* state;      // [batch, channels] or NULL
  const int32_t* lengths;  // [batch] or NULL
  void* y;                 // [batch, time, channels]
  float* last;             // [batch, channels]
  float* saved;            // [batch, blocks of kScanSave frames, channels] or NULL
  // backward
  const void* dy;
  int64_t dys[2];
  const float* dlast;  // or NULL
  void* dx;
  void* df;
  void* dg;
  float* dstate;  // or NULL
  float* part;    // [batch, splits, channels rounded up to a workgroup's, 2]
  int batch, time, channels;
  int splits, chunk;  // time ranges and their length
};

constexpr int kScanSave = 64;   // frames between saved states
constexpr int kScanWaves = 8;   // waves of a workgroup, one time range of a tile each

// Bytes of a frame's row that a workgroup takes (four channels a lane), frames of
// a lane, time ranges and their length.
struct ScanSplit {
  int row, frames, splits, chunk;
};
// Frames of a tile: 8 waves, as many lanes of the same channels, frames of a lane.
constexpr int scan_tile(int row, int frames, int size) { return kScanWaves * (64 * 4 * size / row) * frames; }
inline int64_t scan_blocks(int channels, int row, int size) {
  const int n = row / size;
  return ((int64_t)channels + n - 1) / n;
}
inline ScanSplit scan_split(int batch, int time, int channels, int size, bool backward) {
  ScanSplit p;
  p.row = (int64_t)batch * scan_blocks(channels, 128, size) >= 256 ? 128 : 64;
  const int least = p.row == 128 ? 2 : 1;
  p.frames = time <= scan_tile(p.row, least, size) ? least : backward ? 2 : 4;
  const int64_t units = batch * scan_blocks(channels, p.row, size);
  const int tile = scan_tile(p.row, p.frames, size);
  const int64_t tiles = ((int64_t)time + tile - 1) / tile;
  int64_t s = units > 0 ? 512 / units : 1;
  if (s > tiles / 2) s = tiles / 2;
  if (s < 1) s = 1;
  const int64_t per = tiles > 0 ? (tiles + s - 1) / s : 1;
  p.splits = (int)(tiles > 0 ? (tiles + per - 1) / per : 1);
  p.chunk = (int)(per * tile);
  return p;
}
inline int64_t scan_workspace(int batch, int time, int channels, int size, bool backward) {
  const ScanSplit p = scan_split(batch, time, channels, size, backward);
  return p.splits == 1 ? 0 : 8 * (int64_t)batch * p.splits * scan_blocks(channels, p.row, size) * (p.row / size);
}
// Few frames go one after another through threads that hold four channels.
constexpr int kScanStepFrames = 8;
inline bool scan_steps(const ScanArgs& a) { return a.time <= kScanStepFrames && !a.saved; }

int scan_forward_f32(const ScanArgs& a, void* stream);
int scan_forward_f16(const ScanArgs& a, void* stream);
int scan_forward_bf16(const ScanArgs& a, void* stream);
int scan_backward_f32(const ScanArgs& a, void* stream);
int scan_backward_f16(const ScanArgs& a, void* stream);
int scan_backward_bf16(const ScanArgs& a, void* stream);

// Root-mean-square norm of x, or of x + residual.
struct RmsForward {
  const void* x;
  int64_t x_stride;  // elements between rows
  const void* residual;
  int64_t r_stride;
  const void* weight;  // or NULL
  void* y;
  int out;        // 0 the rows' type, 1 e4m3, 2 int8
  float* scale;   // [rows] with 8-bit output
  void* sum;      // [rows, width] with a residual
  float* rstd;    // or NULL
  int64_t rows;
  int width;
  float eps;
  void* stream;
};
struct RmsBackward {
  const void* dy;
  int64_t dy_stride;
  const void* s;  // what was normed
  int64_t s_stride;
  const void* ds;  // gradient of the sum, or NULL
  int64_t ds_stride;
  const void* weight;
  const float* rstd;
  void* dx;
  void* dw;
  void* workspace;
  int64_t rows;
  int width;
  void* stream;
};
// One translation unit per element type; w32: a float32 weight.
int rms_forward_f32(const RmsForward& a);
int rms_forward_f16(const RmsForward& a, bool w32);
int rms_forward_bf16(const RmsForward& a, bool w32);
int rms_backward_f32(const RmsBackward& a);
int rms_backward_f16(const RmsBackward& a, bool w32);
int rms_backward_bf16(const RmsBackward& a, bool w32);

}  // namespace fm
