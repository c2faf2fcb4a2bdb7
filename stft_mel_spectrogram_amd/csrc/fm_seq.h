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
// Bytes of a frame's row that a workgroup takes (four channels a lane), frames of
// a lane, time ranges and their length.
struct ScanSplit {
  int row, frames, splits, chunk;
};
constexpr int kScanWaves = 8;  // waves of a workgroup, one time range of a tile each
// Frames of a tile: waves, as many lanes of the same channels, frames of a lane.
constexpr int scan_tile(int row, int frames, int size) { return kScanWaves * (64 * 4 * size / row) * frames; }
inline int64_t scan_blocks(int channels, int row, int size) {
  const int n = row / size;
  return ((int64_t)channels + n - 1) / n;
}
// Whole 128-byte lines where that gives a workgroup per compute unit (forward,
// 16 x 1501 x 2048 bf16: 83 us, 64-byte rows 100; backward 168 and 217), 64-byte rows
// where those do for five eighths (8 x 1501 x 1024 bf16: 26 us, 128-byte rows 35, in
// time ranges 32; 4 x 3000 x 1000 f32: 38, 39 and 52).
// The backward of 16-bit frames, two of whose workgroups share a unit, takes time
// ranges instead (50 us, 64-byte rows 55), and so does everything with fewer
// channels: as many ranges as fill the chip, down to one tile each (1 x 1501 x 1024
// bf16: forward 10, unsplit 21; backward 16 and 50; 1 x 100003 x 256 f16: 60 and 1230).
// A first launch then reads x and forget (backward: forget, gate and grad_y) twice.
// Four frames a lane forward (16 x 1501 x 2048: 83, 2 frames the same, 8 x 1501 x 1024: 26
// and 28; float32 in 64-byte rows two, so that two workgroups share a unit: 38, four 42),
// two backward (four do not fit the registers), two for what one tile holds.
// Fewer than four channels have kernels of their own, single frames.
inline ScanSplit scan_split(int batch, int time, int channels, int size, bool backward) {
  ScanSplit p;
  const int64_t wide = (int64_t)batch * scan_blocks(channels, 128, size);
  const int64_t narrow = (int64_t)batch * scan_blocks(channels, 64, size);
  const bool tiny = channels < 4;
  const bool brief = time <= scan_tile(128, 2, size);
  p.row = tiny || (!brief && wide < 256 && narrow >= 160 && (!backward || size == 4)) ? 64 : 128;
  p.frames = tiny ? 1 : backward || brief || (p.row == 64 && size == 4) ? 2 : 4;
  const int64_t units = p.row == 128 ? wide : narrow;
  const int tile = scan_tile(p.row, p.frames, size);
  const int64_t tiles = ((int64_t)time + tile - 1) / tile;
  int64_t s = units > 0 && units < (p.row == 128 ? 256 : 160) ? 512 / units : 1;
  if (s > tiles) s = tiles;
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
// Few frames go one after another through threads that hold four channels (8 x 1 x
// 1024 bf16: 3.2 us, tiles 4.0; 8 frames 7.2 and 4.1).
constexpr int kScanStepFrames = 2;
inline bool scan_steps(const ScanArgs& a) { return a.time <= kScanStepFrames && !a.saved; }
// Bytes between frames below this stay in 32 bits over a tile (256 frames at most).
constexpr int64_t kScanMaxStride = int64_t(1) << 23;
constexpr int kScanMaxChannels = 1 << 20;

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
