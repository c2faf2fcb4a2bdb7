// Host-only stand-ins for the launches of the recurrence, the RMS norm, the
// distillation and the adjusted logits.  Each writes every element of the
// workspace that the kernels' indexing can reach and looks at the split's rules.
// Test infrastructure: never linked into the library.
#include "fm_logit.h"
#include "fm_seq.h"

namespace fm {
namespace {

void fill(float* p, int64_t n) {
  for (int64_t i = 0; i < n; ++i) p[i] = 1.f;
}

int scan(const ScanArgs& a, int size, bool backward) {
  if (!backward && scan_steps(a)) return FM_OK;
  const ScanSplit p = scan_split(a.batch, a.time, a.channels, size, backward);
  const int tile = scan_tile(p.row, p.frames, size);
  if (tile % kScanSave || p.chunk % tile || p.splits < 1) return set_error(FM_E_HIP, "tiles");
  if (int64_t(p.splits) * p.chunk < a.time || (a.time > 0 && int64_t(p.splits - 1) * p.chunk >= a.time))
    return set_error(FM_E_HIP, "ranges do not cover the frames");
  // a wave's range starts at every saved state
  const int span = tile / kScanWaves;
  if (kScanSave % span) return set_error(FM_E_HIP, "saved states inside a wave's range");
  const int64_t blocks = scan_blocks(a.channels, p.row, size);
  if (a.batch * blocks * p.splits * 64 * kScanWaves >= int64_t(1) << 32) return set_error(FM_E_HIP, "grid");
  if (p.splits > 1) fill(a.part, int64_t(a.batch) * p.splits * blocks * (p.row / size) * 2);
  return FM_OK;
}
int rms(const RmsBackward& a, int ve) {
  if (a.dw && a.rows > 0 && !norm_single(a.rows, a.width, ve))
    fill(static_cast<float*>(a.workspace), int64_t(norm_parts(a.rows, a.width, ve)) * a.width);
  return FM_OK;
}
int distill(const DistillArgs& a, int ve) {
  const ScoreSplit p = score_split(a.rows, a.vocab, ve, 0);
  if (p.segs > 1) fill(static_cast<float*>(a.workspace), a.rows * p.segs * 2);
  return FM_OK;
}
int adjust(const AdjustArgs& a, int ve) {
  const int64_t n = int64_t(kAdjustThreads) * ve * adjust_vecs(a.rows, a.vocab, ve);
  if (a.segs != adjust_segments(a.rows, a.vocab, ve) || n * a.segs < a.vocab || n * (a.segs - 1) >= a.vocab)
    return set_error(FM_E_HIP, "segments do not cover the row");
  return a.rows * a.segs * kAdjustThreads < int64_t(1) << 31 ? FM_OK : set_error(FM_E_HIP, "grid");
}

}  // namespace

int scan_forward_f32(const ScanArgs& a, void*) { return scan(a, 4, false); }
int scan_forward_f16(const ScanArgs& a, void*) { return scan(a, 2, false); }
int scan_forward_bf16(const ScanArgs& a, void*) { return scan(a, 2, false); }
int scan_backward_f32(const ScanArgs& a, void*) { return scan(a, 4, true); }
int scan_backward_f16(const ScanArgs& a, void*) { return scan(a, 2, true); }
int scan_backward_bf16(const ScanArgs& a, void*) { return scan(a, 2, true); }
int rms_forward_f32(const RmsForward&) { return FM_OK; }
int rms_forward_f16(const RmsForward&, bool) { return FM_OK; }
int rms_forward_bf16(const RmsForward&, bool) { return FM_OK; }
int rms_backward_f32(const RmsBackward& a) { return rms(a, 4); }
int rms_backward_f16(const RmsBackward& a, bool) { return rms(a, 8); }
int rms_backward_bf16(const RmsBackward& a, bool) { return rms(a, 8); }
int distill_forward_f32(const DistillArgs& a) { return distill(a, 4); }
int distill_forward_f16(const DistillArgs& a) { return distill(a, 8); }
int distill_forward_bf16(const DistillArgs& a) { return distill(a, 8); }
int distill_backward_f32(const DistillArgs&) { return FM_OK; }
int distill_backward_f16(const DistillArgs&) { return FM_OK; }
int distill_backward_bf16(const DistillArgs&) { return FM_OK; }
int adjust_f32(const AdjustArgs& a, void*) { return adjust(a, 4); }
int adjust_f16(const AdjustArgs& a, void*) { return adjust(a, 8); }
int adjust_bf16(const AdjustArgs& a, void*) { return adjust(a, 8); }

}  // namespace fm
