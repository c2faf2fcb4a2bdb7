// C ABI of the gated recurrence and the root-mean-square norm (declared in
// include/fm.h): argument checks on the host, then the launches of the type.
#include "fm_seq.h"

#include <cmath>
#include <cstdint>
#include <limits>

#include "fm_check.h"

namespace fm {
namespace {

int bad(const char* what) { return set_error(FM_E_INVAL, what); }

// Checks what every call shares (a workspace's size depends on no more) and
// translates the public struct.
int recurrence_args(const fm_recurrence_args* p, ScanArgs& a) {
  if (!p) return bad("gated recurrence: args must not be NULL");
  if (!elem_bytes(p->dtype)) return bad("gated recurrence: dtype must be FM_F32, FM_F16 or FM_BF16");
  const int64_t most = int64_t(1) << 30;
  if (p->batch < 0 || p->batch >= most || p->time < 0 || p->time >= most || p->channels < 1)
    return bad("gated recurrence: batch and time must be in [0, 2^30), channels >= 1");
  if (p->channels > kScanMaxChannels)
    return set_error(FM_E_UNSUPPORTED, "gated recurrence: channels must be <= 2^20");
  a = ScanArgs{};
  a.batch = static_cast<int>(p->batch);
  a.time = static_cast<int>(p->time);
  a.channels = static_cast<int>(p->channels);
  a.x = p->x;
  a.f = p->forget;
  a.g = p->gate;
  a.state = p->state;
  a.lengths = p->lengths;
  a.y = p->y;
  a.last = p->last_state;
  a.saved = p->saved;
  a.dy = p->grad_y;
  a.dlast = p->grad_last;
  a.dx = p->grad_x;
  a.df = p->grad_forget;
  a.dg = p->grad_gate;
  a.dstate = p->grad_state;
  for (int i = 0; i < 2; ++i) {
    a.xs[i] = p->x_stride[i];
    a.fs[i] = p->forget_stride[i];
    a.gs[i] = p->gate_stride[i];
    a.dys[i] = p->grad_y_stride[i];
  }
  // one frame has no next one, whatever its stride says
  if (a.time <= 1) a.xs[1] = a.fs[1] = a.gs[1] = a.dys[1] = 0;
  // workgroups of 512 threads and single threads, below 2^32 threads
  const int size = elem_bytes(p->dtype);
  int64_t units = 0;
  for (int row : {64, 128}) {
    const int64_t n = a.batch * scan_blocks(a.channels, row, size);
    units = n > units ? n : units;
  }
  // at most 512 workgroups, or one per unit
  if (units >= (int64_t(1) << 23) || a.batch * ((static_cast<int64_t>(a.channels) + 3) / 4) >= int64_t(1) << 31)
    return bad("gated recurrence: too many channels for one launch");
  return FM_OK;
}

bool scan_strides_fit(const int64_t* s) { return s[0] >= 0 && s[1] >= 0; }

// The strides and pointers of a call: what it reads must exist, elements aligned.
int recurrence_pointers(const ScanArgs& a, int dtype, bool backward) {
  if (!scan_strides_fit(a.xs) || !scan_strides_fit(a.fs) || !scan_strides_fit(a.gs) ||
      (backward && !scan_strides_fit(a.dys)))
    return bad("gated recurrence: strides must be >= 0");
  const int es = elem_bytes(dtype);
  // (few frames are walked with addresses in 64 bits)
  const bool tiles = backward || !scan_steps(a);
  if (tiles &&
      (a.xs[1] >= kScanMaxStride / es || a.fs[1] >= kScanMaxStride / es || (a.g && a.gs[1] >= kScanMaxStride / es) ||
       (backward && a.dys[1] >= kScanMaxStride / es)))
    return set_error(FM_E_UNSUPPORTED, "gated recurrence: frames must be less than 8 MiB apart");
  if (!aligned_to(a.x, es) || !aligned_to(a.f, es) || !aligned_to(a.g, es) || !aligned_to(a.y, es) ||
      !aligned_to(a.dy, es) || !aligned_to(a.dx, es) || !aligned_to(a.df, es) || !aligned_to(a.dg, es) ||
      !aligned_to(a.state, 4) || !aligned_to(a.lengths, 4) || !aligned_to(a.last, 4) || !aligned_to(a.saved, 4) ||
      !aligned_to(a.dlast, 4) || !aligned_to(a.dstate, 4))
    return bad("gated recurrence: misaligned pointer");
  if (a.batch > 0 && a.time > 0) {
    if (!a.x || !a.f) return bad("gated recurrence: x and forget must not be NULL");
    if (backward && (!a.dy || !a.dx || !a.df || !a.saved))
      return bad("gated recurrence: grad_y, saved, grad_x and grad_forget must not be NULL");
    if (backward && a.g && !a.dg) return bad("gated recurrence: grad_gate must not be NULL with a gate");
    if (!backward && !a.y) return bad("gated recurrence: y must not be NULL");
  }
  if (!backward && a.batch > 0 && !a.last) return bad("gated recurrence: last_state must not be NULL");
  return FM_OK;
}

int check_rms(int64_t rows, int64_t width, int dtype) {
  if (!elem_bytes(dtype)) return bad("rms norm: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (rows < 0 || rows >= (int64_t(1) << 31)) return bad("rms norm: rows must be in [0, 2^31)");
  if (width < 1) return bad("rms norm: width must be >= 1");
  if (width > kNormMaxWidth) return set_error(FM_E_UNSUPPORTED, "rms norm: width must be <= 2^20");
  return FM_OK;
}

// In float32; what is above 0 stays so: a row of zeros is normed to zeros.
float rms_eps(double eps) {
  const float e = static_cast<float>(eps);
  return eps > 0.0 && e == 0.f ? std::numeric_limits<float>::denorm_min() : e;
}

int rms_forward(const RmsForward& a, double eps, int dtype, int param_dtype) {
  if (param_dtype != dtype && param_dtype != FM_F32)
    return bad("rms norm: param_dtype must be the rows' dtype or FM_F32");
  if (!(eps >= 0.0) || !std::isfinite(a.eps)) return bad("rms norm: eps must be >= 0 and finite in float32");
  if (a.rows == 0) return FM_OK;
  if (!a.x || !a.y) return bad("rms norm: x and the output must not be NULL");
  if ((a.residual != nullptr) != (a.sum != nullptr)) return bad("rms norm: residual and sum go together");
  if (a.out != 0 && !a.scale) return bad("rms norm: scale must not be NULL");
  if (a.rows > 1 && (a.x_stride < 0 || (a.residual && a.r_stride < 0)))
    return bad("rms norm: strides must be >= 0");
  const int es = elem_bytes(dtype);
  if (!aligned_to(a.x, es) || !aligned_to(a.y, a.out ? 1 : es) || !aligned_to(a.residual, es) ||
      !aligned_to(a.sum, es) || !aligned_to(a.scale, 4) || !aligned_to(a.rstd, 4) ||
      !aligned_to(a.weight, elem_bytes(param_dtype)))
    return bad("rms norm: misaligned pointer");
  const bool w32 = param_dtype == FM_F32;
  if (dtype == FM_F32) return rms_forward_f32(a);
  return dtype == FM_F16 ? rms_forward_f16(a, w32) : rms_forward_bf16(a, w32);
}

}  // namespace
}  // namespace fm

using fm::bad;

extern "C" {

int64_t fm_gated_recurrence_workspace(const fm_recurrence_args* args, int backward) try {
  fm::ScanArgs a;
  if (int st = fm::recurrence_args(args, a)) return st;
  return fm::scan_workspace(a.batch, a.time, a.channels, fm::elem_bytes(args->dtype), backward != 0);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_gated_recurrence_forward(const fm_recurrence_args* args, void* workspace, void* stream) try {
  fm::ScanArgs a;
  if (int st = fm::recurrence_args(args, a)) return st;
  if (int st = fm::recurrence_pointers(a, args->dtype, false)) return st;
  if (a.batch == 0) return FM_OK;
  const int size = fm::elem_bytes(args->dtype);
  if (fm::scan_workspace(a.batch, a.time, a.channels, size, false) > 0 &&
      (!workspace || !fm::aligned_to(workspace, 16)))
    return bad("gated recurrence: the workspace must be 16-byte aligned device memory");
  a.part = static_cast<float*>(workspace);
  if (args->dtype == FM_F32) return fm::scan_forward_f32(a, stream);
  return args->dtype == FM_F16 ? fm::scan_forward_f16(a, stream) : fm::scan_forward_bf16(a, stream);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_gated_recurrence_backward(const fm_recurrence_args* args, void* workspace, void* stream) try {
  fm::ScanArgs a;
  if (int st = fm::recurrence_args(args, a)) return st;
  if (int st = fm::recurrence_pointers(a, args->dtype, true)) return st;
  if (a.batch == 0) return FM_OK;
  const int size = fm::elem_bytes(args->dtype);
  if (fm::scan_workspace(a.batch, a.time, a.channels, size, true) > 0 &&
      (!workspace || !fm::aligned_to(workspace, 16)))
    return bad("gated recurrence: the workspace must be 16-byte aligned device memory");
  a.part = static_cast<float*>(workspace);
  if (args->dtype == FM_F32) return fm::scan_backward_f32(a, stream);
  return args->dtype == FM_F16 ? fm::scan_backward_f16(a, stream) : fm::scan_backward_bf16(a, stream);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_rms_norm_forward(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        const void* weight, void* y, void* sum, float* rstd, int64_t rows, int64_t width,
                        double eps, int dtype, int param_dtype, void* stream) try {
  if (int st = fm::check_rms(rows, width, dtype)) return st;
  const fm::RmsForward a = {x,   x_stride, residual, residual_stride, weight, y, 0, nullptr, sum, rstd, rows,
                            static_cast<int>(width), fm::rms_eps(eps), stream};
  return fm::rms_forward(a, eps, dtype, param_dtype);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_rms_norm_quantized(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          const void* weight, void* q, float* scale, void* sum, int64_t rows, int64_t width,
                          double eps, int dtype, int param_dtype, int out_dtype, void* stream) try {
  if (int st = fm::check_rms(rows, width, dtype)) return st;
  if (out_dtype != FM_E4M3 && out_dtype != FM_I8) return bad("rms norm: out_dtype must be FM_E4M3 or FM_I8");
  const fm::RmsForward a = {x, x_stride, residual, residual_stride, weight, q, out_dtype == FM_E4M3 ? 1 : 2,
                            scale, sum, nullptr, rows, static_cast<int>(width), fm::rms_eps(eps), stream};
  return fm::rms_forward(a, eps, dtype, param_dtype);
} catch (...) {
  return FM_E_NOMEM;
}

int64_t fm_rms_norm_backward_workspace(int64_t rows, int64_t width, int dtype) try {
  if (int st = fm::check_rms(rows, width, dtype)) return st;
  const int ve = 16 / fm::elem_bytes(dtype);
  if (fm::norm_single(rows, static_cast<int>(width), ve)) return 0;
  return fm::norm_parts(rows, static_cast<int>(width), ve) * width * static_cast<int64_t>(sizeof(float));
} catch (...) {
  return FM_E_NOMEM;
}

int fm_rms_norm_backward(const void* dy, int64_t dy_stride, const void* sum, int64_t sum_stride, const void* grad_sum,
                         int64_t grad_sum_stride, const void* weight, const float* rstd, void* dx, void* dw,
                         void* workspace, int64_t rows, int64_t width, int dtype, int param_dtype, void* stream) try {
  if (int st = fm::check_rms(rows, width, dtype)) return st;
  if (param_dtype != dtype && param_dtype != FM_F32)
    return bad("rms norm: param_dtype must be the rows' dtype or FM_F32");
  if (dw && !weight) return bad("rms norm: dw needs the weight");
  const int es = fm::elem_bytes(dtype);
  if (!fm::aligned_to(weight, fm::elem_bytes(param_dtype)) || !fm::aligned_to(dw, fm::elem_bytes(param_dtype)))
    return bad("rms norm: misaligned pointer");
  if (rows > 0) {
    if (!dy || !sum || !dx || !rstd) return bad("rms norm: dy, sum, rstd and dx must not be NULL");
    if (dw && !fm::norm_single(rows, static_cast<int>(width), 16 / es) &&
        (!workspace || !fm::aligned_to(workspace, 16)))
      return bad("rms norm: the workspace must be 16-byte aligned device memory");
    if (rows > 1 && (dy_stride < 0 || sum_stride < 0 || (grad_sum && grad_sum_stride < 0)))
      return bad("rms norm: strides must be >= 0");
    if (!fm::aligned_to(dy, es) || !fm::aligned_to(sum, es) || !fm::aligned_to(grad_sum, es) ||
        !fm::aligned_to(dx, es) || !fm::aligned_to(rstd, 4))
      return bad("rms norm: misaligned pointer");
  }
  const fm::RmsBackward a = {dy,     dy_stride, sum, sum_stride, grad_sum, grad_sum_stride,
                             weight, rstd,      dx,  dw,         workspace, rows,
                             static_cast<int>(width), stream};
  const bool w32 = param_dtype == FM_F32;
  if (dtype == FM_F32) return fm::rms_backward_f32(a);
  return dtype == FM_F16 ? fm::rms_backward_f16(a, w32) : fm::rms_backward_bf16(a, w32);
} catch (...) {
  return FM_E_NOMEM;
}

}  // extern "C"
