// C ABI of the speech-model operators (declared in include/fm.h): argument
// checks on the host, then the launches of the element type.
#include "fm_ops.h"

#include <cmath>
#include <cstdint>
#include <string>

namespace fm {
namespace {

int bad(const char* what) { return set_error(FM_E_INVAL, what); }

int elem_size(int dtype) {
  return dtype == FM_F32 ? 4 : (dtype == FM_F16 || dtype == FM_BF16) ? 2 : 0;
}
int vec_elems(int dtype) { return 16 / elem_size(dtype); }

bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

int check_norm(int64_t rows, int64_t width, int dtype) {
  if (!elem_size(dtype)) return bad("layer norm: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (rows < 0 || rows >= (int64_t(1) << 31)) return bad("layer norm: rows must be in [0, 2^31)");
  if (width < 1) return bad("layer norm: width must be >= 1");
  if (width > kNormMaxWidth)
    return set_error(FM_E_UNSUPPORTED, "layer norm: width must be <= 2^20");
  return FM_OK;
}

int check_params(int dtype, int param_dtype, const void* w, const void* b) {
  if (param_dtype != dtype && param_dtype != FM_F32)
    return bad("layer norm: param_dtype must be the rows' dtype or FM_F32");
  if (!w && b) return bad("layer norm: a bias needs a weight");
  return FM_OK;
}

int check_scores(int64_t rows, int64_t vocab, int top, int dtype) {
  if (!elem_size(dtype)) return bad("token log probabilities: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (rows < 0) return bad("token log probabilities: rows must be >= 0");
  if (vocab < 1 || vocab >= (int64_t(1) << 31) - 65536)
    return bad("token log probabilities: vocab must be in [1, 2^31 - 65536)");
  if (top < 0 || top > kScoreMaxTop || top > vocab)
    return bad("token log probabilities: top must be in [0, min(64, vocab)]");
  const ScoreSplit p = score_split(rows, static_cast<int>(vocab), vec_elems(dtype), top);
  if (rows >= (int64_t(1) << 31) / p.segs)
    return bad("token log probabilities: too many rows for one launch");
  return FM_OK;
}

int check_score_strides(int64_t rows, int64_t stride, int64_t inner, int64_t outer) {
  if (rows > 1 && stride < 0) return bad("token log probabilities: x_stride must be >= 0");
  if (inner < 0 || inner >= int64_t(1) << 31 || (inner > 0 && outer < 0))
    return bad("token log probabilities: x_inner must be in [0, 2^31) and x_outer >= 0");
  return FM_OK;
}

bool strides_fit(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0) return false;
  return true;
}

// Checks what every call shares (a workspace's size depends on no more) and
// translates the public struct.
int attention_args(const fm_attention_args* p, AttnArgs& a) {
  if (!p) return bad("attention: args must not be NULL");
  if (!elem_size(p->dtype)) return bad("attention: dtype must be FM_F32, FM_F16 or FM_BF16");
  if (p->table_dtype != p->dtype && p->table_dtype != FM_F32)
    return bad("attention: table_dtype must be dtype or FM_F32");
  const int64_t most = int64_t(1) << 30;
  if (p->batch < 0 || p->batch >= most || p->heads < 1 || p->heads >= 65536 || p->kv_heads < 1 ||
      p->heads % p->kv_heads != 0)
    return bad("attention: batch >= 0 and heads, a multiple of kv_heads, of at least 1 are wanted");
  if (p->q_len < 0 || p->k_len < 0 || p->q_len >= most || p->k_len >= most)
    return bad("attention: q_len and k_len must be in [0, 2^30)");
  if (p->head_dim < 1) return bad("attention: head_dim must be >= 1");
  if (p->head_dim > kAttnMaxDim) return set_error(FM_E_UNSUPPORTED, "attention: head_dim must be <= 128");
  // its reciprocal times a bias (at most 2^16) or a log sum exp has to stay in float32's range
  if (!(p->scale >= 0x1p-60 && p->scale <= 0x1p60))
    return bad("attention: scale must be in [2^-60, 2^60]");
  if (p->far < 0 || p->num_buckets < 1) return bad("attention: far >= 0 and num_buckets >= 1 are wanted");
  if (p->far > kAttnMaxFar || p->num_buckets > kAttnMaxBuckets)
    return set_error(FM_E_UNSUPPORTED, "attention: far and num_buckets must be <= 1024");
  if (p->query_offset_value < -most || p->query_offset_value > most)
    return bad("attention: query_offset_value must be within +-2^30");
  a = AttnArgs{};
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.table = p->table;
  a.map = p->bucket_map;
  a.key_lengths = p->key_lengths;
  a.query_offset = p->query_offset;
  a.query_offset_value = static_cast<int>(p->query_offset_value);
  a.far = p->far;
  a.num_buckets = p->num_buckets;
  a.table32 = p->table_dtype == FM_F32;
  a.causal = p->causal != 0;
  a.batch = static_cast<int>(p->batch);
  a.heads = static_cast<int>(p->heads);
  a.kv_heads = static_cast<int>(p->kv_heads);
  a.q_len = static_cast<int>(p->q_len);
  a.k_len = static_cast<int>(p->k_len);
  a.dim = static_cast<int>(p->head_dim);
  a.size = elem_size(p->dtype);
  a.scale = static_cast<float>(p->scale);
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = p->q_stride[i];
    a.ks[i] = p->k_stride[i];
    a.vs[i] = p->v_stride[i];
    a.os[i] = p->o_stride[i];
    a.dos[i] = p->grad_o_stride[i];
    a.dqs[i] = p->grad_q_stride[i];
    a.dks[i] = p->grad_k_stride[i];
    a.dvs[i] = p->grad_v_stride[i];
  }
  // grids: query blocks x heads, key blocks x key heads, rows of the join
  if (!attn_fits_grids(a)) return bad("attention: too many rows for one launch");
  a.o = p->o;
  a.lse = p->lse;
  a.d_o = p->grad_o;
  a.dq = p->grad_q;
  a.dk = p->grad_k;
  a.dv = p->grad_v;
  a.d_table = p->grad_table;
  a.splits = attn_splits(a);
  return FM_OK;
}

// The strides and pointers of a call: what it reads must exist, elements aligned.
int attention_pointers(const AttnArgs& a, int dtype, bool backward) {
  if (!strides_fit(a.qs) || !strides_fit(a.ks) || !strides_fit(a.vs) || !strides_fit(a.os) ||
      (backward && (!strides_fit(a.dos) || !strides_fit(a.dqs) || !strides_fit(a.dks) || !strides_fit(a.dvs))))
    return bad("attention: strides must be >= 0");
  if (!a.table || !a.map) return bad("attention: table and bucket_map must not be NULL");
  const int es = elem_size(dtype);
  const bool q = attn_rows(a) > 0, k = q && a.k_len > 0;
  if (q && (!a.q || !a.o)) return bad("attention: q and o must not be NULL");
  if (k && (!a.k || !a.v)) return bad("attention: k and v must not be NULL");
  if (!aligned(a.q, es) || !aligned(a.k, es) || !aligned(a.v, es) || !aligned(a.o, es) ||
      !aligned(a.d_o, es) || !aligned(a.dq, es) || !aligned(a.dk, es) ||
      !aligned(a.dv, es) || !aligned(a.map, 4) || !aligned(a.key_lengths, 4) ||
      !aligned(a.query_offset, 4))
    return bad("attention: misaligned pointer");
  return FM_OK;
}

}  // namespace
}  // namespace fm

using fm::bad;

extern "C" {

int fm_layer_norm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                          void* y, float* mean, float* rstd, int64_t rows, int64_t width,
                          double eps, int dtype, int param_dtype, void* stream) try {
  if (int st = fm::check_norm(rows, width, dtype)) return st;
  if (int st = fm::check_params(dtype, param_dtype, weight, bias)) return st;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return bad("layer norm: eps must be finite and >= 0");
  if (rows == 0) return FM_OK;
  if (!x || !y) return bad("layer norm: x and y must not be NULL");
  if (rows > 1 && x_stride < 0) return bad("layer norm: x_stride must be >= 0");
  const int es = fm::elem_size(dtype);
  if (!fm::aligned(x, es) || !fm::aligned(y, es)) return bad("layer norm: misaligned pointer");
  const fm::NormForward a = {x, x_stride, weight, bias, y, mean, rstd, rows,
                             static_cast<int>(width), static_cast<float>(eps), stream};
  const bool w32 = param_dtype == FM_F32;
  if (dtype == FM_F32) return fm::norm_forward_f32(a);
  return dtype == FM_F16 ? fm::norm_forward_f16(a, w32) : fm::norm_forward_bf16(a, w32);
} catch (...) {
  return FM_E_NOMEM;
}

int64_t fm_layer_norm_backward_workspace(int64_t rows, int64_t width, int dtype) try {
  if (int st = fm::check_norm(rows, width, dtype)) return st;
  if (fm::norm_single(rows, static_cast<int>(width), fm::vec_elems(dtype))) return 0;
  return int64_t(2) * fm::norm_parts(rows, static_cast<int>(width), fm::vec_elems(dtype)) * width *
         static_cast<int64_t>(sizeof(float));
} catch (...) {
  return FM_E_NOMEM;
}

int fm_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                           const void* weight, const float* mean, const float* rstd, void* dx,
                           void* dw, void* db, void* workspace, int64_t rows, int64_t width,
                           int dtype, int param_dtype, void* stream) try {
  if (int st = fm::check_norm(rows, width, dtype)) return st;
  if (int st = fm::check_params(dtype, param_dtype, weight, nullptr)) return st;
  if (db && !dw) return bad("layer norm: db needs dw");
  if (dw && !weight) return bad("layer norm: dw needs the weight");
  if (rows > 0) {
    if (!dy || !x || !dx || !mean || !rstd)
      return bad("layer norm: dy, x, mean, rstd and dx must not be NULL");
    if (dw && !fm::norm_single(rows, static_cast<int>(width), fm::vec_elems(dtype)) &&
        (!workspace || !fm::aligned(workspace, 16)))
      return bad("layer norm: the workspace must be 16-byte aligned device memory");
    if (rows > 1 && (x_stride < 0 || dy_stride < 0)) return bad("layer norm: strides must be >= 0");
    const int es = fm::elem_size(dtype);
    if (!fm::aligned(x, es) || !fm::aligned(dy, es) || !fm::aligned(dx, es))
      return bad("layer norm: misaligned pointer");
  }
  const fm::NormBackward a = {dy, dy_stride, x,  x_stride,  weight, mean,
                              rstd, dx,       dw, db,        workspace, rows,
                              static_cast<int>(width), stream};
  const bool w32 = param_dtype == FM_F32;
  if (dtype == FM_F32) return fm::norm_backward_f32(a);
  return dtype == FM_F16 ? fm::norm_backward_f16(a, w32) : fm::norm_backward_bf16(a, w32);
} catch (...) {
  return FM_E_NOMEM;
}

int64_t fm_token_logprobs_workspace(int64_t rows, int64_t vocab, int top, int dtype) try {
  if (int st = fm::check_scores(rows, vocab, top, dtype)) return st;
  return fm::score_workspace(rows, static_cast<int>(vocab), top, fm::vec_elems(dtype));
} catch (...) {
  return FM_E_NOMEM;
}

int fm_token_logprobs_strided(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer,
                              const void* tokens, int token_bits, float* lp, float* ent, float* lse,
                              int64_t* top_ids, float* top_lp, void* workspace, int64_t rows,
                              int64_t vocab, int top, int dtype, void* stream) try {
  if (int st = fm::check_scores(rows, vocab, top, dtype)) return st;
  if (token_bits != 64 && token_bits != 32)
    return bad("token log probabilities: token_bits must be 32 or 64");
  if (rows == 0) return FM_OK;
  if (!x || !tokens) return bad("token log probabilities: x and tokens must not be NULL");
  if (top > 0 && (!top_ids || !top_lp))
    return bad("token log probabilities: top_ids and top_lp must not be NULL");
  if (int st = fm::check_score_strides(rows, x_stride, x_inner, x_outer)) return st;
  if (!fm::aligned(x, fm::elem_size(dtype)) || !fm::aligned(tokens, token_bits / 8))
    return bad("token log probabilities: misaligned pointer");
  if (fm::score_workspace(rows, static_cast<int>(vocab), top, fm::vec_elems(dtype)) > 0 &&
      (!workspace || !fm::aligned(workspace, 16)))
    return bad("token log probabilities: the workspace must be 16-byte aligned device memory");
  const fm::ScoreForward a = {x, x_stride, x_inner, x_outer, tokens, token_bits == 64, lp, ent, lse, top_ids,
                              top_lp, workspace, rows, static_cast<int>(vocab), top, stream};
  if (dtype == FM_F32) return fm::score_forward_f32(a);
  return dtype == FM_F16 ? fm::score_forward_f16(a) : fm::score_forward_bf16(a);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_token_logprobs_backward_strided(const void* x, int64_t x_stride, int64_t x_inner,
                                       int64_t x_outer, const void* tokens, int token_bits,
                                       const float* lse, const float* ent, const float* g_lp,
                                       const float* g_ent, const int64_t* top_ids, const float* g_top,
                                       void* dx, int64_t rows, int64_t vocab, int top, int dtype,
                                       void* stream) try {
  if (int st = fm::check_scores(rows, vocab, top, dtype)) return st;
  if (token_bits != 64 && token_bits != 32)
    return bad("token log probabilities: token_bits must be 32 or 64");
  if (rows == 0) return FM_OK;
  if (!x || !tokens || !lse || !dx)
    return bad("token log probabilities: x, tokens, lse and dx must not be NULL");
  if (g_ent && !ent) return bad("token log probabilities: g_ent needs ent");
  if (g_top && (!top_ids || top < 1)) return bad("token log probabilities: g_top needs top_ids");
  if (int st = fm::check_score_strides(rows, x_stride, x_inner, x_outer)) return st;
  const int es = fm::elem_size(dtype);
  if (!fm::aligned(x, es) || !fm::aligned(dx, es) || !fm::aligned(tokens, token_bits / 8))
    return bad("token log probabilities: misaligned pointer");
  const fm::ScoreBackward a = {x,   x_stride, x_inner, x_outer, tokens, token_bits == 64,
                               lse, ent,      g_lp,    g_ent,   top_ids, g_top,
                               dx,  rows,     static_cast<int>(vocab), top, stream};
  if (dtype == FM_F32) return fm::score_backward_f32(a);
  return dtype == FM_F16 ? fm::score_backward_f16(a) : fm::score_backward_bf16(a);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_token_logprobs(const void* x, int64_t x_stride, const void* tokens, int token_bits,
                      float* lp, float* ent, float* lse, int64_t* top_ids, float* top_lp,
                      void* workspace, int64_t rows, int64_t vocab, int top, int dtype,
                      void* stream) {
  return fm_token_logprobs_strided(x, x_stride, 0, 0, tokens, token_bits, lp, ent, lse, top_ids, top_lp,
                                   workspace, rows, vocab, top, dtype, stream);
}

int fm_token_logprobs_backward(const void* x, int64_t x_stride, const void* tokens,
                               int token_bits, const float* lse, const float* ent,
                               const float* g_lp, const float* g_ent, const int64_t* top_ids,
                               const float* g_top, void* dx, int64_t rows, int64_t vocab, int top,
                               int dtype, void* stream) {
  return fm_token_logprobs_backward_strided(x, x_stride, 0, 0, tokens, token_bits, lse, ent, g_lp, g_ent,
                                            top_ids, g_top, dx, rows, vocab, top, dtype, stream);
}

int64_t fm_attention_workspace(const fm_attention_args* args, int backward) try {
  fm::AttnArgs a;
  if (int st = fm::attention_args(args, a)) return st;
  return backward ? fm::attn_backward_space(a, args->dtype == FM_F16).total
                  : fm::attn_forward_workspace(a);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_attention_forward(const fm_attention_args* args, void* workspace, void* stream) try {
  fm::AttnArgs a;
  if (int st = fm::attention_args(args, a)) return st;
  if (int st = fm::attention_pointers(a, args->dtype, false)) return st;
  if (fm::attn_rows(a) == 0) return FM_OK;
  if (a.splits > 1) {
    if (!workspace || !fm::aligned(workspace, 16))
      return bad("attention: the workspace must be 16-byte aligned device memory");
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + fm::attn_round16(4 * a.splits * fm::attn_rows(a) * a.dim) / 4;
  }
  if (args->dtype == FM_F32) return fm::attn_forward_f32(a, stream);
  return args->dtype == FM_F16 ? fm::attn_forward_f16(a, stream) : fm::attn_forward_bf16(a, stream);
} catch (...) {
  return FM_E_NOMEM;
}

int fm_attention_backward(const fm_attention_args* args, void* workspace, void* stream) try {
  fm::AttnArgs a;
  if (int st = fm::attention_args(args, a)) return st;
  if (int st = fm::attention_pointers(a, args->dtype, true)) return st;
  const bool rows = fm::attn_rows(a) > 0;
  if (rows && (!a.lse || !a.d_o || !a.dq)) return bad("attention: lse, grad_o and grad_q must not be NULL");
  if (a.batch > 0 && a.k_len > 0 && (!a.k || !a.v || !a.dk || !a.dv))
    return bad("attention: k, v, grad_k and grad_v must not be NULL");
  const fm::AttnBackwardSpace w = fm::attn_backward_space(a, args->dtype == FM_F16);
  if (w.total > 0 && (!workspace || !fm::aligned(workspace, 16)))
    return bad("attention: the workspace must be 16-byte aligned device memory");
  char* base = static_cast<char*>(workspace);
  a.delta = reinterpret_cast<float*>(base);
  a.amax = reinterpret_cast<float*>(base + w.amax);
  a.table_part = reinterpret_cast<float*>(base + w.part);
  a.table_dist = reinterpret_cast<float*>(base + w.dist);
  a.part_dkv = reinterpret_cast<float*>(base + w.dkv);
  a.dkv_splits = fm::attn_dkv_splits(a);
  a.part_dq = reinterpret_cast<float*>(base + w.dq);
  a.part_row = reinterpret_cast<float*>(base + w.row);
  a.dq_splits = fm::attn_dq_splits(a);
  if (args->dtype == FM_F32) return fm::attn_backward_f32(a, stream);
  return args->dtype == FM_F16 ? fm::attn_backward_f16(a, stream) : fm::attn_backward_bf16(a, stream);
} catch (...) {
  return FM_E_NOMEM;
}

}  // extern "C"
