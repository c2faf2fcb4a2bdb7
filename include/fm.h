/*
 * fm.h -- C ABI of the fused mel-spectrogram forward pass for AMD Instinct
 * MI355X (gfx950).
 *
 * The operation is the one the flashmel 0.1.0 page (PyPI sdist diff view)
 * describes: a torchaudio-MelSpectrogram-compatible forward pass -- centre
 * padding, framing at hop_length, periodic Hann window, real-to-complex FFT of
 * size n_fft, |X|^power and a projection onto a sparse triangular mel
 * filterbank -- in a single kernel launch (README "How it works"; argument
 * list and shape contract in README "Usage"; window and filterbank packing in
 * flashmel/filters.py).
 *
 * Conventions for every entry point:
 *   - Return value: FM_OK (0) on success, a negative FM_E_* code otherwise.
 *     On failure a message is kept per thread; fm_last_error() returns it.
 *   - Pointers named `in`/`out` are DEVICE pointers owned by the caller.
 *     Plans own their device tables; fm_plan_destroy frees them.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *   - Nothing here synchronises the device; fm_forward only enqueues.
 */
#ifndef FM_H_
#define FM_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------- */
#define FM_OK 0
#define FM_E_INVAL (-1)       /* invalid argument (bad value, null pointer)  */
#define FM_E_UNSUPPORTED (-2) /* valid for torchaudio, not built here         */
#define FM_E_HIP (-3)         /* a HIP runtime call failed                    */
#define FM_E_NOMEM (-4)       /* host or device allocation failed            */
#define FM_E_NODEVICE (-5)    /* plan has no device tables (host-only plan)  */

/* ---- enumerations -------------------------------------------------------- */
/* pad_mode: how frames read beyond the signal when center != 0 (README "How
 * it works": all four pad modes are index arithmetic).                      */
#define FM_PAD_REFLECT 0   /* x[-i] = x[i], edge sample not repeated         */
#define FM_PAD_CONSTANT 1  /* zeros                                          */
#define FM_PAD_REPLICATE 2 /* edge sample repeated                           */
#define FM_PAD_CIRCULAR 3  /* periodic wrap                                  */

/* mel_scale and norm: passed through to the filterbank construction
 * (flashmel/filters.py pack_fbank).                                        */
#define FM_MEL_HTK 0
#define FM_MEL_SLANEY 1
#define FM_NORM_NONE 0
#define FM_NORM_SLANEY 1

/* sample types.  Input: float32, or int16 PCM that the kernel multiplies by
 * 2^-15 as it loads it (README "Usage" lists both input types and that
 * scale).  Output: float32, or float16 (README "Usage", out_dtype): the
 * float32 result rounded to nearest at the store; values past 65504 become
 * inf.                                                                     */
#define FM_F32 0
#define FM_I16 1
#define FM_F16 2
#define FM_BF16 3 /* the models' operators below only                        */
#define FM_E4M3 4 /* 8-bit outputs of fm_rms_norm_quantized                  */
#define FM_I8 5

/* normalized: STFT normalisation folded into the window (flashmel/filters.py
 * make_window): none, divide by sqrt(sum of the squared window), or divide
 * by sqrt(win_length).                                                     */
#define FM_NORMALIZED_NONE 0
#define FM_NORMALIZED_WINDOW 1
#define FM_NORMALIZED_FRAME_LENGTH 2

typedef struct fm_plan fm_plan;

/*
 * fm_args -- every argument of a plan (torchaudio MelSpectrogram's, README
 * "Usage", plus the output type).  Fill it with fm_args_default, which sets
 * torchaudio's defaults for n_fft = 400 at 16 kHz, then change fields.
 *   sample_rate, n_fft, win_length, hop_length, n_mels, f_min, f_max, power,
 *   center, pad_mode, mel_scale, norm: as for fm_plan_create below;
 *   pad        >= 0 zero samples added on both sides of the signal before the
 *              centre padding (which then reflects / repeats / wraps the
 *              zero-extended signal); at most 2^28;
 *   normalized FM_NORMALIZED_*;
 *   out_dtype  FM_F32 or FM_F16: the element type fm_forward writes.
 */
typedef struct fm_args {
  int sample_rate, n_fft, win_length, hop_length, n_mels;
  double f_min, f_max, power;
  int center, pad_mode, mel_scale, norm;
  int pad, normalized, out_dtype;
} fm_args;

/* sample_rate 16000, n_fft 400, win_length 400, hop_length 200, n_mels 128,
 * f_min 0, f_max 8000, power 2, center 1, reflect, HTK, no norm, pad 0, not
 * normalized, f32 output.  FM_E_INVAL if args is NULL.                      */
int fm_args_default(fm_args* args);

/*
 * fm_plan_create_args / fm_plan_create_args_host -- fm_plan_create and
 * fm_plan_create_host with every argument in one struct (read, not kept).
 * Same ownership, validation and errors; a plan made with out_dtype FM_F16
 * writes float16 from fm_forward.
 */
int fm_plan_create_args(fm_plan** out, const fm_args* args);
int fm_plan_create_args_host(fm_plan** out, const fm_args* args);

/*
 * fm_plan_create -- build a plan on the CURRENT HIP device.
 *
 * Arguments are torchaudio MelSpectrogram's (README "Usage"):
 *   sample_rate > 0; n_fft 400 or a power of two from 64 to 16384 (others:
 *   FM_E_UNSUPPORTED; README "Usage" allows exactly these);
 *   0 < win_length <= n_fft (a shorter window is zero-padded centred,
 *   flashmel/filters.py make_window); hop_length > 0;
 *   1 <= n_mels <= 256 (README "Usage");
 *   0 <= f_min < f_max <= sample_rate/2;  power > 0 (2: power spectrum,
 *   1: magnitude);  center 0/1;  pad_mode FM_PAD_*;  mel_scale FM_MEL_*;
 *   norm FM_NORM_*.
 *
 * The window, the CSR filterbank (per mel: first bin, run length, offset,
 * weights), the FFT twiddle tables and the tile geometry are built in
 * float64 on the host, rounded once to float32 and uploaded.  *out receives
 * a plan that owns that device memory; it is immutable and may be used
 * concurrently from several streams of the same device.
 *
 * Errors: FM_E_INVAL / FM_E_UNSUPPORTED for arguments, FM_E_NOMEM,
 * FM_E_HIP (no device, upload failed).  *out is set to NULL on failure.
 */
int fm_plan_create(fm_plan** out, int sample_rate, int n_fft, int win_length,
                   int hop_length, int n_mels, double f_min, double f_max,
                   double power, int center, int pad_mode, int mel_scale,
                   int norm);

/*
 * fm_plan_create_host -- same arguments and validation as fm_plan_create,
 * but builds only the host tables and touches no GPU.  Such a plan serves
 * fm_plan_info / fm_plan_tables / fm_out_frames; fm_forward on it returns
 * FM_E_NODEVICE.
 */
int fm_plan_create_host(fm_plan** out, int sample_rate, int n_fft,
                        int win_length, int hop_length, int n_mels,
                        double f_min, double f_max, double power, int center,
                        int pad_mode, int mel_scale, int norm);

/*
 * fm_forward -- enqueue one mel-spectrogram forward pass on `stream`.
 *
 * The flashmel 0.1.0 page, README "Usage", defines the call: a batch of
 * signals (..., time) in float32 or int16 on the GPU gives (..., n_mels,
 * n_frames), e.g. [8, 480000] at hop 160 gives [8, 128, 3001]; README "How
 * it works" puts the whole chain (padding as index arithmetic, window, real
 * FFT, |X|^power, sparse mel projection) in one kernel launch.  Here the
 * leading dimensions are flattened into `batch`.
 *
 *   in     device pointer to [batch, length] samples, row-major, contiguous,
 *          of type in_dtype (FM_F32: float, FM_I16: int16_t).
 *   out    device pointer to [batch, n_mels, n_frames] elements of the plan's
 *          out_dtype (float32 unless made with FM_F16: float16), row-major,
 *          contiguous (frames fastest), n_frames = fm_out_frames(plan,
 *          length), aligned to its element size.  Every element is written.
 *   batch  >= 0 (0 is a no-op); length >= 1, and with center + reflect
 *          padding length + 2*pad > n_fft/2 (a single reflection), with
 *          circular padding length + 2*pad >= n_fft/2, otherwise FM_E_INVAL;
 *          without center length + 2*pad >= n_fft.
 *
 * One kernel launch; no allocation, no synchronisation.  Launch errors are
 * reported as FM_E_HIP.  The plan must live on the device that is current.
 */
int fm_forward(const fm_plan* plan, const void* in, int in_dtype,
               int64_t batch, int64_t length, void* out, void* stream);

/*
 * fm_backward -- enqueue the gradient of the forward pass with respect to
 * its float32 input: grad_in = d/dx sum(grad_out * mel(x)).
 *
 * The flashmel 0.1.0 page (README "Usage") leaves the transform
 * inference-only; the specux "Backends" page (section "Gradients") computes
 * a spectrogram's gradient as the analytic adjoint, in kernels of the same
 * family as the forward, with a bitwise-reproducible mode.  This entry point
 * applies that adjoint, always deterministically: the transposed filterbank, the gradient of |X|^power
 * (p |X|^(p-2) X, taken as 0 where X = 0 and power != 2), the adjoint of
 * the one-sided DFT (an inverse real FFT), the window, overlap-add of the
 * frames, and the adjoint of the padding (gradients of padded positions go
 * to the samples they copy).
 *
 *   in        device pointer to the forward input [batch, length], float32,
 *             row-major, contiguous (the spectrum is recomputed from it).
 *   grad_out  device pointer to [batch, n_mels, n_frames] float32 (whatever
 *             the plan's out_dtype), n_frames = fm_out_frames(plan, length).
 *   grad_in   device pointer to [batch, length] float32; every element is
 *             written (not accumulated).  Must not overlap the inputs.
 *   batch, length  as for fm_forward.
 *
 * Any hop: when more frames overlap one sample than one workgroup pass
 * holds, the workgroups take several passes.  FM_E_UNSUPPORTED for n_fft
 * 8192 and 16384 (no backward kernel is built for them), and when the
 * samples one workgroup owns (2 n_fft + 2 pad floats or so) do not fit its
 * LDS next to one frame's pass (a very large `pad`).  One kernel launch; no
 * allocation, no synchronisation.
 */
int fm_backward(const fm_plan* plan, const float* in, int64_t batch, int64_t length,
                const float* grad_out, float* grad_in, void* stream);

/*
 * fm_out_frames -- frames per signal for a given length (L = length + 2*pad),
 * the last dimension of fm_forward's output (README "Usage": the output
 * shape (..., n_mels, n_frames), 480000 samples at hop 160 giving 3001):
 *   center: 1 + floor(L / hop) for even n_fft (generally
 *           1 + floor((L + 2*(n_fft/2) - n_fft) / hop));
 *   else:   1 + floor((L - n_fft) / hop).
 * Returns a negative FM_E_* code if the length is invalid for the plan.
 */
int64_t fm_out_frames(const fm_plan* plan, int64_t length);

/*
 * fm_forward_config -- how fm_forward runs a call of `batch` signals of
 * `length` samples on this plan, without running it: *variant = the kernel
 * (FM_FWD_SPLIT, FM_FWD_ROWS, FM_FWD_PAIRED or FM_FWD_LARGE; never
 * FM_FWD_AUTO), *tile_frames = frames per workgroup tile (PAIRED: frames per
 * chunk at most), *workgroups = workgroups launched (0 for batch 0).  The
 * choice depends on the device the plan was created on (its compute units
 * and the kernels' residency); a host-only plan assumes 256 compute units
 * and one resident workgroup per unit.  Any output pointer may be NULL.
 * Returns FM_OK, FM_E_INVAL (NULL plan, batch < 0) or the negative code of
 * an invalid length (as fm_out_frames).  Operation-wise this is a host-side
 * query of the launch geometry behind the pages' one-launch forward pass
 * (flashmel 0.1.0 README "How it works").
 */
int fm_forward_config(const fm_plan* plan, int64_t batch, int64_t length, int* variant,
                      int* tile_frames, int64_t* workgroups);

/* fm_plan_destroy -- free the plan and its device tables.  NULL is a no-op. */
int fm_plan_destroy(fm_plan* plan);

/* Human-readable text for a status code (static storage).                 */
const char* fm_strerror(int status);

/* Message of the last failure on this thread ("" if none).                */
const char* fm_last_error(void);

/* ---- host-side inspection (used by CPU tests; no GPU needed) ------------ */

typedef struct fm_plan_info {
  int n_fft, win_length, hop_length, n_mels, n_freqs; /* n_freqs = n_fft/2+1 */
  int pad, normalized, out_dtype;
  int nnz;          /* nonzero filterbank weights (CSR length)              */
  int w_max;        /* widest filter (bins)                                 */
  int fft_n1, fft_n2; /* complex FFT of n_fft/2 = fft_n1 * fft_n2 points of
                       the split forward kernel and of the backward          */
  int tile_frames;  /* frames per workgroup tile (paired: per chunk)        */
  int threads;      /* threads per workgroup (FM_FWD_AUTO: of the split
                       kernel; the row kernel runs 512)                    */
  int lds_bytes;    /* dynamic LDS per workgroup                            */
  int has_device;   /* 1 if the plan owns device tables                     */
  int forward_variant; /* FM_FWD_SPLIT, FM_FWD_PAIRED, FM_FWD_LARGE,
                          FM_FWD_ROWS or FM_FWD_AUTO                       */
  int fft_n3;       /* FM_FWD_LARGE: n_fft/2 = fft_n1 * fft_n2 * fft_n3 (three
                       passes); 0 otherwise                                  */
} fm_plan_info;

/* Forward kernel variants.  SPLIT: each frame's real FFT through a complex
 * FFT of n_fft/2 points and the real-spectrum split, one tile of frames per
 * workgroup.  PAIRED: two frames per complex FFT of n_fft points (the
 * pages' packing of two real frames into one complex transform, README "How
 * it works"), persistent workgroups that walk their frames in chunks and load
 * the next chunk while transforming the current one; built for n_fft = 400,
 * taken only when the environment variable FM_FORWARD=paired is set at plan
 * creation (measured slower than SPLIT; kept for A/B measurements).
 * LARGE: n_fft 8192 and 16384, whose complex FFT of n_fft/2 points runs in
 * three passes over one LDS buffer, one frame at a time per workgroup, with
 * the mel projection over the CSR rows (these sizes have no backward).  A
 * SPLIT plan of n_fft 4096 also holds this kernel
 * (2048 = 16 x 16 x 8) and runs a call on it when the SPLIT tiles would
 * outnumber the compute units (fm_forward_config reports LARGE then; the
 * plan's own shape, its info and its backward stay SPLIT); FM_FORWARD=large
 * or split at plan creation forces the choice.
 * ROWS: the SPLIT chain with 512-thread workgroups whose second FFT pass
 * gives each row of fft_n2 points of a frame its own thread (the mirrored
 * row's values exchanged between lanes); built for n_fft 64 ... 2048.
 * AUTO (the default for n_fft 64 ... 2048): ROWS or SPLIT chosen per call
 * from the call's size (fm_forward_config reports the choice):
 * n_fft 256, 400, 512 and 2048 always ROWS; the other sizes ROWS when its
 * workgroups number at most the device's compute units.  FM_FORWARD=rows or
 * FM_FORWARD=split at plan creation forces one of them.  ROWS and SPLIT
 * compute the same operations in the same order: their outputs are
 * identical.                                                             */
#define FM_FWD_SPLIT 0
#define FM_FWD_PAIRED 1
#define FM_FWD_LARGE 2
#define FM_FWD_ROWS 3
#define FM_FWD_AUTO 4

int fm_plan_info_get(const fm_plan* plan, fm_plan_info* info);

/*
 * fm_plan_tables -- copy the host tables of a plan.  Any pointer may be NULL
 * to skip that table.  Sizes: window[n_fft] (float32, with the plan's
 * normalisation; the device copy is further scaled by 1/2 for the real-FFT
 * post-processing);
 * mel_first[n_mels], mel_len[n_mels], mel_off[n_mels] (int32; CSR rows,
 * len 0 for an empty filter); mel_w[nnz] (float32);
 * tw_m[2*(n_fft/2)] interleaved re,im of exp(-2*pi*i*j/(n_fft/2));
 * tw_n[2*(n_fft/2)] interleaved re,im of exp(-2*pi*i*k/n_fft).
 */
int fm_plan_tables(const fm_plan* plan, float* window, int32_t* mel_first,
                   int32_t* mel_len, int32_t* mel_off, float* mel_w,
                   float* tw_m, float* tw_n);

/*
 * fm_plan_mel_blocks -- the mel stage's layout on the matrix cores (host
 * copy, for tests).  The filterbank is cut into blocks of up to 16
 * consecutive filters (16, and the longest blocks split into halves of
 * filters); block j covers bins kb .. kb + 4*ksteps - 1 and its weights are
 * stored dense, 64 floats per 4-bin step, float s*64 + l holding filter
 * mel0 + l%16 at bin kb + 4*s + l/16 (0 outside the filter, and for l%16 >=
 * nrow, the block's filter count).
 *   blocks[4*n_blocks]  int32 {kb, ksteps, w_off, mel0 + 65536*nrow} per
 *                       block, grouped by the workgroup wave that computes
 *                       them;
 *   wave_beg[5]         wave w computes blocks wave_beg[w] .. wave_beg[w+1]-1;
 *   weights[n_weights]  every block's weights (w_off indexes them), plus
 *                       zero slack at the end.
 * Any pointer may be NULL; call once with NULL arrays to learn the sizes.
 */
int fm_plan_mel_blocks(const fm_plan* plan, int32_t* blocks, int32_t* wave_beg,
                       float* weights, int32_t* n_blocks, int64_t* n_weights);

/*
 * fm_plan_mel_quads -- the mel stage's layout on the vector units (host copy,
 * for tests; the same projection as the blocks above, used by tiles of 17
 * frames or more).  Filters in quads of 4 consecutive filters (quad q: filters
 * 4q .. 4q+3, those past n_mels empty); a quad runs L steps of one bin, filter
 * a of the quad over bins start_a .. start_a + L - 1, weight w[4*(off + i) + a]
 * at step i (0 outside the filter).
 *   headers[6*n_quads]   int32 {start_0, start_1, start_2, start_3, L, off}
 *                        per quad;
 *   share_beg[9]         share s holds quads share_beg[s] .. share_beg[s+1]-1
 *                        (a workgroup of w waves gives each wave 8/w shares);
 *   weights[n_weights]   every quad's weights, 4 per step.
 * Any pointer may be NULL; call once with NULL arrays to learn the sizes.
 */
int fm_plan_mel_quads(const fm_plan* plan, int32_t* headers, int32_t* share_beg,
                      float* weights, int32_t* n_quads, int64_t* n_weights);

/* ---- operators of the models on top of the mel front end ------------------
 *
 * Element types are FM_F32, FM_F16 and FM_BF16; sums, statistics and
 * reductions are float32, results are rounded once to the element type.
 * Every call only enqueues on `stream`, allocates nothing and is
 * deterministic.  Workspaces are device memory of the caller, 16-byte
 * aligned, of at least the size that the _workspace function returns
 * (negative: FM_E_*; 0: NULL is accepted), free again when the call's work
 * on the stream is done.
 */

/*
 * fm_layer_norm_forward -- y = (x - mean) / sqrt(var + eps) * weight + bias
 * over the last axis, var the mean squared deviation.
 *   x [rows, width], x_stride elements from row to row, elements of a row
 *   contiguous; y [rows, width] contiguous, same type; weight, bias [width]
 *   of type param_dtype (dtype or FM_F32), both NULL or bias NULL allowed;
 *   mean, rstd [rows] float32, each may be NULL (the backward needs them).
 *   0 <= rows < 2^31, 1 <= width <= 2^20, eps >= 0.
 */
int fm_layer_norm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                          void* y, float* mean, float* rstd, int64_t rows, int64_t width,
                          double eps, int dtype, int param_dtype, void* stream);

/* Bytes of fm_layer_norm_backward's workspace. */
int64_t fm_layer_norm_backward_workspace(int64_t rows, int64_t width, int dtype);

/*
 * fm_layer_norm_backward -- gradients of sum(dy * y).  dy, x as above; dx
 * [rows, width] contiguous; dw, db [width] of type param_dtype: dw NULL
 * leaves both out (workspace unused), db may be NULL by itself.  weight NULL:
 * the forward had none.
 */
int fm_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                           const void* weight, const float* mean, const float* rstd, void* dx,
                           void* dw, void* db, void* workspace, int64_t rows, int64_t width,
                           int dtype, int param_dtype, void* stream);

/* Bytes of fm_token_logprobs's workspace. */
int64_t fm_token_logprobs_workspace(int64_t rows, int64_t vocab, int top, int dtype);

/*
 * fm_token_logprobs -- per row of logits x [rows, vocab] (x_stride elements
 * from row to row): lp [rows] = x[token] - lse, the entropy of softmax(x),
 * lse = log sum exp(x), and the `top` largest entries (0 <= top <= 64, <=
 * vocab) in descending order, ties to the lower index: top_ids [rows, top]
 * int64 and top_lp [rows, top].  tokens [rows]: int64 (token_bits 64) or int32
 * (32); a negative token asks for nothing (lp 0), one >= vocab gives NaN.
 * -inf entries have probability 0; a row of only -inf has lp = lse = -inf
 * and entropy 0.  A NaN or +inf entry makes its row's results NaN.  lp, ent,
 * lse may be NULL.  vocab < 2^31 - 65536, rows * (row segments) < 2^31.
 */
int fm_token_logprobs(const void* x, int64_t x_stride, const void* tokens, int token_bits,
                      float* lp, float* ent, float* lse, int64_t* top_ids, float* top_lp,
                      void* workspace, int64_t rows, int64_t vocab, int top, int dtype,
                      void* stream);

/*
 * fm_token_logprobs_backward -- dx [rows, vocab] contiguous, the gradient of
 * sum(g_lp * lp) + sum(g_ent * ent) + sum(g_top * top_lp) with respect to x;
 * any of g_lp, g_ent, g_top (float32) may be NULL; lse and ent from the
 * forward call, top_ids too where g_top is given.  Rows without a valid token
 * take no g_lp; rows of only -inf have a zero gradient.
 */
int fm_token_logprobs_backward(const void* x, int64_t x_stride, const void* tokens,
                               int token_bits, const float* lse, const float* ent,
                               const float* g_lp, const float* g_ent, const int64_t* top_ids,
                               const float* g_top, void* dx, int64_t rows, int64_t vocab, int top,
                               int dtype, void* stream);

/*
 * fm_token_logprobs_strided, fm_token_logprobs_backward_strided -- the same for
 * logits whose rows lie in groups, such as all but the last position of every
 * entry: x_stride elements from row to row of a group of x_inner rows, x_outer
 * elements from group to group.  x_inner 0: all rows at x_stride.  Everything
 * else is contiguous as above.
 */
int fm_token_logprobs_strided(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer,
                              const void* tokens, int token_bits, float* lp, float* ent, float* lse,
                              int64_t* top_ids, float* top_lp, void* workspace, int64_t rows,
                              int64_t vocab, int top, int dtype, void* stream);
int fm_token_logprobs_backward_strided(const void* x, int64_t x_stride, int64_t x_inner,
                                       int64_t x_outer, const void* tokens, int token_bits,
                                       const float* lse, const float* ent, const float* g_lp,
                                       const float* g_ent, const int64_t* top_ids, const float* g_top,
                                       void* dx, int64_t rows, int64_t vocab, int top, int dtype,
                                       void* stream);

/*
 * fm_attention_args -- attention with a learned relative position bias:
 *
 *   s[i, j] = scale * q[i].k[j] + table[bucket_map[far + clamp(j - pos(i), -far, far)]][head]
 *   o[i] = sum_j softmax_j(s[i, j]) v[j],  pos(i) = query_offset[entry] + i
 *
 * over the keys j < key_lengths[entry], and j <= pos(i) if causal.  A query
 * without any key gives o = 0, lse = -inf and zero gradients; keys and values
 * at or past key_lengths are not read (NaN there does no harm).  Below
 * key_lengths they have to be finite for a causal query too: the keys after it
 * have a probability of 0, which times an infinity or NaN of a value is NaN.
 *   dtype        of q, k, v, o and their gradients;
 *   q, o [batch, heads, q_len, head_dim], k, v [batch, kv_heads, k_len,
 *                head_dim]: strides in elements of (entry, head, time), >= 0,
 *                the last axis contiguous; heads a multiple of kv_heads, query
 *                head h reads key head h / (heads / kv_heads); head_dim <= 128;
 *                batch * heads * (query blocks of 128) and batch * kv_heads *
 *                (key blocks of 128) stay below about 2^24;
 *   scale        in [2^-60, 2^60];
 *   table        [num_buckets, heads] contiguous, table_dtype (dtype or
 *                FM_F32), num_buckets <= 1024; finite values beyond +-65536
 *                count as +-65536, -inf hides a distance;
 *   bucket_map   [2 far + 1] int32, the bucket of each distance key - query
 *                from -far to far (<= 1024), farther ones taken at the ends; a
 *                distance with an entry outside [0, num_buckets) has no bias;
 *   key_lengths  [batch] int32 (clamped to [0, k_len]) or NULL: k_len;
 *   query_offset [batch] int32 or NULL: query_offset_value for every entry;
 *   lse          [batch, heads, q_len] float32, NULL allowed in the forward;
 * backward: grad_o in; grad_q, grad_k, grad_v out (every element written);
 *                grad_table out, [num_buckets, heads] of table_dtype, or NULL.
 */
typedef struct fm_attention_args {
  int dtype, table_dtype, causal, far, num_buckets, reserved;
  int64_t batch, heads, kv_heads, q_len, k_len, head_dim, query_offset_value;
  double scale;
  const void* q;
  const void* k;
  const void* v;
  const void* table;
  const int32_t* bucket_map;
  const int32_t* key_lengths;
  const int32_t* query_offset;
  void* o;
  float* lse;
  const void* grad_o;
  void* grad_q;
  void* grad_k;
  void* grad_v;
  void* grad_table;
  int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];
  int64_t grad_o_stride[3], grad_q_stride[3], grad_k_stride[3], grad_v_stride[3];
} fm_attention_args;

/* Bytes of the workspace of fm_attention_forward (backward 0) or _backward
 * (1); pointers and strides are not looked at. */
int64_t fm_attention_workspace(const fm_attention_args* args, int backward);

/* o (and lse if not NULL). */
int fm_attention_forward(const fm_attention_args* args, void* workspace, void* stream);

/* Gradients of sum(grad_o * o); o and lse as the forward wrote them. */
int fm_attention_backward(const fm_attention_args* args, void* workspace, void* stream);

/*
 * fm_recurrence_args -- a gated linear recurrence over time, per channel:
 *
 *   a = sigmoid(forget[t]), h[t] = a h[t - 1] + (1 - a) x[t], y[t] = h[t] silu(gate[t])
 *
 * from h[-1] = state.  forget of +inf keeps the state, -inf replaces it by x.
 * Without a gate y = h.  Frames at or past lengths[entry] are not part of the
 * sequence: NaN there does no harm, y and the gradients are 0 there and the
 * state stays as it was after the last frame before.
 *   dtype        of x, forget, gate, y and their gradients; states are float32;
 *   x, forget, gate, grad_y [batch, time, channels]: strides in elements of
 *                (entry, time), >= 0, channels contiguous; gate NULL: none;
 *   y, grad_x, grad_forget, grad_gate [batch, time, channels] contiguous;
 *   state, last_state, grad_last, grad_state [batch, channels]: state NULL is
 *                0, and last_state may be the same memory; grad_last NULL is 0,
 *                grad_state NULL is not wanted;
 *   lengths      [batch] int32 (clamped to [0, time]) or NULL: time;
 *   saved        [batch, (time + 63) / 64, channels] float32, the state before
 *                every 64th frame below the entry's length: written by the forward
 *                (NULL: not wanted), read by the backward;
 * backward: grad_y and grad_last in; grad_x, grad_forget, grad_gate (with a
 *                gate) and grad_state out; y and last_state are not looked at.
 * batch, time < 2^30, channels <= 2^20, batch * (blocks of 16 channels) < 2^23;
 * frames of x, forget, gate and grad_y less than 8 MiB apart where there are more than
 * one (more than two in a forward without saved).
 */
typedef struct fm_recurrence_args {
  int dtype, reserved;
  int64_t batch, time, channels;
  const void* x;
  const void* forget;
  const void* gate;
  const float* state;
  const int32_t* lengths;
  void* y;
  float* last_state;
  float* saved;
  const void* grad_y;
  const float* grad_last;
  void* grad_x;
  void* grad_forget;
  void* grad_gate;
  float* grad_state;
  int64_t x_stride[2], forget_stride[2], gate_stride[2], grad_y_stride[2];
} fm_recurrence_args;

/* Bytes of the workspace of fm_gated_recurrence_forward (backward 0) or
 * _backward (1); pointers and strides are not looked at. */
int64_t fm_gated_recurrence_workspace(const fm_recurrence_args* args, int backward);

/* y, last_state (and saved if not NULL). */
int fm_gated_recurrence_forward(const fm_recurrence_args* args, void* workspace, void* stream);

/* Gradients of sum(grad_y * y) + sum(grad_last * last_state). */
int fm_gated_recurrence_backward(const fm_recurrence_args* args, void* workspace, void* stream);

/*
 * fm_rms_norm_forward -- y = s / sqrt(mean(s^2) + eps) * weight over the last
 * axis, s = x, or with a residual s = x + residual rounded to the rows' type.
 *   x, residual [rows, width], strides in elements from row to row, elements of
 *   a row contiguous; y [rows, width] contiguous, same type; sum [rows, width]
 *   contiguous takes s where there is a residual (NULL otherwise) and may be the
 *   residual's own memory if that is contiguous; weight [width] of type
 *   param_dtype (dtype or FM_F32) or NULL; rstd [rows] float32 or NULL (the
 *   backward needs it).  0 <= rows < 2^31, 1 <= width <= 2^20, eps >= 0
 *   and finite in float32.  A row's sum of squares is a float32: past its range
 *   (|s| around 10^19) y is 0.
 */
int fm_rms_norm_forward(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        const void* weight, void* y, void* sum, float* rstd, int64_t rows, int64_t width,
                        double eps, int dtype, int param_dtype, void* stream);

/*
 * fm_rms_norm_quantized -- the same with an output in 8 bits: scale [rows]
 * float32 is the row's largest |y| over 448 (out_dtype FM_E4M3) or 127 (FM_I8),
 * 1 for a row of zeros, at least 2^-126; q [rows, width] is y / scale rounded to
 * nearest from the unrounded y.  A NaN in a row makes its scale NaN.
 */
int fm_rms_norm_quantized(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          const void* weight, void* q, float* scale, void* sum, int64_t rows, int64_t width,
                          double eps, int dtype, int param_dtype, int out_dtype, void* stream);

/* Bytes of fm_rms_norm_backward's workspace. */
int64_t fm_rms_norm_backward_workspace(int64_t rows, int64_t width, int dtype);

/*
 * fm_rms_norm_backward -- gradients of sum(dy * y) + sum(grad_sum * s), s (`sum`)
 * and rstd from the forward (s = x without a residual).  dx [rows, width]
 * contiguous is the gradient of x and of the residual alike; grad_sum may be
 * NULL; dw [width] of type param_dtype, NULL leaves it out (workspace unused).
 */
int fm_rms_norm_backward(const void* dy, int64_t dy_stride, const void* sum, int64_t sum_stride,
                         const void* grad_sum, int64_t grad_sum_stride, const void* weight, const float* rstd,
                         void* dx, void* dw, void* workspace, int64_t rows, int64_t width, int dtype,
                         int param_dtype, void* stream);

/*
 * fm_distill -- how far logits x [rows, vocab] are from a teacher of whom each
 * row's `top` best tokens ids [rows, top] int64 and log probabilities lps
 * [rows, top] float32 are known (1 <= top <= 64):
 *
 *   loss = T^2 sum_k q_k (log q_k - lp[ids_k]),  lp = log_softmax(x / T),
 *   q = softmax(lps / T) over the row's tokens,  T the temperature;
 *
 * with rest != 0 (T has to be 1) q = exp(lps), and the mass that the teacher
 * leaves, r = max(0, 1 - sum q), stands against the student's for all tokens
 * that are not named: + r (log r - log sum of p over those).
 * An entry with a negative id is none (rows with fewer); a row without any has
 * loss 0 and no gradient; an id >= vocab gives NaN and takes no part in the
 * gradient.  The same id twice counts twice.  Teacher entries of -inf have
 * q = 0.  A student that gives a named token no probability (-inf) has loss inf;
 * one that leaves nothing for the others has no rest term.  A row of -inf only
 * has a zero gradient.  NaN or +inf in a row stays in its row.
 *   x: x_stride elements from row to row, or groups of x_inner rows at x_stride
 *   and the groups at x_outer (x_inner 0: none); loss [rows] float32; stats
 *   [rows, 4] float32 or NULL: what the backward needs (the largest x and the log
 *   of the sum of exp((x - largest) / T), both also over the tokens that are not
 *   named).  T in [2^-10, 2^10], the largest |x| / T within float32; vocab <
 *   2^31 - 65536, rows * (row segments) < 2^31.
 */
int64_t fm_distill_workspace(int64_t rows, int64_t vocab, int dtype);
int fm_distill(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer, const int64_t* ids,
               const float* lps, float* loss, float* stats, void* workspace, int64_t rows, int64_t vocab, int top,
               double temperature, int rest, int dtype, void* stream);

/*
 * fm_distill_backward -- dx [rows, vocab] contiguous, the gradient of
 * sum(grad_loss * loss) with respect to x: T grad (p - q) and, with the rest,
 * the others' p (1 - r / their sum) grad.  stats from the forward.
 */
int fm_distill_backward(const void* x, int64_t x_stride, int64_t x_inner, int64_t x_outer, const int64_t* ids,
                        const float* lps, const float* stats, const float* grad_loss, void* dx, int64_t rows,
                        int64_t vocab, int top, double temperature, int rest, int dtype, void* stream);

/*
 * fm_adjust_args -- logits before a token is chosen from them; per row and token
 *
 *   x = x > 0 ? x * (1 / repetition) : x * repetition   if it is in the history
 *   x = x - frequency * count - presence * (count > 0)
 *   x = x + the sum of the token's biases, in their order
 *   x = -inf                                       if its bit of `allowed` is 0
 *
 * in float32, rounded once.  count is how often the token is in the history from
 * prompt_lengths[row] on (0 without).
 *   x [rows, vocab]: x_stride elements from row to row; out [rows, vocab]
 *   contiguous, same type, may be x's own memory if that is contiguous;
 *   history [rows, history_len] of history_bits (32 or 64) wide integers,
 *   history_stride from row to row; history_lengths, prompt_lengths [rows] int32
 *   (clamped to [0, history_len]) or NULL: history_len, 0.  Tokens outside
 *   [0, vocab) are none;
 *   repetition, frequency, presence [rows] float32 or NULL: the *_value for all
 *   rows (repetition > 0, finite in float32 like its reciprocal);
 *   bias_ids [rows, biases] int64, bias [rows, biases] float32, contiguous; ids
 *   outside [0, vocab) are none; the same one twice counts twice;
 *   allowed: rows of (vocab + 31) / 32 words of 32 bits, lowest first,
 *   allowed_stride words from row to row (0: one for all rows), or NULL.
 * rows < 2^31, vocab < 2^31 - 65536, rows * (row segments of 2048) < 2^22,
 * history_len < 2^20, biases <= 1024.
 */
typedef struct fm_adjust_args {
  int dtype, history_bits;
  int64_t rows, vocab, history_len, biases;
  int64_t x_stride, history_stride, allowed_stride;
  double repetition_value, frequency_value, presence_value;
  const void* x;
  void* out;
  const void* history;
  const int32_t* history_lengths;
  const int32_t* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int64_t* bias_ids;
  const float* bias;
  const int32_t* allowed;
} fm_adjust_args;

int fm_adjust_logits(const fm_adjust_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FM_H_ */
