/*
 * attnres.h - C ABI of the GB300 (sm_103a) AttnRes depth-wise aggregation.
 *
 * Attention Residuals replace the additive residual of a pre-norm Transformer
 * with a softmax-weighted sum over depth. For one token and one read (the
 * input of one sublayer, or of the LM head):
 *
 *     e_i = w^T RMSNorm_key(v_i)              (no 1/sqrt(d), temperature 1)
 *     a_i = exp(e_i) / sum_j exp(e_j)
 *     z   = sum_i a_i v_i
 *
 * (DepthBench reading notes, section 2.3 "Full AttnRes", paper Appendix A;
 * LLMRes blog, section "Kimi AttnRes": phi(q, k) = exp(q^T RMSNorm(k)),
 * q = w_l, k_i = v_i, with RMSNorm applied to the keys only.) RMSNorm is not
 * written out on the pages; this library uses the plain form
 * RMSNorm(x)_k = gamma_k x_k / sqrt(mean_k x_k^2 + eps).
 *
 * Full AttnRes: the sources of read l are the embedding v_0 and every earlier
 * sublayer output. Block AttnRes (DepthBench reading notes section 2.5; LLMRes
 * blog "Block Attention Residuals"; datacamp explainer "block attention
 * residuals"): the sublayers are cut into blocks of S; a read attends over the
 * embedding, the sums of the completed blocks, and the running sum of the
 * current block when it is non-empty. The two-stage computation (datacamp
 * explainer, "two-stage computation") batches the S pseudo-queries of a block
 * against the cross-block sources (stage 1) and folds in the running sum with
 * an online-softmax merge (stage 2).
 *
 * Conventions for every entry point:
 *   - Pointers named as device pointers must point to device memory of the
 *     current CUDA device; the library reads and writes them only from
 *     kernels. Host arrays are marked "host".
 *   - The caller owns all memory. The library keeps no per-call state and
 *     allocates no device memory.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL is
 *     the legacy default stream) and is asynchronous: the call returns before
 *     the kernels finish. No call synchronises, except attnres_device_status.
 *   - Tensors are row-major. A [T, d] tensor has row stride d (contiguous);
 *     "sources" of a read are consecutive [T, d] slices `src_stride` elements
 *     apart, src_stride >= T*d.
 *   - dtype arguments take attnres_dtype values. Storage is fp32 or bf16;
 *     arithmetic is fp32 throughout; bf16 results are rounded to nearest even.
 *     w and gamma are always fp32; eps is a host scalar (>= 0).
 *   - T == 0 is valid and launches nothing.
 *   - Fast kernels need 16-byte aligned pointers and d a multiple of 128
 *     (full read), of the per-warp slice (stage 1) or of 8 (merge); any other
 *     valid input runs on a general kernel with the same results.
 *   - Errors: ATTNRES_ERR_INVALID_ARG for bad arguments (nothing launched),
 *     ATTNRES_ERR_UNSUPPORTED for valid requests beyond a stated limit,
 *     ATTNRES_ERR_CUDA when a launch fails (the CUDA error is consumed).
 *     Device-side waits are bounded; a wait that runs out makes the kernel
 *     stop and is reported by attnres_device_status as ATTNRES_ERR_TIMEOUT.
 *   - Outputs must not overlap inputs unless a function says otherwise.
 */
#ifndef ATTNRES_H
#define ATTNRES_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ATTNRES_F32 = 0, ATTNRES_BF16 = 1 } attnres_dtype;

typedef enum {
  ATTNRES_OK = 0,
  ATTNRES_ERR_INVALID_ARG = 1,
  ATTNRES_ERR_UNSUPPORTED = 2,
  ATTNRES_ERR_CUDA = 3,
  ATTNRES_ERR_TIMEOUT = 4
} attnres_status;

/* Largest number of pseudo-queries one stage-1 call batches. */
#define ATTNRES_MAX_QUERIES 16

/*
 * attnres_full_fwd - one Full AttnRes read (DepthBench reading notes section
 * 2.3, paper Appendix A; LLMRes blog "Kimi AttnRes", h_l = sum_i alpha_{i->l} v_i).
 *
 *   V          device, [n_src, T, d] sources (slice i at V + i*src_stride
 *              elements), dtype v_dtype. Slice 0 is the embedding.
 *   src_stride elements between consecutive sources, >= T*d.
 *   n_src      number of sources, >= 1 (n_src == 1 returns v_0 exactly).
 *   w, gamma   device, fp32 [d]: the read's pseudo-query and key-RMSNorm gain.
 *   eps        RMSNorm epsilon, >= 0.
 *   out        device, [T, d] of out_dtype; must not overlap V.
 */
int attnres_full_fwd(const void* V, int64_t src_stride, int32_t n_src, int64_t T,
                     int32_t d, int32_t v_dtype, const float* w, const float* gamma,
                     float eps, void* out, int32_t out_dtype, void* stream);

/*
 * attnres_full_pass - R consecutive Full AttnRes reads over one stored
 * history: read r aggregates V[0 .. r] (r + 1 sources) with W[r], Gamma[r]
 * and writes out + r*out_stride. This is the read sequence of a Full AttnRes
 * model whose sublayer r's output is V[r + 1] (DepthBench reading notes
 * section 2.3: the first sublayer reads the embedding alone; with R = 2L + 1
 * the last read is the LM-head read).
 *
 *   V        device, [R, T, d] history, dtype v_dtype, src_stride >= T*d.
 *   W, Gamma device, fp32 [R, d].
 *   out      device, R outputs [T, d] of out_dtype, out_stride >= T*d
 *            elements apart; must not overlap V.
 */
int attnres_full_pass(const void* V, int64_t src_stride, int32_t R, int64_t T,
                      int32_t d, int32_t v_dtype, const float* W, const float* Gamma,
                      float eps, void* out, int64_t out_stride, int32_t out_dtype,
                      void* stream);

/*
 * attnres_full_fwd_prenorm / attnres_full_pass_prenorm - the same reads,
 * each also emitting the consuming sublayer's pre-norm of its result
 * (DepthBench reading notes section 2.3: the sublayer computes
 * f_l = F_l(RMSNorm_pre,l(z_l)) from the aggregated z_l). The row is
 * normalised while it is still in registers, which saves the sublayer a read
 * of z:
 *
 *   out_normed[t, k] = gamma_pre[k] * z[t, k] / sqrt(mean_k z[t, k]^2 + eps_pre)
 *
 * from z in fp32 before it is rounded to out_dtype.
 *
 *   gamma_pre   device, fp32 [d] (pass: [R, d], row r for read r).
 *   eps_pre     >= 0.
 *   out         as for the plain read, or NULL: z itself is then not stored.
 *   out_normed  device, [T, d] of out_dtype (pass: R of them, out_stride
 *               elements apart, like out); must not overlap V, out, W,
 *               Gamma or gamma_pre. Not NULL.
 */
int attnres_full_fwd_prenorm(const void* V, int64_t src_stride, int32_t n_src, int64_t T,
                             int32_t d, int32_t v_dtype, const float* w, const float* gamma,
                             float eps, const float* gamma_pre, float eps_pre, void* out,
                             void* out_normed, int32_t out_dtype, void* stream);
int attnres_full_pass_prenorm(const void* V, int64_t src_stride, int32_t R, int64_t T,
                              int32_t d, int32_t v_dtype, const float* W, const float* Gamma,
                              float eps, const float* Gamma_pre, float eps_pre, void* out,
                              void* out_normed, int64_t out_stride, int32_t out_dtype,
                              void* stream);

/*
 * attnres_query_projection / attnres_full_fwd_dynq - the input-dependent
 * query (the ablation the pages report: LLMRes blog, on the paper's ablation:
 * a query projected from the current hidden state by a per-layer d x d matrix
 * instead of the fixed learned pseudo-query).
 *
 * attnres_query_projection: Q[t, j] = sum_k Wq[j, k] H[t, k], i.e. Q = H Wq^T,
 * on the tensor cores (bf16 inputs, fp32 sums).
 *   H    device, [T, d] of h_dtype (ATTNRES_BF16 only; else UNSUPPORTED).
 *   Wq   device, bf16 [d, d], row j the weights of query feature j.
 *   Q    device, fp32 [T, d]; must not overlap H or Wq.
 *
 * attnres_full_fwd_dynq: the Full read with token t scored by its own query:
 * e_i(t) = Q[t] . (gamma * v_i(t)) / rms(v_i(t)); otherwise as
 * attnres_full_fwd (there is no shared w).
 *   Q    device, fp32 [T, d]; must not overlap out.
 */
int attnres_query_projection(const void* H, int64_t T, int32_t d, int32_t h_dtype, const void* Wq,
                             float* Q, void* stream);
int attnres_full_fwd_dynq(const void* V, int64_t src_stride, int32_t n_src, int64_t T, int32_t d,
                          int32_t v_dtype, const float* Q, const float* gamma, float eps, void* out,
                          int32_t out_dtype, void* stream);

/*
 * 8-bit rows. The history of a Full read, and the hidden states its queries are
 * projected from, may be held in 8 bits: half the bytes of bf16. A read, bound
 * by the conversion of the codes, takes as long as one of bf16 rows (3 sources)
 * or less (by 7 % for 141 sources of 640 features, a quarter to a third at most
 * other sizes). The pages have no counterpart; they name the
 * history's memory as the cost of Full AttnRes (DepthBench reading notes,
 * section 4.7 and Fig. 11).
 *
 * A row of d features is cut into groups of ATTNRES_Q8_GROUP = 128 (the last
 * may be short). With a_g the largest finite magnitude of group g, its scale is
 * 2^e_g with e_g the smallest integer >= -126 such that a_g <= 448 * 2^e_g (448
 * is the largest e4m3 number), and feature k is held as
 *   c_k = x_k * 2^-e_g rounded to e4m3 (to nearest, ties to even),
 * so it stands for v_k = c_k * 2^e_g. A power of two scales exactly: the codes
 * follow from x alone, and writing what was read back gives the same values. A
 * magnitude below 2^-117 keeps fewer than four bits. Where e_g = 120 codes stop
 * at 240, so that v_k stays finite. An element that is not finite becomes NaN.
 * With the row goes mean_k v_k^2 (fp32), the mean square its key RMSNorm needs
 * in every read (infinite, and the row's score 0, where squares of its values
 * add up past fp32's range: magnitudes of some 1e19; for queries whose
 * magnitudes, times gamma, add up to less than 2^32).
 *
 * A source is `cap` rows in attnres_q8_source_bytes(cap, d) bytes, with G = ceil(d / 128):
 *   cap rows of 128 G bytes: the codes, zero from feature d on;
 *   cap tails of 16 ceil((4 ceil(G / 4) + 4) / 16) bytes: e_g + 127 of each
 *   group, one byte each; on the next 4-byte boundary the mean square (fp32);
 *   zeros;
 *   what is left up to a multiple of 128 bytes is not looked at.
 * Sources follow each other. Calls take `cap` and the number T <= cap of rows in use (a batch may be
 * smaller than the history was made for). Pointers to sources must be 16-byte
 * aligned (128-byte aligned ones stream fastest): else INVALID_ARG.
 */
#define ATTNRES_Q8_GROUP 128

/* Bytes of a source of cap rows; -1 for cap < 0, d < 1 or d > 2^24. */
int64_t attnres_q8_source_bytes(int64_t cap, int32_t d);

/*
 * attnres_q8_write - n sources of T rows each into 8-bit rows (a history, one
 * source at a time as sublayers finish, or as a whole).
 *
 *   x           device, n slices [T, d] of dtype, x_stride elements apart
 *               (>= T*d; not looked at when n == 1).
 *   rows, cap   device, n sources of cap >= T rows. The codes and tails of the
 *               first T rows are written whole, nothing else. Must not overlap x.
 * Any d; d a multiple of 8 (bf16) or 4 (fp32) in 16-byte aligned storage
 * streams fastest.
 */
int attnres_q8_write(const void* x, int64_t x_stride, int32_t n, int64_t T, int32_t d,
                     int32_t dtype, void* rows, int64_t cap, void* stream);

/*
 * attnres_q8_read - the values 8-bit rows stand for: out = c * 2^e. In bf16
 * they are exact (codes have four significant bits) down to bf16's smallest
 * number, so attnres_full_bwd over them is the backward of attnres_full_fwd_q8
 * with the shared query w, up to z (the pre-norm's is attnres_rmsnorm_bwd).
 * There is no backward for the queries of tokens, Q.
 *
 *   rows, cap, n, T, d   as attnres_q8_write.
 *   out         device, n slices [T, d] of out_dtype, out_stride elements
 *               apart (>= T*d; not looked at when n == 1). Must not overlap rows.
 */
int attnres_q8_read(const void* rows, int64_t cap, int32_t n, int64_t T, int32_t d, void* out,
                    int64_t out_stride, int32_t out_dtype, void* stream);

/*
 * attnres_full_fwd_q8 - the Full read (attnres_full_fwd) over 8-bit rows: the
 * sources are the values the rows stand for, and rms(v_i) comes from the
 * rows' mean squares.
 *
 *   rows, cap   device, n_src sources of cap >= T rows.
 *   w           device, fp32 [d], the shared query, or NULL with Q.
 *   Q           device, fp32 [T, d], a query for each token
 *               (attnres_full_fwd_dynq), or NULL with w. One of the two.
 *   gamma, eps  as attnres_full_fwd.
 *   gamma_pre, eps_pre, out_normed   the consuming sublayer's pre-norm, as
 *               attnres_full_fwd_prenorm; gamma_pre and out_normed both given
 *               or both NULL.
 *   out         device, [T, d] of out_dtype; NULL (z not stored) only with
 *               out_normed.
 * Outputs overlap nothing. Which kernel runs, and how many warps and CTAs share
 * a token's sources, depends on T, n_src and d; so do the last bits of z.
 * Nothing overflows on the way to z, which is finite where the values and the
 * scores are; the pre-norm of a z whose squares add up past fp32's range is 0.
 * d up to 2048 takes streaming kernels; wider rows take a general one, for
 * which ATTNRES_ERR_UNSUPPORTED means that
 * 4 (n_src + 512 ceil(G / 4)) bytes are over 200 KB.
 */
int attnres_full_fwd_q8(const void* rows, int64_t cap, int32_t n_src, int64_t T, int32_t d,
                        const float* w, const float* Q, const float* gamma, float eps,
                        const float* gamma_pre, float eps_pre, void* out, void* out_normed,
                        int32_t out_dtype, void* stream);

/*
 * attnres_q8_weight - a weight matrix in 8 bits with one scale for each block
 * of 128 x 128 weights (the last ones of a row or column may be short), by the
 * rule of the rows: a power of two from the block's largest finite magnitude.
 *
 *   W           device, [m, d] of dtype, row-major (m output features).
 *   W8          device, attnres_q8_weight_bytes(m, d) bytes, 16-byte aligned:
 *               m rows of 128 G codes (zero from d on), then, for each 128
 *               output features, 16 ceil(G / 16) bytes: e + 127 of its G
 *               blocks, then zeros. Must not overlap W.
 */
int attnres_q8_weight(const void* W, int32_t m, int32_t d, int32_t dtype, void* W8, void* stream);
/* -1 for sizes below 1 or above 2^24. */
int64_t attnres_q8_weight_bytes(int32_t m, int32_t d);

/*
 * attnres_query_projection_q8 - the input-dependent query's projection
 * (attnres_query_projection) of 8-bit rows by an 8-bit weight matrix:
 * Q[t, j] = sum_k v[t, k] W[j, k], summed in fp32 in an order that is not
 * specified: with G = ceil(d / 128) the result is within (d + 2 G + 4) 2^-24 of
 * sum_k |v[t, k] W[j, k]|. (On tensor cores products of 32 features, scaled, are
 * added to one sum over all of d; for few tokens the sums of 16 features are
 * scaled and added.) Which kernel runs, and so the last bits, depends on T, d
 * and m.
 *
 *   rows, cap   device, one source of cap >= T rows of d features.
 *   W8          device, [m, d] as attnres_q8_weight laid it out, 16-byte aligned. m need not be
 *               d: the queries of several reads may be projected at once.
 *   Q           device, fp32 [T, m]; must not overlap rows or W8.
 * The mean squares of the rows are not looked at.
 */
int attnres_query_projection_q8(const void* rows, int64_t cap, int64_t T, int32_t d, const void* W8,
                                int32_t m, float* Q, void* stream);

/*
 * attnres_rmsnorm - RMSNorm of each row, out = gamma * x / sqrt(mean(x^2) + eps)
 * in fp32, stored in dtype: the sublayer pre-norm for a row no aggregation
 * call produces with it (the first sublayer of a block, whose output is
 * stage 1's O[0]).
 *
 *   x, out   device, [T, d] of dtype; out may be x (in place) but must not
 *            otherwise overlap it.
 *   gamma    device, fp32 [d].  eps >= 0.
 */
int attnres_rmsnorm(const void* x, int64_t T, int32_t d, int32_t dtype, const float* gamma,
                    float eps, void* out, void* stream);

/*
 * attnres_gated_residual - what lies between a sublayer's output f and the
 * next sublayer's input: the norm after the sublayer, its gate, the residual
 * scale, the addition to the stream and the next sublayer's pre-norm, in one
 * pass over the rows:
 *
 *   y[t, k]      = gamma_post[k] f[t, k] / sqrt(mean_k f[t, k]^2 + eps_post)
 *   x_out[t, k]  = x[t, k] + scale * act(gate[t / gate_rows, k]) * y[t, k]
 *   normed[t, k] = gamma_pre[k] x_out[t, k] / sqrt(mean_k x_out[t, k]^2 + eps_pre)
 *
 * all in fp32, x_out and normed each rounded once (normed from the fp32 row,
 * before x_out is rounded, as in the pre-norm epilogues). With x NULL the
 * result is the sublayer's AttnRes source itself; with x an fp32 running sum
 * of a block it is the sum advanced by the sublayer.
 *
 *   f           device, [T, d] of dtype: the sublayer's output.
 *   x           device, [T, d] of x_dtype: the stream, or NULL (x = 0).
 *   gamma_post  device, fp32 [d], or NULL: no post-norm (y = f).
 *   gate        device, [ceil(T / gate_rows), d] of gate_dtype, or NULL (1).
 *               Token t takes row t / gate_rows: gate_rows 1 is a gate per
 *               token, gate_rows >= T one row for all of them (a learned gain
 *               per feature), anything between one row per run of tokens (the
 *               last run may be short).
 *   gate_rows   >= 1 (not looked at without a gate).
 *   gate_act    ATTNRES_GATE_IDENTITY, or ATTNRES_GATE_SIGMOID: 1/(1+exp(-g)).
 *   scale       host, finite; so is scale * gamma_post, which the fast kernel
 *               forms first.
 *   x_out       device, [T, d] of x_dtype; may be x (in place).
 *   gamma_pre   device, fp32 [d], and normed, device, [T, d] of dtype: both
 *               given, or both NULL (no pre-norm).
 *   dtype BF16 takes x_dtype BF16 or F32; dtype F32 takes x_dtype F32. The
 *   gate may be of either type.
 * Outputs overlap nothing but, for x_out, x itself. Rows whose squares
 * overflow fp32 (elements of about 1e19) are outside what RMSNorm computes
 * here, as in attnres_rmsnorm. Any d >= 1; d a multiple of 8 up to 8192 with
 * 16-byte aligned pointers takes the fast kernel. Others take a general one,
 * here and in the two backwards below: about 3 times as long forward, 6 to 8
 * times backward, where measured.
 */
typedef enum { ATTNRES_GATE_IDENTITY = 0, ATTNRES_GATE_SIGMOID = 1 } attnres_gate_act;

int attnres_gated_residual(const void* f, const void* x, const float* gamma_post, float eps_post,
                           const void* gate, int64_t gate_rows, int32_t gate_dtype,
                           int32_t gate_act, float scale, int64_t T, int32_t d, int32_t dtype,
                           int32_t x_dtype, void* x_out, const float* gamma_pre, float eps_pre,
                           void* normed, void* stream);

/*
 * attnres_gated_residual_bwd - its gradients, given dL/dx_out and dL/dnormed.
 * With r = 1/sqrt(mean(x_out^2) + eps_pre), u = r x_out, q = r_f f (r_f the
 * same of f; q = f without a post-norm), h = gamma_pre dnormed and, per token,
 * <a> the mean over features:
 *   D          = dx_out + r (h - u <h u>)                   dL/dx = D
 *   dy         = scale act(gate) D
 *   df         = r_f (gamma_post dy - q <gamma_post dy q>)  (dy without a post-norm)
 *   dgate      = sum over the row's tokens of scale act'(gate) gamma_post q D
 *   dgamma_post = sum_t dy q,   dgamma_pre = sum_t dnormed u.
 * Everything is recomputed from f, the gate and the stored x_out: the forward
 * keeps nothing else.
 *
 *   f, gamma_post, eps_post, gate, gate_rows, gate_dtype, gate_act, scale, T,
 *   d, dtype, x_dtype, gamma_pre, eps_pre   as the forward's.
 *   x_out      device, [T, d] of x_dtype, as the forward left it. Read only
 *              with dnormed; may be NULL without.
 *   dx_out     device, [T, d] of dx_dtype, or NULL (0): dL/dx_out by every way
 *              other than normed.
 *   dnormed    device, [T, d] of dtype, or NULL (0; gamma_pre is then not
 *              looked at). dx_out or dnormed must be given.
 *   dx_dtype   F32, or with dtype BF16 also BF16.
 *   df         device, [T, d] of dtype, or NULL (not wanted).
 *   dx         device, [T, d] of dx_dtype, or NULL; may be dx_out (in place).
 *   dgate      device, like gate, or NULL: written (not added to), summed over
 *              its tokens in fp32 and rounded once.
 *   dgamma_post, dgamma_pre   device, fp32 [d], or NULL: added to, or with
 *              accumulate 0 written. Without a post-norm (dnormed) the
 *              dgamma_post (dgamma_pre) gradient is zero.
 *   scratch    device, fp32, at least attnres_gated_residual_bwd_scratch_floats
 *              floats; need not be initialised, contents on return unspecified.
 *              Calls that may overlap on the GPU need scratches of their own.
 * Sums run in a fixed order: the same call gives the same bits. Outputs
 * overlap nothing but, for dx, dx_out itself. T == 0 launches nothing unless
 * accumulate is 0, which writes zeros to the gains' gradients.
 */
int attnres_gated_residual_bwd(const void* f, const float* gamma_post, float eps_post,
                               const void* gate, int64_t gate_rows, int32_t gate_dtype,
                               int32_t gate_act, float scale, int64_t T, int32_t d, int32_t dtype,
                               int32_t x_dtype, const void* x_out, const float* gamma_pre,
                               float eps_pre, const void* dx_out, int32_t dx_dtype,
                               const void* dnormed, void* df, void* dx, void* dgate,
                               float* dgamma_post, float* dgamma_pre, int32_t accumulate,
                               float* scratch, int64_t scratch_floats, void* stream);
/* Scratch the call above needs, in floats; -1 for bad sizes (gate_rows 1 without a gate). */
int64_t attnres_gated_residual_bwd_scratch_floats(int64_t T, int32_t d, int64_t gate_rows);

/*
 * attnres_rmsnorm_bwd - gradients of attnres_rmsnorm, and of the pre-norm of
 * any *_prenorm call with respect to the row it normalised (x: the stored z):
 *   dx = dres + r (h - u <h u>),  h = gamma dy, u = r x;   dgamma = sum_t dy u.
 *
 *   x, dy      device, [T, d] of dtype.
 *   dres       device, [T, d] of dx_dtype, or NULL (0): the gradient of x by
 *              its other uses (attnres_full_bwd's dV slice, for one).
 *   dx         device, [T, d] of dx_dtype; may be dres (in place).
 *   dgamma     device, fp32 [d], or NULL: added to, or with accumulate 0
 *              written.
 *   dx_dtype, scratch, overlaps and T == 0   as attnres_gated_residual_bwd.
 */
int attnres_rmsnorm_bwd(const void* x, int64_t T, int32_t d, int32_t dtype, const float* gamma,
                        float eps, const void* dy, const void* dres, int32_t dx_dtype, void* dx,
                        float* dgamma, int32_t accumulate, float* scratch, int64_t scratch_floats,
                        void* stream);
int64_t attnres_rmsnorm_bwd_scratch_floats(int64_t T, int32_t d);

/*
 * attnres_grad_norm / attnres_grad_clip - the global norm of a list of
 * gradients, norm = sqrt(sum over all elements of all tensors of g^2), and the
 * list scaled so that its norm is at most max_norm:
 *   out_i = c g_i,  c = max_norm / norm if max_norm < norm < inf, else 1.
 * A norm that is not finite thus changes no gradient and is there to be read.
 *
 *   grads      host array of n device pointers: tensor i holds counts[i]
 *              consecutive elements of dtypes[i] (each F32 or BF16).
 *   counts, dtypes   host arrays; counts[i] >= 0 (0: grads[i] not looked at).
 *   n          >= 0. The host arrays are read before the call returns.
 *   outs, out_dtypes   host arrays like grads and dtypes: where the scaled
 *              tensors go (all elements are written; outs[i] may be grads[i]
 *              with the same type). outs NULL: in place; with c = 1 nothing is
 *              then written. Outputs overlap no gradient but their own and no
 *              other output, so a tensor is listed once.
 *   max_norm   host, >= 0 (may be infinite: the norm alone, or a conversion).
 *   norm       device, fp32 [1]: the norm before clipping.
 *   scratch    device, fp32, at least attnres_grad_norm_scratch_floats(n)
 *              floats; as for attnres_gated_residual_bwd.
 * The squares are summed in fp32, in three scales and in a fixed order, with
 * the rounding of long sums carried along: the norm is right for gradients anywhere in
 * fp32's normal range, also where g^2 would overflow or vanish, and the same
 * call gives the same bits. attnres_grad_norm may list a tensor twice; it then
 * counts twice. Tensors of 16-byte aligned storage stream fastest.
 */
int attnres_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                      int32_t n, float* norm, float* scratch, int64_t scratch_floats, void* stream);
int attnres_grad_clip(const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                      void* const* outs, const int32_t* out_dtypes, int32_t n, float max_norm,
                      float* norm, float* scratch, int64_t scratch_floats, void* stream);
int64_t attnres_grad_norm_scratch_floats(int32_t n);

/*
 * attnres_full_bwd - backward of one read over V[0 .. n_src): given
 * dz = dL/dz of its result, ADD the gradients with respect to the sources,
 * the query and the key-norm gain into dV, dw and dgamma. The read is
 * e_i = r_i (u . v_i), u = w * gamma, r_i = 1 / sqrt(mean_k v_ik^2 + eps),
 * a = softmax_i(e), z = sum_i a_i v_i (DepthBench reading notes section 2.3);
 * by the chain rule, per token:
 *   dL/da_i = dz . v_i,  dL/de_i = a_i (dL/da_i - sum_j a_j dL/da_j),
 *   dL/dv_i = a_i dz + dL/de_i (r_i u - e_i r_i^2 v_i / d),
 *   dL/du = sum over tokens and i of dL/de_i r_i v_i, dw = dL/du * gamma,
 *   dgamma = dL/du * w.
 * Accumulation (+=) lets a model's backward add every later read's share to
 * a source's gradient; zero the buffers before the first call.
 *
 *   V, src_stride, n_src, T, d, v_dtype, w, gamma, eps   as attnres_full_fwd.
 *   dz         device, [T, d] of dz_dtype.
 *   dV         device, fp32, n_src slices [T, d] dv_stride elements apart
 *              (>= T*d when n_src > 1); added to with atomic adds.
 *   dw, dgamma device, fp32 [d], added to; either may be NULL (skipped).
 * None of dV, dw, dgamma may overlap each other or an input. Returns
 * ATTNRES_ERR_UNSUPPORTED for shapes no kernel covers (d > 16384 off the
 * fast path). Results depend on the order of atomic additions only within
 * fp32 rounding.
 */
int attnres_full_bwd(const void* V, int64_t src_stride, int32_t n_src, int64_t T, int32_t d,
                     int32_t v_dtype, const float* w, const float* gamma, float eps,
                     const void* dz, int32_t dz_dtype, float* dV, int64_t dv_stride, float* dw,
                     float* dgamma, void* stream);

/*
 * attnres_block_bwd - gradients of a whole Block pass (the pass of
 * attnres_block_pass) with respect to the embedding, every sublayer output,
 * and every read's query and key gain, given dL/dout_k for every sublayer k.
 * Block AttnRes (DepthBench reading notes section 2.5; LLMRes blog, "Block
 * Attention Residuals"): sublayer k = n * S + j reads {embedding, b_1 .. b_n,
 * P_k if j >= 1}, with b_m the plain sum of block (m-1)'s outputs and P_k the
 * sum of block n's outputs before k. By the chain rule the gradient of b_m
 * reaches every member of block m-1 unchanged and that of P_k every output of
 * block n before k. All dL/dout_k are inputs (the vector-Jacobian product of
 * the pass with F given, as the forward defines it; a model whose sublayers
 * make F from the outputs runs the read backward per sublayer instead). For d
 * a multiple of 128 up to 1024, at most 8 blocks and 8 sublayers per block,
 * each block's S reads run in one batched pass over the tokens; otherwise the
 * reads run in reverse order through the Full read's backward over fp32
 * copies of their sources. Either way the running sums are rebuilt by the
 * same fp32 additions the forward made.
 *
 *   Src       device, [N][T][d] dtype, rows src_stride apart: Src[0] the
 *             embedding, Src[m] the frozen summary b_m (as the forward pass
 *             left them); row N (if any) is not read.
 *   F         device, [N*S][T][d] dtype: the sublayer outputs, f_stride apart.
 *   W, Gamma  device, fp32 [N*S][d]: each read's query and key gain.
 *   dOut      device, [N*S][T][d] dout_dtype: dL/dout_k, dout_stride apart.
 *   dEmb      device, fp32 [T][d], +=.
 *   dF        device, fp32 [N*S][T][d], +=, df_stride apart.
 *   dW, dGamma device, fp32 [N*S][d], +=; may be NULL.
 *   scratch   device, fp32, at least attnres_block_bwd_scratch_floats(N, S,
 *             T, d) floats (the caller's; contents on return unspecified).
 * Returns ATTNRES_ERR_INVALID_ARG for bad sizes, strides, a short scratch or
 * outputs overlapping inputs or each other; launch errors as ATTNRES_ERR_CUDA.
 */
int attnres_block_bwd(const void* Src, int64_t src_stride, const void* F, int64_t f_stride, int32_t N,
                      int32_t S, int64_t T, int32_t d, int32_t dtype, const float* W, const float* Gamma,
                      float eps, const void* dOut, int64_t dout_stride, int32_t dout_dtype, float* dEmb,
                      float* dF, int64_t df_stride, float* dW, float* dGamma, float* scratch,
                      int64_t scratch_floats, void* stream);
/* Scratch attnres_block_bwd needs: (2 (N + 1) + S + 1) * T * d floats; -1 for bad sizes. */
int64_t attnres_block_bwd_scratch_floats(int32_t N, int32_t S, int64_t T, int32_t d);

/*
 * attnres_block_stage1 - stage 1 of the two-stage Block AttnRes computation
 * (datacamp explainer, "two-stage computation"): the S pseudo-queries of one
 * block against the cross-block sources, each source row read once for all S.
 *
 *   Src        device, [n_src, T, d] cross-block sources (embedding, then the
 *              completed block sums), dtype, src_stride >= T*d.
 *   W, Gamma   device, fp32 [S, d], one row per sublayer of the block.
 *   S          1 <= S <= ATTNRES_MAX_QUERIES.
 *   O          host array of S device pointers; O[j] receives the normalised
 *              read of query j over Src, [T, d] of dtype. For the first
 *              sublayer of a block (empty running sum) O[0] is its final
 *              output. O[j] must not overlap Src or each other.
 *   lse        device, fp32 [S, T] (row j at lse + j*T): log sum_i exp(e_ij),
 *              the softmax mass stage 2 merges on. May be NULL (not written).
 */
int attnres_block_stage1(const void* Src, int64_t src_stride, int32_t n_src, int64_t T,
                         int32_t d, int32_t dtype, const float* W, const float* Gamma,
                         int32_t S, float eps, void* const* O, float* lse, void* stream);

/*
 * attnres_stage1_dsplit_partials / attnres_stage1_dsplit_finish - stage 1 with
 * the features split into shards (datacamp explainer, system optimisations,
 * "memory-efficient prefill": block representations sharded across
 * tensor-parallel devices; read as a feature split, where each device keeps a
 * slice of every source row and only score statistics cross devices). A score needs
 * ss = sum_k v_k^2 and dot_j = sum_k w_jk gamma_jk v_k over all d features;
 * both are sums, so each shard forms its part and the parts are added (the one
 * exchange step: an all-reduce of (1 + S) floats per (source, token)). With the
 * totals, each shard finishes the softmax and its own features of the outputs.
 *
 * partials:
 *   Src       device, [n_src, T, d_shard] the shard's features, src_stride >= T*d_shard.
 *   W, Gamma  device, fp32 [S, d_shard], the shard's slice of each query row.
 *   partials  device, fp32 [T][n_src][S + 1]: for token t and source i, entry 0
 *             holds ss, entry 1 + j dot_j. accumulate != 0 adds to it (the
 *             shards of one GPU in turn); 0 overwrites.
 * finish:
 *   Src       as above; d_total the full feature count (mean of squares).
 *   partials  the totals over all shards.
 *   O         host array of S device pointers, [T, d_shard] each: the shard's
 *             features of each query's normalised read.
 *   lse       device, fp32 [S, T] or NULL.
 * Kernels: bf16 shards whose width is a multiple of 64 stream the sources by
 * TMA and take the dots, sum v^2 and (with at most 16 sources) the weighted
 * sums on the tensor cores; other shapes take FMA kernels.
 * Shards wider than 512 features, or unaligned buffers, return
 * ATTNRES_ERR_UNSUPPORTED.
 */
int attnres_stage1_dsplit_partials(const void* Src, int64_t src_stride, int32_t n_src, int64_t T,
                                   int32_t d_shard, int32_t dtype, const float* W,
                                   const float* Gamma, int32_t S, float* partials,
                                   int32_t accumulate, void* stream);
int attnres_stage1_dsplit_finish(const void* Src, int64_t src_stride, int32_t n_src, int64_t T,
                                 int32_t d_shard, int32_t d_total, int32_t dtype,
                                 const float* partials, int32_t S, float eps, void* const* O,
                                 float* lse, void* stream);

/*
 * attnres_block_merge - stage 2 for one sublayer: extend the block's running
 * sum and merge it, as one more softmax source, with the stage-1 result
 * (datacamp explainer, "two-stage computation": online-softmax merge of the
 * intra-block dependency; DepthBench reading notes section 2.5: a read sees
 * the embedding, the frozen blocks and the current running sum).
 *
 *   O_j, lse_j device, stage-1 output [T, d] (dtype) and fp32 [T] of this query.
 *   P          device, fp32 [T, d] running sum, read and written in place.
 *   f_prev     device, [T, d] dtype, or NULL. Non-NULL: P <- P + f_prev first
 *              (P <- f_prev when p_is_empty != 0). NULL: P is used as it is
 *              and is not written; p_is_empty must then be 0.
 *   w, gamma   device, fp32 [d] of this sublayer.
 *   out        device, [T, d] dtype: the sublayer's aggregated input.
 *              out must not overlap O_j, P or f_prev.
 */
int attnres_block_merge(const void* O_j, const float* lse_j, float* P, const void* f_prev,
                        int32_t p_is_empty, const float* w, const float* gamma, float eps,
                        int64_t T, int32_t d, int32_t dtype, void* out, void* stream);

/*
 * attnres_block_merge_prenorm - the same merge, also emitting the sublayer's
 * pre-norm of the merged row (see attnres_full_fwd_prenorm):
 * out_normed = gamma_pre * z / sqrt(mean(z^2) + eps_pre) from z in fp32.
 * out may be NULL (z not stored); out_normed ([T, d] dtype, not NULL) must not
 * overlap out, O_j, lse_j, P or f_prev.
 */
int attnres_block_merge_prenorm(const void* O_j, const float* lse_j, float* P,
                                const void* f_prev, int32_t p_is_empty, const float* w,
                                const float* gamma, float eps, const float* gamma_pre,
                                float eps_pre, int64_t T, int32_t d, int32_t dtype, void* out,
                                void* out_normed, void* stream);

/*
 * attnres_block_summary_accumulate - running sum of a block and the block
 * summary (LLMRes blog "Block Attention Residuals": a block is represented by
 * the sum of its sublayer outputs; datacamp explainer: b_n = sum of the
 * outputs of the layers in block n, with b_0 the embedding).
 *
 *   P            device, fp32 [T, d] running sum.
 *   f            device, [T, d] dtype: a sublayer output to add.
 *   p_is_empty   non-zero: the running sum is empty (treated as 0, P not read).
 *   summary_out  NULL: accumulate, P <- P + f.
 *                non-NULL: freeze, summary_out <- P + f rounded to dtype
 *                ([T, d] dtype, device); P is then not written.
 */
int attnres_block_summary_accumulate(float* P, const void* f, int32_t p_is_empty,
                                     void* summary_out, int64_t T, int32_t d, int32_t dtype,
                                     void* stream);

/*
 * attnres_block_merge_parts - the stage-2 merge with the running sum given in
 * parts: P_j = P_base + f_0 + ... + f_{n_parts-1}, the sum of the block's
 * first j outputs (LLMRes blog "Block Attention Residuals": the running sum
 * of the current block is one more softmax source, DepthBench reading notes
 * section 2.5), formed in fp32 and added in that order. This is the order in
 * which the one-step calls above build it, so keeping a sum in P or forming
 * it again from the outputs gives the same bits. Re-reading a few bf16
 * outputs moves fewer bytes than storing and reloading an fp32 sum; the Block
 * pass chooses by attnres_block_running_sum_plan.
 *
 *   O_j, lse_j  as in attnres_block_merge.
 *   P_base      device, fp32 [T, d]: a stored running sum to start from, or
 *               NULL (the sum starts from the first part; n_parts >= 1).
 *   F_parts     device, the n_parts outputs [T, d] dtype, part_stride >= T*d
 *               elements apart (part_stride unused when n_parts <= 1); n_parts
 *               from 0 (P_base used as it is) to 16.
 *   P_out       device, fp32 [T, d], or NULL: where P_j is stored. It may be
 *               P_base itself (in place) but must not overlap anything else.
 *   w, gamma    device, fp32 [d] of this sublayer.
 *   out         device, [T, d] dtype; overlaps no other argument.
 *   summary_out device, [T, d] dtype, or NULL. When given, F_parts holds one
 *               output more (n_parts + 1 of them, at most 16) and summary_out
 *               receives P_j + f_{n_parts}, added in fp32 after the others
 *               and rounded: the block's summary, frozen by its last merge
 *               (the same bits as attnres_block_summary_parts over all
 *               n_parts + 1 parts). Overlaps no other argument.
 * Errors as attnres_block_merge.
 */
int attnres_block_merge_parts(const void* O_j, const float* lse_j, const float* P_base,
                              const void* F_parts, int64_t part_stride, int32_t n_parts,
                              float* P_out, const float* w, const float* gamma, float eps,
                              int64_t T, int32_t d, int32_t dtype, void* out, void* summary_out,
                              void* stream);

/*
 * attnres_block_summary_parts - a running sum from parts (as in
 * attnres_block_merge_parts, n_parts from 1 to 16): summary_out <- P_base +
 * f_0 + ... rounded to dtype (the freeze of a block summary), or, with
 * summary_out NULL, P_out <- that sum in fp32 (P_out may be P_base).
 */
int attnres_block_summary_parts(const float* P_base, const void* F_parts, int64_t part_stride,
                                int32_t n_parts, float* P_out, void* summary_out, int64_t T,
                                int32_t d, int32_t dtype, void* stream);

/*
 * attnres_block_running_sum_plan - which running sums attnres_block_pass keeps
 * in P_scratch for blocks of S sublayers stored as dtype: stored[j] = 1 for
 * each 1 <= j < S whose P_j is written (stored[0] = stored[S] = 0). Every
 * other P_j is formed from the last kept one, or from nothing, plus the
 * outputs since; the plan minimises the bytes each element moves (an output
 * re-read costs 2 or 4 bytes, a kept fp32 sum 4 to write and 4 to read).
 * Example: bf16, S = 6 keeps P_4 only. stored has S + 1 entries (host).
 */
int attnres_block_running_sum_plan(int32_t S, int32_t dtype, int32_t* stored);

/*
 * attnres_block_pass - the reads of N blocks of S sublayers by the two-stage
 * computation, for stored sublayer outputs F (the synthetic sequencing a
 * model would interleave with its sublayers). Block n (0-based) runs stage 1
 * over Src[0 .. n], S - 1 merges and, unless it is the last block and
 * freeze_last == 0, freezes its summary into Src[n + 1].
 *
 *   F           device, [N*S, T, d] sublayer outputs, dtype, f_stride >= T*d.
 *   W, Gamma    device, fp32 [N*S, d].
 *   Src         device, [N + freeze_last, T, d] dtype, src_stride >= T*d.
 *               Src[0] holds the embedding (input); Src[1 ..] are written.
 *   O_scratch   device, [max(S-1,1), T, d] dtype workspace (stage-1 results).
 *   lse_scratch device, fp32 [S, T] workspace.
 *   P_scratch   device, fp32 [T, d] workspace (the running sums that
 *               attnres_block_running_sum_plan says to keep).
 *   out         device, N*S outputs [T, d] dtype, out_stride >= T*d apart.
 * Merge j of a block takes its running sum as the last kept one plus the
 * outputs since (attnres_block_merge_parts); the freeze likewise
 * (attnres_block_summary_parts).
 */
int attnres_block_pass(const void* F, int64_t f_stride, int32_t N, int32_t S, int64_t T,
                       int32_t d, int32_t dtype, const float* W, const float* Gamma,
                       float eps, void* Src, int64_t src_stride, int32_t freeze_last,
                       void* O_scratch, float* lse_scratch, float* P_scratch,
                       void* out, int64_t out_stride, void* stream);

/*
 * attnres_block_pass_noalloc - attnres_block_pass for callers that cannot
 * allocate device memory. (The pages have no counterpart: this is a library
 * convenience, not part of the method.)
 *
 * Some callers have no device memory to lend as workspace and may not call
 * cudaMalloc: a serving process that reserves and budgets all device memory
 * up front and forbids allocation afterwards, or a caller running on a thread
 * that must never make a call that can implicitly synchronise the device,
 * which cudaMalloc and cudaFree can do. This entry point takes the same
 * inputs and outputs as attnres_block_pass (F, W, Gamma, Src, out) but no
 * workspace: the stage-1 results, their log-masses and the fp32 running sum
 * live in one array of ATTNRES_NOALLOC_SCRATCH_BYTES bytes that the library
 * defines at file scope. It calls no cudaMalloc, cudaFree or other
 * allocating routine.
 *
 *   - Size limit: the workspace of a call needs
 *     (S > 1 ? (S-1)*T*d*es + 4*T*d : 0) + 4*S*T bytes (es = 2 for bf16, 4
 *     for fp32; each part rounded up to 256 bytes). A call that needs more
 *     than ATTNRES_NOALLOC_SCRATCH_BYTES returns ATTNRES_ERR_UNSUPPORTED and
 *     launches nothing. Example: bf16, d = 1024, S = 8 fits up to T = 3634.
 *     The pointer, dtype, eps and stride checks come first, so a call that is
 *     both malformed and too large returns ATTNRES_ERR_INVALID_ARG (except
 *     when T or d alone exceeds the array's size: ATTNRES_ERR_UNSUPPORTED).
 *   - Memory: every CUDA context that loads the library's device code holds
 *     the array (64 MiB) until the context is destroyed or the process
 *     exits. With lazy module loading (the CUDA default) the array is
 *     allocated when this entry point first runs in a context, and that first
 *     call may synchronise the device while the module loads; with
 *     CUDA_MODULE_LOADING=EAGER it is allocated when the context is created,
 *     in every process that loads the library. A caller that budgets device
 *     memory up front, or that must not synchronise later, should therefore
 *     make one small warm-up call (for example T = 1) at start-up, before it
 *     reserves its memory or starts its no-sync thread.
 *   - Set-up: the first call in a CUDA context, with that context current,
 *     looks up the array's device address (cudaGetSymbolAddress) and caches
 *     it under the context's id. Make that first call before any stream
 *     capture begins. After cudaDeviceReset, or when a primary context is
 *     released and created again, the array is a new one: the next call looks
 *     its address up again (and is then such a first call).
 *   - Sharing: all calls in a context share the one array, and it keeps the
 *     contents of the last call. Nothing in it needs to start at zero (every
 *     byte a call reads was written earlier in the same call). Calls whose
 *     work overlaps on the GPU (for example on two streams) race on the
 *     array: order them on one stream or with events.
 *   - Otherwise as attnres_block_pass (same arguments, checks and statuses).
 */
#define ATTNRES_NOALLOC_SCRATCH_BYTES (64ull * 1024ull * 1024ull)
int attnres_block_pass_noalloc(const void* F, int64_t f_stride, int32_t N, int32_t S, int64_t T,
                               int32_t d, int32_t dtype, const float* W, const float* Gamma,
                               float eps, void* Src, int64_t src_stride, int32_t freeze_last,
                               void* out, int64_t out_stride, void* stream);

/*
 * attnres_device_status - synchronise `stream` and report device-side
 * failures of earlier calls on the current device: ATTNRES_ERR_TIMEOUT if a
 * kernel gave up a bounded wait since the last call (the record is then
 * cleared), ATTNRES_ERR_CUDA on a pending CUDA error, else ATTNRES_OK.
 */
int attnres_device_status(void* stream);

/*
 * attnres_selftest_wait_timeout - checks the bounded-wait failure path on the
 * current device: launches one CTA whose mbarrier wait is never satisfied (no
 * thread arrives and no copy is issued), so the wait runs out after its limit
 * (about 2 s), records a timeout and returns. A following
 * attnres_device_status(stream) reports ATTNRES_ERR_TIMEOUT and clears the
 * record; the context stays usable. Returns the launch status.
 */
int attnres_selftest_wait_timeout(void* stream);

/*
 * Failure-path test hooks. The pages define no error handling; these exist so
 * that tests can drive the library's error paths without faulting a GPU. Both
 * are off by default, process-wide (all devices and threads), and meant for
 * tests only.
 *
 * attnres_test_fail_launch - arms a simulated launch failure: after `after`
 * more launches succeed (kernels, and the memsets and copies of the Block
 * backward), the next launch is not made and its call returns
 * ATTNRES_ERR_CUDA, as a real launch error would; the hook then disarms
 * itself. A call that makes several launches (a Full or Block pass) stops at
 * the failed one: the launches before it ran, nothing after it is enqueued.
 * after < 0 disarms. Returns the previous setting (-1 once an armed failure
 * has fired), so a test can tell whether it was consumed.
 */
int64_t attnres_test_fail_launch(int64_t after);

/*
 * attnres_test_withhold_stage - makes the copy producer of one pipelined
 * kernel leave one stage unfilled, so the consumers' bounded wait for it runs
 * out (after about 2 s): the kernel records a timeout and returns, and
 * attnres_device_status reports ATTNRES_ERR_TIMEOUT. kernel: 0 = off, 1 = the
 * Full-read bulk kernel (index counts the (tile, source) copies of each CTA),
 * 2 = the tensor-core stage 1 (index counts each CTA's tiles), 3 = the tiled
 * merge (index counts each CTA's tiles; tiles fetched before the previous
 * kernel finishes, in a Block pass, are never withheld), 4 = the gated residual
 * and its backward (index counts each team's rows), 5 = the streaming read over
 * 8-bit rows (index counts each CTA's stages, of one or more sources), 6 = the
 * 8-bit projection on tensor cores (index counts each CTA's stages, of one or
 * two blocks of 128 features). Every CTA (4: team) with more than `index` copies
 * withholds its copy number `index`; its other copies are issued and waited for
 * before the CTA exits. Stays set until changed.
 * Returns ATTNRES_ERR_INVALID_ARG for an unknown kernel or a negative index.
 */
int attnres_test_withhold_stage(int32_t kernel, int64_t index);

/* Static description of a status code (never NULL). */
const char* attnres_status_string(int32_t status);

/*
 * attnres_kernel_path - which kernel a call with these arguments would use:
 * 1 = the fast kernel, 0 = the general kernel, negative = invalid arguments.
 * op: 0 full read, 1 stage 1, 2 merge, 3 accumulate, 5 gated residual, 6 its
 * backward (5 and 6: every array at src or out and of dtype, all of them given,
 * a gate per token; scratch at out), 7 the RMSNorm backward, 4 query projection
 * (attnres_query_projection with H = Wq = src and Q = out; dtype must be
 * ATTNRES_BF16): 2 = tensor-core tiles shared by pairs of CTAs, 1 = tensor-core
 * tiles of one CTA, 0 = another kernel. Pointers are only inspected for
 * alignment; n_or_s is n_src for op 0 and 1, ignored otherwise; s is S for
 * op 1. Op 4 asks the device how many CTA pairs fit, so it wants one.
 */
int attnres_kernel_path(int32_t op, const void* src, const void* out, int32_t n_or_s,
                        int32_t s, int64_t T, int32_t d, int32_t dtype);

/* ABI version of this header: 1. */
int attnres_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTNRES_H */
