/*
 * ma_layers.h -- C ABI of the operators that a layer's forward and backward
 * passes are made of, beside those of ma_grads.h, whose 8-bit form of an
 * activation (codes and exps) they share.
 *
 *   ma_rms_norm_forward     s = x + residual, y = norm(s) (w + offset), y held in 8 bits
 *   ma_rms_norm_backward    ds and dw (+)= from dy, s and the saved 1 / rms
 *   ma_rotary               feature pairs turned by positions of several axes, and back
 *   ma_token_logprob_forward    log probabilities of given tokens, entropies, top alternatives
 *   ma_token_logprob_backward   the gradient of the logits
 *   ma_attention_forward    softmax(scale q k^T) v over packed sequences with grouped heads
 *   ma_attention_backward   dq, dk and dv
 *
 * Conventions are those of ma_grads.h: return codes and messages, checks
 * before any launch, caller-owned memory, the caller's HIP stream, capturable,
 * a workspace of its own for each of two calls that may run at once, float32
 * arithmetic with one rounding to an array's type (attention in bfloat16 rounds what
 * its matrix instructions take once more, as its functions say), results that do not
 * depend on timing, strides in elements.  Written arrays overlap neither each other
 * nor an input, unless a function allows it.
 */
#ifndef MA_LAYERS_H_
#define MA_LAYERS_H_

#include "ma_grads.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- root-mean-square norm ------------------------------------------------- */

/* Most columns of a norm: a row is kept in one workgroup's registers. */
#define MA_NORM_MAX_COLS 8192

/* For every row: s = x + residual, inv_rms = 1 / sqrt(mean(s^2) + eps) and
 * y = s * inv_rms * (weight + weight_offset).
 *   residual, sum   both or neither NULL; without them s is x.  sum receives s rounded
 *                   to dtype (the norm is that of the unrounded s).
 *   y               may be NULL where codes are given
 *   codes, exps     both or neither NULL: y as rounded to dtype, held in 8 bits: the
 *                   bytes ma_act_pack gives for y
 * x, residual, sum and y are rows x cols of one dtype, weight has cols entries of
 * weight_dtype, inv_rms rows float32 values.  eps is a finite float32, at least
 * 2^-100.  A row whose squares leave float32's range is summed scaled, so only
 * a row that holds an infinity or a NaN gives such values.  rows may be 0.
 * Errors: INVALID_ARG, SHAPE (cols above MA_NORM_MAX_COLS), HIP. */
int ma_rms_norm_forward(const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, int32_t dtype, int64_t rows, int64_t cols,
                        const void* weight, int32_t weight_dtype, double weight_offset, double eps,
                        void* sum, int64_t sum_stride, void* y, int64_t y_stride, int8_t* codes,
                        uint8_t* exps, float* inv_rms, void* stream);

/* Bytes of workspace (256-byte aligned) a ma_rms_norm_backward call with a
 * dweight needs (without one none).  Errors: INVALID_ARG (null), SHAPE. */
int ma_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes);

/* The gradient of y in s and the weight, at the s and inv_rms of the forward pass:
 * with h = s * inv_rms and g = dy * (weight + weight_offset),
 *   ds = inv_rms * (g - h * mean(g * h)) + dsum
 *   dweight = sum over rows of dy * h   (with accumulate = 1, added to dweight)
 * dsum (NULL for none) is the gradient that reaches s past the norm; ds is the
 * gradient of x and of the residual alike.  dweight, contiguous in dweight_dtype,
 * may be NULL.  rows may be 0 (dweight's sum is then zero).  The sums over
 * rows are float32, in an order that follows from rows and cols alone.  Errors:
 * INVALID_ARG, SHAPE, WORKSPACE, HIP. */
int ma_rms_norm_backward(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride,
                         const void* dsum, int64_t dsum_stride, int32_t dtype, int64_t rows,
                         int64_t cols, const float* inv_rms, const void* weight,
                         int32_t weight_dtype, double weight_offset, void* ds, int64_t ds_stride,
                         void* dweight, int32_t dweight_dtype, int32_t accumulate,
                         void* workspace, size_t ws_bytes, void* stream);

/* ---- rotary positions -------------------------------------------------------- */

#define MA_ROTARY_MAX_PAIRS 256
#define MA_ROTARY_MAX_AXES  4

/* Where pair i of `pairs` lies in a head's features */
#define MA_ROTARY_HALF  0   /* features i and pairs + i   */
#define MA_ROTARY_PAIRS 1   /* features 2 i and 2 i + 1   */

/* Which axis a pair belongs to */
#define MA_ROTARY_BLOCKS 0  /* the axes' pairs one axis after the other             */
#define MA_ROTARY_CYCLED 1  /* the axes in turn, without those that are used up     */

/* Fills frequencies (radians per position) and pair_axis, both host arrays of
 * sum(sections) entries, for axes that own sections[0 .. axes) pairs each.  Pair i
 * of all `pairs` turns at theta^(-i / pairs); with restart = 1 the j-th pair of an
 * axis with n turns at theta^(-j / n).  Errors: INVALID_ARG, SHAPE. */
int ma_rotary_frequencies(const int32_t* sections, int32_t axes, double theta, int32_t order,
                          int32_t restart, double* frequencies, uint8_t* pair_axis);

/* For token t, head h and pair i, with the angle a = positions[pair_axis[i]][t] *
 * frequencies[i] and the pair's features (u, v):
 *   (u, v) -> (u cos a - v sin a, u sin a + v cos a)
 * and with inverse = 1 by -a, which is the backward pass.  Features past
 * 2 * pairs are copied.  x and out are n_tokens x heads x head_dim of one dtype, each
 * head's features contiguous, with strides between tokens and between heads; positions
 * is axes x n_tokens signed integers of position_bytes (4 or 8), axis_stride from axis
 * to axis.  out may be x itself with x's strides.  frequencies and pair_axis are
 * host arrays, read before the call returns.  Angles are formed and reduced in 64 bits.
 * n_tokens may be 0.  Errors: INVALID_ARG, SHAPE, HIP. */
int ma_rotary(const void* x, int32_t dtype, int64_t n_tokens, int64_t heads, int64_t head_dim,
              int64_t x_token_stride, int64_t x_head_stride, const void* positions,
              int32_t position_bytes, int32_t axes, int64_t axis_stride,
              const double* frequencies, const uint8_t* pair_axis, int64_t pairs, int32_t layout,
              int32_t inverse, void* out, int64_t out_token_stride, int64_t out_head_stride,
              void* stream);

/* ---- log probabilities of tokens ---------------------------------------------- */

#define MA_LOGPROB_MAX_TOP 64

/* Bytes of workspace (256-byte aligned; 0: none, NULL may be passed) a forward call
 * needs.  Errors: INVALID_ARG (null), SHAPE. */
int ma_token_logprob_workspace_size(int64_t n_tokens, int64_t vocab, int32_t top, size_t* bytes);

/* For every row of logits (n_tokens x vocab), with z = scale * logits[t], scale > 0:
 *   lse[t]      = ln sum exp z
 *   logprob[t]  = z[tokens[t]] - lse[t]   (a token outside [0, vocab) selects none: 0)
 *   entropy[t]  = -sum p ln p, p = exp(z - lse[t])
 *   top_ids[t][j], top_logprobs[t][j], j < top: the ids of the highest logits, falling,
 *                 of equal ones the lowest id first, and their z - lse[t]
 * tokens and top_ids are signed integers of token_bytes (4 or 8); the results are
 * float32 and contiguous.  logprob (with tokens) and entropy may be NULL, and with
 * top = 0 top_ids and top_logprobs.  An entry of -infinity has no probability; a row of
 * nothing else has lse and log probabilities of -infinity and entropy 0.  A row with a
 * NaN or +infinity gives NaN, and its top ids are some distinct ids.  0 <= top <=
 * min(MA_LOGPROB_MAX_TOP, vocab).  n_tokens may be 0.  Errors: INVALID_ARG, SHAPE,
 * WORKSPACE, HIP. */
int ma_token_logprob_forward(const void* logits, int32_t dtype, int64_t n_tokens, int64_t vocab,
                             int64_t stride, const void* tokens, int32_t token_bytes, double scale,
                             float* logprob, float* entropy, float* lse, int32_t top,
                             void* top_ids, float* top_logprobs, void* workspace, size_t ws_bytes,
                             void* stream);

/* With p = exp(z - lse[t]), the gradient of sum_t dlogprob[t] * logprob[t] +
 * dentropy[t] * entropy[t] in the logits:
 *   dlogits[t][v] = scale * (dlogprob[t] * ([v = tokens[t]] - p[v])
 *                            - dentropy[t] * p[v] * (ln p[v] + entropy[t]))
 * p errs by |lse[t]| 2^-24 of itself, by which lse is rounded: a row of nothing but a finite
 * mask value of -1e8, say, has lost its ln vocab there (give it dlogprob and dentropy of 0).
 * A token outside [0, vocab) takes dlogprob as 0.  lse and entropy are the forward pass';
 * dentropy (with entropy) may be NULL.  A row of nothing but -infinity has gradient 0.
 * dlogits may be logits itself, with its type and stride.  n_tokens may be 0.
 * Errors: INVALID_ARG, SHAPE, HIP. */
int ma_token_logprob_backward(const void* logits, int32_t dtype, int64_t n_tokens, int64_t vocab,
                              int64_t stride, const void* tokens, int32_t token_bytes,
                              double scale, const float* lse, const float* entropy,
                              const float* dlogprob, const float* dentropy, void* dlogits,
                              int32_t dlogits_dtype, int64_t dlogits_stride, void* stream);

/* ---- attention ------------------------------------------------------------------- */

#define MA_ATTN_MAX_DIM 256

/* tokens x heads x head_dim, each head's features contiguous: strides in elements
 * between tokens and between heads. */
typedef struct ma_heads {
    void*   p;                 /* (not written where a function only reads it) */
    int64_t token_stride;
    int64_t head_stride;
} ma_heads;

/* Packed sequences: queries [cu_q[s], cu_q[s + 1]) attend to keys [cu_k[s], cu_k[s + 1]),
 * s < n_seqs.  cu_q and cu_k are device arrays of n_seqs + 1 rising int32 values; both NULL for
 * one sequence of everything (n_seqs = 1).  Queries and keys outside every sequence (behind the
 * last one) have no effect, and their results are not written.  Offsets that fall or leave [0, n] are cut to the
 * arrays: no access leaves them, but what is then computed is not defined.
 * Query head h reads key head h / (heads / kv_heads).  With causal = 1 the last query of a
 * sequence sees its last key: query i of nq sees keys 0 .. i + nk - nq. */
typedef struct ma_attention {
    int32_t dtype;             /* of q, k, v, o and their gradients */
    int32_t heads, kv_heads;   /* heads a multiple of kv_heads */
    int32_t head_dim;          /* 1 .. MA_ATTN_MAX_DIM */
    int32_t causal;            /* 0 or 1 */
    int32_t n_seqs;            /* may be 0 */
    int64_t n_queries, n_keys;
    double  scale;             /* of the scores, > 0 */
    const int32_t* cu_q;
    const int32_t* cu_k;
    ma_heads q, k, v;
    ma_heads o;                /* forward: written; backward: read */
    float*   lse;              /* heads x n_queries: ln of the softmax's sums; backward: read */
    ma_heads dout, dq, dk, dv; /* backward only */
} ma_attention;

/* Bytes of workspace (256-byte aligned; 0: none, NULL may be passed) a forward call of these
 * arrays needs (nothing is read): calls of few rows cut their walk over the keys into pieces and
 * join them, and inputs whose heads are not whole 16-byte chunks at 16-byte addresses with
 * token strides from head_dim to 2^22 are copied.  Errors: INVALID_ARG, SHAPE. */
int ma_attention_forward_workspace_size(const ma_attention* a, size_t* bytes);

/* o = softmax(scale q k^T) v and lse.  A query that sees no key has o = 0 and lse =
 * -infinity.  Sums, maxima and lse are float32; a bfloat16 call rounds the probabilities
 * to bfloat16 (at up to 2^8 of the row's largest) for their product with v, as its matrix
 * instructions take them.  A NaN or infinity in a sequence may make that head of that whole
 * sequence NaN, and reaches no other.  Errors: INVALID_ARG, SHAPE (n_queries * heads or
 * n_keys * heads above 2^28, n_seqs * heads above 2^22), WORKSPACE, HIP. */
int ma_attention_forward(const ma_attention* a, void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace (256-byte aligned) a backward call of these arrays needs.  Errors:
 * INVALID_ARG, SHAPE. */
int ma_attention_backward_workspace_size(const ma_attention* a, size_t* bytes);

/* dq, dk and dv from dout and the forward pass' o and lse.  dk and dv sum over the query heads
 * that share them; keys that no query sees get 0.  The probabilities and the scores' gradients
 * of a bfloat16 call are rounded to bfloat16 for their products.  The probabilities are formed
 * from lse and err by |lse| 2^-24 of themselves, by which it is rounded.  No atomics: reruns are
 * bitwise equal.  Errors: as ma_attention_forward. */
int ma_attention_backward(const ma_attention* a, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MA_LAYERS_H_ */
