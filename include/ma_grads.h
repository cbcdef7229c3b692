/*
 * ma_grads.h -- C ABI of the operators that produce the gradients an
 * optimizer step (muon_adamw.h) consumes, and of the 8-bit form in which the
 * activations those gradients need are kept between forward and backward.
 *
 *   ma_embedding_lookup   out[t] = scale * table[tokens[t]]
 *   ma_embedding_grad     dtable[v] (+)= scale * sum of dout[t] over tokens[t] = v
 *   ma_act_pack/_unpack   an activation matrix held in 8 bits, and read back
 *   ma_linear_grad        dW (+)= dY^T X from an X held in 8 bits
 *   ma_glu_forward        h = act(gate) * up, holding gate and up in 8 bits
 *   ma_glu_backward       dgate, dup (and h held in 8 bits) from those
 *
 * The gradients land in float32 or bfloat16 arrays laid out like the
 * parameters (the two parameter storages of a plan), so they can be passed to
 * muon_adamw_step as they are; `accumulate` adds a micro-batch to what an
 * array holds.
 *
 * Conventions are those of muon_adamw.h: 0 (MA_OK) or a negative MA_ERR_*
 * code with a message in muon_adamw_last_error(); arguments are checked
 * before anything is launched; no exception crosses the boundary; the caller
 * owns all device memory, scratch included; work is asynchronous on the
 * caller's HIP stream, with no other stream used, and may be captured into a
 * HIP graph.  The current device must be the one that holds the buffers.  A
 * call writes every part of its workspace that it reads, so the workspace
 * holds nothing between calls; two calls that may run at the same time (two
 * streams, two graphs) need a workspace each.  Results do not depend on timing: every sum
 * is taken in a fixed order, and reruns are bitwise equal.
 *
 * Types: `dtype` arguments are MA_PARAM_FP32 or MA_PARAM_BF16.  Arithmetic
 * is float32 whatever they are, and a result is rounded once, to its
 * array's type (to nearest, ties to even).
 *
 * Matrices are row-major, `*_stride` elements from row to row.  An input's
 * stride may be any value >= 0 (0 repeats one row) and below 2^31; an output's is at least
 * its columns.  Addresses are multiples of the element size.  Outputs and
 * the workspace must overlap neither each other nor an input, except that
 * rows may interleave (gate and up as two halves of one array, both with its
 * stride).
 */
#ifndef MA_GRADS_H_
#define MA_GRADS_H_

#include <stddef.h>
#include <stdint.h>

#include "muon_adamw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- activations held in 8 bits ------------------------------------------ */

/* Features of a token that share one scale. */
#define MA_ACT_GROUP 32

/* An activation matrix of rows x cols (tokens x features) is held as
 *   codes  int8   [rows][code_pitch], code_pitch = cols rounded up to 32
 *   exps   uint8  [rows][exp_pitch],  exp_pitch = code_pitch / 32 rounded up to 4
 * and stands for codes[t][k] * 2^(exps[t][k / 32] - 127).  The exponent of a
 * group of 32 features is the smallest, from -126 to 121, for which every
 * quotient x / 2^e rounds (to nearest even) to at most 127 (at 121 quotients
 * are cut at 127 instead, so a finite value stays finite).  The error of a
 * value is at most half a step, the step being between 1/127 and 1/64 of the
 * group's largest magnitude, and every value is exact in bfloat16.  A group that
 * holds a NaN or an infinity has exponent byte 255 and codes 0, and stands for
 * NaN throughout.  Codes past the last column are 0.  A token's form depends on that
 * token alone.  codes must be 16-byte and exps 4-byte aligned.
 *
 * The two pitches for `cols`.  Errors: INVALID_ARG (null), SHAPE (cols < 1 or
 * above 2^30). */
int ma_act_pitch(int64_t cols, int64_t* code_pitch, int64_t* exp_pitch);

/* x (rows x cols) into codes and exps.  rows may be 0.  Errors: INVALID_ARG,
 * SHAPE, HIP. */
int ma_act_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                int8_t* codes, uint8_t* exps, void* stream);

/* The values codes and exps stand for, into out.  Errors: as ma_act_pack. */
int ma_act_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                  void* out, int32_t dtype, int64_t out_stride, void* stream);

/* ---- embedding table ------------------------------------------------------ */

/* out[t] = scale * table[tokens[t]] for n_tokens tokens of token_bytes (4 or
 * 8) bytes each, signed; table is vocab x hidden.  A token outside [0, vocab)
 * selects no row: its output row is zero.  n_tokens may be 0.  Errors: INVALID_ARG, SHAPE
 * (vocab or hidden < 1, counts above 2^30), HIP. */
int ma_embedding_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t hidden,
                        int64_t table_stride, const void* tokens, int32_t token_bytes,
                        int64_t n_tokens, double scale, void* out, int32_t out_dtype,
                        int64_t out_stride, void* stream);

/* Bytes of workspace (256-byte aligned) one ma_embedding_grad call needs.
 * Errors: INVALID_ARG (null), SHAPE. */
int ma_embedding_grad_workspace_size(int64_t n_tokens, int64_t vocab, int64_t hidden,
                                     size_t* bytes);

/* grad[v] = scale * sum of dout[t] over the tokens t with tokens[t] = v, for
 * every row v of the contiguous vocab x hidden array grad (a row of no token becomes
 * zero); with accumulate = 1 the sum is added to grad[v], and rows of no token
 * are not touched.  Tokens outside [0, vocab), and those equal to
 * padding_token (any value outside the vocabulary for none), add to no row.
 * The sums are float32, over the tokens in rising order within pieces that depend
 * only on the tokens and sizes.  Errors: INVALID_ARG, SHAPE, WORKSPACE, HIP. */
int ma_embedding_grad(const void* dout, int32_t dout_dtype, int64_t dout_stride,
                      const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t vocab,
                      int64_t hidden, double scale, int64_t padding_token, void* grad,
                      int32_t grad_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                      void* stream);

/* ---- linear layer ----------------------------------------------------------- */

/* Bytes of workspace (256-byte aligned; 0: none, NULL may be passed) one
 * ma_linear_grad call needs, whatever dy's address and stride.  A large product
 * takes 2 bytes per element of x in it and, of a float32 dy or one with odd rows, 6 or
 * 2 per element of dy.  Errors: INVALID_ARG, SHAPE. */
int ma_linear_grad_workspace_size(int64_t n_tokens, int64_t n_out, int64_t n_in,
                                  int32_t dy_dtype, size_t* bytes);

/* The same for a dy at this address (its alignment counts; nothing is read) and of this
 * stride: never more, and without the copy of dy where its rows are aligned.  Errors:
 * INVALID_ARG, SHAPE. */
int ma_linear_grad_workspace_size_at(const void* dy, int32_t dy_dtype, int64_t n_tokens,
                                     int64_t n_out, int64_t dy_stride, int64_t n_in,
                                     size_t* bytes);

/* grad[n][k] = sum over t of dy[t][n] * x[t][k] (with accumulate = 1, added
 * to grad): the gradient of y = x W^T in the contiguous n_out x n_in W, from dy
 * (n_tokens x n_out) and x (n_tokens x n_in) held in 8 bits.  No factor is
 * rounded: a bfloat16 dy and x as held enter the matrix cores as they are, a
 * float32 dy as three bfloat16 parts that add up to it (below 2^-110 in magnitude less
 * its bits under 2^-133); sums are float32, in an order that follows from the sizes,
 * dy's type and, for a bfloat16 dy, its alignment and stride (the same values elsewhere
 * may give other last bits).
 * n_tokens may be 0 (the sum is then zero).  Errors: INVALID_ARG, SHAPE,
 * WORKSPACE, HIP. */
int ma_linear_grad(const void* dy, int32_t dy_dtype, int64_t n_tokens, int64_t n_out,
                   int64_t dy_stride, const int8_t* codes, const uint8_t* exps, int64_t n_in,
                   void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace,
                   size_t ws_bytes, void* stream);

/* ---- gated activation ------------------------------------------------------- */

#define MA_ACT_SILU      0   /* g * sigmoid(g)                                        */
#define MA_ACT_GELU_TANH 1   /* g/2 * (1 + tanh(sqrt(2/pi) * (g + 0.044715 g^3)))      */

/* h = act(gate) * up from gate and up as given, and both of them held in 8
 * bits for the backward pass.  All matrices rows x cols of one dtype.  rows may be 0.
 * Errors: INVALID_ARG, SHAPE, UNSUPPORTED (unknown act), HIP. */
int ma_glu_forward(const void* gate, const void* up, int32_t dtype, int64_t rows, int64_t cols,
                   int64_t gate_stride, int64_t up_stride, int32_t act, void* h,
                   int64_t h_stride, int8_t* gate_codes, uint8_t* gate_exps, int8_t* up_codes,
                   uint8_t* up_exps, void* stream);

/* dgate = dh * up * act'(gate) and dup = dh * act(gate) at gate and up as
 * held; h_codes and h_exps (both or neither NULL) receive act(gate) * up at
 * the held values, itself held in 8 bits: the down projection's x for
 * ma_linear_grad.  Errors: as ma_glu_forward. */
int ma_glu_backward(const void* dh, int32_t dtype, int64_t rows, int64_t cols, int64_t dh_stride,
                    const int8_t* gate_codes, const uint8_t* gate_exps, const int8_t* up_codes,
                    const uint8_t* up_exps, int32_t act, void* dgate, int64_t dgate_stride,
                    void* dup, int64_t dup_stride, int8_t* h_codes, uint8_t* h_exps,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MA_GRADS_H_ */
