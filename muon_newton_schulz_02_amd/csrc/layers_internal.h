// Internal declarations of the layer operators (include/ma_layers.h): the
// split rules their host code and kernels share, and the kernel launchers.
// Not part of the C ABI.
#pragma once

#include "../../include/ma_layers.h"
#include "grads_internal.h"

namespace ma {

// Each launcher returns a hipError_t as int.

// ---------------------------------------------------------------- norm --
struct NormArgs {
    const void *x, *res, *dy, *dsum;      // forward: x, res; backward: s (as x), dy, dsum
    void *sum, *y, *ds, *dw;
    const void* weight;
    int8_t* codes;
    uint8_t* exps;
    float* inv;
    float* partials;
    int64_t x_stride, res_stride, dy_stride, dsum_stride, sum_stride, y_stride, ds_stride;
    int64_t rows, cols;
    float offset, eps;
    int32_t dtype, weight_dtype, dw_dtype, accumulate;
};
// Workgroups of a backward pass, each of which leaves one partial sum of dw.
int64_t norm_backward_groups(int64_t rows, int64_t cols);
int launch_rms_norm_forward(const NormArgs& a, void* stream);
int launch_rms_norm_backward(const NormArgs& a, void* stream);

// -------------------------------------------------------------- rotary --
// Frequencies in turns per position, and the axis of each pair; they travel as a
// kernel argument, so a captured launch holds its own copy.
struct RotaryTable {
    double turns[MA_ROTARY_MAX_PAIRS];
    uint8_t axis[MA_ROTARY_MAX_PAIRS];
};
struct RotaryArgs {
    const void *x, *positions;
    void* out;
    int64_t x_token, x_head, out_token, out_head, axis_stride, n_tokens;
    int32_t heads, dim, pairs, layout, inverse, position_bytes, dtype;
};
int launch_rotary(const RotaryArgs& a, const RotaryTable& t, void* stream);

// ------------------------------------------- token log probabilities --
struct LogprobArgs {
    const void *logits, *tokens;
    float *logprob, *entropy, *lse;                // (backward: lse is read)
    const float *ent, *dlogprob, *dentropy;
    void *top_ids, *dlogits;
    float* top_logprobs;
    float* sums;                                   // of a row's pieces: m, s, t, unused
    uint64_t* keys;                                // and their highest
    int64_t rows, vocab, stride, dstride, piece;
    float scale;
    int32_t top, token_bytes, dtype, ddtype;
};
// Pieces a row is cut into.
int64_t logprob_pieces(int64_t rows, int64_t vocab);
int launch_logprob_forward(const LogprobArgs& a, void* stream);
int launch_logprob_backward(const LogprobArgs& a, void* stream);

// ------------------------------------------------------------ attention --
// tokens x heads x dim, with strides between tokens and between heads.
struct AttnArray {
    const void* p;
    int64_t token, head;
};
struct AttnArgs {
    AttnArray q, k, v, o, dout, dq, dk, dv;
    float *lse;
    float *stats;          // forward: m and l of every row of a piece; backward: lse in base 2 and delta of every row
    float *parts;          // float32 results of pieces
    char *packed;          // copies of inputs with aligned rows
    const int32_t *cu_q, *cu_k;
    int64_t n_queries, n_keys;
    float scale;
    int32_t heads, kv_heads, dim, n_seqs, causal, dtype;
    int32_t cols;          // of the inputs' rows: dim in whole chunks
    bool wide;             // whether results are stored 4 at a time
};
// Which of q, k, v and dout are copied first, and where to.
struct AttnPack {
    bool copied[4] = {false, false, false, false};
    int64_t at[4] = {0, 0, 0, 0}, total = 0;
};
AttnPack attention_pack(const AttnArgs& a, bool back);
// How many rows a workgroup takes, and how many pieces its walk over the other side is cut
// into.
struct AttnSplit {
    int32_t rows = 128, pieces = 1;
};
AttnSplit attention_query_split(const AttnArgs& a, bool back);
AttnSplit attention_key_split(const AttnArgs& a);
int launch_attention_forward(const AttnArgs& a, void* stream);
int launch_attention_backward(const AttnArgs& a, void* stream);
// Its two walks, over inputs with aligned rows.
int launch_attention_dq(const AttnArgs& a, const AttnSplit& sp, void* stream);
int launch_attention_dkv(const AttnArgs& a, const AttnSplit& sp, void* stream);

}  // namespace ma
