// Internal declarations of the gradient operators (include/ma_grads.h): the
// split rules their host code and kernels share, and the kernel launchers.
// Not part of the C ABI.
#pragma once

#include "../../include/ma_grads.h"
#include "ma_internal.h"

namespace ma {

constexpr int64_t kMaxCount = int64_t(1) << 30;   // most rows, columns, tokens or ids of a call

// Whether a stream of this many elements goes past the caches: it could not stay
// in the 32 MB of L2 or much of the 256 MB behind it until it is read, and leaves them to
// the launch's other data.  Measured: a lookup of 65536 x 2048 bf16 rows (268 MB) 89 us
// through the caches and 78 past them, packing 32768 x 8192 bf16 143 and 128 us,
// the gated activation's backward pass at 16384 x 4096 94 and 84; at 33 MB it is no
// faster.  Only where one instruction covers whole lines: units of 8 floats are two
// interleaved halves, and a zeroing of 1.2 GB in them took 560 us against 250.
inline bool streams_past_caches(int64_t elems, int32_t dtype) {
    return dtype == MA_PARAM_BF16 && elems > (int64_t(32) << 20);
}

// --------------------------------------------------- 8-bit activations --
inline int64_t act_code_pitch(int64_t cols) { return round_up(cols, MA_ACT_GROUP); }
inline int64_t act_exp_pitch(int64_t cols) {
    return round_up(ceil_div(cols, MA_ACT_GROUP), 4);
}

struct GluArgs {
    const void *gate, *up, *dh;           // forward: gate, up; backward: dh
    void *h, *dgate, *dup;                // forward: h; backward: dgate, dup
    int64_t gate_stride, up_stride, dh_stride, h_stride, dgate_stride, dup_stride;
    int8_t *gate_codes, *up_codes, *h_codes;
    uint8_t *gate_exps, *up_exps, *h_exps;
    int64_t rows, cols;
    int32_t act, dtype;
};

// Each launcher returns a hipError_t as int.
int launch_act_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                    int8_t* codes, uint8_t* exps, void* stream);
int launch_act_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                      void* out, int32_t dtype, int64_t stride, void* stream);
int launch_glu_forward(const GluArgs& a, void* stream);
int launch_glu_backward(const GluArgs& a, void* stream);

// ---------------------------------------------------------- embedding --
// How ma_embedding_grad splits its work: a radix sort of (row, position)
// pairs in `passes` passes of `bits` bits (over `blocks` blocks of `per`
// tokens, where one workgroup does not do it), then chunks of `chunk` sorted
// entries.  All zero for so few tokens that no sort is needed.
struct EmbPlan {
    int32_t bits = 0, passes = 0;
    int64_t per = 0, blocks = 0;
    int64_t chunk = 0, n_chunks = 0;
    int64_t pitch = 0;            // columns of a partial sum
    int32_t lane_bits = 0;        // threads (log2) that take a row's columns
    // workspace offsets: a flag byte per row, two pairs of (row, position)
    // arrays, the digit counts of a pass, and of runs that cross chunks which
    // ones do and their partial sums
    size_t flags = 0, keys[2] = {0, 0}, pos[2] = {0, 0}, counts = 0, tails = 0, through = 0,
           partials = 0, total = 0;
};
EmbPlan embedding_plan(int64_t n_tokens, int64_t vocab, int64_t hidden);

struct EmbGradArgs {
    const void* dout;
    const void* tokens;
    void* grad;
    char* ws;
    int64_t dout_stride, n_tokens, vocab, hidden, padding_token;
    float scale;
    int32_t dout_dtype, grad_dtype, token_bytes, accumulate;
};
int launch_embedding_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t hidden,
                            int64_t table_stride, const void* tokens, int32_t token_bytes,
                            int64_t n_tokens, float scale, void* out, int32_t out_dtype,
                            int64_t out_stride, void* stream);
int launch_embedding_grad(const EmbGradArgs& a, const EmbPlan& p, void* stream);

// -------------------------------------------------------- linear grad --
// Output tiles (256 x 256 for a large product, else 128 x 128), the token axis
// cut into `slices` of `per` stages of kLgStage tokens; more than one slice
// leaves float32 partial sums in the workspace for a last launch to add in order.
// A large product also keeps X in the workspace as bf16, at xt_off, and at dy_off a copy of
// dY with aligned rows where it needs one (`align`), or a float32 dY's three bf16 parts
// (`split`), which it takes one after the other: three times the stages.
constexpr int kLgStage = 32;
struct LgPlan {
    bool big = false, align = false, split = false;
    int64_t tiles_n = 0, tiles_k = 0;
    int64_t slices = 1, per = 1;
    size_t xt_off = 0, dy_off = 0, total = 0;
};
// Whether dY's rows can be copied in aligned 16-byte pieces, as a large product does.
bool linear_grad_big_rows(const void* dy, int64_t n_out, int64_t stride);
LgPlan linear_grad_plan(int64_t n_tokens, int64_t n_out, int64_t n_in, int32_t dy_dtype,
                        bool big_rows);

struct LgArgs {
    const void* dy;
    const int8_t* codes;
    const uint8_t* exps;
    void* grad;
    float* partials;
    int64_t n_tokens, n_out, n_in, dy_stride;
    int32_t dy_dtype, grad_dtype, accumulate;
};
int launch_linear_grad(const LgArgs& a, const LgPlan& p, void* stream);

}  // namespace ma
