// The C entry points of the gradient operators: argument checks and the
// calls of their kernels' launchers.  Nothing is launched before every
// argument has been checked.

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <initializer_list>

#include "grads_internal.h"

using namespace ma;

namespace {

int hip_fail(const char* what, int err) {
    set_error("%s: %s", what, hipGetErrorString((hipError_t)err));
    return MA_ERR_HIP;
}

size_t type_size(int32_t dtype) { return dtype == MA_PARAM_BF16 ? 2 : 4; }

int check_dtype(const char* fn, const char* what, int32_t dtype) {
    if (dtype == MA_PARAM_FP32 || dtype == MA_PARAM_BF16) return MA_OK;
    set_error("%s: unknown %s dtype %d", fn, what, dtype);
    return MA_ERR_INVALID_ARG;
}

int check_flag(const char* fn, const char* what, int32_t v) {
    if (v == 0 || v == 1) return MA_OK;
    set_error("%s: %s must be 0 or 1", fn, what);
    return MA_ERR_INVALID_ARG;
}

int check_size(const char* fn, const char* what, int64_t v, int64_t least, int64_t most) {
    if (v >= least && v <= most) return MA_OK;
    set_error("%s: %s %lld outside [%lld, %lld]", fn, what, (long long)v, (long long)least,
              (long long)most);
    return MA_ERR_SHAPE;
}

// A row stride of at least `least` elements and below 2^31; `rows` of them stay below 2^40.
int check_stride(const char* fn, const char* what, int64_t stride, int64_t least, int64_t rows) {
    if (stride >= least && stride < (int64_t(1) << 31) &&
        stride <= (int64_t(1) << 40) / (rows > 1 ? rows : 1))
        return MA_OK;
    set_error("%s: %s stride %lld for %lld rows (at least %lld, below 2^31, 2^40 elements in all)", fn,
              what, (long long)stride, (long long)rows, (long long)least);
    return MA_ERR_INVALID_ARG;
}

// One array of a call: `rows` rows of `row_bytes`, `stride` bytes apart.
struct Span {
    const char* name;
    const void* p;
    int64_t rows, row_bytes, stride;
    size_t align;
    bool written;
};

Span matrix(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols,
            int64_t stride, bool written) {
    const int64_t e = (int64_t)type_size(dtype);
    return {name, p, rows, cols * e, stride * e, (size_t)e, written};
}

Span flat(const char* name, const void* p, int64_t bytes, size_t align, bool written) {
    return {name, p, bytes > 0 ? 1 : 0, bytes, bytes, align, written};
}

Span codes_of(const char* name, const void* p, int64_t rows, int64_t cols, bool written) {
    return flat(name, p, rows * act_code_pitch(cols), 16, written);
}
Span exps_of(const char* name, const void* p, int64_t rows, int64_t cols, bool written) {
    return flat(name, p, rows * act_exp_pitch(cols), 4, written);
}

bool overlap(const Span& a, const Span& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const uintptr_t ea = pa + (uintptr_t)((a.rows - 1) * a.stride + a.row_bytes);
    const uintptr_t eb = pb + (uintptr_t)((b.rows - 1) * b.stride + b.row_bytes);
    if (ea <= pb || eb <= pa) return false;
    // rows that interleave at one stride
    if (a.stride == b.stride && a.stride > 0) {
        const int64_t s = a.stride;
        const int64_t d = pb >= pa ? (int64_t)((pb - pa) % (uintptr_t)s)
                                   : (s - (int64_t)((pa - pb) % (uintptr_t)s)) % s;
        return !(d >= a.row_bytes && d + b.row_bytes <= s);
    }
    return true;
}

// Null, misaligned and overlapping arrays.  Arrays of no element may be null.
int check_spans(const char* fn, std::initializer_list<Span> spans) {
    for (const Span& s : spans) {
        if (s.rows == 0) continue;
        if (!s.p) {
            set_error("%s: %s is NULL", fn, s.name);
            return MA_ERR_INVALID_ARG;
        }
        if ((uintptr_t)s.p % s.align != 0) {
            set_error("%s: %s must be %zu-byte aligned", fn, s.name, s.align);
            return MA_ERR_INVALID_ARG;
        }
    }
    for (const Span& s : spans) {
        if (!s.written) continue;
        for (const Span& o : spans) {
            if (&o == &s || (o.written && &o < &s)) continue;
            if (overlap(s, o)) {
                set_error("%s: %s overlaps %s", fn, s.name, o.name);
                return MA_ERR_INVALID_ARG;
            }
        }
    }
    return MA_OK;
}

int check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
    if (need == 0) return MA_OK;
    if (!ws || bytes < need) {
        set_error("%s: workspace of %zu bytes, need %zu", fn, ws ? bytes : (size_t)0, need);
        return MA_ERR_WORKSPACE;
    }
    if ((uintptr_t)ws % 256 != 0) {
        set_error("%s: workspace must be 256-byte aligned", fn);
        return MA_ERR_WORKSPACE;
    }
    return MA_OK;
}

int check_tokens(const char* fn, int32_t token_bytes) {
    if (token_bytes == 4 || token_bytes == 8) return MA_OK;
    set_error("%s: token_bytes %d (4 or 8)", fn, token_bytes);
    return MA_ERR_INVALID_ARG;
}

int check_scale(const char* fn, double scale) {
    if (std::isfinite(scale) && std::isfinite((float)scale)) return MA_OK;
    set_error("%s: scale must be a finite float32", fn);
    return MA_ERR_INVALID_ARG;
}

constexpr int64_t kMaxHidden = int64_t(1) << 20;   // most columns of an embedding table
// Most elements of one array: its bytes stay far inside 63 bits.
constexpr int64_t kMaxElems = int64_t(1) << 40;

int check_elems(const char* fn, const char* what, int64_t a, int64_t b) {
    if (a == 0 || b <= kMaxElems / a) return MA_OK;
    set_error("%s: %s has more than 2^40 elements", fn, what);
    return MA_ERR_SHAPE;
}

#define TRY(x)                          \
    do {                                \
        const int rc_ = (x);            \
        if (rc_ != MA_OK) return rc_;   \
    } while (0)

int check_act_shape(const char* fn, int64_t rows, int64_t cols) {
    TRY(check_size(fn, "rows", rows, 0, kMaxCount));
    TRY(check_size(fn, "cols", cols, 1, kMaxCount));
    return check_elems(fn, "the matrix", rows, cols);
}

int check_act_kind(const char* fn, int32_t act) {
    if (act == MA_ACT_SILU || act == MA_ACT_GELU_TANH) return MA_OK;
    set_error("%s: unknown act %d", fn, act);
    return MA_ERR_UNSUPPORTED;
}

int done(const char* fn, int err) {
    if (err) return hip_fail(fn, err);
    clear_error();
    return MA_OK;
}

}  // namespace

extern "C" {

int ma_act_pitch(int64_t cols, int64_t* code_pitch, int64_t* exp_pitch) {
    const char* fn = "ma_act_pitch";
    if (!code_pitch || !exp_pitch) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_size(fn, "cols", cols, 1, kMaxCount));
    *code_pitch = act_code_pitch(cols);
    *exp_pitch = act_exp_pitch(cols);
    clear_error();
    return MA_OK;
}

int ma_act_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                int8_t* codes, uint8_t* exps, void* stream) {
    const char* fn = "ma_act_pack";
    TRY(check_dtype(fn, "x", dtype));
    TRY(check_act_shape(fn, rows, cols));
    TRY(check_stride(fn, "x", x_stride, 0, rows));
    TRY(check_spans(fn, {matrix("x", x, dtype, rows, cols, x_stride, false),
                         codes_of("codes", codes, rows, cols, true),
                         exps_of("exps", exps, rows, cols, true)}));
    return done(fn, launch_act_pack(x, dtype, rows, cols, x_stride, codes, exps, stream));
}

int ma_act_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                  void* out, int32_t dtype, int64_t out_stride, void* stream) {
    const char* fn = "ma_act_unpack";
    TRY(check_dtype(fn, "out", dtype));
    TRY(check_act_shape(fn, rows, cols));
    TRY(check_stride(fn, "out", out_stride, cols, rows));
    TRY(check_spans(fn, {matrix("out", out, dtype, rows, cols, out_stride, true),
                         codes_of("codes", codes, rows, cols, false),
                         exps_of("exps", exps, rows, cols, false)}));
    return done(fn, launch_act_unpack(codes, exps, rows, cols, out, dtype, out_stride, stream));
}

int ma_embedding_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t hidden,
                        int64_t table_stride, const void* tokens, int32_t token_bytes,
                        int64_t n_tokens, double scale, void* out, int32_t out_dtype,
                        int64_t out_stride, void* stream) {
    const char* fn = "ma_embedding_lookup";
    TRY(check_dtype(fn, "table", table_dtype));
    TRY(check_dtype(fn, "out", out_dtype));
    TRY(check_tokens(fn, token_bytes));
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "vocab", vocab, 1, kMaxCount));
    TRY(check_size(fn, "hidden", hidden, 1, kMaxHidden));
    TRY(check_elems(fn, "table", vocab, hidden));
    TRY(check_elems(fn, "out", n_tokens, hidden));
    TRY(check_stride(fn, "table", table_stride, 0, vocab));
    TRY(check_stride(fn, "out", out_stride, hidden, n_tokens));
    TRY(check_scale(fn, scale));
    TRY(check_spans(fn, {matrix("table", table, table_dtype, vocab, hidden, table_stride, false),
                         flat("tokens", tokens, n_tokens * token_bytes, (size_t)token_bytes, false),
                         matrix("out", out, out_dtype, n_tokens, hidden, out_stride, true)}));
    return done(fn, launch_embedding_lookup(table, table_dtype, vocab, hidden, table_stride, tokens,
                                            token_bytes, n_tokens, (float)scale, out, out_dtype,
                                            out_stride, stream));
}

int ma_embedding_grad_workspace_size(int64_t n_tokens, int64_t vocab, int64_t hidden,
                                     size_t* bytes) {
    const char* fn = "ma_embedding_grad_workspace_size";
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "vocab", vocab, 1, kMaxCount));
    TRY(check_size(fn, "hidden", hidden, 1, kMaxHidden));
    *bytes = embedding_plan(n_tokens, vocab, hidden).total;
    clear_error();
    return MA_OK;
}

int ma_embedding_grad(const void* dout, int32_t dout_dtype, int64_t dout_stride,
                      const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t vocab,
                      int64_t hidden, double scale, int64_t padding_token, void* grad,
                      int32_t grad_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                      void* stream) {
    const char* fn = "ma_embedding_grad";
    TRY(check_dtype(fn, "dout", dout_dtype));
    TRY(check_dtype(fn, "grad", grad_dtype));
    TRY(check_tokens(fn, token_bytes));
    TRY(check_flag(fn, "accumulate", accumulate));
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "vocab", vocab, 1, kMaxCount));
    TRY(check_size(fn, "hidden", hidden, 1, kMaxHidden));
    TRY(check_elems(fn, "grad", vocab, hidden));
    TRY(check_elems(fn, "dout", n_tokens, hidden));
    TRY(check_stride(fn, "dout", dout_stride, 0, n_tokens));
    TRY(check_scale(fn, scale));
    const EmbPlan p = embedding_plan(n_tokens, vocab, hidden);
    TRY(check_workspace(fn, workspace, ws_bytes, p.total));
    TRY(check_spans(fn, {matrix("dout", dout, dout_dtype, n_tokens, hidden, dout_stride, false),
                         flat("tokens", tokens, n_tokens * token_bytes, (size_t)token_bytes, false),
                         matrix("grad", grad, grad_dtype, vocab, hidden, hidden, true),
                         flat("workspace", workspace, (int64_t)p.total, 1, true)}));
    EmbGradArgs a{};
    a.dout = dout;
    a.tokens = tokens;
    a.grad = grad;
    a.ws = static_cast<char*>(workspace);
    a.dout_stride = dout_stride;
    a.n_tokens = n_tokens;
    a.vocab = vocab;
    a.hidden = hidden;
    a.padding_token = padding_token;
    a.scale = (float)scale;
    a.dout_dtype = dout_dtype;
    a.grad_dtype = grad_dtype;
    a.token_bytes = token_bytes;
    a.accumulate = accumulate;
    return done(fn, launch_embedding_grad(a, p, stream));
}

static int check_lg_shape(const char* fn, int64_t n_tokens, int64_t n_out, int64_t n_in,
                          int32_t dy_dtype) {
    TRY(check_dtype(fn, "dy", dy_dtype));
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "n_out", n_out, 1, kMaxHidden));
    TRY(check_size(fn, "n_in", n_in, 1, kMaxHidden));
    TRY(check_elems(fn, "dy", n_tokens, n_out));
    TRY(check_elems(fn, "x", n_tokens, n_in));
    // (about 2^22 tiles at most: a launch's threads stay below 2^32)
    if (n_out > (int64_t(1) << 36) / n_in) {
        set_error("%s: grad has more than 2^36 elements", fn);
        return MA_ERR_SHAPE;
    }
    return MA_OK;
}

int ma_linear_grad_workspace_size(int64_t n_tokens, int64_t n_out, int64_t n_in,
                                  int32_t dy_dtype, size_t* bytes) {
    const char* fn = "ma_linear_grad_workspace_size";
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_lg_shape(fn, n_tokens, n_out, n_in, dy_dtype));
    // enough for any dy address and stride
    const size_t a = linear_grad_plan(n_tokens, n_out, n_in, dy_dtype, false).total;
    const size_t b = linear_grad_plan(n_tokens, n_out, n_in, dy_dtype, n_out % 8 == 0).total;
    *bytes = a > b ? a : b;
    clear_error();
    return MA_OK;
}

int ma_linear_grad_workspace_size_at(const void* dy, int32_t dy_dtype, int64_t n_tokens,
                                     int64_t n_out, int64_t dy_stride, int64_t n_in,
                                     size_t* bytes) {
    const char* fn = "ma_linear_grad_workspace_size_at";
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_lg_shape(fn, n_tokens, n_out, n_in, dy_dtype));
    TRY(check_stride(fn, "dy", dy_stride, 0, n_tokens));
    *bytes = linear_grad_plan(n_tokens, n_out, n_in, dy_dtype,
                              linear_grad_big_rows(dy, n_out, dy_stride)).total;
    clear_error();
    return MA_OK;
}

int ma_linear_grad(const void* dy, int32_t dy_dtype, int64_t n_tokens, int64_t n_out,
                   int64_t dy_stride, const int8_t* codes, const uint8_t* exps, int64_t n_in,
                   void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace,
                   size_t ws_bytes, void* stream) {
    const char* fn = "ma_linear_grad";
    TRY(check_dtype(fn, "grad", grad_dtype));
    TRY(check_flag(fn, "accumulate", accumulate));
    TRY(check_lg_shape(fn, n_tokens, n_out, n_in, dy_dtype));
    TRY(check_stride(fn, "dy", dy_stride, 0, n_tokens));
    const LgPlan p = linear_grad_plan(n_tokens, n_out, n_in, dy_dtype,
                                      linear_grad_big_rows(dy, n_out, dy_stride));
    TRY(check_workspace(fn, workspace, ws_bytes, p.total));
    TRY(check_spans(fn, {matrix("dy", dy, dy_dtype, n_tokens, n_out, dy_stride, false),
                         codes_of("codes", codes, n_tokens, n_in, false),
                         exps_of("exps", exps, n_tokens, n_in, false),
                         matrix("grad", grad, grad_dtype, n_out, n_in, n_in, true),
                         flat("workspace", workspace, (int64_t)p.total, 1, true)}));
    LgArgs a{};
    a.dy = dy;
    a.codes = codes;
    a.exps = exps;
    a.grad = grad;
    a.partials = static_cast<float*>(workspace);
    a.n_tokens = n_tokens;
    a.n_out = n_out;
    a.n_in = n_in;
    a.dy_stride = dy_stride;
    a.dy_dtype = dy_dtype;
    a.grad_dtype = grad_dtype;
    a.accumulate = accumulate;
    return done(fn, launch_linear_grad(a, p, stream));
}

int ma_glu_forward(const void* gate, const void* up, int32_t dtype, int64_t rows, int64_t cols,
                   int64_t gate_stride, int64_t up_stride, int32_t act, void* h,
                   int64_t h_stride, int8_t* gate_codes, uint8_t* gate_exps, int8_t* up_codes,
                   uint8_t* up_exps, void* stream) {
    const char* fn = "ma_glu_forward";
    TRY(check_dtype(fn, "matrix", dtype));
    TRY(check_act_kind(fn, act));
    TRY(check_act_shape(fn, rows, cols));
    TRY(check_stride(fn, "gate", gate_stride, 0, rows));
    TRY(check_stride(fn, "up", up_stride, 0, rows));
    TRY(check_stride(fn, "h", h_stride, cols, rows));
    TRY(check_spans(fn, {matrix("gate", gate, dtype, rows, cols, gate_stride, false),
                         matrix("up", up, dtype, rows, cols, up_stride, false),
                         matrix("h", h, dtype, rows, cols, h_stride, true),
                         codes_of("gate_codes", gate_codes, rows, cols, true),
                         exps_of("gate_exps", gate_exps, rows, cols, true),
                         codes_of("up_codes", up_codes, rows, cols, true),
                         exps_of("up_exps", up_exps, rows, cols, true)}));
    GluArgs a{};
    a.gate = gate;
    a.up = up;
    a.h = h;
    a.gate_stride = gate_stride;
    a.up_stride = up_stride;
    a.h_stride = h_stride;
    a.gate_codes = gate_codes;
    a.gate_exps = gate_exps;
    a.up_codes = up_codes;
    a.up_exps = up_exps;
    a.rows = rows;
    a.cols = cols;
    a.act = act;
    a.dtype = dtype;
    return done(fn, launch_glu_forward(a, stream));
}

int ma_glu_backward(const void* dh, int32_t dtype, int64_t rows, int64_t cols, int64_t dh_stride,
                    const int8_t* gate_codes, const uint8_t* gate_exps, const int8_t* up_codes,
                    const uint8_t* up_exps, int32_t act, void* dgate, int64_t dgate_stride,
                    void* dup, int64_t dup_stride, int8_t* h_codes, uint8_t* h_exps,
                    void* stream) {
    const char* fn = "ma_glu_backward";
    TRY(check_dtype(fn, "matrix", dtype));
    TRY(check_act_kind(fn, act));
    TRY(check_act_shape(fn, rows, cols));
    TRY(check_stride(fn, "dh", dh_stride, 0, rows));
    TRY(check_stride(fn, "dgate", dgate_stride, cols, rows));
    TRY(check_stride(fn, "dup", dup_stride, cols, rows));
    if ((h_codes == nullptr) != (h_exps == nullptr)) {
        set_error("%s: h_codes and h_exps go together", fn);
        return MA_ERR_INVALID_ARG;
    }
    const int64_t hr = h_codes ? rows : 0;
    TRY(check_spans(fn, {matrix("dh", dh, dtype, rows, cols, dh_stride, false),
                         codes_of("gate_codes", gate_codes, rows, cols, false),
                         exps_of("gate_exps", gate_exps, rows, cols, false),
                         codes_of("up_codes", up_codes, rows, cols, false),
                         exps_of("up_exps", up_exps, rows, cols, false),
                         matrix("dgate", dgate, dtype, rows, cols, dgate_stride, true),
                         matrix("dup", dup, dtype, rows, cols, dup_stride, true),
                         codes_of("h_codes", h_codes, hr, cols, true),
                         exps_of("h_exps", h_exps, hr, cols, true)}));
    GluArgs a{};
    a.dh = dh;
    a.dgate = dgate;
    a.dup = dup;
    a.dh_stride = dh_stride;
    a.dgate_stride = dgate_stride;
    a.dup_stride = dup_stride;
    a.gate_codes = const_cast<int8_t*>(gate_codes);
    a.gate_exps = const_cast<uint8_t*>(gate_exps);
    a.up_codes = const_cast<int8_t*>(up_codes);
    a.up_exps = const_cast<uint8_t*>(up_exps);
    a.h_codes = h_codes;
    a.h_exps = h_exps;
    a.rows = rows;
    a.cols = cols;
    a.act = act;
    a.dtype = dtype;
    return done(fn, launch_glu_backward(a, stream));
}

}  // extern "C"
