// The C entry points of the layer operators: argument checks and the calls of
// their kernels' launchers.  Nothing is launched before every argument has
// been checked.

#include <cstring>

#include "arg_checks.h"
#include "layers_internal.h"

using namespace ma;

namespace {

constexpr int64_t kMaxHeads = int64_t(1) << 16;

// tokens x heads x dim with strides between tokens and between heads: none
// negative or of 2^31 elements or more, and the array within 2^40.
int check_heads(const char* fn, const char* what, int64_t tokens, int64_t heads, int64_t dim,
                int64_t token, int64_t head) {
    const int64_t most = int64_t(1) << 31;
    if (token < 0 || token >= most || head < 0 || head >= most ||
        (tokens > 0 && (tokens - 1) * token + (heads - 1) * head + dim > kMaxElems)) {
        set_error("%s: %s strides %lld and %lld (at least 0, below 2^31, 2^40 elements in all)", fn, what,
                  (long long)token, (long long)head);
        return MA_ERR_INVALID_ARG;
    }
    return MA_OK;
}

// Whether no two elements share an address: rows of whole tokens, or of whole heads.
bool token_rows(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head) {
    return (heads == 1 || head >= dim) && (tokens == 1 || token >= (heads - 1) * head + dim);
}
bool head_rows(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head) {
    return (tokens == 1 || token >= dim) && (heads == 1 || head >= (tokens - 1) * token + dim);
}

int check_heads_out(const char* fn, const char* what, int64_t tokens, int64_t heads, int64_t dim,
                    int64_t token, int64_t head) {
    TRY(check_heads(fn, what, tokens, heads, dim, token, head));
    if (tokens <= 0 || token_rows(tokens, heads, dim, token, head) || head_rows(tokens, heads, dim, token, head))
        return MA_OK;
    set_error("%s: %s strides %lld and %lld: its elements overlap", fn, what, (long long)token, (long long)head);
    return MA_ERR_INVALID_ARG;
}

Span heads_of(const char* name, const void* p, int32_t dtype, int64_t tokens, int64_t heads, int64_t dim,
              int64_t token, int64_t head, bool written) {
    const int64_t e = (int64_t)type_size(dtype);
    if (tokens <= 0) return {name, p, 0, 0, 0, (size_t)e, written};
    if (token_rows(tokens, heads, dim, token, head))
        return {name, p, tokens, ((heads - 1) * head + dim) * e, token * e, (size_t)e, written};
    if (head_rows(tokens, heads, dim, token, head))
        return {name, p, heads, ((tokens - 1) * token + dim) * e, head * e, (size_t)e, written};
    const int64_t all = ((tokens - 1) * token + (heads - 1) * head + dim) * e;
    return {name, p, 1, all, all, (size_t)e, written};
}

int check_pair(const char* fn, const char* one, const void* a, const char* two, const void* b) {
    if (!a == !b) return MA_OK;
    set_error("%s: %s and %s must both be given or both be NULL", fn, one, two);
    return MA_ERR_INVALID_ARG;
}

int check_norm_shape(const char* fn, int64_t rows, int64_t cols) {
    TRY(check_size(fn, "rows", rows, 0, kMaxCount));
    TRY(check_size(fn, "cols", cols, 1, MA_NORM_MAX_COLS));
    return MA_OK;
}

int64_t norm_ws_bytes(int64_t rows, int64_t cols) {
    return round_up(norm_backward_groups(rows, cols) * cols * 4, 256);
}

int check_logprob(const char* fn, int32_t dtype, int64_t n_tokens, int64_t vocab, int64_t stride,
                  int32_t token_bytes, double scale) {
    TRY(check_dtype(fn, "logits", dtype));
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "vocab", vocab, 1, kMaxCount));
    TRY(check_elems(fn, "logits", n_tokens, vocab));
    TRY(check_stride(fn, "logits", stride, 0, n_tokens));
    TRY(check_tokens(fn, token_bytes));
    if (!(scale >= 0x1p-100) || !std::isfinite((float)scale)) {
        set_error("%s: scale must be a positive float32, at least 2^-100", fn);
        return MA_ERR_INVALID_ARG;
    }
    return MA_OK;
}

// Elements of a row's piece: whole units of 8.
int64_t logprob_piece(int64_t rows, int64_t vocab) {
    return round_up(ceil_div(vocab, logprob_pieces(rows, vocab)), 8);
}

struct LogprobSpace {
    size_t sums = 0, keys = 0, total = 0;
};
LogprobSpace logprob_space(int64_t rows, int64_t vocab, int64_t top) {
    LogprobSpace s;
    const int64_t pieces = ceil_div(vocab, logprob_piece(rows, vocab));
    if (pieces == 1 || rows == 0) return s;
    s.keys = (size_t)round_up(rows * pieces * 16, 256);
    s.total = s.keys + (size_t)round_up(rows * pieces * top * 8, 256);
    return s;
}

int check_attention(const char* fn, const ma_attention* a, bool back) {
    if (!a) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_dtype(fn, "q", a->dtype));
    TRY(check_size(fn, "kv_heads", a->kv_heads, 1, kMaxHeads));
    TRY(check_size(fn, "heads", a->heads, 1, kMaxHeads));
    TRY(check_size(fn, "head_dim", a->head_dim, 1, MA_ATTN_MAX_DIM));
    TRY(check_flag(fn, "causal", a->causal));
    if (a->heads % a->kv_heads) {
        set_error("%s: %d heads are no multiple of %d key heads", fn, a->heads, a->kv_heads);
        return MA_ERR_SHAPE;
    }
    // (a launch has fewer than 2^32 threads)
    TRY(check_size(fn, "n_seqs", a->n_seqs, 0, (int64_t(1) << 22) / a->heads));
    TRY(check_size(fn, "n_queries", a->n_queries, 0, kMaxCount / 4 / a->heads));
    TRY(check_size(fn, "n_keys", a->n_keys, 0, kMaxCount / 4 / a->heads));
    if (!(a->scale >= 0x1p-100) || !std::isfinite((float)a->scale)) {
        set_error("%s: scale must be a positive float32, at least 2^-100", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_pair(fn, "cu_q", a->cu_q, "cu_k", a->cu_k));
    if (!a->cu_q && a->n_seqs != 1) {
        set_error("%s: %d sequences without offsets", fn, a->n_seqs);
        return MA_ERR_INVALID_ARG;
    }
    struct {
        const char* name;
        const ma_heads* x;
        int64_t n;
        int32_t heads;
        bool out;
    } all[] = {{"q", &a->q, a->n_queries, a->heads, false},  {"k", &a->k, a->n_keys, a->kv_heads, false},
               {"v", &a->v, a->n_keys, a->kv_heads, false},  {"o", &a->o, a->n_queries, a->heads, !back},
               {"dout", &a->dout, a->n_queries, a->heads, false}, {"dq", &a->dq, a->n_queries, a->heads, true},
               {"dk", &a->dk, a->n_keys, a->kv_heads, true}, {"dv", &a->dv, a->n_keys, a->kv_heads, true}};
    for (int i = 0; i < (back ? 8 : 4); ++i) {
        const auto& e = all[i];
        TRY((e.out ? check_heads_out : check_heads)(fn, e.name, e.n, e.heads, a->head_dim, e.x->token_stride,
                                                    e.x->head_stride));
    }
    return MA_OK;
}

Span attention_span(const ma_attention* a, const char* name, const ma_heads& x, bool keys, bool written) {
    return heads_of(name, x.p, a->dtype, keys ? a->n_keys : a->n_queries, keys ? a->kv_heads : a->heads, a->head_dim,
                    x.token_stride, x.head_stride, written);
}

AttnArgs attention_args(const ma_attention* a) {
    const auto arr = [](const ma_heads& x) { return AttnArray{x.p, x.token_stride, x.head_stride}; };
    AttnArgs g{};
    g.q = arr(a->q);
    g.k = arr(a->k);
    g.v = arr(a->v);
    g.o = arr(a->o);
    g.lse = a->lse;
    g.cu_q = a->cu_q;
    g.cu_k = a->cu_k;
    g.n_queries = a->n_queries;
    g.n_keys = a->n_keys;
    g.scale = (float)a->scale;
    g.heads = a->heads;
    g.kv_heads = a->kv_heads;
    g.dim = a->head_dim;
    g.n_seqs = a->n_seqs;
    g.causal = a->causal;
    g.dtype = a->dtype;
    return g;
}

// Workspace: the rows' numbers, then the pieces' results, then copies of inputs.
struct AttnSpace {
    int64_t parts = 0, packed = 0, total = 0;
};
AttnSpace attention_space(const AttnArgs& g, bool back) {
    AttnSpace s;
    const int64_t rows = g.heads * g.n_queries, keys = (int64_t)g.kv_heads * g.n_keys;
    const int64_t pq = attention_query_split(g, back).pieces, pk = attention_key_split(g).pieces;
    int64_t floats = pq > 1 ? pq * rows * g.dim : 0;
    if (back && pk > 1 && 2 * pk * keys * g.dim > floats) floats = 2 * pk * keys * g.dim;
    s.parts = round_up(back ? rows * 8 : pq > 1 ? pq * rows * 8 : 0, 256);
    s.packed = s.parts + round_up(floats * 4, 256);
    s.total = s.packed + attention_pack(g, back).total;
    return s;
}

int attention_size(const char* fn, const ma_attention* a, bool back, size_t* bytes) {
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_attention(fn, a, back));
    AttnArgs g = attention_args(a);
    g.dout = {a->dout.p, a->dout.token_stride, a->dout.head_stride};
    *bytes = (size_t)attention_space(g, back).total;
    clear_error();
    return MA_OK;
}

int check_top(const char* fn, int32_t top, int64_t vocab) {
    return check_size(fn, "top", top, 0, vocab < MA_LOGPROB_MAX_TOP ? vocab : MA_LOGPROB_MAX_TOP);
}

}  // namespace

extern "C" {

int ma_rms_norm_forward(const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, int32_t dtype, int64_t rows, int64_t cols,
                        const void* weight, int32_t weight_dtype, double weight_offset, double eps,
                        void* sum, int64_t sum_stride, void* y, int64_t y_stride, int8_t* codes,
                        uint8_t* exps, float* inv_rms, void* stream) {
    const char* fn = "ma_rms_norm_forward";
    TRY(check_dtype(fn, "x", dtype));
    TRY(check_dtype(fn, "weight", weight_dtype));
    TRY(check_norm_shape(fn, rows, cols));
    TRY(check_stride(fn, "x", x_stride, 0, rows));
    TRY(check_scale(fn, weight_offset));
    if (!(eps >= 0x1p-100) || !std::isfinite((float)eps)) {
        set_error("%s: eps must be a finite float32, at least 2^-100", fn);
        return MA_ERR_INVALID_ARG;
    }
    if (rows > 0) {
        TRY(check_pair(fn, "residual", residual, "sum", sum));
        TRY(check_pair(fn, "codes", codes, "exps", exps));
        if (!y && !codes) {
            set_error("%s: y and codes are both NULL", fn);
            return MA_ERR_INVALID_ARG;
        }
    }
    if (residual) {
        TRY(check_stride(fn, "residual", residual_stride, 0, rows));
        TRY(check_stride(fn, "sum", sum_stride, cols, rows));
    }
    if (y) TRY(check_stride(fn, "y", y_stride, cols, rows));
    const int64_t r = residual ? rows : 0;
    TRY(check_spans(fn, {matrix("x", x, dtype, rows, cols, x_stride, false),
                         matrix("residual", residual, dtype, r, cols, residual_stride, false),
                         flat("weight", weight, rows ? cols * (int64_t)type_size(weight_dtype) : 0,
                              type_size(weight_dtype), false),
                         matrix("sum", sum, dtype, r, cols, sum_stride, true),
                         matrix("y", y, dtype, y ? rows : 0, cols, y_stride, true),
                         codes_of("codes", codes, codes ? rows : 0, cols, true),
                         exps_of("exps", exps, codes ? rows : 0, cols, true),
                         flat("inv_rms", inv_rms, rows * 4, 4, true)}));
    NormArgs a{};
    a.x = x;
    a.res = residual;
    a.sum = sum;
    a.y = y;
    a.weight = weight;
    a.codes = codes;
    a.exps = exps;
    a.inv = inv_rms;
    a.x_stride = x_stride;
    a.res_stride = residual_stride;
    a.sum_stride = sum_stride;
    a.y_stride = y_stride;
    a.rows = rows;
    a.cols = cols;
    a.offset = (float)weight_offset;
    a.eps = (float)eps;
    a.dtype = dtype;
    a.weight_dtype = weight_dtype;
    return done(fn, launch_rms_norm_forward(a, stream));
}

int ma_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
    const char* fn = "ma_rms_norm_backward_workspace_size";
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_norm_shape(fn, rows, cols));
    *bytes = (size_t)norm_ws_bytes(rows, cols);
    clear_error();
    return MA_OK;
}

int ma_rms_norm_backward(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride,
                         const void* dsum, int64_t dsum_stride, int32_t dtype, int64_t rows,
                         int64_t cols, const float* inv_rms, const void* weight,
                         int32_t weight_dtype, double weight_offset, void* ds, int64_t ds_stride,
                         void* dweight, int32_t dweight_dtype, int32_t accumulate,
                         void* workspace, size_t ws_bytes, void* stream) {
    const char* fn = "ma_rms_norm_backward";
    TRY(check_dtype(fn, "dy", dtype));
    TRY(check_dtype(fn, "weight", weight_dtype));
    TRY(check_norm_shape(fn, rows, cols));
    TRY(check_stride(fn, "dy", dy_stride, 0, rows));
    TRY(check_stride(fn, "s", s_stride, 0, rows));
    if (dsum) TRY(check_stride(fn, "dsum", dsum_stride, 0, rows));
    TRY(check_stride(fn, "ds", ds_stride, cols, rows));
    TRY(check_scale(fn, weight_offset));
    TRY(check_flag(fn, "accumulate", accumulate));
    const int64_t need = dweight ? norm_ws_bytes(rows, cols) : 0;
    if (dweight) {
        TRY(check_dtype(fn, "dweight", dweight_dtype));
        TRY(check_workspace(fn, workspace, ws_bytes, (size_t)need));
    }
    const int64_t we = (int64_t)type_size(dweight_dtype);
    TRY(check_spans(fn, {matrix("dy", dy, dtype, rows, cols, dy_stride, false),
                         matrix("s", s, dtype, rows, cols, s_stride, false),
                         matrix("dsum", dsum, dtype, dsum ? rows : 0, cols, dsum_stride, false),
                         flat("inv_rms", inv_rms, rows * 4, 4, false),
                         flat("weight", weight, rows ? cols * (int64_t)type_size(weight_dtype) : 0,
                              type_size(weight_dtype), false),
                         matrix("ds", ds, dtype, rows, cols, ds_stride, true),
                         flat("dweight", dweight, dweight ? cols * we : 0, (size_t)we, true),
                         flat("workspace", workspace, need, 1, true)}));
    NormArgs a{};
    a.x = s;
    a.dy = dy;
    a.dsum = dsum;
    a.ds = ds;
    a.dw = dweight;
    a.weight = weight;
    a.inv = const_cast<float*>(inv_rms);
    a.partials = dweight ? static_cast<float*>(workspace) : nullptr;
    a.x_stride = s_stride;
    a.dy_stride = dy_stride;
    a.dsum_stride = dsum_stride;
    a.ds_stride = ds_stride;
    a.rows = rows;
    a.cols = cols;
    a.offset = (float)weight_offset;
    a.dtype = dtype;
    a.weight_dtype = weight_dtype;
    a.dw_dtype = dweight_dtype;
    a.accumulate = accumulate;
    return done(fn, launch_rms_norm_backward(a, stream));
}

int ma_rotary_frequencies(const int32_t* sections, int32_t axes, double theta, int32_t order,
                          int32_t restart, double* frequencies, uint8_t* pair_axis) {
    const char* fn = "ma_rotary_frequencies";
    if (!sections || !frequencies || !pair_axis) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_size(fn, "axes", axes, 1, MA_ROTARY_MAX_AXES));
    TRY(check_flag(fn, "restart", restart));
    if (order != MA_ROTARY_BLOCKS && order != MA_ROTARY_CYCLED) {
        set_error("%s: unknown order %d", fn, order);
        return MA_ERR_INVALID_ARG;
    }
    if (!(theta > 0) || !std::isfinite(theta)) {
        set_error("%s: theta must be positive and finite", fn);
        return MA_ERR_INVALID_ARG;
    }
    int64_t pairs = 0;
    for (int a = 0; a < axes; ++a) {
        TRY(check_size(fn, "a section", sections[a], 0, MA_ROTARY_MAX_PAIRS));
        pairs += sections[a];
    }
    TRY(check_size(fn, "pairs", pairs, 1, MA_ROTARY_MAX_PAIRS));
    int used[MA_ROTARY_MAX_AXES] = {0}, axis = 0;
    for (int i = 0; i < (int)pairs; ++i) {
        while (used[axis] == sections[axis]) axis = (axis + 1) % axes;
        const int j = used[axis]++;
        pair_axis[i] = (uint8_t)axis;
        frequencies[i] = std::pow(theta, restart ? -(double)j / sections[axis] : -(double)i / (double)pairs);
        if (order == MA_ROTARY_CYCLED) axis = (axis + 1) % axes;
    }
    clear_error();
    return MA_OK;
}

int ma_rotary(const void* x, int32_t dtype, int64_t n_tokens, int64_t heads, int64_t head_dim,
              int64_t x_token_stride, int64_t x_head_stride, const void* positions,
              int32_t position_bytes, int32_t axes, int64_t axis_stride,
              const double* frequencies, const uint8_t* pair_axis, int64_t pairs, int32_t layout,
              int32_t inverse, void* out, int64_t out_token_stride, int64_t out_head_stride,
              void* stream) {
    const char* fn = "ma_rotary";
    TRY(check_dtype(fn, "x", dtype));
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "heads", heads, 1, kMaxHeads));
    TRY(check_size(fn, "head_dim", head_dim, 1, 2 * MA_ROTARY_MAX_PAIRS));
    TRY(check_size(fn, "pairs", pairs, 1, head_dim / 2));
    TRY(check_size(fn, "axes", axes, 1, MA_ROTARY_MAX_AXES));
    TRY(check_flag(fn, "inverse", inverse));
    if (position_bytes != 4 && position_bytes != 8) {
        set_error("%s: position_bytes %d (4 or 8)", fn, position_bytes);
        return MA_ERR_INVALID_ARG;
    }
    if (layout != MA_ROTARY_HALF && layout != MA_ROTARY_PAIRS) {
        set_error("%s: unknown layout %d", fn, layout);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_heads(fn, "x", n_tokens, heads, head_dim, x_token_stride, x_head_stride));
    TRY(check_heads_out(fn, "out", n_tokens, heads, head_dim, out_token_stride, out_head_stride));
    if (axis_stride < 0 || axis_stride > (int64_t(1) << 31)) {
        set_error("%s: axis stride %lld (at least 0, at most 2^31)", fn, (long long)axis_stride);
        return MA_ERR_INVALID_ARG;
    }
    if (!frequencies || !pair_axis) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    RotaryTable tab;
    std::memset(&tab, 0, sizeof(tab));
    for (int i = 0; i < (int)pairs; ++i) {
        if (pair_axis[i] >= axes || !std::isfinite(frequencies[i])) {
            set_error("%s: pair %d has axis %d of %d and frequency %g", fn, i, pair_axis[i], axes, frequencies[i]);
            return MA_ERR_INVALID_ARG;
        }
        tab.axis[i] = pair_axis[i];
        tab.turns[i] = (double)(frequencies[i] / 6.283185307179586476925286766559005768L);
    }
    const int64_t reach = n_tokens > 0 ? (axes - 1) * axis_stride + n_tokens : 0;
    const bool same = out == x && out_token_stride == x_token_stride && out_head_stride == x_head_stride;
    TRY(check_spans(fn, {heads_of("x", x, dtype, same ? 0 : n_tokens, heads, head_dim, x_token_stride, x_head_stride,
                                  false),
                         flat("positions", positions, reach * position_bytes, (size_t)position_bytes, false),
                         heads_of("out", out, dtype, n_tokens, heads, head_dim, out_token_stride, out_head_stride,
                                  true)}));
    RotaryArgs a{};
    a.x = x;
    a.positions = positions;
    a.out = out;
    a.x_token = x_token_stride;
    a.x_head = x_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.axis_stride = axis_stride;
    a.n_tokens = n_tokens;
    a.heads = (int32_t)heads;
    a.dim = (int32_t)head_dim;
    a.pairs = (int32_t)pairs;
    a.layout = layout;
    a.inverse = inverse;
    a.position_bytes = position_bytes;
    a.dtype = dtype;
    return done(fn, launch_rotary(a, tab, stream));
}

int ma_token_logprob_workspace_size(int64_t n_tokens, int64_t vocab, int32_t top, size_t* bytes) {
    const char* fn = "ma_token_logprob_workspace_size";
    if (!bytes) {
        set_error("%s: NULL argument", fn);
        return MA_ERR_INVALID_ARG;
    }
    TRY(check_size(fn, "n_tokens", n_tokens, 0, kMaxCount));
    TRY(check_size(fn, "vocab", vocab, 1, kMaxCount));
    TRY(check_top(fn, top, vocab));
    *bytes = logprob_space(n_tokens, vocab, top).total;
    clear_error();
    return MA_OK;
}

int ma_token_logprob_forward(const void* logits, int32_t dtype, int64_t n_tokens, int64_t vocab,
                             int64_t stride, const void* tokens, int32_t token_bytes, double scale,
                             float* logprob, float* entropy, float* lse, int32_t top,
                             void* top_ids, float* top_logprobs, void* workspace, size_t ws_bytes,
                             void* stream) {
    const char* fn = "ma_token_logprob_forward";
    TRY(check_logprob(fn, dtype, n_tokens, vocab, stride, token_bytes, scale));
    TRY(check_top(fn, top, vocab));
    if (n_tokens > 0) TRY(check_pair(fn, "tokens", tokens, "logprob", logprob));
    const LogprobSpace sp = logprob_space(n_tokens, vocab, top);
    TRY(check_workspace(fn, workspace, ws_bytes, sp.total));
    const int64_t n4 = n_tokens * 4;
    TRY(check_spans(fn, {matrix("logits", logits, dtype, n_tokens, vocab, stride, false),
                         flat("tokens", tokens, tokens ? n_tokens * token_bytes : 0, (size_t)token_bytes, false),
                         flat("logprob", logprob, logprob ? n4 : 0, 4, true),
                         flat("entropy", entropy, entropy ? n4 : 0, 4, true), flat("lse", lse, n4, 4, true),
                         flat("top_ids", top_ids, n_tokens * top * token_bytes, (size_t)token_bytes, true),
                         flat("top_logprobs", top_logprobs, n4 * top, 4, true),
                         flat("workspace", workspace, (int64_t)sp.total, 1, true)}));
    LogprobArgs a{};
    a.logits = logits;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.lse = lse;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.sums = static_cast<float*>(workspace);
    a.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + sp.keys);
    a.rows = n_tokens;
    a.vocab = vocab;
    a.stride = stride;
    a.piece = logprob_piece(n_tokens, vocab);
    a.scale = (float)scale;
    a.top = top;
    a.token_bytes = token_bytes;
    a.dtype = dtype;
    return done(fn, launch_logprob_forward(a, stream));
}

int ma_token_logprob_backward(const void* logits, int32_t dtype, int64_t n_tokens, int64_t vocab,
                              int64_t stride, const void* tokens, int32_t token_bytes,
                              double scale, const float* lse, const float* entropy,
                              const float* dlogprob, const float* dentropy, void* dlogits,
                              int32_t dlogits_dtype, int64_t dlogits_stride, void* stream) {
    const char* fn = "ma_token_logprob_backward";
    TRY(check_logprob(fn, dtype, n_tokens, vocab, stride, token_bytes, scale));
    TRY(check_dtype(fn, "dlogits", dlogits_dtype));
    TRY(check_stride(fn, "dlogits", dlogits_stride, vocab, n_tokens));
    if (n_tokens > 0) TRY(check_pair(fn, "entropy", entropy, "dentropy", dentropy));
    const bool same = logits == dlogits && dtype == dlogits_dtype && stride == dlogits_stride;
    const int64_t n4 = n_tokens * 4;
    TRY(check_spans(fn, {matrix("logits", logits, dtype, same ? 0 : n_tokens, vocab, stride, false),
                         flat("tokens", tokens, n_tokens * token_bytes, (size_t)token_bytes, false),
                         flat("lse", lse, n4, 4, false), flat("entropy", entropy, entropy ? n4 : 0, 4, false),
                         flat("dlogprob", dlogprob, n4, 4, false),
                         flat("dentropy", dentropy, dentropy ? n4 : 0, 4, false),
                         matrix("dlogits", dlogits, dlogits_dtype, n_tokens, vocab, dlogits_stride, true)}));
    LogprobArgs a{};
    a.logits = logits;
    a.tokens = tokens;
    a.lse = const_cast<float*>(lse);
    a.ent = entropy;
    a.dlogprob = dlogprob;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    a.rows = n_tokens;
    a.vocab = vocab;
    a.stride = stride;
    a.dstride = dlogits_stride;
    a.piece = logprob_piece(n_tokens, vocab);
    a.scale = (float)scale;
    a.token_bytes = token_bytes;
    a.dtype = dtype;
    a.ddtype = dlogits_dtype;
    return done(fn, launch_logprob_backward(a, stream));
}

int ma_attention_forward_workspace_size(const ma_attention* a, size_t* bytes) {
    return attention_size("ma_attention_forward_workspace_size", a, false, bytes);
}

int ma_attention_forward(const ma_attention* a, void* workspace, size_t ws_bytes, void* stream) {
    const char* fn = "ma_attention_forward";
    TRY(check_attention(fn, a, false));
    AttnArgs g = attention_args(a);
    const AttnSpace sp = attention_space(g, false);
    TRY(check_workspace(fn, workspace, ws_bytes, (size_t)sp.total));
    const int64_t cu = a->cu_q ? ((int64_t)a->n_seqs + 1) * 4 : 0;
    TRY(check_spans(fn, {attention_span(a, "q", a->q, false, false), attention_span(a, "k", a->k, true, false),
                         attention_span(a, "v", a->v, true, false), flat("cu_q", a->cu_q, cu, 4, false),
                         flat("cu_k", a->cu_k, cu, 4, false), attention_span(a, "o", a->o, false, true),
                         flat("lse", a->lse, a->heads * a->n_queries * 4, 4, true),
                         flat("workspace", workspace, sp.total, 1, true)}));
    g.stats = static_cast<float*>(workspace);
    g.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + sp.parts);
    g.packed = static_cast<char*>(workspace) + sp.packed;
    return done(fn, launch_attention_forward(g, stream));
}

int ma_attention_backward_workspace_size(const ma_attention* a, size_t* bytes) {
    return attention_size("ma_attention_backward_workspace_size", a, true, bytes);
}

int ma_attention_backward(const ma_attention* a, void* workspace, size_t ws_bytes, void* stream) {
    const char* fn = "ma_attention_backward";
    TRY(check_attention(fn, a, true));
    AttnArgs g = attention_args(a);
    g.dout = {a->dout.p, a->dout.token_stride, a->dout.head_stride};
    g.dq = {a->dq.p, a->dq.token_stride, a->dq.head_stride};
    g.dk = {a->dk.p, a->dk.token_stride, a->dk.head_stride};
    g.dv = {a->dv.p, a->dv.token_stride, a->dv.head_stride};
    const AttnSpace sp = attention_space(g, true);
    TRY(check_workspace(fn, workspace, ws_bytes, (size_t)sp.total));
    const int64_t cu = a->cu_q ? ((int64_t)a->n_seqs + 1) * 4 : 0;
    TRY(check_spans(fn, {attention_span(a, "q", a->q, false, false), attention_span(a, "k", a->k, true, false),
                         attention_span(a, "v", a->v, true, false), attention_span(a, "o", a->o, false, false),
                         attention_span(a, "dout", a->dout, false, false), flat("cu_q", a->cu_q, cu, 4, false),
                         flat("cu_k", a->cu_k, cu, 4, false),
                         flat("lse", a->lse, a->heads * a->n_queries * 4, 4, false),
                         attention_span(a, "dq", a->dq, false, true), attention_span(a, "dk", a->dk, true, true),
                         attention_span(a, "dv", a->dv, true, true), flat("workspace", workspace, sp.total, 1, true)}));
    g.stats = static_cast<float*>(workspace);
    g.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + sp.parts);
    g.packed = static_cast<char*>(workspace) + sp.packed;
    return done(fn, launch_attention_backward(g, stream));
}

}  // extern "C"
