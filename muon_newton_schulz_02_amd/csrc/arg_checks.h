// Argument checks shared by the C entry points of ma_grads.h and ma_layers.h.
// A failed check leaves its message for muon_adamw_last_error() and gives the
// call's return code.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <initializer_list>

#include "grads_internal.h"

namespace ma {
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

int done(const char* fn, int err) {
    if (err) return hip_fail(fn, err);
    clear_error();
    return MA_OK;
}

}  // namespace
}  // namespace ma
