// Activations held in 8 bits, and the gated activation that holds its
// inputs so, on gfx950.
//
// All four kernels stream: a thread takes 8 features of a token, four
// neighbouring lanes form one group of 32, whose largest magnitude they find
// with two lane exchanges.  A packing thread covers the padding up to the
// exponents' pitch (a multiple of 128 features), so every code and exponent
// byte of a row is written.
//
// Large ones are bound by HBM.  Measured on 32768 x 8192 bf16: packing 128 us (0.82 GB,
// 6.3 TB/s), unpacking 131 us (6.2); on 32768 x 8192 gated pairs (silu), holding both
// inputs: forward 346 to 380 us (2.17 GB, 5.7 to 6.3 TB/s), backward 343 to 415 us (2.17
// GB, 5.2 to 6.4 TB/s; a copy of 1 GB runs at 5.15).  On a few dozen rows each is one
// launch of 2.2 to 3.7 us.  Between them the vector instructions count: the codes' fused
// division and rounding, exponent bytes by permutation instead of a lane exchange through
// LDS and one division per thread left 73 instructions per 8 features
// packed of 183 (16384 x 4096: 41 -> 37 us).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "grads_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

// The units (8 features) a thread takes: its own index, then every gridDim *
// kThreads-th.  A matrix has `upr` units per row; the step between a thread's units is
// given as whole rows and units, so that only its first unit takes a division.
struct Walk {
    uint32_t upr, step_rows, step_units;
    uint32_t rows;
};
struct At {
    uint32_t row, unit;
    __device__ __forceinline__ At(const Walk& w) {
        const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
        row = u / w.upr;
        unit = u - row * w.upr;
    }
    __device__ __forceinline__ void next(const Walk& w) {
        row += w.step_rows;
        unit += w.step_units;
        if (unit >= w.upr) {
            unit -= w.upr;
            ++row;
        }
    }
    __device__ __forceinline__ int col() const { return (int)unit * 8; }
    // offset of this unit's row in a matrix of the given row length or stride
    __device__ __forceinline__ int64_t row_at(uint32_t stride) const {
        return (int64_t)((uint64_t)row * stride);
    }
};

// 8 features from column `col` on, zeros past the last column.
template <typename T, bool AL, bool NT>
__device__ __forceinline__ void load8(const T* row, int col, int cols, float* v) {
    if (col < cols) {
        load_unit<T, AL, NT>(row + col, cols - col, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
}

template <typename T, bool AL, bool NT>
__device__ __forceinline__ void store8(T* row, int col, int cols, const float* v) {
    if (col < cols) store_unit<T, AL, NT>(row + col, cols - col, v);
}

// Hold 8 features of each lane: codes and exponent byte of its group of four
// lanes (active together: every row has a multiple of 16 units), into the held
// matrix's row.
template <bool NT>
__device__ __forceinline__ void hold8(const float* v, int8_t* codes, uint8_t* exps, const At& at,
                                      int code_pitch, int exp_pitch) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
    // the largest of four neighbouring lanes, by lane permutation within them
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));     // 1, 0, 3, 2
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));     // 2, 3, 0, 1
    const uint32_t b = act_exp_byte(top);
    const u32x2 w = act_codes(v, b);
    const int col = at.col();
    if (col < code_pitch) {
        u32x2* p = reinterpret_cast<u32x2*>(codes + at.row_at(code_pitch) + col);
        if constexpr (NT) __builtin_nontemporal_store(w, p);
        else *p = w;
    }
    if ((col & 31) == 0) exps[at.row_at(exp_pitch) + (col >> 5)] = (uint8_t)b;
}

__device__ __forceinline__ void held8(const int8_t* codes, const uint8_t* exps, const At& at,
                                      int code_pitch, int exp_pitch, float* v) {
    const int col = at.col();
    const u32x2 w = *reinterpret_cast<const u32x2*>(codes + at.row_at(code_pitch) + col);
    const float s = act_scale(exps[at.row_at(exp_pitch) + (col >> 5)]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = act_value(w[0], e, s);
        v[4 + e] = act_value(w[1], e, s);
    }
}

template <typename T, bool AL, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_pack(const T* __restrict__ x, uint32_t stride,
                                                       int8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ exps, int cols,
                                                       int code_pitch, int exp_pitch, Walk w) {
    for (At at(w); at.row < w.rows; at.next(w)) {
        float v[8];
        load8<T, AL, NT>(x + at.row_at(stride), at.col(), cols, v);
        hold8<NT>(v, codes, exps, at, code_pitch, exp_pitch);
    }
}

template <typename T, bool AL, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_unpack(const int8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ exps,
                                                         T* __restrict__ out, uint32_t stride,
                                                         int cols, int code_pitch, int exp_pitch,
                                                         Walk w) {
    for (At at(w); at.row < w.rows; at.next(w)) {
        float v[8];
        held8(codes, exps, at, code_pitch, exp_pitch, v);
        store8<T, AL, NT>(out + at.row_at(stride), at.col(), cols, v);
    }
}

// ------------------------------------------------------ gated activation --
// h = act(g) u, with g and u held in the same pass; and dg = dh u act'(g), du = dh act(g)
// from the held forms: 3 values read or written per feature each way beside the
// codes, so the two passes of a backbone's 32768 x 8192 pairs move 4.3 GB in 0.70 to 0.76 ms.
// 1 / (1 + 2^(-x log2 e)): saturates to 0 and 1, NaN stays NaN.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __expf(-x));
}

// act(g) = g s with s = sigmoid(a(g)), and its derivative s + g s (1 - s) a'(g):
// a(g) = g for SiLU; GELU's tanh form is g sigmoid(2 z), z = sqrt(2/pi) (g +
// 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ float act_sig(float g) {
    if (ACT == MA_ACT_SILU) return sigmoid(g);
    return sigmoid(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.f));
}
// Where s (1 - s) has run out to 0 the second term is 0, although g a'(g) may
// have overflowed.
template <int ACT>
__device__ __forceinline__ float act_slope(float g, float s) {
    const float da =
        ACT == MA_ACT_SILU ? 1.f : 1.5957691216057308f * fmaf(3.f * 0.044715f * g, g, 1.f);
    const float p = s * (1.f - s);
    return p > 0.f ? fmaf(p, g * da, s) : s;
}

template <typename T, bool AL, bool NT, int ACT>
__global__ __launch_bounds__(kThreads) void k_glu_forward(GluArgs a, int cols, int code_pitch,
                                                          int exp_pitch, Walk w) {
    const T* gate = static_cast<const T*>(a.gate);
    const T* up = static_cast<const T*>(a.up);
    T* h = static_cast<T*>(a.h);
    const uint32_t gs = (uint32_t)a.gate_stride, us = (uint32_t)a.up_stride, hs = (uint32_t)a.h_stride;
    for (At at(w); at.row < w.rows; at.next(w)) {
        float gv[8], uv[8], hv[8];
        load8<T, AL, NT>(gate + at.row_at(gs), at.col(), cols, gv);
        load8<T, AL, NT>(up + at.row_at(us), at.col(), cols, uv);
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = gv[e] * act_sig<ACT>(gv[e]) * uv[e];
        store8<T, AL, NT>(h + at.row_at(hs), at.col(), cols, hv);
        hold8<NT>(gv, a.gate_codes, a.gate_exps, at, code_pitch, exp_pitch);
        hold8<NT>(uv, a.up_codes, a.up_exps, at, code_pitch, exp_pitch);
    }
}

template <typename T, bool AL, bool NT, int ACT, bool HOLD>
__global__ __launch_bounds__(kThreads) void k_glu_backward(GluArgs a, int cols, int code_pitch,
                                                           int exp_pitch, Walk w) {
    const T* dh = static_cast<const T*>(a.dh);
    T* dgate = static_cast<T*>(a.dgate);
    T* dup = static_cast<T*>(a.dup);
    const uint32_t ds = (uint32_t)a.dh_stride, gs = (uint32_t)a.dgate_stride, us = (uint32_t)a.dup_stride;
    for (At at(w); at.row < w.rows; at.next(w)) {
        const int col = at.col();
        float gv[8], uv[8], dv[8], o[8], hv[8];
        load8<T, AL, NT>(dh + at.row_at(ds), col, cols, dv);
        if (!HOLD || col < code_pitch) {
            held8(a.gate_codes, a.gate_exps, at, code_pitch, exp_pitch, gv);
            held8(a.up_codes, a.up_exps, at, code_pitch, exp_pitch, uv);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) gv[e] = uv[e] = 0.f;
        }
        float sv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sv[e] = act_sig<ACT>(gv[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = dv[e] * uv[e] * act_slope<ACT>(gv[e], sv[e]);
        store8<T, AL, NT>(dgate + at.row_at(gs), col, cols, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float av = gv[e] * sv[e];
            o[e] = dv[e] * av;
            hv[e] = col + e < cols ? av * uv[e] : 0.f;
        }
        store8<T, AL, NT>(dup + at.row_at(us), col, cols, o);
        if (HOLD) hold8<NT>(hv, a.h_codes, a.h_exps, at, code_pitch, exp_pitch);
    }
}

// A streaming launch over rows of `upr` units: every unit once, in at most 16
// rounds of a full GPU (8 workgroups per CU).
struct Grid {
    dim3 dim;
    Walk walk;
    Grid(int64_t rows, int64_t upr) {
        const int64_t n = std::min<int64_t>(ceil_div(rows * upr, kThreads), (int64_t)kCus * 8 * 16);
        dim = dim3((unsigned)n);
        walk.upr = (uint32_t)upr;
        walk.rows = (uint32_t)rows;
        walk.step_rows = (uint32_t)(n * kThreads / upr);
        walk.step_units = (uint32_t)(n * kThreads % upr);
    }
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// 16-byte accesses to rows of 8-element units: every row starts 16-byte aligned
// and holds whole units.
bool al_rows(const void* p, int64_t stride, int64_t cols, int32_t dtype) {
    const int64_t per = dtype == MA_PARAM_BF16 ? 8 : 4;
    return aligned16(p) && stride % per == 0 && cols % 8 == 0;
}

// Calls f(T{}, aligned, past the caches) with a launch's type and paths (only
// aligned bf16 streams go past the caches).
template <typename F>
int by_paths(int32_t dtype, bool al, bool nt, F f) {
    if (dtype == MA_PARAM_BF16) {
        if (al && nt) f(__bf16{}, std::true_type{}, std::true_type{});
        else if (al) f(__bf16{}, std::true_type{}, std::false_type{});
        else f(__bf16{}, std::false_type{}, std::false_type{});
    } else {
        if (al) f(float{}, std::true_type{}, std::false_type{});
        else f(float{}, std::false_type{}, std::false_type{});
    }
    return (int)hipGetLastError();
}

// The same with the activation function.
template <typename F>
int by_act(int32_t act, int32_t dtype, bool al, bool nt, F f) {
    return by_paths(dtype, al, nt, [&](auto t, auto a, auto n) {
        if (act == MA_ACT_SILU) f(t, a, n, std::integral_constant<int, MA_ACT_SILU>{});
        else f(t, a, n, std::integral_constant<int, MA_ACT_GELU_TANH>{});
    });
}

}  // namespace

int launch_act_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                    int8_t* codes, uint8_t* exps, void* stream) {
    if (rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(cols), ep = (int)act_exp_pitch(cols);
    const Grid grid(rows, (int64_t)ep * 4);
    return by_paths(dtype, al_rows(x, stride, cols, dtype), streams_past_caches(rows * cols, dtype),
                    [&](auto t, auto al, auto nt) {
        using T = decltype(t);
        hipLaunchKernelGGL((k_act_pack<T, decltype(al)::value, decltype(nt)::value>), grid.dim, dim3(kThreads), 0,
                           (hipStream_t)stream, static_cast<const T*>(x), (uint32_t)stride, codes, exps, (int)cols, cp,
                           ep, grid.walk);
    });
}

int launch_act_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                      void* out, int32_t dtype, int64_t stride, void* stream) {
    if (rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(cols), ep = (int)act_exp_pitch(cols);
    const Grid grid(rows, cp / 8);
    return by_paths(dtype, al_rows(out, stride, cols, dtype), streams_past_caches(rows * cols, dtype),
                    [&](auto t, auto al, auto nt) {
        using T = decltype(t);
        hipLaunchKernelGGL((k_act_unpack<T, decltype(al)::value, decltype(nt)::value>), grid.dim, dim3(kThreads), 0,
                           (hipStream_t)stream, codes, exps, static_cast<T*>(out), (uint32_t)stride, (int)cols, cp, ep,
                           grid.walk);
    });
}

int launch_glu_forward(const GluArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    const Grid grid(a.rows, (int64_t)ep * 4);
    const bool al = al_rows(a.gate, a.gate_stride, a.cols, a.dtype) &&
                    al_rows(a.up, a.up_stride, a.cols, a.dtype) &&
                    al_rows(a.h, a.h_stride, a.cols, a.dtype);
    return by_act(a.act, a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype),
                  [&](auto t, auto w, auto nt, auto act) {
        hipLaunchKernelGGL((k_glu_forward<decltype(t), decltype(w)::value, decltype(nt)::value, decltype(act)::value>),
                           grid.dim, dim3(kThreads), 0, (hipStream_t)stream, a, (int)a.cols, cp, ep, grid.walk);
    });
}

int launch_glu_backward(const GluArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    const bool hold = a.h_codes != nullptr;
    const Grid grid(a.rows, hold ? (int64_t)ep * 4 : cp / 8);
    const bool al = al_rows(a.dh, a.dh_stride, a.cols, a.dtype) &&
                    al_rows(a.dgate, a.dgate_stride, a.cols, a.dtype) &&
                    al_rows(a.dup, a.dup_stride, a.cols, a.dtype);
    return by_act(a.act, a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype),
                  [&](auto t, auto w, auto nt, auto act) {
        using T = decltype(t);
        constexpr bool AL = decltype(w)::value, NT = decltype(nt)::value;
        constexpr int ACT = decltype(act)::value;
        if (hold)
            hipLaunchKernelGGL((k_glu_backward<T, AL, NT, ACT, true>), grid.dim, dim3(kThreads), 0, (hipStream_t)stream,
                               a, (int)a.cols, cp, ep, grid.walk);
        else
            hipLaunchKernelGGL((k_glu_backward<T, AL, NT, ACT, false>), grid.dim, dim3(kThreads), 0, (hipStream_t)stream,
                               a, (int)a.cols, cp, ep, grid.walk);
    });
}

}  // namespace ma
