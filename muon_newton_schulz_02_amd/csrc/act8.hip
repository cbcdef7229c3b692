// Activations held in 8 bits, and the gated activation that holds its
// inputs so, on gfx950.
//
// All four kernels stream: a thread takes 8 features of a token, four
// neighbouring lanes form one group of 32, whose largest magnitude they find
// with two lane exchanges.  A packing thread covers the padding up to the
// exponents' pitch (a multiple of 128 features), so every code and exponent
// byte of a row is written.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "grads_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

// Where unit u (8 features) of a matrix with `upr` units per row lies.
struct Unit {
    int64_t row;
    int col;
};
__device__ __forceinline__ Unit unit_at(int64_t u, uint32_t upr) {
    Unit r;
    if (u < (int64_t(1) << 32)) {
        const uint32_t q = (uint32_t)u / upr;
        r.row = q;
        r.col = (int)((uint32_t)u - q * upr) * 8;
    } else {
        r.row = u / upr;
        r.col = (int)(u - r.row * upr) * 8;
    }
    return r;
}

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
// lanes, into the held matrix's row.
template <bool NT>
__device__ __forceinline__ void hold8(const float* v, int8_t* codes, uint8_t* exps, int64_t row,
                                      int col, int code_pitch, int exp_pitch) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    const uint32_t b = act_exp_byte(top);
    const float inv = act_inv_scale(b);
    u32x2 w = {0u, 0u};
    if (b != 255u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[0] |= act_code(v[e], inv) << (8 * e);
            w[1] |= act_code(v[4 + e], inv) << (8 * e);
        }
    }
    if (col < code_pitch) {
        u32x2* p = reinterpret_cast<u32x2*>(codes + row * code_pitch + col);
        if constexpr (NT) __builtin_nontemporal_store(w, p);
        else *p = w;
    }
    if ((col & 31) == 0) exps[row * exp_pitch + (col >> 5)] = (uint8_t)b;
}

__device__ __forceinline__ void held8(const int8_t* codes, const uint8_t* exps, int64_t row,
                                      int col, int code_pitch, int exp_pitch, float* v) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(codes + row * code_pitch + col);
    const float s = act_scale(exps[row * exp_pitch + (col >> 5)]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = act_value(w[0], e, s);
        v[4 + e] = act_value(w[1], e, s);
    }
}

template <typename T, bool AL, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_pack(const T* __restrict__ x, int64_t stride,
                                                       int8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ exps, int cols,
                                                       int code_pitch, int exp_pitch,
                                                       uint32_t upr, int64_t units) {
    // (a group's four lanes share a row and are active together: units is a
    // multiple of 16)
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * kThreads) {
        const Unit at = unit_at(u, upr);
        float v[8];
        load8<T, AL, NT>(x + at.row * stride, at.col, cols, v);
        hold8<NT>(v, codes, exps, at.row, at.col, code_pitch, exp_pitch);
    }
}

template <typename T, bool AL, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_unpack(const int8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ exps,
                                                         T* __restrict__ out, int64_t stride,
                                                         int cols, int code_pitch, int exp_pitch,
                                                         uint32_t upr, int64_t units) {
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * kThreads) {
        const Unit at = unit_at(u, upr);
        float v[8];
        held8(codes, exps, at.row, at.col, code_pitch, exp_pitch, v);
        store8<T, AL, NT>(out + at.row * stride, at.col, cols, v);
    }
}

// ------------------------------------------------------ gated activation --
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
                                                          int exp_pitch, uint32_t upr,
                                                          int64_t units) {
    const T* gate = static_cast<const T*>(a.gate);
    const T* up = static_cast<const T*>(a.up);
    T* h = static_cast<T*>(a.h);
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * kThreads) {
        const Unit at = unit_at(u, upr);
        float gv[8], uv[8], hv[8];
        load8<T, AL, NT>(gate + at.row * a.gate_stride, at.col, cols, gv);
        load8<T, AL, NT>(up + at.row * a.up_stride, at.col, cols, uv);
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = gv[e] * act_sig<ACT>(gv[e]) * uv[e];
        store8<T, AL, NT>(h + at.row * a.h_stride, at.col, cols, hv);
        hold8<NT>(gv, a.gate_codes, a.gate_exps, at.row, at.col, code_pitch, exp_pitch);
        hold8<NT>(uv, a.up_codes, a.up_exps, at.row, at.col, code_pitch, exp_pitch);
    }
}

template <typename T, bool AL, bool NT, int ACT, bool HOLD>
__global__ __launch_bounds__(kThreads) void k_glu_backward(GluArgs a, int cols, int code_pitch,
                                                           int exp_pitch, uint32_t upr,
                                                           int64_t units) {
    const T* dh = static_cast<const T*>(a.dh);
    T* dgate = static_cast<T*>(a.dgate);
    T* dup = static_cast<T*>(a.dup);
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * kThreads) {
        const Unit at = unit_at(u, upr);
        float gv[8], uv[8], dv[8], o[8], hv[8];
        if (!HOLD || at.col < code_pitch) {
            held8(a.gate_codes, a.gate_exps, at.row, at.col, code_pitch, exp_pitch, gv);
            held8(a.up_codes, a.up_exps, at.row, at.col, code_pitch, exp_pitch, uv);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) gv[e] = uv[e] = 0.f;
        }
        load8<T, AL, NT>(dh + at.row * a.dh_stride, at.col, cols, dv);
        float sv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sv[e] = act_sig<ACT>(gv[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = dv[e] * uv[e] * act_slope<ACT>(gv[e], sv[e]);
        store8<T, AL, NT>(dgate + at.row * a.dgate_stride, at.col, cols, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float av = gv[e] * sv[e];
            o[e] = dv[e] * av;
            hv[e] = at.col + e < cols ? av * uv[e] : 0.f;
        }
        store8<T, AL, NT>(dup + at.row * a.dup_stride, at.col, cols, o);
        if (HOLD) hold8<NT>(hv, a.h_codes, a.h_exps, at.row, at.col, code_pitch, exp_pitch);
    }
}

// Workgroups of a streaming launch: every unit once, at most 16 rounds of a
// full GPU (8 workgroups per CU); longer matrices loop.
int64_t stream_grid(int64_t units) {
    return std::min<int64_t>(ceil_div(units, kThreads), (int64_t)kCus * 8 * 16);
}

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
    const uint32_t upr = (uint32_t)ep * 4;
    const int64_t units = rows * upr;
    const dim3 grid((unsigned)stream_grid(units));
    return by_paths(dtype, al_rows(x, stride, cols, dtype), streams_past_caches(rows * cols, dtype),
                    [&](auto t, auto al, auto nt) {
        using T = decltype(t);
        hipLaunchKernelGGL((k_act_pack<T, decltype(al)::value, decltype(nt)::value>), grid, dim3(kThreads), 0,
                           (hipStream_t)stream, static_cast<const T*>(x), stride, codes, exps, (int)cols, cp,
                           ep, upr, units);
    });
}

int launch_act_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                      void* out, int32_t dtype, int64_t stride, void* stream) {
    if (rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(cols), ep = (int)act_exp_pitch(cols);
    const uint32_t upr = (uint32_t)cp / 8;
    const int64_t units = rows * upr;
    const dim3 grid((unsigned)stream_grid(units));
    return by_paths(dtype, al_rows(out, stride, cols, dtype), streams_past_caches(rows * cols, dtype),
                    [&](auto t, auto al, auto nt) {
        using T = decltype(t);
        hipLaunchKernelGGL((k_act_unpack<T, decltype(al)::value, decltype(nt)::value>), grid, dim3(kThreads), 0,
                           (hipStream_t)stream, codes, exps, static_cast<T*>(out), stride, (int)cols, cp, ep,
                           upr, units);
    });
}

int launch_glu_forward(const GluArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    const uint32_t upr = (uint32_t)ep * 4;
    const int64_t units = a.rows * upr;
    const dim3 grid((unsigned)stream_grid(units));
    const bool al = al_rows(a.gate, a.gate_stride, a.cols, a.dtype) &&
                    al_rows(a.up, a.up_stride, a.cols, a.dtype) &&
                    al_rows(a.h, a.h_stride, a.cols, a.dtype);
    return by_act(a.act, a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype),
                  [&](auto t, auto w, auto nt, auto act) {
        hipLaunchKernelGGL((k_glu_forward<decltype(t), decltype(w)::value, decltype(nt)::value, decltype(act)::value>),
                           grid, dim3(kThreads), 0, (hipStream_t)stream, a, (int)a.cols, cp, ep, upr, units);
    });
}

int launch_glu_backward(const GluArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    const bool hold = a.h_codes != nullptr;
    const uint32_t upr = hold ? (uint32_t)ep * 4 : (uint32_t)cp / 8;
    const int64_t units = a.rows * upr;
    const dim3 grid((unsigned)stream_grid(units));
    const bool al = al_rows(a.dh, a.dh_stride, a.cols, a.dtype) &&
                    al_rows(a.dgate, a.dgate_stride, a.cols, a.dtype) &&
                    al_rows(a.dup, a.dup_stride, a.cols, a.dtype);
    return by_act(a.act, a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype),
                  [&](auto t, auto w, auto nt, auto act) {
        using T = decltype(t);
        constexpr bool AL = decltype(w)::value, NT = decltype(nt)::value;
        constexpr int ACT = decltype(act)::value;
        if (hold)
            hipLaunchKernelGGL((k_glu_backward<T, AL, NT, ACT, true>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                               a, (int)a.cols, cp, ep, upr, units);
        else
            hipLaunchKernelGGL((k_glu_backward<T, AL, NT, ACT, false>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                               a, (int)a.cols, cp, ep, upr, units);
    });
}

}  // namespace ma
