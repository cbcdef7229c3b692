// Root-mean-square norm with the residual's addition and an output held in 8
// bits, and its backward pass, on gfx950.
//
// Both stream rows: TPR threads keep one row in registers, U units of 8
// columns each, so every array is read and written once and the mean costs one
// reduction over those threads (lane exchanges up to a wave, one LDS round above).
// A wave per row up to 4096 columns (2048 backward) needs no barrier; a workgroup
// takes the longer rows.  Rows go to workgroups in a fixed order, the weights
// stay in registers from row to row.  The weight's gradient is summed in registers
// over a workgroup's rows, then over its waves, and by a second launch over
// the workgroups' partial sums, each in a fixed order.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "layers_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

// Sum over the TPR threads of a row; `slot` is LDS of kThreads / 64 floats that no
// earlier sum still reads.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v += slot[w];
    }
    return v;
}

// The columns of this thread's unit u: first column, and how many exist.
template <int TPR>
__device__ __forceinline__ int unit_col(int u) {
    return (u * TPR + (int)(threadIdx.x & (TPR - 1))) * 8;
}

template <typename T, bool AL, bool NT>
__device__ __forceinline__ void load_cols(const T* row, int col, int cols, float* v) {
    if (col < cols) {
        load_unit<T, AL, NT>(row + col, cols - col, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
}

// weight + offset for this thread's columns, zeros past the last.
template <int TPR, int U>
__device__ __forceinline__ void load_weight(const NormArgs& a, int cols, float (*w)[8]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = unit_col<TPR>(u);
        if (a.weight_dtype == MA_PARAM_BF16)
            load_cols<__bf16, false, false>(static_cast<const __bf16*>(a.weight), col, cols, w[u]);
        else
            load_cols<float, false, false>(static_cast<const float*>(a.weight), col, cols, w[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[u][e] = col + e < cols ? w[u][e] + a.offset : 0.f;
    }
}

template <typename T, bool AL, bool NT, int TPR, int U>
__global__ __launch_bounds__(kThreads) void k_rms_norm_forward(NormArgs a, int cols, int code_pitch,
                                                               int exp_pitch) {
    __shared__ float slots[3][kThreads / 64];
    constexpr int kRows = kThreads / TPR;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.res);
    T* sum = static_cast<T*>(a.sum);
    T* y = static_cast<T*>(a.y);
    float w[U][8];
    load_weight<TPR, U>(a, cols, w);
    const float mean_of = 1.f / (float)cols;
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + threadIdx.x / TPR;
        const bool here = TPR >= kThreads || row < a.rows;
        const int n = here ? cols : 0;           // (the lanes past the last row hold zeros)
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load_cols<T, AL, NT>(x + row * a.x_stride, unit_col<TPR>(u), n, v[u]);
        if (res) {
            float r[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) load_cols<T, AL, NT>(res + row * a.res_stride, unit_col<TPR>(u), n, r[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[u][e] += r[u][e];
                const int col = unit_col<TPR>(u);
                if (col < n) store_unit<T, AL, NT>(sum + row * a.sum_stride + col, n - col, v[u]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[u][e], v[u][e], ss);
        ss = row_sum<TPR>(ss, slots[turn]);
        float inv = rsqrtf(fmaf(ss, mean_of, a.eps));
        // squares beyond float32: the same sum of values scaled by 2^-80, in which
        // the largest are at least 2^-24 (and eps counts for nothing)
        const bool over = !(ss < __builtin_inff());
        if (TPR >= 64 ? over : (bool)__any(over)) {
            float s2 = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = v[u][e] * 0x1p-80f;
                    s2 = fmaf(t, t, s2);
                }
            s2 = row_sum<TPR>(s2, slots[2]);
            if (over) inv = rsqrtf(s2 * mean_of) * 0x1p-80f;
            if (TPR > 64) __syncthreads();
        }
        turn ^= 1;
        if (here && (threadIdx.x & (TPR - 1)) == 0) a.inv[row] = inv;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = unit_col<TPR>(u);
            // what is held is y as it is stored
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = (float)(T)(v[u][e] * inv * w[u][e]);
            if (y && col < n) store_unit<T, AL, NT>(y + row * a.y_stride + col, n - col, v[u]);
            if (a.codes) {
                if (col + 8 > n)         // (a NaN row is none in the columns past its end)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[u][e] = col + e < n ? v[u][e] : 0.f;
                uint32_t b;
                const u32x2 q = hold_unit(v[u], b);
                if (here && col < code_pitch) {
                    u32x2* p = reinterpret_cast<u32x2*>(a.codes + row * code_pitch + col);
                    if constexpr (NT) __builtin_nontemporal_store(q, p);
                    else *p = q;
                }
                if (here && (col & 31) == 0 && (col >> 5) < exp_pitch)
                    a.exps[row * exp_pitch + (col >> 5)] = (uint8_t)b;
            }
        }
    }
}

template <typename T, bool AL, bool NT, int TPR, int U>
__global__ __launch_bounds__(kThreads) void k_rms_norm_backward(NormArgs a, int cols) {
    constexpr int kRows = kThreads / TPR;
    constexpr int kCols = TPR * U * 8;
    __shared__ float slots[2][kThreads / 64];
    __shared__ float joined[TPR <= 64 ? kThreads / 64 - 1 : 1][TPR <= 64 ? kCols : 1];
    const T* s = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    const T* dsum = static_cast<const T*>(a.dsum);
    T* ds = static_cast<T*>(a.ds);
    float w[U][8], acc[U][8];
    load_weight<TPR, U>(a, cols, w);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[u][e] = 0.f;
    const float mean_of = 1.f / (float)cols;
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + threadIdx.x / TPR;
        const bool here = TPR >= kThreads || row < a.rows;
        const int n = here ? cols : 0;
        float h[U][8], d[U][8];
        const float inv = here ? a.inv[row] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) load_cols<T, AL, NT>(s + row * a.x_stride, unit_col<TPR>(u), n, h[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) load_cols<T, AL, NT>(dy + row * a.dy_stride, unit_col<TPR>(u), n, d[u]);
        float dot = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[u][e] *= inv;
                acc[u][e] = fmaf(d[u][e], h[u][e], acc[u][e]);
                d[u][e] *= w[u][e];
                dot = fmaf(d[u][e], h[u][e], dot);
            }
        dot = row_sum<TPR>(dot, slots[turn]) * mean_of;
        turn ^= 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = unit_col<TPR>(u);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = inv * fmaf(-h[u][e], dot, d[u][e]);
            if (dsum) {
                float r[8];
                load_cols<T, AL, NT>(dsum + row * a.dsum_stride, col, n, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += r[e];
            }
            if (col < n) store_unit<T, AL, NT>(ds + row * a.ds_stride + col, n - col, o);
        }
    }
    if (!a.partials) return;
    // this workgroup's sum: over the rows side by side in a wave, then over the waves
#pragma unroll
    for (int m = TPR; m < 64; m <<= 1)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[u][e] += __shfl_xor(acc[u][e], m, 64);
    const int wave = threadIdx.x >> 6;
    if constexpr (TPR <= 64) {
        const bool lead = (threadIdx.x & 63) < TPR;
        if (wave > 0 && lead)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) joined[wave - 1][unit_col<TPR>(u) + e] = acc[u][e];
        __syncthreads();
        if (wave > 0 || !lead) return;
#pragma unroll
        for (int k = 0; k < kThreads / 64 - 1; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[u][e] += joined[k][unit_col<TPR>(u) + e];
    }
    float* out = a.partials + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = unit_col<TPR>(u);
        if (col < cols) store_unit<float, false>(out + col, cols - col, acc[u]);
    }
}

// dw (+)= the sum of `groups` partial sums: 32 columns a workgroup, whose 32 rows of
// threads take every 32nd partial sum each.
constexpr int kJoin = 32;
template <typename TW>
__global__ __launch_bounds__(kJoin * kJoin) void k_norm_weight_grad(const float* __restrict__ partials, int groups,
                                                                    int cols, TW* __restrict__ dw, int accumulate) {
    __shared__ float part[kJoin][kJoin + 1];
    const int c = threadIdx.x % kJoin, g = threadIdx.x / kJoin;
    const int col = blockIdx.x * kJoin + c;
    float v = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int k = g; k < groups; k += kJoin) v += partials[(int64_t)k * cols + col];
    part[g][c] = v;
    __syncthreads();
    if (g != 0 || col >= cols) return;
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) t += part[k][c];
    if (accumulate) t += (float)dw[col];
    dw[col] = (TW)t;
}

bool al_rows(const void* p, int64_t stride, int64_t cols, int32_t dtype) {
    const int64_t per = dtype == MA_PARAM_BF16 ? 8 : 4;
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % per == 0 && cols % 8 == 0);
}

// Calls f(T{}, aligned, past the caches).
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

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f(threads per row, units per thread) for a row length.
template <typename F>
void by_forward_row(int64_t cols, F f) {
    if (cols <= 128) f(Int<16>{}, Int<1>{});
    else if (cols <= 256) f(Int<32>{}, Int<1>{});
    else if (cols <= 512) f(Int<64>{}, Int<1>{});
    else if (cols <= 1024) f(Int<64>{}, Int<2>{});
    else if (cols <= 2048) f(Int<64>{}, Int<4>{});
    else if (cols <= 4096) f(Int<64>{}, Int<8>{});
    else if (cols <= 8192) f(Int<256>{}, Int<4>{});
    else f(Int<256>{}, Int<8>{});
}
// (the backward pass holds four arrays of a row's length: half the columns a thread)
template <typename F>
void by_backward_row(int64_t cols, F f) {
    if (cols <= 128) f(Int<16>{}, Int<1>{});
    else if (cols <= 256) f(Int<32>{}, Int<1>{});
    else if (cols <= 512) f(Int<64>{}, Int<1>{});
    else if (cols <= 1024) f(Int<64>{}, Int<2>{});
    else if (cols <= 2048) f(Int<64>{}, Int<4>{});
    else if (cols <= 4096) f(Int<256>{}, Int<2>{});
    else if (cols <= 8192) f(Int<256>{}, Int<4>{});
    else f(Int<256>{}, Int<8>{});
}

}  // namespace

int64_t norm_backward_groups(int64_t rows, int64_t cols) {
    int64_t per = 1;
    by_backward_row(cols, [&](auto tpr, auto) { per = kThreads / decltype(tpr)::value; });
    return std::min<int64_t>(ceil_div(rows, per), kCus * 3);
}

int launch_rms_norm_forward(const NormArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const bool al = al_rows(a.x, a.x_stride, a.cols, a.dtype) && al_rows(a.res, a.res_stride, a.cols, a.dtype) &&
                    al_rows(a.sum, a.sum_stride, a.cols, a.dtype) && al_rows(a.y, a.y_stride, a.cols, a.dtype);
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    return by_paths(a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype), [&](auto t, auto w, auto nt) {
        by_forward_row(a.cols, [&](auto tpr, auto u) {
            constexpr int TPR = decltype(tpr)::value, U = decltype(u)::value;
            const int64_t n = std::min<int64_t>(ceil_div(a.rows, kThreads / TPR), kCus * 8);
            hipLaunchKernelGGL((k_rms_norm_forward<decltype(t), decltype(w)::value, decltype(nt)::value, TPR, U>),
                               dim3((unsigned)n), dim3(kThreads), 0, (hipStream_t)stream, a, (int)a.cols, cp, ep);
        });
    });
}

int launch_rms_norm_backward(const NormArgs& a, void* stream) {
    const int64_t groups = norm_backward_groups(a.rows, a.cols);
    const bool al = al_rows(a.x, a.x_stride, a.cols, a.dtype) && al_rows(a.dy, a.dy_stride, a.cols, a.dtype) &&
                    al_rows(a.dsum, a.dsum_stride, a.cols, a.dtype) && al_rows(a.ds, a.ds_stride, a.cols, a.dtype);
    if (groups > 0) {
        const int rc = by_paths(a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype),
                                [&](auto t, auto w, auto nt) {
            by_backward_row(a.cols, [&](auto tpr, auto u) {
                hipLaunchKernelGGL((k_rms_norm_backward<decltype(t), decltype(w)::value, decltype(nt)::value,
                                                        decltype(tpr)::value, decltype(u)::value>),
                                   dim3((unsigned)groups), dim3(kThreads), 0, (hipStream_t)stream, a, (int)a.cols);
            });
        });
        if (rc != (int)hipSuccess) return rc;
    }
    if (!a.dw) return (int)hipSuccess;
    const dim3 grid((unsigned)ceil_div(a.cols, kJoin)), block(kJoin * kJoin);
    if (a.dw_dtype == MA_PARAM_BF16)
        hipLaunchKernelGGL(k_norm_weight_grad<__bf16>, grid, block, 0, (hipStream_t)stream, a.partials, (int)groups,
                           (int)a.cols, static_cast<__bf16*>(a.dw), a.accumulate);
    else
        hipLaunchKernelGGL(k_norm_weight_grad<float>, grid, block, 0, (hipStream_t)stream, a.partials, (int)groups,
                           (int)a.cols, static_cast<float*>(a.dw), a.accumulate);
    return (int)hipGetLastError();
}

}  // namespace ma
