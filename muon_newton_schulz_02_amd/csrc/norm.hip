// Root-mean-square norm with the residual's addition and an output held in 8
// bits, and its backward pass, on gfx950.
//
// Both stream rows: TPR threads keep one row in registers, a unit of 8 columns
// each, so every array is read and written once and the mean costs one reduction
// over those threads (lane exchanges up to a wave, one LDS round and barrier above).
// Rows go to workgroups in a fixed order, the weights stay in registers from row
// to row.  The weight's gradient is summed in registers over a workgroup's rows,
// then over its waves, and by a second launch over the workgroups' partial sums,
// each in a fixed order.
//
// Bound by HBM: forward of 32768 x 2048 bf16 rows with residual and held output 0.61 GB
// in 110 us (5.6 TB/s), backward with the stream's gradient 0.54 GB in 95 us
// (5.6 TB/s, the partial sums' 3 us with it); a large copy reaches 5.2.  One unit a
// thread keeps enough waves on a CU for its loads: a wave of four units each took 177
// and 173 us (172 and 224 registers).  Odd rows (2001 columns) take 1.5 times as long:
// 16-byte accesses at any address, and a last unit element by element.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "layers_internal.h"

namespace ma {
namespace {

// Threads of a workgroup: several rows of up to a wave each, or one longer row.
template <int TPR>
constexpr int kThreads = TPR <= 64 ? 256 : TPR;

// Sum over the TPR threads of a row; `slot` is LDS of TPR / 64 floats that no
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

// 1 / sqrt(m): the hardware's estimate (off by one step or so) and one step of
// Newton's method, r + r (1 - m r^2) / 2; 0 and infinity stay what they are.
__device__ __forceinline__ float inv_root(float m) {
    const float r = rsqrtf(m);
    const float e = fmaf(-(m * r), r, 1.f);
    return m < __builtin_inff() ? fmaf(0.5f * r, e, r) : r;
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

// weight + offset of a unit's columns, zeros past the last.
__device__ __forceinline__ void load_weight(const NormArgs& a, int col, int cols, float* w) {
    if (a.weight_dtype == MA_PARAM_BF16)
        load_cols<__bf16, false, false>(static_cast<const __bf16*>(a.weight), col, cols, w);
    else
        load_cols<float, false, false>(static_cast<const float*>(a.weight), col, cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = col + e < cols ? w[e] + a.offset : 0.f;
}

template <typename T, bool AL, bool NT, int TPR>
__global__ __launch_bounds__(kThreads<TPR>) void k_rms_norm_forward(NormArgs a, int cols, int code_pitch,
                                                                    int exp_pitch) {
    __shared__ float slots[3][kThreads<TPR> / 64];
    constexpr int kRows = kThreads<TPR> / TPR;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.res);
    T* sum = static_cast<T*>(a.sum);
    T* y = static_cast<T*>(a.y);
    const int col = (int)(threadIdx.x & (TPR - 1)) * 8;
    float w[8];
    load_weight(a, col, cols, w);
    const float mean_of = 1.f / (float)cols;
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + threadIdx.x / TPR;
        const bool here = kRows == 1 || row < a.rows;
        const int n = here ? cols : 0;           // (the lanes past the last row hold zeros)
        float v[8];
        load_cols<T, AL, NT>(x + row * a.x_stride, col, n, v);
        if (res) {
            float r[8];
            load_cols<T, AL, NT>(res + row * a.res_stride, col, n, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
            if (col < n) store_unit<T, AL, NT>(sum + row * a.sum_stride + col, n - col, v);
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
        ss = row_sum<TPR>(ss, slots[turn]);
        float inv = inv_root(fmaf(ss, mean_of, a.eps));
        // squares beyond float32: the same sum of values scaled by 2^-80, in which
        // the largest are at least 2^-24 (and eps counts for nothing)
        const bool over = !(ss < __builtin_inff());
        if (TPR >= 64 ? over : (bool)__any(over)) {
            float s2 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = v[e] * 0x1p-80f;
                s2 = fmaf(t, t, s2);
            }
            s2 = row_sum<TPR>(s2, slots[2]);
            if (over) inv = inv_root(s2 * mean_of) * 0x1p-80f;
            if (TPR > 64) __syncthreads();
        }
        turn ^= 1;
        if (here && col == 0) a.inv[row] = inv;
        // the product with inv keeps its rounding error, so y is rounded once beside inv and
        // the weight; what is held is y as it is stored
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = v[e] * inv, lost = fmaf(v[e], inv, -t);
            v[e] = (float)(T)(fabsf(t) < __builtin_inff() ? fmaf(t, w[e], lost * w[e]) : t * w[e]);
        }
        if (y && col < n) store_unit<T, AL, NT>(y + row * a.y_stride + col, n - col, v);
        if (a.codes) {
            if (col + 8 > n)         // (a NaN row is none in the columns past its end)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = col + e < n ? v[e] : 0.f;
            uint32_t b;
            const u32x2 q = hold_unit(v, b);
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

template <typename T, bool AL, bool NT, int TPR>
__global__ __launch_bounds__(kThreads<TPR>) void k_rms_norm_backward(NormArgs a, int cols) {
    constexpr int kRows = kThreads<TPR> / TPR, kWaves = kThreads<TPR> / 64;
    __shared__ float slots[2][kWaves];
    __shared__ float joined[TPR <= 64 ? kWaves - 1 : 1][TPR <= 64 ? TPR * 8 : 1];
    const T* s = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    const T* dsum = static_cast<const T*>(a.dsum);
    T* ds = static_cast<T*>(a.ds);
    const int col = (int)(threadIdx.x & (TPR - 1)) * 8;
    float w[8], acc[8];
    load_weight(a, col, cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    const float mean_of = 1.f / (float)cols;
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + threadIdx.x / TPR;
        const bool here = kRows == 1 || row < a.rows;
        const int n = here ? cols : 0;
        float h[8], d[8], r[8];
        const float inv = here ? a.inv[row] : 0.f;
        load_cols<T, AL, NT>(s + row * a.x_stride, col, n, h);
        load_cols<T, AL, NT>(dy + row * a.dy_stride, col, n, d);
        if (dsum) load_cols<T, AL, NT>(dsum + row * a.dsum_stride, col, n, r);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] *= inv;
            acc[e] = fmaf(d[e], h[e], acc[e]);
            d[e] *= w[e];
            dot = fmaf(d[e], h[e], dot);
        }
        dot = row_sum<TPR>(dot, slots[turn]) * mean_of;
        turn ^= 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            d[e] = inv * fmaf(-h[e], dot, d[e]);
            if (dsum) d[e] += r[e];
        }
        if (col < n) store_unit<T, AL, NT>(ds + row * a.ds_stride + col, n - col, d);
    }
    if (!a.partials) return;
    // this workgroup's sum: over the rows side by side in a wave, then over the waves
#pragma unroll
    for (int m = TPR; m < 64; m <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor(acc[e], m, 64);
    if constexpr (TPR <= 64) {
        const int wave = threadIdx.x >> 6;
        const bool lead = (threadIdx.x & 63) < TPR;
        if (wave > 0 && lead)
#pragma unroll
            for (int e = 0; e < 8; ++e) joined[wave - 1][col + e] = acc[e];
        __syncthreads();
        if (wave > 0 || !lead) return;
#pragma unroll
        for (int k = 0; k < kWaves - 1; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += joined[k][col + e];
    }
    if (col < cols) store_unit<float, false>(a.partials + (int64_t)blockIdx.x * cols + col, cols - col, acc);
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

// Calls f(threads per row) for a row length.
template <typename F>
void by_row(int64_t cols, F f) {
    if (cols <= 128) f(Int<16>{});
    else if (cols <= 256) f(Int<32>{});
    else if (cols <= 512) f(Int<64>{});
    else if (cols <= 1024) f(Int<128>{});
    else if (cols <= 2048) f(Int<256>{});
    else if (cols <= 4096) f(Int<512>{});
    else f(Int<1024>{});
}

}  // namespace

// As many workgroups as are on a CU at once for rows of whole units (24 waves: 32768 x 2048
// bf16 101 us with 16, 95 with 24, 120 with 32), fewer for others, whose kernel takes more
// registers (x 2001: 159, 200, 166); but four rounds of rows at least where that leaves one
// for every CU, since each costs a partial sum.
int64_t norm_backward_groups(int64_t rows, int64_t cols) {
    int64_t n = 0;
    by_row(cols, [&](auto tpr) {
        constexpr int TPR = decltype(tpr)::value, T = kThreads<TPR>;
        const int64_t rounds = ceil_div(rows, T / TPR);
        const int64_t per_cu = std::max(1, (cols % 8 == 0 ? 24 : 16) * 64 / T);
        n = std::min({rounds, std::max<int64_t>(kCus, rounds / 4), kCus * per_cu});
    });
    return n;
}

int launch_rms_norm_forward(const NormArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const bool al = al_rows(a.x, a.x_stride, a.cols, a.dtype) && al_rows(a.res, a.res_stride, a.cols, a.dtype) &&
                    al_rows(a.sum, a.sum_stride, a.cols, a.dtype) && al_rows(a.y, a.y_stride, a.cols, a.dtype);
    const int cp = (int)act_code_pitch(a.cols), ep = (int)act_exp_pitch(a.cols);
    return by_paths(a.dtype, al, streams_past_caches(a.rows * a.cols, a.dtype), [&](auto t, auto w, auto nt) {
        by_row(a.cols, [&](auto tpr) {
            constexpr int TPR = decltype(tpr)::value;
            const int64_t n = std::min<int64_t>(ceil_div(a.rows, kThreads<TPR> / TPR), (int64_t)kCus * 2048 / kThreads<TPR>);
            hipLaunchKernelGGL((k_rms_norm_forward<decltype(t), decltype(w)::value, decltype(nt)::value, TPR>),
                               dim3((unsigned)n), dim3(kThreads<TPR>), 0, (hipStream_t)stream, a, (int)a.cols, cp, ep);
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
            by_row(a.cols, [&](auto tpr) {
                constexpr int TPR = decltype(tpr)::value;
                hipLaunchKernelGGL((k_rms_norm_backward<decltype(t), decltype(w)::value, decltype(nt)::value, TPR>),
                                   dim3((unsigned)groups), dim3(kThreads<TPR>), 0, (hipStream_t)stream, a, (int)a.cols);
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
