// Rotary positions of several axes on gfx950: a stream of x with one sine and
// cosine for every token and feature pair.
//
// A workgroup takes a few whole tokens.  It first forms their sines and cosines
// in LDS, once for all heads: the angle in turns, position times turns per
// position, is rounded to whole turns in 64 bits (the remainder by a fused
// multiply-add, so only the frequency's own rounding counts: 2^-54 of the angle)
// and only the remainder goes to 32 bits.  Then it streams the tokens' heads, 8
// pairs (or 8 features of neighbouring pairs) a thread.
//
// Bound by HBM: 32768 tokens of 20 heads of 128 bf16, 0.34 GB, in 62 us (5.4 TB/s; a large copy
// reaches 4.5 to 5.2).  The sines are formed behind the stream; read as a table they would add
// 5 % to those bytes, and 50 % with two heads.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "layers_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;        // most (token, pair) angles a workgroup holds: 8 KB
static_assert(kAngles >= MA_ROTARY_MAX_PAIRS, "a token's angles fit");

// Turns v in place: pairs (v[e], w[e]) by angles cs[0 .. n), none past n.
__device__ __forceinline__ void turn8(float* v, float* w, const float2* cs, int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 c = cs[min(e, n - 1)];
        const float a = v[e], b = w[e];
        v[e] = fmaf(a, c.x, -b * c.y);
        w[e] = fmaf(a, c.y, b * c.x);
    }
}

template <typename T, bool AL, bool NT, int LAYOUT>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a, RotaryTable tab, int per, int units, int turned) {
    __shared__ float2 cs[kAngles];
    const T* x = static_cast<const T*>(a.x);
    T* out = static_cast<T*>(a.out);
    const int per_token = a.heads * units;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.n_tokens; t0 += (int64_t)gridDim.x * per) {
        const int nt = (int)min<int64_t>(per, a.n_tokens - t0);
        for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
            const int t = i / a.pairs, p = i - t * a.pairs;
            const int64_t at = (int64_t)tab.axis[p] * a.axis_stride + t0 + t;
            const double pos = a.position_bytes == 8 ? (double)static_cast<const int64_t*>(a.positions)[at]
                                                     : (double)static_cast<const int32_t*>(a.positions)[at];
            const double turns = tab.turns[p];
            const float part = (float)fma(pos, turns, -rint(pos * turns));
            float s, c;
            sincospif(2.f * part, &s, &c);
            cs[i] = make_float2(c, a.inverse ? -s : s);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
            const int t = i / per_token, r = i - t * per_token;
            const int h = r / units, u = r - h * units;
            const T* px = x + (t0 + t) * a.x_token + h * a.x_head;
            T* po = out + (t0 + t) * a.out_token + h * a.out_head;
            float v[8], w[8];
            if (u >= turned) {               // features past the pairs
                const int c = 2 * a.pairs + 8 * (u - turned);
                load_unit<T, AL, NT>(px + c, a.dim - c, v);
                store_unit<T, AL, NT>(po + c, a.dim - c, v);
            } else if (LAYOUT == MA_ROTARY_HALF) {
                const int p = 8 * u, n = a.pairs - p;
                load_unit<T, AL, NT>(px + p, n, v);
                load_unit<T, AL, NT>(px + a.pairs + p, n, w);
                turn8(v, w, cs + t * a.pairs + p, min(n, 8));
                store_unit<T, AL, NT>(po + p, n, v);
                store_unit<T, AL, NT>(po + a.pairs + p, n, w);
            } else {
                const int p = 4 * u, n = a.pairs - p;
                load_unit<T, AL, NT>(px + 2 * p, 2 * n, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 c = cs[t * a.pairs + p + min(e, n - 1)];
                    w[2 * e] = fmaf(v[2 * e], c.x, -v[2 * e + 1] * c.y);
                    w[2 * e + 1] = fmaf(v[2 * e], c.y, v[2 * e + 1] * c.x);
                }
                store_unit<T, AL, NT>(po + 2 * p, 2 * n, w);
            }
        }
        __syncthreads();         // (the next tokens' angles take this LDS)
    }
}

bool al16(const void* p, int64_t token, int64_t head, int32_t dtype) {
    const int64_t per = dtype == MA_PARAM_BF16 ? 8 : 4;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && token % per == 0 && head % per == 0;
}

}  // namespace

int launch_rotary(const RotaryArgs& a, const RotaryTable& tab, void* stream) {
    if (a.n_tokens == 0) return (int)hipSuccess;
    const bool half = a.layout == MA_ROTARY_HALF;
    const int turned = (int)ceil_div(half ? a.pairs : 2 * a.pairs, 8);
    // (in place, the features past the pairs stay where they are)
    const int rest = a.out == a.x ? 0 : a.dim - 2 * a.pairs;
    const int units = turned + (int)ceil_div(rest, 8);
    // about four units a thread, as long as that leaves a few workgroups per CU, and
    // no more tokens than the angles' LDS holds
    const int64_t per_token = (int64_t)a.heads * units;
    int64_t per = std::max<int64_t>(1, 4 * kThreads / per_token);
    per = std::min<int64_t>(per, std::max<int64_t>(1, ceil_div(a.n_tokens, kCus * 4)));
    per = std::min<int64_t>(per, kAngles / a.pairs);
    const bool al = al16(a.x, a.x_token, a.x_head, a.dtype) && al16(a.out, a.out_token, a.out_head, a.dtype) &&
                    a.pairs % (half ? 8 : 4) == 0 && (a.dim - 2 * a.pairs) % 8 == 0;
    const bool nt = streams_past_caches(a.n_tokens * a.heads * a.dim, a.dtype);
    // (a launch has fewer than 2^32 threads: more tokens than that come round again)
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(a.n_tokens, per), int64_t(1) << 20));
    auto go = [&](auto t, auto w, auto n) {
        using T = decltype(t);
        constexpr bool AL = decltype(w)::value, NT = decltype(n)::value;
        if (half)
            hipLaunchKernelGGL((k_rotary<T, AL, NT, MA_ROTARY_HALF>), grid, dim3(kThreads), 0, (hipStream_t)stream, a,
                               tab, (int)per, units, turned);
        else
            hipLaunchKernelGGL((k_rotary<T, AL, NT, MA_ROTARY_PAIRS>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                               a, tab, (int)per, units, turned);
    };
    if (a.dtype == MA_PARAM_BF16) {
        if (al && nt) go(__bf16{}, std::true_type{}, std::true_type{});
        else if (al) go(__bf16{}, std::true_type{}, std::false_type{});
        else go(__bf16{}, std::false_type{}, std::false_type{});
    } else {
        if (al) go(float{}, std::true_type{}, std::false_type{});
        else go(float{}, std::false_type{}, std::false_type{});
    }
    return (int)hipGetLastError();
}

}  // namespace ma
