// Weight gradient of a linear layer, dW = dY^T X, from an X held in 8 bits, as
// MFMA GEMMs on gfx950.
//
// The reduction runs over tokens, along the rows of both operands, so both
// are staged in LDS as they lie in memory (a stage: 32 tokens by the tile's
// columns, bf16) and their fragments read with the transposing LDS load
// (ds_read_b64_tr_b16).  X is turned from codes into bf16 once per workgroup
// while it is staged: a held value is exact in bf16.  Products of two bf16
// values are exact in the matrix cores' float32, so a bf16 dY enters with
// nothing rounded; a float32 dY is cut into three bf16 parts of 8 bits
// each, which add up to it, and enters as three products.  Sums are float32.
//
// LDS layout of a stage operand of W columns: token row t at t * 2 W bytes,
// its 16-byte chunk c (8 columns) at slot c ^ ((t & 3) << 2), so the four
// rows of 64 bytes that half a wave reads together fall in distinct banks.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "grads_device.h"
#include "grads_internal.h"

namespace ma {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kTile = 128;                       // output tile side
constexpr int kRow = 2 * kTile;                  // LDS bytes of a token row
constexpr int kRegion = kLgStage * kRow;         // LDS bytes of an operand's stage

__device__ __forceinline__ u32x2 lds_tr8(const char* p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
    return __builtin_bit_cast(u32x2, v);
}

// Which tile and token slice a workgroup takes.  Consecutive workgroups go to
// the XCDs in turn; each XCD gets a contiguous range of the work list, in which
// tiles that share operand columns are neighbours.
struct Work {
    int64_t tn, tk, slice;
};
__device__ __forceinline__ Work work_of(int64_t id, int64_t total, int64_t tiles_n, int64_t tiles_k) {
    const int64_t q = total / kXcds, r = total % kXcds;
    const int64_t xcd = id % kXcds, local = id / kXcds;
    const int64_t i = xcd * q + min(xcd, r) + local;
    Work w;
    const int64_t tiles = tiles_n * tiles_k;
    w.slice = i / tiles;
    const int64_t t = i - w.slice * tiles;
    // blocks of four tile rows, walked column by column
    const int64_t band = t / (4 * tiles_k);
    const int64_t rows = min<int64_t>(4, tiles_n - band * 4);
    const int64_t in = t - band * 4 * tiles_k;
    w.tk = in / rows;
    w.tn = band * 4 + in % rows;
    return w;
}

// 16 held values of a token as bf16 (exact), packed in pairs.
__device__ __forceinline__ void held16(u32x4 codes, float scale, u32x4& lo, u32x4& hi) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t a = pack_bf16(act_value(codes[w], 0, scale), act_value(codes[w], 1, scale));
        const uint32_t b = pack_bf16(act_value(codes[w], 2, scale), act_value(codes[w], 3, scale));
        if (w < 2) {
            lo[2 * w] = a;
            lo[2 * w + 1] = b;
        } else {
            hi[2 * (w - 2)] = a;
            hi[2 * (w - 2) + 1] = b;
        }
    }
}

// The three bf16 parts of a float, as the high halves of words: x = h + m + l
// exactly (each takes the next 8 bits of the significand, cut, so none can
// overflow).  An infinity or NaN is all in the first part.
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
    const uint32_t b = __float_as_uint(x);
    const bool finite = (b & 0x7f800000u) != 0x7f800000u;
    h = b & 0xffff0000u;
    const float r1 = x - __uint_as_float(h);
    m = __float_as_uint(r1) & 0xffff0000u;
    l = __float_as_uint(r1 - __uint_as_float(m));
    if (!finite) {
        if (b & 0x007fffffu) h = 0x7fc00000u;
        m = l = 0u;
    }
}

__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {
    return (lo >> 16) | (hi & 0xffff0000u);
}

// The simple kernel: 128 x 128 tiles, four waves of 64 x 64, two LDS stages,
// operands staged through registers.  It takes any types, strides and sizes.
template <typename TD, bool VEC, typename TG>
__global__ __launch_bounds__(kThreads) void k_linear_grad(LgArgs a, int64_t tiles_n,
                                                          int64_t tiles_k, int64_t slices,
                                                          int64_t per) {
    constexpr int NP = sizeof(TD) == 4 ? 3 : 1;         // bf16 parts of dY
    constexpr int kStageBytes = (NP + 1) * kRegion;
    __shared__ __attribute__((aligned(1024))) char ring[2 * kStageBytes];
    const Work wk = work_of(blockIdx.x, (int64_t)gridDim.x, tiles_n, tiles_k);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t n0 = wk.tn * kTile, k0 = wk.tk * kTile;
    const int64_t t0 = wk.slice * per * kLgStage;
    const int64_t t1 = min(a.n_tokens, t0 + per * kLgStage);
    const int64_t cp = (a.n_in + 31) / 32 * 32, ep = ((cp / 32) + 3) / 4 * 4;

    // staging: this thread's token row and first of 16 columns
    const int srow = tid >> 3, scol = (tid & 7) * 16;
    const uint32_t s0 = (uint32_t)(srow * kRow + ((((scol >> 3)) ^ ((srow & 3) << 2)) << 4));
    const uint32_t s1 = (uint32_t)(srow * kRow + ((((scol >> 3) + 1) ^ ((srow & 3) << 2)) << 4));
    // fragments: block 0 of this wave, per operand
    uint32_t fa[2], fb[2];
    {
        const int g = lane >> 4, j = lane & 15, sw = (j >> 2) & 3;
        const int row = 8 * (g >> 1) + (j >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int in = 2 * (g & 1) + ((j & 3) >> 1);
            fa[i] = (uint32_t)(row * kRow + (((((wm * 2 + i) ^ sw) << 2) + in) << 4) + 8 * (j & 1));
            fb[i] = (uint32_t)(row * kRow + (((((wn * 2 + i) ^ sw) << 2) + in) << 4) + 8 * (j & 1));
        }
    }

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    float dv[16];
    u32x4 xc;
    uint32_t xe;
    auto load = [&](int64_t t) {
        const bool in = t + srow < t1;
        const TD* d = static_cast<const TD*>(a.dy) + (t + srow) * a.dy_stride + n0 + scol;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (VEC) {
                if (in && n0 + scol + 8 * h < a.n_out) {
                    load_v<TD, 8>(d + 8 * h, dv + 8 * h);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dv[8 * h + e] = 0.f;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dv[8 * h + e] = in && n0 + scol + 8 * h + e < a.n_out ? (float)d[8 * h + e] : 0.f;
            }
        }
        xc = (u32x4){0u, 0u, 0u, 0u};
        xe = 0;
        if (in && k0 + scol < cp) {
            xc = *reinterpret_cast<const u32x4*>(a.codes + (t + srow) * cp + k0 + scol);
            xe = a.exps[(t + srow) * ep + ((k0 + scol) >> 5)];
        }
    };
    auto put = [&](char* buf) {
        uint32_t w[NP][8];
        if constexpr (NP == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[0][e] = high_halves(__float_as_uint(dv[2 * e]), __float_as_uint(dv[2 * e + 1]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t h0, m0, l0, h1, m1, l1;
                split3(dv[2 * e], h0, m0, l0);
                split3(dv[2 * e + 1], h1, m1, l1);
                w[0][e] = high_halves(h0, h1);
                w[1][e] = high_halves(m0, m1);
                w[2][e] = high_halves(l0, l1);
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            *reinterpret_cast<u32x4*>(buf + p * kRegion + s0) = (u32x4){w[p][0], w[p][1], w[p][2], w[p][3]};
            *reinterpret_cast<u32x4*>(buf + p * kRegion + s1) = (u32x4){w[p][4], w[p][5], w[p][6], w[p][7]};
        }
        u32x4 lo, hi;
        held16(xc, act_scale(xe), lo, hi);
        *reinterpret_cast<u32x4*>(buf + NP * kRegion + s0) = lo;
        *reinterpret_cast<u32x4*>(buf + NP * kRegion + s1) = hi;
    };
    auto frag = [&](const char* p) {
        const u32x2 lo = lds_tr8(p), hi = lds_tr8(p + 4 * kRow);
        return __builtin_bit_cast(bf16x8, (u32x4){lo[0], lo[1], hi[0], hi[1]});
    };

    const int stages = (int)((t1 - t0 + kLgStage - 1) / kLgStage);   // (0 or less: no token)
    if (stages > 0) load(t0);
    for (int s = 0; s < stages; ++s) {
        // (the buffer was last read two stages ago, before the barrier in between)
        char* buf = ring + (s & 1) * kStageBytes;
        put(buf);
        if (s + 1 < stages) load(t0 + (int64_t)(s + 1) * kLgStage);
        __syncthreads();
#pragma unroll
        for (int kg = 0; kg < 2; ++kg) {
            bf16x8 b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = frag(buf + NP * kRegion + fb[j] + kg * 16 * kRow);
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) {      // smallest part first
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 f = frag(buf + p * kRegion + fa[i] + kg * 16 * kRow);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, b[j], acc[i][j], 0, 0, 0);
                }
            }
        }
    }

    // accumulator register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4,
    // column l % 32: a wave stores two row pieces of 32 columns at a time
    float* part = slices > 1 ? a.partials + wk.slice * a.n_out * a.n_in : nullptr;
    TG* grad = static_cast<TG*>(a.grad);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t col = k0 + wn * 64 + j * 32 + (lane & 31);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t row = n0 + wm * 64 + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row >= a.n_out || col >= a.n_in) continue;
                const int64_t o = row * a.n_in + col;
                if (part) part[o] = acc[i][j][r];
                else if (a.accumulate) grad[o] = (TG)((float)grad[o] + acc[i][j][r]);
                else grad[o] = (TG)acc[i][j][r];
            }
        }
}

// The slices' partial sums, added in slice order.
template <typename TG, int V>
__global__ __launch_bounds__(kThreads) void k_linear_join(const float* __restrict__ partials,
                                                          TG* __restrict__ grad, int64_t units,
                                                          int64_t slices, int accumulate) {
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;
    float acc[V];
    load_v<float, V>(partials + u * V, acc);
#pragma unroll 4
    for (int64_t s = 1; s < slices; ++s) {
        float v[V];
        load_v<float, V>(partials + (s * units + u) * V, v);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += v[e];
    }
    if (accumulate) {
        float old[V];
        load_v<TG, V>(grad + u * V, old);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += old[e];
    }
    store_v<TG, V>(grad + u * V, acc);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

LgPlan linear_grad_plan(int64_t n_tokens, int64_t n_out, int64_t n_in, int32_t dy_dtype) {
    (void)dy_dtype;
    LgPlan p;
    p.tile = kTile;
    p.tiles_n = ceil_div(n_out, kTile);
    p.tiles_k = ceil_div(n_in, kTile);
    const int64_t stages = ceil_div(n_tokens, kLgStage);
    const int64_t tiles = p.tiles_n * p.tiles_k;
    // enough slices for two workgroups per CU, of at least 8 stages each
    int64_t slices = std::max<int64_t>(1, std::min<int64_t>(ceil_div(2 * kCus, tiles), stages / 8));
    p.per = std::max<int64_t>(1, ceil_div(stages, slices));
    p.slices = std::max<int64_t>(1, ceil_div(stages, p.per));
    if (p.slices > 1) p.total = (size_t)p.slices * (size_t)n_out * (size_t)n_in * 4;
    return p;
}

int launch_linear_grad(const LgArgs& a, const LgPlan& p, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    const bool bd = a.dy_dtype == MA_PARAM_BF16, bg = a.grad_dtype == MA_PARAM_BF16;
    const bool vec = aligned16(a.dy) && a.n_out % 8 == 0 && a.dy_stride % (bd ? 8 : 4) == 0;
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_k * p.slices));
#define GO(TD, V, TG)                                                                           \
    hipLaunchKernelGGL((k_linear_grad<TD, V, TG>), grid, dim3(kThreads), 0, st, a, p.tiles_n,   \
                       p.tiles_k, p.slices, p.per)
#define GO_G(TD, V)                                                                             \
    do {                                                                                        \
        if (bg) GO(TD, V, __bf16);                                                              \
        else GO(TD, V, float);                                                                  \
    } while (0)
    if (bd) {
        if (vec) GO_G(__bf16, true); else GO_G(__bf16, false);
    } else {
        if (vec) GO_G(float, true); else GO_G(float, false);
    }
#undef GO_G
#undef GO
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.slices == 1) return (int)e;
    const int64_t n = a.n_out * a.n_in;
    const bool v8 = n % 8 == 0 && aligned16(a.grad);
    const int64_t units = v8 ? n / 8 : n;
    const dim3 jgrid((unsigned)ceil_div(units, kThreads));
#define GO(TG)                                                                                  \
    do {                                                                                        \
        if (v8)                                                                                 \
            hipLaunchKernelGGL((k_linear_join<TG, 8>), jgrid, dim3(kThreads), 0, st, a.partials, \
                               static_cast<TG*>(a.grad), units, p.slices, a.accumulate);        \
        else                                                                                    \
            hipLaunchKernelGGL((k_linear_join<TG, 1>), jgrid, dim3(kThreads), 0, st, a.partials, \
                               static_cast<TG*>(a.grad), units, p.slices, a.accumulate);        \
    } while (0)
    if (bg) GO(__bf16);
    else GO(float);
#undef GO
    return (int)hipGetLastError();
}

}  // namespace ma
