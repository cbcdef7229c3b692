// Attention over packed sequences with grouped heads, and its backward pass, on
// gfx950.
//
// Forward: a workgroup takes 32 query rows a wave of one head and walks the keys in
// tiles, copied into LDS one tile ahead.  Scores are formed transposed (keys by queries), so
// a lane holds one query's scores, the running maximum and sum of the softmax cost one
// exchange between the wave's halves, and the probabilities are the next product's
// operand where they are.
//
// Backward, without atomics: delta = sum(dout o) a row; one kernel over key tiles (dk, dv:
// a wave holds 32 keys and walks every query of the heads that share them) and one over
// query tiles (dq).  Both recompute the scores, seven products instead of five, and
// every sum has one owner and one order.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention_tile.h"

namespace ma {
namespace {

constexpr int kNt = 256;                 // threads: 4 waves of 32 rows
constexpr int kBlock = 128;              // query or key rows of a workgroup

// One workgroup's sequence, head and first row.
struct Job {
    int q_at, q_len, k_at, k_len, head, row0;
    bool any;
};
template <bool KEYS>
__device__ __forceinline__ Job job_of(const AttnArgs& a, int slots) {
    const int slot = blockIdx.x % slots;
    Job j;
    j.head = blockIdx.x / slots;
    const Place p = KEYS ? place_of(a.cu_k, a.n_seqs, a.n_keys, kBlock, slot)
                         : place_of(a.cu_q, a.n_seqs, a.n_queries, kBlock, slot);
    j.q_at = seq_at(a.cu_q, p.seq, a.n_seqs, a.n_queries);
    j.q_len = max(0, seq_at(a.cu_q, p.seq + 1, a.n_seqs, a.n_queries) - j.q_at);
    j.k_at = seq_at(a.cu_k, p.seq, a.n_seqs, a.n_keys);
    j.k_len = max(0, seq_at(a.cu_k, p.seq + 1, a.n_seqs, a.n_keys) - j.k_at);
    j.any = p.tile >= 0 && (int64_t)p.tile * kBlock < (KEYS ? j.k_len : j.q_len);
    j.row0 = j.any ? p.tile * kBlock : 0;
    return j;
}

template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const AttnArray& x, int head, int at, int len, int dim) {
    return {static_cast<const T*>(x.p) + (int64_t)at * x.token + (int64_t)head * x.head, x.token, len, dim};
}
template <typename T>
__device__ __forceinline__ T* row_of(const AttnArray& x, int head, int64_t row) {
    return static_cast<T*>(const_cast<void*>(x.p)) + row * x.token + (int64_t)head * x.head;
}

// Keys of a tile that query `q` sees: those before this one (counted from the tile's first).
__device__ __forceinline__ int seen(const AttnArgs& a, const Job& j, int q, int key0) {
    const int end = a.causal ? min(j.k_len, q + 1 + j.k_len - j.q_len) : j.k_len;
    return end - key0;
}

template <typename T, int DP, int KV, bool AL, int PER>
__global__ __launch_bounds__(kNt, PER) void k_attention_forward(AttnArgs a, int slots) {
    using KT = Tile<T, DP, KV, kNt>;
    __shared__ __attribute__((aligned(1024))) char lds[2][2][KT::kBytes];
    const Job j = job_of<false>(a, slots);
    if (!j.any) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
    const int kvh = j.head / (a.heads / a.kv_heads);
    const Rows<T> qx = rows_of<T>(a.q, j.head, j.q_at, j.q_len, a.dim);
    const Rows<T> kx = rows_of<T>(a.k, kvh, j.k_at, j.k_len, a.dim);
    const Rows<T> vx = rows_of<T>(a.v, kvh, j.k_at, j.k_len, a.dim);
    const int q = j.row0 + 32 * wave + (lane & 31);
    Frag<T> qf[DP / 16];
    load_row<T, DP, AL>(qx, q, qf);

    f32x16 o[DP / 32];
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) o[b] = zero16();
    float m = -kInf, l = 0.f;
    const float k = a.scale * kLog2e;
    // key tiles that some row of the workgroup sees
    const int last = min(j.row0 + kBlock, j.q_len) - 1;
    const int tiles = max(0, seen(a, j, last, 0) + KV - 1) / KV;
    if (tiles > 0) {
        KT::template copy<AL>(lds[0][0], kx, 0);
        KT::template copy<AL>(lds[0][1], vx, 0);
    }
    for (int t = 0; t < tiles; ++t) {
        copies_barrier();
        const char* kt = lds[t & 1][0];
        const char* vt = lds[t & 1][1];
        if (t + 1 < tiles) {
            KT::template copy<AL>(lds[(t + 1) & 1][0], kx, (t + 1) * KV);
            KT::template copy<AL>(lds[(t + 1) & 1][1], vx, (t + 1) * KV);
        }
        f32x16 s[KV / 32];
#pragma unroll
        for (int n = 0; n < KV / 32; ++n) {
            s[n] = zero16();
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) s[n] = mma(KT::rows(kt, 32 * n, d), qf[d], s[n]);
        }
        // what the rows of this wave do not all see
        const int sees = seen(a, j, q, t * KV);
        if (__any(sees < KV)) {
#pragma unroll
            for (int n = 0; n < KV / 32; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[n][i] = 32 * n + result_row(i, h) < sees ? s[n][i] : -kInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int n = 0; n < KV / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
        top = fmaxf(top, other_half(top));
        // The reference m follows the largest score only where that is 2^8 above it: a
        // probability of up to 2^8 is as exact, and most tiles then leave the sums alone.
        if (__any((top - m) * k > 8.f)) {
            const float to = fmaxf(m, top);
            const float c = to == -kInf ? 1.f : __builtin_amdgcn_exp2f((m - to) * k);
            m = to;
            l *= c;
#pragma unroll
            for (int b = 0; b < DP / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= c;
        }
        const float mk = m == -kInf ? 0.f : m * k;
#pragma unroll
        for (int n = 0; n < KV / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], k, -mk));
                l += s[n][i];
            }
#pragma unroll
        for (int n = 0; n < KV / 16; ++n) {
            const Frag<T> p = frag_of<T>(s[n / 2], n % 2);
#pragma unroll
            for (int b = 0; b < DP / 32; ++b) o[b] = mma(KT::cols(vt, 16 * n, 32 * b), p, o[b]);
        }
    }
    l += other_half(l);
    if (q >= j.q_len) return;
    const int64_t row = (int64_t)j.q_at + q;
    store_row<T, DP / 32>(row_of<T>(a.o, j.head, row), a.dim, o, l > 0.f ? 1.f / l : l == 0.f ? 0.f : l, AL);
    if (h == 0) a.lse[(int64_t)j.head * a.n_queries + row] = l == 0.f ? -kInf : fmaf(m, a.scale, logf(l));
}

// delta of a row: sum(dout o) over a head's features, 16 lanes a row.
template <typename T, bool AL>
__global__ __launch_bounds__(kNt) void k_attention_delta(AttnArgs a, int64_t rows) {
    const int64_t r = (int64_t)blockIdx.x * (kNt / 16) + threadIdx.x / 16;
    if (r >= rows) return;
    const int64_t t = r / a.heads;
    const int head = (int)(r - t * a.heads);
    const T* x = row_of<T>(a.dout, head, t);
    const T* y = row_of<T>(a.o, head, t);
    float s = 0.f;
    for (int c = 8 * (threadIdx.x & 15); c < a.dim; c += 128) {
        float u[8], v[8];
        load_unit<T, AL>(x + c, a.dim - c, u);
        load_unit<T, AL>(y + c, a.dim - c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(u[e], c + e < a.dim ? v[e] : 0.f, s);
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) s += __shfl_xor(s, m, 64);
    if ((threadIdx.x & 15) == 0) a.delta[(int64_t)head * a.n_queries + t] = s;
}

// lse in base 2 (infinity where a row sees nothing: its probabilities are then 0).
__device__ __forceinline__ float lse2(float lse) { return lse == -kInf ? kInf : lse * kLog2e; }

template <typename T, int DP, int KV, bool AL, int PER>
__global__ __launch_bounds__(kNt, PER) void k_attention_dq(AttnArgs a, int slots) {
    using KT = Tile<T, DP, KV, kNt>;
    __shared__ __attribute__((aligned(1024))) char lds[2][2][KT::kBytes];
    const Job j = job_of<false>(a, slots);
    if (!j.any) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
    const int kvh = j.head / (a.heads / a.kv_heads);
    const Rows<T> kx = rows_of<T>(a.k, kvh, j.k_at, j.k_len, a.dim);
    const Rows<T> vx = rows_of<T>(a.v, kvh, j.k_at, j.k_len, a.dim);
    const int q = j.row0 + 32 * wave + (lane & 31);
    Frag<T> qf[DP / 16], df[DP / 16];
    load_row<T, DP, AL>(rows_of<T>(a.q, j.head, j.q_at, j.q_len, a.dim), q, qf);
    load_row<T, DP, AL>(rows_of<T>(a.dout, j.head, j.q_at, j.q_len, a.dim), q, df);
    const int64_t at = (int64_t)j.head * a.n_queries + j.q_at + q;
    const float ls = q < j.q_len ? lse2(a.lse[at]) : kInf;
    const float delta = q < j.q_len ? a.delta[at] : 0.f;

    f32x16 dq[DP / 32];
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) dq[b] = zero16();
    const float k = a.scale * kLog2e;
    const int last = min(j.row0 + kBlock, j.q_len) - 1;
    const int tiles = max(0, seen(a, j, last, 0) + KV - 1) / KV;
    if (tiles > 0) {
        KT::template copy<AL>(lds[0][0], kx, 0);
        KT::template copy<AL>(lds[0][1], vx, 0);
    }
    for (int t = 0; t < tiles; ++t) {
        copies_barrier();
        const char* kt = lds[t & 1][0];
        const char* vt = lds[t & 1][1];
        if (t + 1 < tiles) {
            KT::template copy<AL>(lds[(t + 1) & 1][0], kx, (t + 1) * KV);
            KT::template copy<AL>(lds[(t + 1) & 1][1], vx, (t + 1) * KV);
        }
        const int sees = seen(a, j, q, t * KV);
        const bool part = __any(sees < KV);
#pragma unroll
        for (int n = 0; n < KV / 32; ++n) {
            f32x16 s = zero16(), p = zero16();
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                s = mma(KT::rows(kt, 32 * n, d), qf[d], s);
                p = mma(KT::rows(vt, 32 * n, d), df[d], p);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], k, -ls)) * (p[i] - delta);
            if (part)
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = 32 * n + result_row(i, h) < sees ? p[i] : 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const Frag<T> f = frag_of<T>(p, u);
#pragma unroll
                for (int b = 0; b < DP / 32; ++b) dq[b] = mma(KT::cols(kt, 32 * n + 16 * u, 32 * b), f, dq[b]);
            }
        }
    }
    if (q >= j.q_len) return;
    store_row<T, DP / 32>(row_of<T>(a.dq, j.head, (int64_t)j.q_at + q), a.dim, dq, a.scale, AL);
}

template <typename T, int DP, int QT, bool AL, int PER>
__global__ __launch_bounds__(kNt, PER) void k_attention_dkv(AttnArgs a, int slots) {
    using QTile = Tile<T, DP, QT, kNt>;
    __shared__ __attribute__((aligned(1024))) char lds[2][2][QTile::kBytes];
    __shared__ __attribute__((aligned(16))) float stat[2][2][QT];
    const Job j = job_of<true>(a, slots);        // (its head is a key head)
    if (!j.any) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
    const int group = a.heads / a.kv_heads;
    const int key = j.row0 + 32 * wave + (lane & 31);
    Frag<T> kf[DP / 16], vf[DP / 16];
    load_row<T, DP, AL>(rows_of<T>(a.k, j.head, j.k_at, j.k_len, a.dim), key, kf);
    load_row<T, DP, AL>(rows_of<T>(a.v, j.head, j.k_at, j.k_len, a.dim), key, vf);
    f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int b = 0; b < DP / 32; ++b) dk[b] = dv[b] = zero16();
    const float k = a.scale * kLog2e;
    // the first query that sees this workgroup's first key, and the tiles from its on
    const int off = j.k_len - j.q_len;
    const int first = a.causal ? max(0, j.row0 - off) / QT * QT : 0;
    const int per = first < j.q_len ? (j.q_len - first + QT - 1) / QT : 0, tiles = per * group;
    auto fetch = [&](int t) {
        const int head = j.head * group + t / per, q0 = first + t % per * QT, b = t & 1;
        QTile::template copy<AL>(lds[b][0], rows_of<T>(a.q, head, j.q_at, j.q_len, a.dim), q0);
        QTile::template copy<AL>(lds[b][1], rows_of<T>(a.dout, head, j.q_at, j.q_len, a.dim), q0);
        if (threadIdx.x < QT) {
            const int q = q0 + threadIdx.x;
            const int64_t at = (int64_t)head * a.n_queries + j.q_at + q;
            stat[b][0][threadIdx.x] = q < j.q_len ? lse2(a.lse[at]) : kInf;
            stat[b][1][threadIdx.x] = q < j.q_len ? a.delta[at] : 0.f;
        }
    };
    if (tiles > 0) fetch(0);
    for (int t = 0; t < tiles; ++t) {
        copies_barrier();
        const char* qt = lds[t & 1][0];
        const char* dt = lds[t & 1][1];
        const float* ls = stat[t & 1][0];
        const float* dl = stat[t & 1][1];
        if (t + 1 < tiles) fetch(t + 1);
        const int q0 = first + t % per * QT;
        // the first query of the tile that sees this lane's key
        const int from = a.causal ? key - off - q0 : 0;
        const bool part = __any(from > 0);
#pragma unroll
        for (int n = 0; n < QT / 32; ++n) {
            f32x16 s = zero16(), p = zero16();
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                s = mma(QTile::rows(qt, 32 * n, d), kf[d], s);
                p = mma(QTile::rows(dt, 32 * n, d), vf[d], p);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 l4 = *reinterpret_cast<const f32x4*>(ls + 32 * n + 8 * g + 4 * h);
                const f32x4 d4 = *reinterpret_cast<const f32x4*>(dl + 32 * n + 8 * g + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * g + e;
                    s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], k, -l4[e]));
                    p[i] = s[i] * (p[i] - d4[e]);
                }
            }
            if (part)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool in = 32 * n + result_row(i, h) >= from;
                    s[i] = in ? s[i] : 0.f;
                    p[i] = in ? p[i] : 0.f;
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const Frag<T> fs = frag_of<T>(s, u), fp = frag_of<T>(p, u);
#pragma unroll
                for (int b = 0; b < DP / 32; ++b) {
                    dv[b] = mma(QTile::cols(dt, 32 * n + 16 * u, 32 * b), fs, dv[b]);
                    dk[b] = mma(QTile::cols(qt, 32 * n + 16 * u, 32 * b), fp, dk[b]);
                }
            }
        }
    }
    if (key >= j.k_len) return;
    const int64_t row = (int64_t)j.k_at + key;
    store_row<T, DP / 32>(row_of<T>(a.dk, j.head, row), a.dim, dk, a.scale, AL);
    store_row<T, DP / 32>(row_of<T>(a.dv, j.head, row), a.dim, dv, 1.f, AL);
}

// Whole 16-byte chunks: what copies into LDS and wide stores need.
bool al_heads(const AttnArray& x, int32_t dim, int32_t dtype) {
    const int64_t per = dtype == MA_PARAM_BF16 ? 8 : 4;
    // (a copy's offsets within a tile of 64 rows stay below 2^31 bytes)
    return (reinterpret_cast<uintptr_t>(x.p) & 15) == 0 && x.token % per == 0 && x.head % per == 0 && dim % 8 == 0 &&
           x.token <= (int64_t(1) << 22);
}

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f(T{}, padded dim, aligned).
template <typename F>
int by_kind(const AttnArgs& a, bool al, F f) {
    auto dims = [&](auto t) {
        auto go = [&](auto dp) {
            if (al) f(t, dp, std::true_type{});
            else f(t, dp, std::false_type{});
        };
        if (a.dim <= 64) go(Int<64>{});
        else if (a.dim <= 128) go(Int<128>{});
        else go(Int<256>{});
    };
    if (a.dtype == MA_PARAM_BF16) dims(__bf16{});
    else dims(float{});
    return (int)hipGetLastError();
}

int slots_of(int64_t total, int32_t n_seqs) { return (int)(total / kBlock + n_seqs); }

}  // namespace

int launch_attention_forward(const AttnArgs& a, void* stream) {
    if (a.n_queries == 0 || a.n_seqs == 0) return (int)hipSuccess;
    const bool al = al_heads(a.q, a.dim, a.dtype) && al_heads(a.k, a.dim, a.dtype) && al_heads(a.v, a.dim, a.dtype) &&
                    al_heads(a.o, a.dim, a.dtype);
    const int slots = slots_of(a.n_queries, a.n_seqs);
    return by_kind(a, al, [&](auto t, auto dp, auto w) {
        using T = decltype(t);
        constexpr int DP = decltype(dp)::value;
        // two key tiles of K and V in LDS, two workgroups a CU where registers allow
        constexpr int KV = sizeof(T) == 2 ? 64 : 32;
        constexpr int PER = DP * (int)sizeof(T) <= 256 ? 2 : 1;
        hipLaunchKernelGGL((k_attention_forward<T, DP, KV, decltype(w)::value, PER>), dim3((unsigned)(slots * a.heads)),
                           dim3(kNt), 0, (hipStream_t)stream, a, slots);
    });
}

int launch_attention_backward(const AttnArgs& a, void* stream) {
    const bool al = al_heads(a.q, a.dim, a.dtype) && al_heads(a.k, a.dim, a.dtype) && al_heads(a.v, a.dim, a.dtype) &&
                    al_heads(a.o, a.dim, a.dtype) && al_heads(a.dout, a.dim, a.dtype) &&
                    al_heads(a.dq, a.dim, a.dtype) && al_heads(a.dk, a.dim, a.dtype) && al_heads(a.dv, a.dim, a.dtype);
    if (a.n_seqs == 0) return (int)hipSuccess;
    const int64_t rows = a.n_queries * a.heads;
    if (rows > 0) {
        const int rc = by_kind(a, al, [&](auto t, auto dp, auto w) {
            using T = decltype(t);
            constexpr bool AL = decltype(w)::value;
            constexpr int DP = decltype(dp)::value;
            hipLaunchKernelGGL((k_attention_delta<T, AL>), dim3((unsigned)ceil_div(rows, kNt / 16)), dim3(kNt), 0,
                               (hipStream_t)stream, a, rows);
            constexpr int KV = sizeof(T) == 2 ? 64 : 32;
            const int slots = slots_of(a.n_queries, a.n_seqs);
            hipLaunchKernelGGL((k_attention_dq<T, DP, KV, AL, 1>), dim3((unsigned)(slots * a.heads)), dim3(kNt), 0,
                               (hipStream_t)stream, a, slots);
        });
        if (rc != (int)hipSuccess) return rc;
    }
    if (a.n_keys == 0) return (int)hipSuccess;
    return by_kind(a, al, [&](auto t, auto dp, auto w) {
        using T = decltype(t);
        constexpr int DP = decltype(dp)::value;
        constexpr int QT = sizeof(T) == 2 ? 64 : 32;
        const int slots = slots_of(a.n_keys, a.n_seqs);
        hipLaunchKernelGGL((k_attention_dkv<T, DP, QT, decltype(w)::value, 1>), dim3((unsigned)(slots * a.kv_heads)),
                           dim3(kNt), 0, (hipStream_t)stream, a, slots);
    });
}

}  // namespace ma
