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
//
// Few rows do not fill the GPU: each row block's walk is then cut into pieces, whose float32
// results a last launch joins in order.  This file has the forward kernel, what is before and
// behind the others, and the rules for pieces.
//
// 20011 tokens of 7 sequences, 16 / 4 heads of 128, bf16: forward 251 GFLOP in 290 to 325 us (0.77 to
// 0.86 PFLOP/s; a library product of 8192 x 8192 matrices reaches 1.2 to 1.4).  Bound by matrix and vector
// work that hardly overlap: 48 and 44 % of a SIMD's cycles.  A tile of 32 queries and 64 keys is 32
// matrix instructions of 32 cycles a wave, and (masked tiles and the prologue shared out) some 205
// vector ones for the maximum, exponential, sum and rounding of 2048 scores, of whose time the
// exponentials, of 8 cycles each, take 28 %.  The next tile's scores formed step by step between this
// one's exponentials: 318 -> 328 us.  One sequence of 14336 tokens with 8 heads: 0.95 to 1.0
// PFLOP/s.  Backward (dq, dkv and what is around them) 627 GFLOP counted as five products,
// seven done, in 1.0 to 1.06 ms.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention_tile.h"

namespace ma {
namespace {

constexpr float kFine = 0x1p24f;         // a product below it is rounded by at most 1 / 2

template <typename T, int DP, int KV, int WAVES>
__global__ __launch_bounds__(64 * WAVES * kHalves<DP>, (kPer<T, DP>)) void k_attention_forward(AttnArgs a,
                                                                                            AttnGrid grid) {
    constexpr int BLOCK = 32 * WAVES, HALVES = kHalves<DP>, DW = DP / HALVES;
    using KT = Tile<T, DP, KV, 64 * WAVES * HALVES>;
    __shared__ __attribute__((aligned(1024))) char lds[2][2][KT::kBytes];
    __shared__ Exchange<HALVES == 2 ? 2 * WAVES : 0> exchange;
    const Job j = job_of<false, BLOCK>(a, grid);
    if (!j.any) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
    const int half = __builtin_amdgcn_readfirstlane(wave % HALVES);
    const int kvh = j.head / (a.heads / a.kv_heads);
    const Rows<T> qx = rows_of<T>(a.q, j.head, j.q_at, j.q_len, a.cols);
    const Rows<T> kx = rows_of<T>(a.k, kvh, j.k_at, j.k_len, a.cols);
    const Rows<T> vx = rows_of<T>(a.v, kvh, j.k_at, j.k_len, a.cols);
    const int q = j.row0 + 32 * (wave / HALVES) + (lane & 31);
    Frag<T> qf[DW / 16];
    load_row<T, DW / 16>(qx, q, half * (DW / 16), qf);

    f32x16 o[DW / 32];
#pragma unroll
    for (int b = 0; b < DW / 32; ++b) o[b] = zero16();
    // The running maximum, m k as it is taken off the scores, and the sum.  Lanes whose m k is too coarse once
    // rounded (from 2^31 on the rounding alone leaves the range of 2^x) take m off first.
    float m = -kInf, mk = 0.f, l = 0.f;
    uint64_t coarse = 0;
    const float k = a.scale * kLog2e;
    // key tiles that some row of the workgroup sees
    const int end = min(j.row0 + BLOCK, j.q_len) - 1;
    const Share sh(max(0, seen(a, j, end) + KV - 1) / KV, j.piece, grid.pieces);
    const typename KT::Copy copy_k(kx), copy_v(vx);
    if (sh.first < sh.last) {
        copy_k(lds[0][0], kx, sh.first * KV);
        copy_v(lds[0][1], vx, sh.first * KV);
    }
    const int sees = seen(a, j, q);
    // One tile; PART: some row of the workgroup does not see all of it.  (Two bodies: as a
    // condition the masks would be computed for every tile.)
    auto tile = [&](int t, auto slot, auto part) {
        copies_barrier<0>();
        constexpr int AT = decltype(slot)::value;
        const char* kt = lds[AT][0];
        const char* vt = lds[AT][1];
        if (t + 1 < sh.last) {
            copy_k(lds[AT ^ 1][0], kx, (t + 1) * KV);
            copy_v(lds[AT ^ 1][1], vx, (t + 1) * KV);
        }
        f32x16 s[KV / 32];
        constexpr int ND = DW / 16, NB = DW / 32;
#pragma unroll
        for (int n = 0; n < KV / 32; ++n) s[n] = zero16();
        read_ahead<KV / 32 * ND, kAhead<T>>(
            [&](int i) { return KT::rows(kt, 32 * (i / ND), half * ND + i % ND); },
            [&](int i, const Frag<T>& f) { s[i / ND] = mma(f, qf[i % ND], s[i / ND]); });
        if constexpr (HALVES == 2) {         // (the sums over either half of the features)
            static_assert(KV == 32, "one exchange a tile");
            s[0] += exchange(s[0]);
        }
        if constexpr (decltype(part)::value) {
#pragma unroll
            for (int n = 0; n < KV / 32; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[n][i] = t * KV + 32 * n + result_row(i, h) < sees ? s[n][i] : -kInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int n = 0; n < KV / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
        top = fmaxf(top, other_half(top));
        // The reference m follows the largest score only where that is 2^8 above it: a
        // probability of up to 2^8 is as exact, and most tiles then leave the sums alone.
        if (__ballot((top - m) * k > 8.f) | coarse) {
            const float to = fmaxf(m, top);
            const float c = to == -kInf ? 1.f : __builtin_amdgcn_exp2f((m - to) * k);
            m = to;
            mk = m == -kInf ? 0.f : m * k;
            l *= c;
#pragma unroll
            for (int b = 0; b < DW / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= c;
            const bool far = fabsf(mk) >= kFine;
            coarse = __ballot(far);
            if (coarse) {
#pragma unroll
                for (int n = 0; n < KV / 32; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[n][i] -= far ? m : 0.f;
                mk = far ? 0.f : mk;
            }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < KV / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], k, -mk));
                sum[i & 3] += s[n][i];
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        Frag<T> p[KV / 16];
#pragma unroll
        for (int n = 0; n < KV / 16; ++n) p[n] = frag_of<T>(s[n / 2], n % 2);
        read_ahead<KV / 16 * NB, kAhead<T>>(
            [&](int i) { return KT::cols(vt, 16 * (i / NB), half * DW + 32 * (i % NB)); },
            [&](int i, const Frag<T>& f) { o[i % NB] = mma(f, p[i / NB], o[i % NB]); });
    };
    const int whole = min(max(seen(a, j, j.row0), 0) / KV, sh.last);
    // Two tiles a turn: with LDS slots as constants addresses differ by constants too, which reads
    // hold themselves (28 additions a tile less: 323 -> 313 us).
    int t = sh.first;
    for (; t + 1 < whole; t += 2) {
        tile(t, Int<0>{}, std::false_type{});
        tile(t + 1, Int<1>{}, std::false_type{});
    }
    for (; t < sh.last; t += 2) {
        tile(t, Int<0>{}, std::true_type{});
        if (t + 1 < sh.last) tile(t + 1, Int<1>{}, std::true_type{});
    }
    l += other_half(l);
    if (q >= j.q_len) return;
    const int64_t row = (int64_t)j.q_at + q;
    const bool lead = h == 0 && half == 0;
    if (grid.pieces > 1) {
        store_row<float, DW / 32>(part_row(a.parts, j.piece, a.heads, j.head, a.n_queries, row, a.dim), a.dim,
                                  half * DW, o, 1.f, a.dim % 4 == 0);
        if (lead) {
            float* s = a.stats + (((int64_t)j.piece * a.heads + j.head) * a.n_queries + row) * 2;
            s[0] = m;
            s[1] = l;
        }
        return;
    }
    store_row<T, DW / 32>(row_of<T>(a.o, j.head, row), a.dim, half * DW, o, l > 0.f ? 1.f / l : l == 0.f ? 0.f : l,
                         a.wide);
    if (lead) a.lse[(int64_t)j.head * a.n_queries + row] = l == 0.f ? -kInf : fmaf(m, a.scale, logf(l));
}

// What a launch that joins pieces walks: rows inside sequences x heads, 64 threads a row.
struct JoinRow {
    int64_t row;
    int head;
    bool in;
};
__device__ __forceinline__ JoinRow join_row(const int32_t* cu, int n_seqs, int64_t total, int heads) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    JoinRow j;
    j.row = r / heads;
    j.head = (int)(r - j.row * heads);
    j.in = j.row < total && j.row >= seq_at(cu, 0, n_seqs, total) && j.row < seq_at(cu, n_seqs, n_seqs, total);
    return j;
}

// put(c, v) for every column c of a row, v = add(p, x, v) over its pieces' x in order: four
// columns a lane where they are whole 16-byte chunks.
template <typename A, typename P>
__device__ __forceinline__ void each_column(int dim, const float* x, int pieces, int64_t step, A add, P put) {
    const int lane = threadIdx.x & 63;
    if (dim % 4 == 0) {
        const int c = 4 * lane;          // (a head has at most 256)
        const float* y = x + min(c, dim - 4);
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int p = 0; p < pieces; ++p) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(y + p * step);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = add(p, w[e], v[e]);
        }
        if (c < dim)
#pragma unroll
            for (int e = 0; e < 4; ++e) put(c + e, v[e]);
    } else {
        for (int c0 = 0; c0 < dim; c0 += 64) {
            const float* y = x + min(c0 + lane, dim - 1);
            float v = 0.f;
#pragma unroll 8
            for (int p = 0; p < pieces; ++p) v = add(p, y[p * step], v);
            if (c0 + lane < dim) put(c0 + lane, v);
        }
    }
}

// o and lse of a row from its pieces' sums: as one running softmax would have joined them.
// Lane p holds what piece p (of at most 64) brings; every piece is added in its order.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_join(AttnArgs a, int pieces) {
    const JoinRow j = join_row(a.cu_q, a.n_seqs, a.n_queries, a.heads);
    if (!j.in) return;
    const int lane = threadIdx.x & 63;
    const float k = a.scale * kLog2e;
    const int64_t step = (int64_t)a.heads * a.n_queries, at = (int64_t)j.head * a.n_queries + j.row;
    const float* s = a.stats + (lane * step + at) * 2;
    const float mp = lane < pieces ? s[0] : -kInf, lp = lane < pieces ? s[1] : 0.f;
    float m = mp;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    // (a piece whose keys are all hidden has m = -infinity and sums of 0)
    const float w = mp == -kInf ? 0.f : __builtin_amdgcn_exp2f((mp - m) * k);
    float l = mp == -kInf ? lp : w * lp;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x, 64);
    const float r = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    T* o = row_of<T>(a.o, j.head, j.row);
    each_column(a.dim, a.parts + at * a.dim, pieces, step * a.dim, [&](int p, float x, float v) {
        const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), p));
        return u == 0.f ? v : fmaf(u, x, v);
    }, [&](int c, float v) { o[c] = (T)(v * r); });
    if (lane == 0) a.lse[at] = l == 0.f ? -kInf : fmaf(m, a.scale, logf(l));
}

// The sum of a row's pieces: dq, or dk and dv.
template <typename T, bool KEYS>
__global__ __launch_bounds__(256) void k_attention_sum(AttnArgs a, int pieces) {
    const int heads = KEYS ? a.kv_heads : a.heads;
    const int64_t rows = KEYS ? a.n_keys : a.n_queries;
    const JoinRow j = join_row(KEYS ? a.cu_k : a.cu_q, a.n_seqs, rows, heads);
    if (!j.in) return;
    const int64_t step = (int64_t)heads * rows * a.dim, at = ((int64_t)j.head * rows + j.row) * a.dim;
    auto add = [](int, float x, float v) { return v + x; };
    if (KEYS) {
        T* dk = row_of<T>(a.dk, j.head, j.row);
        T* dv = row_of<T>(a.dv, j.head, j.row);
        each_column(a.dim, a.parts + at, pieces, step, add, [&](int c, float v) { dk[c] = (T)v; });
        each_column(a.dim, a.parts + pieces * step + at, pieces, step, add, [&](int c, float v) { dv[c] = (T)v; });
    } else {
        T* dq = row_of<T>(a.dq, j.head, j.row);
        each_column(a.dim, a.parts + at, pieces, step, add, [&](int c, float v) { dq[c] = (T)v; });
    }
}

// What a row brings to the backward pass: lse in base 2 (infinity where it sees nothing: its
// probabilities are then 0) and delta = sum(dout o) over a head's features, 16 lanes a row.
template <typename T, bool AL>
__global__ __launch_bounds__(256) void k_attention_delta(AttnArgs a, int64_t rows) {
    for (int64_t r = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; r < rows; r += (int64_t)gridDim.x * 16) {
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
        if ((threadIdx.x & 15) == 0) {
            const float lse = a.lse[(int64_t)head * a.n_queries + t];
            float* o = a.stats + ((int64_t)head * a.n_queries + t) * 2;
            o[0] = lse == -kInf ? kInf : lse * kLog2e;
            o[1] = s;
        }
    }
}

}  // namespace

// Rows of a workgroup, and pieces of its walk, for `rows` rows of n_seqs sequences and `heads`
// heads against `walk` rows of the other side.
//
// Pieces: as many as fill the GPU, which runs `at_once` workgroups; each has at least 128 rows
// to walk, in float32, whose products take 16 times as long, 32.  More cost their joining:
// twice as many for causal queries would make 102 us of 60 (10000 tokens of 7 sequences, 8 heads
// of 128, bf16), 75 of 32 (of 40 sequences), 292 of 258 (10700 of one).  Twice as many, since the
// longest walk of a causal call is twice the mean one or, of sequences with lengths unlike, more,
// pay in float32 (4000 tokens of 3 sequences, 8 / 2 heads of 128, backward: 787 us without,
// 567) and for key blocks, each of which walks every query of its group, where a piece keeps
// 2048 rows (20011 tokens of 7 sequences, 16 / 4 heads, backward: of 64 features 727 us without,
// 609; of 128 1097 and 1030; 16000 of 2 with 8 / 1 heads 1228 and 1074), but not for one
// sequence that fills the GPU (10700 tokens: 855 without, 887).
static AttnSplit split_of(const AttnArgs& a, int64_t rows, int64_t walk, int64_t heads, int most, bool halve,
                          int at_once, bool keys) {
    AttnSplit s;
    if (rows == 0 || a.n_seqs == 0) return s;
    const int64_t each = ceil_div(rows, a.n_seqs), seen = ceil_div(walk, a.n_seqs);
    s.rows = halve && each <= most / 2 ? most / 2 : most;
    const int64_t blocks = ceil_div(each, s.rows) * a.n_seqs * heads;
    const bool wide = a.dtype == MA_PARAM_FP32;
    int64_t n = std::min(at_once / blocks, ceil_div(seen, wide ? 32 : 128));
    if (a.causal && (wide || (keys && (blocks < at_once || a.n_seqs > 1))))
        n = std::max(n, std::min(ceil_div(2 * at_once, blocks), seen / (wide ? 128 : 2048)));
    s.pieces = (int32_t)std::max<int64_t>(1, std::min<int64_t>(n, 32));
    return s;
}
// Workgroups of 4 waves (8 for the keys of 256 bfloat16 features): two on a CU where a lane
// has 256 registers.  Where sequences have no more than half a workgroup's rows it takes half
// as many (400 sequences of 50, 16 / 4 heads, backward: 267 us, 311 without), in the forward pass
// only where its LDS lets a CU run twice as many (float32 of 128 features 83 us, 130 without, but
// bfloat16 of 128 188 and 155, float32 of 256 139 and 116).
AttnSplit attention_query_split(const AttnArgs& a, bool back) {
    const bool bf16 = a.dtype == MA_PARAM_BF16;
    return split_of(a, a.n_queries, a.n_keys, a.heads, a.dim > 128 ? 64 : 128, back || a.dim <= (bf16 ? 64 : 128),
                    kCus * (bf16 || a.dim <= 64 ? 2 : 1), false);
}
AttnSplit attention_key_split(const AttnArgs& a) {
    const bool bf16 = a.dtype == MA_PARAM_BF16;
    return split_of(a, a.n_keys, a.n_queries * (a.heads / a.kv_heads), a.kv_heads, a.dim > 128 && !bf16 ? 64 : 128,
                    true, kCus * (a.dim <= (bf16 ? 128 : 64) ? 2 : 1), true);
}

// Workgroups of 256 threads for n of them, in rounds where a launch does not hold so many.
static unsigned capped(int64_t n) { return (unsigned)std::min<int64_t>(n, int64_t(1) << 22); }

static unsigned join_grid(int64_t rows, int64_t heads) { return (unsigned)ceil_div(rows * heads, 4); }

// The inputs that have no aligned rows of whole chunks (every one where dim is not a multiple of
// 8), and where their copies lie in the workspace.
AttnPack attention_pack(const AttnArgs& a, bool back) {
    AttnPack p;
    const int64_t cols = round_up(a.dim, 8), size = a.dtype == MA_PARAM_BF16 ? 2 : 4;
    const AttnArray* in[] = {&a.q, &a.k, &a.v, &a.dout};
    for (int i = 0; i < (back ? 4 : 3); ++i) {
        const bool keys = i == 1 || i == 2;
        if (al_heads(*in[i], a.dim, a.dtype)) continue;
        p.copied[i] = true;
        p.at[i] = p.total;
        p.total += round_up((keys ? a.n_keys * a.kv_heads : a.n_queries * a.heads) * cols * size, 256);
    }
    return p;
}

// Rows (token, head) of x as rows of `cols` columns, zeros past dim: 16 bytes a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_pack(AttnArray x, T* out, int64_t rows, int heads, int dim, int cols) {
    constexpr int kPer = 16 / (int)sizeof(T);
    const int per_row = cols / kPer;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per_row; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per_row;
        const int c = (int)(i - r * per_row) * kPer;
        const int64_t t = r / heads;
        const T* p = row_of<T>(x, (int)(r - t * heads), t);
        T v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const T w = p[min(c + e, dim - 1)];
            v[e] = c + e < dim ? w : (T)0.f;
        }
        *reinterpret_cast<u32x4*>(out + i * kPer) = __builtin_bit_cast(u32x4, v);
    }
}

// The call's inputs with aligned rows.
static int pack_inputs(AttnArgs& g, bool back, void* stream) {
    const AttnPack p = attention_pack(g, back);
    g.cols = g.dim;
    if (p.total == 0) return (int)hipSuccess;
    const int cols = (int)round_up(g.dim, 8);
    AttnArray* in[] = {&g.q, &g.k, &g.v, &g.dout};
    for (int i = 0; i < 4; ++i) {
        const int heads = i == 1 || i == 2 ? g.kv_heads : g.heads;
        const int64_t rows = heads * (i == 1 || i == 2 ? g.n_keys : g.n_queries);
        if (!p.copied[i]) continue;
        char* out = g.packed + p.at[i];
        auto go = [&](auto t) {
            using T = decltype(t);
            const int64_t n = rows * (cols * (int64_t)sizeof(T) / 16);
            if (n > 0)
                hipLaunchKernelGGL((k_attention_pack<T>), dim3(capped(ceil_div(n, 256))), dim3(256), 0,
                                   (hipStream_t)stream, *in[i], reinterpret_cast<T*>(out), rows, heads, g.dim, cols);
        };
        if (g.dtype == MA_PARAM_BF16) go(__bf16{});
        else go(float{});
        *in[i] = {out, (int64_t)heads * cols, cols};
    }
    g.cols = cols;
    return (int)hipGetLastError();
}

int launch_attention_forward(const AttnArgs& a, void* stream) {
    if (a.n_queries == 0 || a.n_seqs == 0) return (int)hipSuccess;
    AttnArgs g = a;
    g.wide = al_heads(a.o, a.dim, a.dtype);
    int rc = pack_inputs(g, false, stream);
    if (rc != (int)hipSuccess) return rc;
    const AttnSplit sp = attention_query_split(a, false);
    const AttnGrid grid = grid_of(a.n_queries, a.n_seqs, a.heads, sp.rows, sp.pieces);
    rc = by_kind(a, sp.rows, [&](auto t, auto dp, auto wv) {
        using T = decltype(t);
        constexpr int DP = decltype(dp)::value, WAVES = decltype(wv)::value;
        constexpr int KV = sizeof(T) == 2 && kHalves<DP> == 1 ? 64 : 32;
        // (workgroups of 4 waves, or of 2 where the rule above halves them)
        constexpr bool HALVE = DP <= (sizeof(T) == 2 ? 64 : 128);
        if constexpr (WAVES * kHalves<DP> == 4 || (HALVE && WAVES == 2))
            hipLaunchKernelGGL((k_attention_forward<T, DP, KV, WAVES>),
                               dim3((unsigned)grid.slots * a.heads * grid.pieces), dim3(64 * WAVES * kHalves<DP>), 0,
                               (hipStream_t)stream, g, grid);
    });
    if (rc != (int)hipSuccess || sp.pieces == 1) return rc;
    const dim3 rows(join_grid(a.n_queries, a.heads)), block(256);
    if (a.dtype == MA_PARAM_BF16)
        hipLaunchKernelGGL(k_attention_join<__bf16>, rows, block, 0, (hipStream_t)stream, a, sp.pieces);
    else
        hipLaunchKernelGGL(k_attention_join<float>, rows, block, 0, (hipStream_t)stream, a, sp.pieces);
    return (int)hipGetLastError();
}

int launch_attention_backward(const AttnArgs& a, void* stream) {
    if (a.n_seqs == 0) return (int)hipSuccess;
    AttnArgs g = a;
    g.wide = al_heads(a.dq, a.dim, a.dtype) && al_heads(a.dk, a.dim, a.dtype) && al_heads(a.dv, a.dim, a.dtype);
    const bool al = al_heads(a.o, a.dim, a.dtype) && al_heads(a.dout, a.dim, a.dtype);
    int rc = pack_inputs(g, true, stream);
    if (rc != (int)hipSuccess) return rc;
    // a sum of pieces: the partial sums of dq, then those of dk and dv, take the same space
    auto join = [&](auto keys, int pieces) {
        constexpr bool KEYS = decltype(keys)::value;
        const dim3 grid(KEYS ? join_grid(a.n_keys, a.kv_heads) : join_grid(a.n_queries, a.heads)), block(256);
        if (a.dtype == MA_PARAM_BF16)
            hipLaunchKernelGGL((k_attention_sum<__bf16, KEYS>), grid, block, 0, (hipStream_t)stream, a, pieces);
        else
            hipLaunchKernelGGL((k_attention_sum<float, KEYS>), grid, block, 0, (hipStream_t)stream, a, pieces);
        return (int)hipGetLastError();
    };
    const int64_t rows = a.n_queries * a.heads;
    if (rows > 0) {
        const dim3 grid(capped(ceil_div(rows, 16))), block(256);
        auto delta = [&](auto t) {
            if (al) hipLaunchKernelGGL((k_attention_delta<decltype(t), true>), grid, block, 0, (hipStream_t)stream, a, rows);
            else hipLaunchKernelGGL((k_attention_delta<decltype(t), false>), grid, block, 0, (hipStream_t)stream, a, rows);
        };
        if (a.dtype == MA_PARAM_BF16) delta(__bf16{});
        else delta(float{});
        rc = (int)hipGetLastError();
        const AttnSplit sp = attention_query_split(a, true);
        if (rc == (int)hipSuccess) rc = launch_attention_dq(g, sp, stream);
        if (rc == (int)hipSuccess && sp.pieces > 1) rc = join(std::false_type{}, sp.pieces);
        if (rc != (int)hipSuccess) return rc;
    }
    if (a.n_keys == 0) return (int)hipSuccess;
    const AttnSplit sp = attention_key_split(a);
    rc = launch_attention_dkv(g, sp, stream);
    if (rc == (int)hipSuccess && sp.pieces > 1) return join(std::true_type{}, sp.pieces);
    return rc;
}

}  // namespace ma
