// What the attention kernels share: operand fragments of the 32 x 32 matrix
// instructions, tiles of rows in LDS, and which packed sequence a workgroup works on.
//
// Every product is a sum of 32 x 32 x 16 steps.  A lane (column or row l = lane % 32, half
// h = lane / 32) holds 8 elements of an operand; the step's reduction index of
// element j is one of two orders, the same for both operands:
//   straight   8 h + j                       rows of a tile, 16 bytes of a row
//   crossed    8 (j / 4) + 4 h + j % 4       columns of a tile, and what a result holds:
//              a lane's 16 results of a 32 x 32 product are column l, rows 8 (i / 4) + 4 h
//              + i % 4, so its results 8 s .. 8 s + 7 are step s's operand as they are
// So scores and their gradients go from one product into the next in registers.
// bfloat16 steps are one v_mfma_f32_32x32x16_bf16, float32 steps 8 v_mfma_f32_32x32x2_f32
// (element j of both halves each).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "grads_device.h"
#include "layers_internal.h"
#include "lds_copy.h"

namespace ma {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_inff();

template <typename T>
using Frag = std::conditional_t<sizeof(T) == 2, bf16x8, f32x8>;

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ f32x16 zero16() {
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    return v;
}

// Results 8 s .. 8 s + 7 as an operand.
template <typename T>
__device__ __forceinline__ Frag<T> frag_of(const f32x16& v, int s) {
    Frag<T> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (T)v[8 * s + j];
    return f;
}

// The row of a result's element i, and the first of the four rows of its group i / 4.
__device__ __forceinline__ int result_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// All but the last N of this wave's copies have landed, its LDS accesses are done, and so
// is every wave's.  (A release fence would wait for all copies; the empty statement keeps the
// compiler from moving LDS accesses over the wait, which it takes for no access to memory.)
template <int N>
__device__ __forceinline__ void copies_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4 << 14));      // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    __builtin_amdgcn_sched_barrier(0);
}

// The same for LDS alone: copies may still be under way.
__device__ __forceinline__ void lds_barrier() { copies_barrier<63>(); }

// One head of a packed array, as the rows of one sequence: whole 16-byte chunks at
// 16-byte addresses (other inputs are copied into such rows first).
template <typename T>
struct Rows {
    const T* p;          // the sequence's first row
    int64_t stride;      // elements from row to row
    int len, dim;
};

// A tile of ROWS rows of DP columns (the head's, padded with zeros) in LDS, NT threads' work.
// A row's 16-byte chunk c lies at slot c ^ turn(row): chosen so that the 16 rows at one
// chunk that straight reads take at a time, and the 4 rows by 64 bytes of a crossed read, lie
// in different banks.
template <typename T, int DP, int ROWS, int NT>
struct Tile {
    static constexpr int kRow = DP * (int)sizeof(T);
    static constexpr int kBytes = ROWS * kRow;
    static constexpr int kChunks = kRow / 16;
    static constexpr int kCopies = kBytes / (NT * 16);       // 16-byte copies a thread
    static_assert(kBytes % (NT * 16) == 0 && ROWS % 16 == 0, "whole copies");

    __device__ static __forceinline__ int turn(int row) {
        if constexpr (kChunks >= 16) return (row & 3) << 2 | (row >> 2 & 3);
        else return (row >> 1 & 1) << 2 | (row >> 2 & 3);
    }

    // Copies of rows of one array into LDS by all threads, which have landed after copies_barrier.
    struct Copy {
        uint32_t from[kCopies];          // byte offset of this thread's chunk; past any extent where there is none
        __device__ __forceinline__ explicit Copy(const Rows<T>& x) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int s = i * NT + (int)threadIdx.x, row = s / kChunks;
                const int col = ((s % kChunks) ^ turn(row)) * (16 / (int)sizeof(T));
                from[i] = col < x.dim ? (uint32_t)row * (uint32_t)(x.stride * sizeof(T)) + (uint32_t)(col * sizeof(T))
                                      : 0x80000000u;
            }
        }
        // Rows [row0, row0 + ROWS) of x into `lds`; rows past x.len and columns past x.dim become
        // zeros.
        __device__ __forceinline__ void operator()(char* lds, const Rows<T>& x, int row0) const {
            const int left = min(x.len - row0, ROWS);
            const u32x4 rsrc = make_rsrc(x.p + (int64_t)row0 * x.stride,
                                         left > 0 ? ((int64_t)(left - 1) * x.stride + x.dim) * (int64_t)sizeof(T) : 0);
            const uint32_t at = lds_addr(lds) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024u;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) dma16(rsrc, at + (uint32_t)(i * NT * 16), from[i]);
        }
    };

    // Straight operand: row row0 + l (row0 a multiple of 32), columns 16 step + 8 h + j.
    __device__ static __forceinline__ Frag<T> rows(const char* lds, int row0, int step) {
        const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5, x = turn(l & 15);
        const char* p = lds + (row0 + l) * kRow;
        if constexpr (sizeof(T) == 2) {
            return __builtin_bit_cast(Frag<T>, *reinterpret_cast<const u32x4*>(p + (((h ^ x) * 16) ^ (step * 32))));
        } else {
            const int c = 4 * step + 2 * h;
            const f32x4 a = *reinterpret_cast<const f32x4*>(p + ((c ^ x) * 16));
            const f32x4 b = *reinterpret_cast<const f32x4*>(p + (((c + 1) ^ x) * 16));
            return {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        }
    }

    // Crossed operand: column col0 + l (col0 a multiple of 32), rows row0 + crossed order
    // (row0 a multiple of 16).
    __device__ static __forceinline__ Frag<T> cols(const char* lds, int row0, int col0) {
        const int lane = threadIdx.x & 63, h = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            // ds_read_b64_tr_b16: within 16 lanes, lane i receives element i % 4 of the 8-byte
            // pieces that lanes i / 4 + 4 e point at: four rows by 16 columns, a column a lane
            const int g = lane >> 4, a = lane & 15, row = 4 * h + (a >> 2);
            const int c = 2 * (g & 1) + ((a & 3) >> 1);
            const int at = (row0 + row) * kRow + (((c ^ turn(row)) * 16) ^ (col0 * 2)) + 8 * (a & 1);
            const u32x2 lo = tr(lds + at), hi = tr(lds + ((at + 8 * kRow) ^ 32));
            return __builtin_bit_cast(Frag<T>, (u32x4){lo[0], lo[1], hi[0], hi[1]});
        } else {
            const int d = col0 + (lane & 31);
            Frag<T> f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = 8 * (j >> 2) + 4 * h + (j & 3);
                f[j] = *reinterpret_cast<const float*>(lds + (row0 + row) * kRow + (((d >> 2) ^ turn(row)) * 16) +
                                                       4 * (d & 3));
            }
            return f;
        }
    }
    __device__ static __forceinline__ u32x2 tr(const char* p) {
        const s16x4 v =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
        return __builtin_bit_cast(u32x2, v);
    }
};

// The straight operand of step s of row `row` of x (zeros past its length, at least 1, and dim), from
// global memory; all of them.  Without a branch around them (they would be waited for one by one) all
// loads are under way together: a row or column that is not there reads another's and drops it.
template <typename T>
__device__ __forceinline__ Frag<T> load_step(const Rows<T>& x, int row, int s) {
    const int col = 16 * s + 8 * ((threadIdx.x & 63) >> 5);
    const bool in = row < x.len && col < x.dim;
    float v[8];
    load_unit<T, true>(x.p + (int64_t)min(row, x.len - 1) * x.stride + min(col, x.dim - 8), 8, v);
    Frag<T> f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (T)(in ? v[e] : 0.f);
    return f;
}
template <typename T, int N>
__device__ __forceinline__ void load_row(const Rows<T>& x, int row, int first, Frag<T>* f) {
#pragma unroll
    for (int s = 0; s < N; ++s) f[s] = load_step<T>(x, row, first + s);
}

// Stores a wave's transposed results (columns of x by rows of 32 at a time) as row `row`:
// acc[b] element i is column col0 + 32 b + result_row(i, h).
template <typename T, int NB>
__device__ __forceinline__ void store_row(T* p, int dim, int col0, const f32x16* acc, float scale, bool wide) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = col0 + 32 * b + 8 * g + 4 * h;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[b][4 * g + e] * scale;
            if (wide) {
                if (col < dim) {
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<u32x2*>(p + col) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                    else
                        *reinterpret_cast<f32x4*>(p + col) = (f32x4){v[0], v[1], v[2], v[3]};
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < dim) p[col + e] = (T)v[e];
            }
        }
}

// N steps use(i, f) of matrix instructions whose LDS operands f = load(i) are read AHEAD steps
// earlier. Left to itself the compiler, short of registers, reads each operand right before its
// use and waits for LDS every time.
template <int N, int AHEAD, typename L, typename U>
__device__ __forceinline__ void read_ahead(L load, U use) {
    decltype(load(0)) f[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD && i < N; ++i) f[i] = load(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        use(i, f[i % AHEAD]);
        if (i + AHEAD < N) f[i % AHEAD] = load(i + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Four bfloat16 steps ahead where the registers allow it, two float32 ones (a step of float32 is
// eight instructions of 64 cycles).
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;

// A value of lane ^ 32 (a swap of registers; through LDS a forward pass takes 2 % longer).
__device__ __forceinline__ float other_half(float v) {
    const uint32_t x = __float_as_uint(v);
    const auto both = __builtin_amdgcn_permlane32_swap(x, x, false, false);    // lanes 0 .. 31, 32 .. 63
    return __uint_as_float(threadIdx.x & 32 ? both[0] : both[1]);
}

// Offsets of sequence s, kept inside the array whatever the device holds.
__device__ __forceinline__ int seq_at(const int32_t* cu, int s, int n_seqs, int64_t total) {
    if (!cu) return s == 0 ? 0 : (int)total;
    return max(0, (int)min<int64_t>(cu[s], total));
}

// Which tile of which sequence slot `slot` is.  Sequence s owns slots from at(s) / tile + s on,
// as many as its length needs at most, so floor(total / tile) + n_seqs slots hold every
// tile without anyone having counted the tiles; a slot past its sequence's end is empty.
struct Place {
    int seq, tile;
};
__device__ __forceinline__ Place place_of(const int32_t* cu, int n_seqs, int64_t total, int tile, int slot) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_at(cu, mid, n_seqs, total) / tile + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return {lo, slot - (seq_at(cu, lo, n_seqs, total) / tile + lo)};
}

// The same in falling order of work: slot 0 is a tile of the largest number, tiles of one number
// (counted from a sequence's first, from 1) are neighbours, in the order of the sequences.  A tile
// of number r lies behind the sum over sequences of max(0, tiles - r) others, which a wave
// counts and searches for the slot's r.
constexpr int kOrderedSeqs = 512;
__device__ __forceinline__ Place ordered_place_of(const int32_t* cu, int n_seqs, int64_t total, int tile, int slot) {
    const int lane = threadIdx.x & 63;
    int own[kOrderedSeqs / 64], most = 0;
#pragma unroll
    for (int i = 0; i < kOrderedSeqs / 64; ++i) {
        const int s = 64 * i + lane;
        own[i] = s < n_seqs ? max(0, seq_at(cu, s + 1, n_seqs, total) - seq_at(cu, s, n_seqs, total) + tile - 1) / tile : 0;
        most = max(most, own[i]);
    }
    auto all = [](int v) {
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
        return v;
    };
    auto above = [&](int r) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kOrderedSeqs / 64; ++i) n += max(0, own[i] - r);
        return all(n);
    };
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) most = max(most, __shfl_xor(most, m, 64));
    int lo = 0, hi = most;               // the smallest r with above(r) <= slot
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (above(mid) <= slot) hi = mid;
        else lo = mid + 1;
    }
    if (lo == 0) return {0, -1};         // more slots than tiles
    int left = slot - above(lo);         // which of the sequences with lo tiles or more
    Place p = {0, -1};
#pragma unroll
    for (int i = 0; i < kOrderedSeqs / 64; ++i) {
        const uint64_t who = __ballot(own[i] >= lo);
        const int n = __popcll(who);
        if (p.tile < 0 && left < n) {
            uint64_t w = who;
            for (; left > 0; --left) w &= w - 1;
            p = {64 * i + __ffsll((unsigned long long)w) - 1, lo - 1};
        } else if (p.tile < 0) {
            left -= n;
        }
    }
    return p;
}

// How a launch's workgroups are laid out.
struct AttnGrid {
    int32_t slots, pieces;
    bool ordered;
};

// One workgroup's sequence, head, first row and piece of its walk.
struct Job {
    int q_at, q_len, k_at, k_len, head, row0, piece;
    bool any;
};
template <bool KEYS, int BLOCK>
__device__ __forceinline__ Job job_of(const AttnArgs& a, const AttnGrid& g) {
    Job j;
    // Heads are neighbours in the launch, those that share keys a multiple of the key heads
    // apart: workgroups go to the XCDs in turn, so fewer XCDs read each key head.
    const int heads = KEYS ? a.kv_heads : a.heads;
    const int head = blockIdx.x % heads, rest = blockIdx.x / heads;
    const int slot = rest % g.slots;
    j.head = KEYS ? head : head % a.kv_heads * (a.heads / a.kv_heads) + head / a.kv_heads;
    j.piece = rest / g.slots;
    const int32_t* cu = KEYS ? a.cu_k : a.cu_q;
    const int64_t total = KEYS ? a.n_keys : a.n_queries;
    Place p = g.ordered ? ordered_place_of(cu, a.n_seqs, total, BLOCK, slot) : place_of(cu, a.n_seqs, total, BLOCK, slot);
    if (KEYS && g.ordered && p.tile >= 0) {
        // (the first keys have the most queries behind them)
        const int n = seq_at(cu, p.seq + 1, a.n_seqs, total) - seq_at(cu, p.seq, a.n_seqs, total);
        p.tile = (n + BLOCK - 1) / BLOCK - 1 - p.tile;
    }
    // (the same in every lane: kept in scalar registers, where buffer descriptors need them)
    p.seq = __builtin_amdgcn_readfirstlane(p.seq);
    p.tile = __builtin_amdgcn_readfirstlane(p.tile);
    j.q_at = seq_at(a.cu_q, p.seq, a.n_seqs, a.n_queries);
    j.q_len = max(0, seq_at(a.cu_q, p.seq + 1, a.n_seqs, a.n_queries) - j.q_at);
    j.k_at = seq_at(a.cu_k, p.seq, a.n_seqs, a.n_keys);
    j.k_len = max(0, seq_at(a.cu_k, p.seq + 1, a.n_seqs, a.n_keys) - j.k_at);
    j.any = p.tile >= 0 && (int64_t)p.tile * BLOCK < (KEYS ? j.k_len : j.q_len);
    j.row0 = j.any ? p.tile * BLOCK : 0;
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

// Keys that query `q` sees: those before this one.
__device__ __forceinline__ int seen(const AttnArgs& a, const Job& j, int q) {
    return a.causal ? min(j.k_len, q + 1 + j.k_len - j.q_len) : j.k_len;
}

// This piece's share [first, last) of n tiles.
struct Share {
    int first, last;
    __device__ __forceinline__ Share(int n, int piece, int pieces)
        : first((int)((int64_t)n * piece / pieces)), last((int)((int64_t)n * (piece + 1) / pieces)) {}
};

// A row of a piece's float32 results.
__device__ __forceinline__ float* part_row(float* parts, int piece, int heads, int head, int64_t rows, int64_t row,
                                           int dim) {
    return parts + (((int64_t)piece * heads + head) * rows + row) * dim;
}

// Two waves share 32 rows of 256 features: the sums of one's half of the features, and what
// leads there, fit its registers (in float32 only so, in bfloat16 twice as many waves are on a
// CU).  The products before the softmax are shared out, and their results go to the other wave
// through LDS.
template <int DP>
constexpr int kHalves = DP > 128 ? 2 : 1;

// Waves on a SIMD, which bounds the registers: 256 or 512 a lane.
template <typename T, int DP>
constexpr int kPer = sizeof(T) == 2 || DP <= 64 ? 2 : 1;

// N results from the wave that shares this one's rows; `mine` is what it gets.
template <int WAVES>
struct Exchange {
    f32x4 at[WAVES][4][64];
    __device__ __forceinline__ f32x16 operator()(const f32x16& mine) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            at[wave][g][lane] = (f32x4){mine[4 * g], mine[4 * g + 1], mine[4 * g + 2], mine[4 * g + 3]};
        lds_barrier();
        f32x16 v;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 w = at[wave ^ 1][g][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * g + e] = w[e];
        }
        return v;
    }
};
template <>
struct Exchange<0> {};

// Whether rows are whole 16-byte chunks at 16-byte addresses, which copies into LDS and wide
// stores need.
inline bool al_heads(const AttnArray& x, int32_t dim, int32_t dtype) {
    const int64_t per = dtype == MA_PARAM_BF16 ? 8 : 4;
    // (a copy's offsets within a tile of at most 128 rows stay below 2^31 bytes, and its rows past
    // the last lie past its extent)
    return (reinterpret_cast<uintptr_t>(x.p) & 15) == 0 && x.token % per == 0 && x.head % per == 0 && dim % 8 == 0 &&
           x.token >= dim && x.token <= (int64_t(1) << 22);
}

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f(T{}, padded dim, waves of 32 rows): those of `rows` rows.
template <typename F>
int by_kind(const AttnArgs& a, int rows, F f) {
    auto each = [&](auto t, auto dp) {
        if (rows == 128) f(t, dp, Int<4>{});
        else if (rows == 64) f(t, dp, Int<2>{});
        else f(t, dp, Int<1>{});
    };
    auto dims = [&](auto t) {
        if (a.dim <= 64) each(t, Int<64>{});
        else if (a.dim <= 128) each(t, Int<128>{});
        else each(t, Int<256>{});
    };
    if (a.dtype == MA_PARAM_BF16) dims(__bf16{});
    else dims(float{});
    return (int)hipGetLastError();
}

// A launch's slots for blocks of `block` rows, and how they are taken: in falling order of
// work where more workgroups are queued than run at once, so that the last to begin are
// short (one sequence of 10700 tokens, 8 heads of 128: forward 314 -> 262 us, backward 937 -> 870;
// 7 sequences of 20011, 16 / 4 heads: 329 -> 331 and 1101 -> 1056).
inline AttnGrid grid_of(int64_t total, int64_t n_seqs, int64_t heads, int block, int pieces) {
    AttnGrid g;
    g.slots = (int32_t)(total / block + n_seqs);
    g.pieces = pieces;
    g.ordered = n_seqs <= kOrderedSeqs && (int64_t)g.slots * heads * pieces > 2 * kCus;
    return g;
}

}  // namespace
}  // namespace ma
