// Log probabilities of given tokens with entropy and the highest alternatives,
// and the gradient of the logits, on gfx950.
//
// Forward: one pass over a row with running maximum m, sum s of e^(z - m) and sum t of
// (z - m) e^(z - m), each in every thread and joined at the end (base 2 inside):
//   lse = m + ln s,   log p = (z - m) - ln s,   entropy = ln s - t / s.
// A workgroup takes a row, or a piece of one where there are few; a second launch then
// joins the pieces.
//
// The highest `top` come from the same pass.  Every thread knows its largest value's
// place; the top-th largest of those keys (value, then lowest id) is a bound
// that at least `top` keys of the row reach, all of them in the `top` threads whose own
// largest does.  Those threads' units that hold a value so high (each knows its second largest too, so
// hardly more than one each) are read again, the keys that reach the bound are listed in
// LDS and ranked by counting.  Keys are distinct, so the result does not depend on the order of the list.
//
// Backward: a stream with the row's numbers in registers.
//
// Bound by HBM: 4096 rows of 151000 bf16 with the top 20, 1.24 GB, in 237 us (5.2 TB/s), their
// gradient, 2.47 GB, in 500 us (4.9; a large copy reaches 4.5 to 5.2).  In the forward pass each
// bf16 value costs a conversion, a multiply-add, an exponential and two sums; the loads of the next six
// rounds go on meanwhile.  Few rows are bound by latency: 37 of 32003 fp32 in pieces 11 us and 4 to join.
//
// Units of 8 elements begin at 16-byte addresses: a row's first and last elements, where
// they are not a whole unit, are taken by one thread each.  So which elements a thread sums follows
// from the row's address modulo 16 too: the same values elsewhere may differ in their last bits.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "layers_internal.h"

namespace ma {
namespace {

// Most listed keys of a workgroup of NT threads before the slow way is taken.
template <int NT>
constexpr int kList = NT > 288 ? 2 * NT : 576;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// (far below the smallest power of two: 2^kFar is 0, and 0 * kFar is 0)
constexpr float kFar = -1000.f;
static_assert(MA_LOGPROB_MAX_TOP <= 64, "a wave's lane for each of the top");

// Which elements of a row piece [first, last) each (thread, round) takes: `full` whole
// units from `base` on in rounds of a workgroup's NT threads, and as round `rounds` thread 0
// the elements before them and thread 1 those after.
template <int NT>
struct Piece {
    int first, last, base, full, rounds;
    __device__ __forceinline__ Piece(const char* row, int size, int a, int b) : first(a), last(b) {
        const int mis = (int)((reinterpret_cast<uintptr_t>(row) + (uintptr_t)a * size) & 15);
        base = min(b, a + (mis ? (16 - mis) / size : 0));
        full = (b - base) >> 3;
        rounds = (full + NT - 1) / NT;
    }
    __device__ __forceinline__ int start(int thread, int round) const {
        if (round < rounds) return base + 8 * (round * NT + thread);
        return thread == 0 ? first : base + 8 * full;
    }
    __device__ __forceinline__ int count(int thread, int round) const {
        if (round < rounds) return round * NT + thread < full ? 8 : 0;
        return thread == 0 ? base - first : thread == 1 ? last - base - 8 * full : 0;
    }
};

// Values as integers in their order; zeros alike, a NaN below everything.
__device__ __forceinline__ uint32_t ordered(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    if (z != z) return 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// The larger key is the higher value, of equal ones the lower id.
__device__ __forceinline__ uint64_t key_of(float z, uint32_t id) { return (uint64_t)ordered(z) << 32 | (uint32_t)~id; }

// (a product of 2^24 is rounded to whole numbers: beyond, its rounding alone soon leaves the range of 2^u)
constexpr float kFine = 0x1p24f;

__device__ __forceinline__ float max3(float a, float b, float c) {
    float v;         // (the builtin maximum would first quieten each input)
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(v) : "v"(a), "v"(b), "v"(c));
    return v;
}

// A running softmax: m the largest value (at least -FLT_MAX), s and t the sums of 2^u and u 2^u.
// u = z k - mk is one multiply-add from a reference that is m k rounded; what the rounding
// left out is made up for once, in ln s.  Where |m k| is 2^24 or more (a row of mask values only,
// say) the reference is m k itself, and u is (z - m) k instead.
struct Soft {
    float m, mk, s, t;
    __device__ __forceinline__ void begin() {
        m = -__FLT_MAX__;
        mk = -0.5f * kFine;          // (sums of 0 have any reference: one that needs no care)
        s = t = 0.f;
    }
    __device__ __forceinline__ bool far() const { return !(fabsf(mk) < kFine); }
    // what the reference's rounding left out
    __device__ __forceinline__ float left(float k) const { return far() ? 0.f : fmaf(m, k, -mk); }
    // this reference less the one of `o`, in units of 2^: at most 0.  Two rounded ones are products rounded by
    // themselves: as a fused multiply-add the difference would be that of a rounded and an exact one.
    __device__ __forceinline__ float below(const Soft& o, float k) const {
#pragma clang fp contract(off)
        float d = mk - o.mk;
        // (whether one of them is far: o is not below this one)
        if (__builtin_expect(!(fmaxf(-mk, o.mk) < kFine), 0)) d = (m - o.m) * k - left(k) + o.left(k);
        return __builtin_amdgcn_fmed3f(d, kFar, 0.f);
    }
    // another reference, not below m
    __device__ __forceinline__ void raise(float to, float k) {
        const Soft o = {to, to * k, 0.f, 0.f};
        const float d = below(o, k), c = __builtin_amdgcn_exp2f(d);
        t = fmaf(s, d, t) * c;
        s *= c;
        m = o.m;
        mk = o.mk;
    }
    __device__ __forceinline__ void add(float u) {
        const float e = __builtin_amdgcn_exp2f(u);
        s += e;
        t = fmaf(e, fmaxf(u, kFar), t);          // (a NaN is in e)
    }
    __device__ __forceinline__ void add8(const float* z, float k) {
        if (__builtin_expect(__any(far()), 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) add(far() ? (z[e] - m) * k : fmaf(z[e], k, -mk));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) add(fmaf(z[e], k, -mk));
        }
    }
    // of N neighbouring lanes, in each of them
    template <int N>
    __device__ __forceinline__ void join(float k) {
        float to = m;
#pragma unroll
        for (int x = 1; x < N; x <<= 1) to = fmaxf(to, __shfl_xor(to, x, 64));
        raise(to, k);
#pragma unroll
        for (int x = 1; x < N; x <<= 1) {
            s += __shfl_xor(s, x, 64);
            t += __shfl_xor(t, x, 64);
        }
    }
    // ln of the sum of e^(scale (z - m))
    __device__ __forceinline__ float log_sum(float k) const {
        return logf(s) - kLn2 * left(k);
    }
};

__device__ __forceinline__ Soft soft_of(const float* x, float k) { return {x[0], x[0] * k, x[1], x[2]}; }

// One row's numbers from its joined sums.
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Soft& f, float zt, bool in) {
    const float ls = f.log_sum(a.scale * kLog2e);
    const bool none = f.s == 0.f;                // nothing but -infinity
    a.lse[row] = none ? -__builtin_inff() : fmaf(f.m, a.scale, ls);
    if (a.logprob) {
        const float lp = fmaf(zt - f.m, a.scale, -ls);
        a.logprob[row] = !in ? 0.f : none ? -__builtin_inff() : lp;
    }
    if (a.entropy) a.entropy[row] = none ? 0.f : fmaf(-kLn2, f.t / f.s, logf(f.s));
}

__device__ __forceinline__ int64_t token_of(const LogprobArgs& a, int64_t row) {
    return a.token_bytes == 8 ? static_cast<const int64_t*>(a.tokens)[row]
                              : (int64_t)static_cast<const int32_t*>(a.tokens)[row];
}

template <typename T>
__device__ __forceinline__ void write_target(const LogprobArgs& a, const T* z, int64_t row, const Soft& f) {
    const int64_t tok = a.tokens ? token_of(a, row) : -1;
    const bool in = tok >= 0 && tok < a.vocab;
    write_row(a, row, f, in ? (float)z[tok] : 0.f, in);
}

__device__ __forceinline__ void write_top(const LogprobArgs& a, int64_t row, int rank, uint64_t key, const Soft& f) {
    const int64_t at = row * a.top + rank;
    const uint32_t id = ~(uint32_t)key;
    if (a.token_bytes == 8) static_cast<int64_t*>(a.top_ids)[at] = id;
    else static_cast<int32_t*>(a.top_ids)[at] = (int32_t)id;
    const uint32_t u = (uint32_t)(key >> 32);
    const float z = u ? unordered(u) : __builtin_nanf("");
    a.top_logprobs[at] = f.s == 0.f ? -__builtin_inff() : fmaf(z - f.m, a.scale, -f.log_sum(a.scale * kLog2e));
}

// The largest of a workgroup's keys, in every thread.
template <int NT>
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* slot) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
        v = max(v, o);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < NT / 64; ++w) v = max(v, slot[w]);
    return v;
}

template <int NT>
struct TopLds {
    uint64_t best[NT];           // every thread's largest key
    uint64_t list[kList<NT>];
    uint64_t slot[NT / 64];
    uint32_t second[NT];         // the value of its largest in another round than that one's,
    int round[NT];               // which this is
    int chosen[64];              // the threads whose largest reaches the bound
    uint64_t bound;
    int n_chosen, n;
    bool more;                   // whether one of them has another value that high
};

// Writes the `top` largest keys of the piece through put(rank, key).  `best`: this thread's
// largest key, 0 for none, from round `at`; `second`: the largest value of its other rounds.  The
// piece has at least `top` elements.
template <int NT, typename T, typename F>
__device__ __forceinline__ void select_top(const T* z, const Piece<NT>& p, int top, uint64_t best, int at,
                                           float second, TopLds<NT>& l, F put) {
    constexpr int kThreads = NT, kWaves = NT / 64, kList = ma::kList<NT>;
    const int tid = threadIdx.x, size = p.last - p.first;
    if (tid == 0) l.n = l.n_chosen = 0;
    l.best[tid] = best;
    l.round[tid] = at;
    l.second[tid] = ordered(second);
    __syncthreads();
    // (with fewer units than `top` not enough threads have a key: every key is listed)
    const bool all = min(p.full, kThreads) < top;
    uint64_t bound = 0;
    if (all) {
        for (int i = tid; i < size; i += kThreads) l.list[i] = key_of((float)z[p.first + i], p.first + i);
        __syncthreads();
    } else {
        if (tid < 64) {
            // the top-th largest of the threads' keys, bit by bit: the largest b that `top` of
            // them reach, found early where exactly `top` do
            uint64_t k[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) k[w] = l.best[w * 64 + tid];
            uint64_t b = 0;
            bool more = false;
            for (int bit = 63; bit >= 0; --bit) {
                const uint64_t at = b | 1ull << bit;
                int n = 0;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) n += __popcll(__ballot(k[w] >= at));
                if (n >= top) b = at;
                if (n == top) break;
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const bool in = k[w] >= b;
                const uint64_t who = __ballot(in);
                int at = 0;
                if (tid == 0) {
                    at = l.n_chosen;
                    l.n_chosen = at + __popcll(who);
                }
                at = __shfl(at, 0, 64) + __popcll(who & ((1ull << tid) - 1));
                if (in && at < 64) l.chosen[at] = w * 64 + tid;
                more |= in && l.second[w * 64 + tid] >= (uint32_t)(b >> 32);
            }
            more = __any(more);
            if (tid == 0) l.more = more;
            if (tid == 0) l.bound = b;
        }
        __syncthreads();
        bound = l.bound;
        auto list = [&](int who, int round) {
            const int cnt = p.count(who, round), s = p.start(who, round);
            if (cnt <= 0) return;
            float v[8];
            load_unit<T, false, false>(z + s, cnt, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t k = key_of(v[e], s + e);
                if (e < cnt && k >= bound) {
                    const int at = atomicAdd(&l.n, 1);
                    if (at < kList) l.list[at] = k;
                }
            }
        };
        if (tid < l.n_chosen) list(l.chosen[tid], l.round[l.chosen[tid]]);
        for (int c = 0; l.more && c < l.n_chosen; ++c) {
            const int who = l.chosen[c];
            if (l.second[who] < (uint32_t)(bound >> 32)) continue;
            for (int round = tid; round <= p.rounds; round += kThreads)
                if (round != l.round[who]) list(who, round);
        }
        __syncthreads();
    }
    const int n = all ? size : l.n;
    if (n <= kList) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = l.list[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) rank += l.list[j] > k;
            if (rank < top) put(rank, k);
        }
    } else {
        // so many keys reach the bound that the list does not hold them: one after the other,
        // the largest below the last, from the chosen threads' units
        const int per = p.rounds + 1, units = l.n_chosen * per;
        uint64_t last = ~0ull;
        for (int r = 0; r < top; ++r) {
            uint64_t k = 0;
            for (int i = tid; i < units; i += kThreads) {
                const int who = l.chosen[i / per], round = i % per;
                const int cnt = p.count(who, round), s = p.start(who, round);
                if (cnt <= 0) continue;
                float v[8];
                load_unit<T, false, false>(z + s, cnt, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint64_t c = key_of(v[e], s + e);
                    if (e < cnt && c < last) k = max(k, c);
                }
            }
            last = block_max<NT>(k, l.slot);
            if (tid == 0) put(r, last);
        }
    }
    __syncthreads();             // (the next row's keys take this LDS)
}

template <typename T, bool TOP, int NT>
__global__ __launch_bounds__(NT) void k_logprob_forward(LogprobArgs a) {
    constexpr int kThreads = NT, kWaves = NT / 64;
    __shared__ float part[kWaves][3];
    __shared__ std::conditional_t<TOP, TopLds<NT>, int> lds;
    const int tid = threadIdx.x;
    const float k = a.scale * kLog2e;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* z = static_cast<const T*>(a.logits) + row * a.stride;
        const int from = (int)min<int64_t>((int64_t)blockIdx.y * a.piece, a.vocab);
        const Piece<NT> p(reinterpret_cast<const char*>(z), sizeof(T), from, (int)min<int64_t>(from + a.piece, a.vocab));
        Soft f;
        f.begin();
        // the largest value, the round that held it, and the largest of the other rounds
        float top = -__builtin_inff(), second = -__builtin_inff();
        // (the elements before the whole units come first, so of equal values a thread's first
        // in its rounds is the lowest)
        const bool head = tid == 0 && p.base > p.first;
        int at = head ? p.rounds : 0;
        auto take = [&](const float* v, int round) {
            const float mu = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7]));
            second = __builtin_amdgcn_fmed3f(mu, top, second);
            if (mu > top) {
                top = mu;
                at = round;
                f.raise(fmaxf(mu, f.m), k);
            }
            f.add8(v, k);
        };
        auto part_of = [&](int round) {
            const int cnt = p.count(tid, round);
            if (cnt <= 0) return;
            float v[8];
            load_unit<T, false>(z + p.start(tid, round), cnt, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < cnt ? v[e] : -__builtin_inff();
            take(v, round);
        };
        if (head) part_of(p.rounds);
        // Whole units in batches, the next one's loads under way while one is worked on.  In the last
        // round threads without a unit read the last and drop it: no branch by lane around a load.
        constexpr int kAhead = 6 / (sizeof(T) / 2), kWords = sizeof(T) / 2;
        u32x4 w[kAhead][kWords];
        auto load = [&](int round) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (round + i < p.rounds) {
                    const T* q = z + p.base + 8 * (int64_t)min((round + i) * kThreads + tid, p.full - 1);
#pragma unroll
                    for (int h = 0; h < kWords; ++h) w[i][h] = reinterpret_cast<const u32x4*>(q)[h];
                }
        };
        if (p.rounds > 0) load(0);
        for (int r = 0; r < p.rounds; r += kAhead) {
            u32x4 now[kAhead][kWords];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int h = 0; h < kWords; ++h) now[i][h] = w[i][h];
            load(r + kAhead);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (r + i < p.rounds) {
                    float v[8];
                    widen<T>(now[i], v);
                    if (r + i == p.rounds - 1) {
                        const bool in = (r + i) * kThreads + tid < p.full;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = in ? v[e] : -__builtin_inff();
                    }
                    take(v, r + i);
                }
        }
        if (tid == 1) part_of(p.rounds);
        uint64_t best = 0;
        if constexpr (TOP) {
            // the key of this thread's largest value: its first place in the round that held it
            const int cnt = p.count(tid, at), s = p.start(tid, at);
            if (cnt > 0) {
                float v[8];
                load_unit<T, false>(z + s, cnt, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < cnt) best = max(best, key_of(v[e], s + e));
            }
        }
        f.join<64>(k);
        if constexpr (kWaves > 1) {
            if ((tid & 63) == 0) {
                part[tid >> 6][0] = f.m;
                part[tid >> 6][1] = f.s;
                part[tid >> 6][2] = f.t;
            }
            __syncthreads();
            f = soft_of(part[tid & (kWaves - 1)], k);
            f.join<kWaves>(k);
        }
        const int64_t slot = row * gridDim.y + blockIdx.y;
        if (tid == 0) {
            if (gridDim.y == 1) {
                write_target(a, z, row, f);
            } else {
                float* o = a.sums + slot * 4;
                o[0] = f.m;
                o[1] = f.s;
                o[2] = f.t;
            }
        }
        if constexpr (TOP) {
            const int n = min(a.top, p.last - p.first);
            uint64_t* keys = a.keys + slot * a.top;
            if (gridDim.y > 1 && tid >= n && tid < a.top) keys[tid] = 0;      // (a last piece of fewer elements)
            select_top<NT>(z, p, n, best, at, second, lds, [&](int rank, uint64_t key) {
                if (gridDim.y == 1) write_top(a, row, rank, key, f);
                else keys[rank] = key;
            });
        }
        __syncthreads();
    }
}

// Joins the pieces of a row: their sums in order, and the largest of their keys.
template <typename T>
__global__ __launch_bounds__(512) void k_logprob_join(LogprobArgs a, int pieces) {
    constexpr int kThreads = 512;
    __shared__ uint64_t keys[kThreads];
    const float k = a.scale * kLog2e;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float* s = a.sums + row * pieces * 4;
        // (at most 64 pieces, one a lane)
        const int lane = threadIdx.x & 63;
        const float none[3] = {-__FLT_MAX__, 0.f, 0.f};
        Soft f = soft_of(lane < pieces ? s + 4 * lane : none, k);
        f.join<64>(k);
        if (threadIdx.x == 0)
            write_target(a, static_cast<const T*>(a.logits) + row * a.stride, row, f);
        if (a.top == 0) continue;
        const int n = pieces * a.top;
        const uint64_t* g = a.keys + row * n;
        // ranks by counting, a workgroup's keys at a time (keys of 0 stand for none; at least
        // `top` others are there)
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            const uint64_t mine = i < n ? g[i] : 0;
            int rank = 0;
            for (int j0 = 0; j0 < n; j0 += kThreads) {
                __syncthreads();
                keys[threadIdx.x] = j0 + (int)threadIdx.x < n ? g[j0 + threadIdx.x] : 0;
                __syncthreads();
#pragma unroll 8
                for (int j = 0; j < min(kThreads, n - j0); ++j) rank += keys[j] > mine;
            }
            if (mine && rank < a.top) write_top(a, row, rank, mine, f);
        }
    }
}

template <typename T, typename TG, int NT>
__global__ __launch_bounds__(NT) void k_logprob_backward(LogprobArgs a) {
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* z = static_cast<const T*>(a.logits) + row * a.stride;
        TG* d = static_cast<TG*>(a.dlogits) + row * a.dstride;
        const int from = (int)min<int64_t>((int64_t)blockIdx.y * a.piece, a.vocab);
        const Piece<NT> p(reinterpret_cast<const char*>(z), sizeof(T), from, (int)min<int64_t>(from + a.piece, a.vocab));
        const float lse = a.lse[row];
        const int64_t tok = token_of(a, row);
        const bool in = tok >= 0 && tok < a.vocab;
        const float gs = in ? a.dlogprob[row] * a.scale : 0.f;
        const float hs = a.dentropy ? a.dentropy[row] * a.scale : 0.f;
        const float c0 = a.dentropy ? fmaf(hs, a.ent[row], gs) : gs;
        // -p (g + h (log p + H)), and g at the token; log p is z scale - lse.  A row of nothing has
        // gradient 0, one whose lse is NaN is NaN throughout.
        const bool none = lse == -__builtin_inff();
        const float c = none ? 0.f : lse != lse ? lse : c0, hc = none ? 0.f : hs, gc = none ? 0.f : gs;
        auto unit = [&](const float* v, int at, float* o) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float lp = fmaxf(fmaf(v[e], a.scale, -lse), kFar);
                o[e] = -__builtin_amdgcn_exp2f(lp * kLog2e) * fmaf(hc, lp, c);
            }
            const int64_t t = tok - at;
            if (in && t >= 0 && t < 8)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += e == (int)t ? gc : 0.f;
        };
        auto part_of = [&](int round) {
            const int cnt = p.count(tid, round), at = p.start(tid, round);
            if (cnt <= 0) return;
            float v[8], o[8];
            load_unit<T, false>(z + at, cnt, v);
            unit(v, at, o);
            store_unit<TG, false>(d + at, cnt, o);
        };
        int r = 0;
        constexpr int kAhead = 2;
        for (; (r + kAhead) * NT <= p.full; r += kAhead) {
            float v[kAhead][8], o[8];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load_unit<T, true>(z + p.start(tid, r + i), 8, v[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int at = p.start(tid, r + i);
                unit(v[i], at, o);
                store_unit<TG, false>(d + at, 8, o);
            }
        }
        for (; r <= p.rounds; ++r) part_of(r);
    }
}

}  // namespace

// A workgroup for every row, or pieces of rows until the GPU has about four for each CU; a
// piece has at least 8192 elements (one row of 151000: 18 pieces 24 us, 36 of them 39, most of it joining).
int64_t logprob_pieces(int64_t rows, int64_t vocab) {
    if (rows == 0) return 1;
    const int64_t want = std::max<int64_t>(1, kCus * 4 / rows);
    return std::max<int64_t>(1, std::min<int64_t>({want, vocab / 8192, 64}));
}

static unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, int64_t(1) << 20); }

// Calls f(threads of a workgroup): the more elements the more, 256 where there is less than one
// workgroup a CU.  What a row costs beside its elements (joining sums, telling the top ids)
// grows with its waves, and goes on beside other rows' loads in several small workgroups a CU:
// 30000 x 8000 bf16 237 us with 256 threads, 151 with 128, 100 with 64; 4096 x 151000 285 with
// 512 (and 301 without loads ahead), 236 with 256, 271 with 128.
template <typename F>
static void by_piece(int64_t piece, int64_t blocks, F f) {
    if (blocks < kCus || piece > 32768) f(std::integral_constant<int, 256>{});
    else if (piece > 16384) f(std::integral_constant<int, 128>{});
    else f(std::integral_constant<int, 64>{});
}

int launch_logprob_forward(const LogprobArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const int pieces = (int)ceil_div(a.vocab, a.piece);
    const dim3 grid(row_grid(a.rows), (unsigned)pieces);
    auto go = [&](auto t) {
        using T = decltype(t);
        by_piece(a.piece, a.rows * pieces, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            if (a.top > 0)
                hipLaunchKernelGGL((k_logprob_forward<T, true, NT>), grid, dim3(NT), 0, (hipStream_t)stream, a);
            else
                hipLaunchKernelGGL((k_logprob_forward<T, false, NT>), grid, dim3(NT), 0, (hipStream_t)stream, a);
        });
        if (pieces > 1)
            hipLaunchKernelGGL((k_logprob_join<T>), dim3(row_grid(a.rows)), dim3(512), 0, (hipStream_t)stream, a,
                               pieces);
    };
    if (a.dtype == MA_PARAM_BF16) go(__bf16{});
    else go(float{});
    return (int)hipGetLastError();
}

int launch_logprob_backward(const LogprobArgs& a, void* stream) {
    if (a.rows == 0) return (int)hipSuccess;
    const dim3 grid(row_grid(a.rows), (unsigned)ceil_div(a.vocab, a.piece));
    auto go = [&](auto t, auto g) {
        // (4096 x 151000 bf16: 536 us with 512 threads, 499 with 1024)
        if (a.piece > 32768) {
            hipLaunchKernelGGL((k_logprob_backward<decltype(t), decltype(g), 1024>), grid, dim3(1024), 0,
                               (hipStream_t)stream, a);
            return;
        }
        by_piece(a.piece, a.rows * grid.y, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            hipLaunchKernelGGL((k_logprob_backward<decltype(t), decltype(g), NT>), grid, dim3(NT), 0,
                               (hipStream_t)stream, a);
        });
    };
    if (a.dtype == MA_PARAM_BF16) {
        if (a.ddtype == MA_PARAM_BF16) go(__bf16{}, __bf16{});
        else go(__bf16{}, float{});
    } else {
        if (a.ddtype == MA_PARAM_BF16) go(float{}, __bf16{});
        else go(float{}, float{});
    }
    return (int)hipGetLastError();
}

}  // namespace ma
