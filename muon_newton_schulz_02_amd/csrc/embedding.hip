// Embedding table: rows looked up and scaled, and the table's gradient from
// sorted tokens, on gfx950.
//
// Gradient.  The rows of dout that belong to one row of the table are summed
// in rising token order.  (row, position) pairs are sorted by row with a stable
// radix sort, and the sorted sequence is cut into chunks of a fixed number of
// entries, whatever rows they belong to, so one row that most tokens share (a
// padding or image token) is spread over the GPU like any other.  A run of
// equal rows inside one chunk is summed in registers and written; the pieces
// of a run that crosses chunks go to the workspace as float32 partial sums,
// and a last launch adds them in order.  Rows without a token are zeroed by
// further workgroups of the sort's launches, which leave most of the GPU idle, and of the
// chunks' launch.  No atomic touches a sum, so reruns are bitwise equal.
//
// Three sizes of sort: up to kDirectTokens tokens none at all (one launch, in which
// every workgroup picks its own few rows' tokens out of all of them); up to
// kLdsSortTokens one workgroup sorts in its LDS; above, passes over many
// workgroups.
//
// A row is handled in units of 8 columns, one thread each: kAligned, whole
// 16-byte aligned units; kShifted, rows at any address, whose last unit begins
// early enough to end with the row, so that every load is whole and none sits
// behind a branch (two threads then write the same values to the columns they
// share, and to add only the owner writes); kTiny, rows of fewer than 8 columns.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "grads_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

enum { kAligned = 0, kShifted = 1, kTiny = 2 };

// Columns of unit u: the first one, how many there are, and how many of the first
// belong to the unit before.
template <int MODE>
struct Cols {
    int at, cnt, shared;
    __device__ __forceinline__ Cols(int u, int hidden) {
        at = u * 8;
        cnt = 8;
        shared = 0;
        if (MODE == kShifted) {
            at = min(u * 8, hidden - 8);
            shared = u * 8 - at;
        } else if (MODE == kTiny) {
            cnt = hidden;
        }
    }
};

// ------------------------------------------------------------- lookup --
// A row of the output is taken by `lanes` threads (a power of two), each of
// which moves its column units of kLookRows rows at a time, so that many
// gathered rows are in flight per thread.  Bound by HBM: 65536 rows of 2048 bf16 out of
// 151000 take 76 to 82 us (155 MB read, since tokens repeat, and 268 MB written: 5.3 TB/s), 37 rows of
// 256 2.6 us.
constexpr int kLookRows = 4;

template <typename TI, typename TO, typename TOK, int MODE, bool NT>
__global__ __launch_bounds__(kThreads) void k_emb_lookup(const TI* __restrict__ table,
                                                         int64_t table_stride, int64_t vocab,
                                                         const TOK* __restrict__ tokens,
                                                         int64_t n, float scale,
                                                         TO* __restrict__ out, int64_t out_stride,
                                                         int hidden, int lane_bits) {
    const int lanes = 1 << lane_bits, per = kThreads >> lane_bits;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x >> lane_bits;
    const int64_t t0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * per * kLookRows + sub;
    int64_t row[kLookRows];
#pragma unroll
    for (int r = 0; r < kLookRows; ++r) {
        const int64_t t = t0 + (int64_t)r * per;
        row[r] = -1;
        if (t < n) {
            row[r] = (int64_t)tokens[t];
            if (row[r] < 0 || row[r] >= vocab) row[r] = -1;
        }
    }
    for (int u = lane; u * 8 < hidden; u += lanes) {
        const Cols<MODE> c(u, hidden);
        float v[kLookRows][8];
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            if (row[r] >= 0) {
                load_unit<TI, MODE == kAligned>(table + row[r] * table_stride + c.at, c.cnt, v[r]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[r][e] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            const int64_t t = t0 + (int64_t)r * per;
            if (t >= n) continue;
            if (row[r] >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[r][e] *= scale;
            }
            store_unit<TO, MODE == kAligned, NT>(out + t * out_stride + c.at, c.cnt, v[r]);
        }
    }
}

// --------------------------------------------------------------- sort --
// Sort key of a token: its table row, or `vocab` (which sorts last) where it
// adds to none.
template <typename TOK>
__device__ __forceinline__ uint32_t token_key(const TOK* tokens, int64_t i, int64_t vocab,
                                              int64_t pad) {
    const int64_t t = (int64_t)tokens[i];
    return (t < 0 || t >= vocab || t == pad) ? (uint32_t)vocab : (uint32_t)t;
}

constexpr int kMaxDigits = 1024;    // digits of a pass: at most 10 bits
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// Where a pass reads its keys and positions: the tokens themselves (pass 0) or
// the previous pass's output.
struct SortIn {
    const void* tokens;
    const uint32_t* keys;
    const int32_t* pos;
    uint8_t* flags;         // one byte per table row: has it a token?
    int64_t n, vocab, pad;
    int32_t token_bytes;    // 4, 8; 0: keys and pos
    int32_t shift, bits;
    int32_t blocks;
    int64_t per;            // entries per block
};

__device__ __forceinline__ uint32_t sort_key(const SortIn& s, int64_t i) {
    if (s.token_bytes == 8) return token_key((const int64_t*)s.tokens, i, s.vocab, s.pad);
    if (s.token_bytes == 4) return token_key((const int32_t*)s.tokens, i, s.vocab, s.pad);
    return s.keys[i];
}

// Exclusive prefix over the digits, digit `tid` each (nd <= kSortThreads).
__device__ __forceinline__ uint32_t digit_prefix(uint32_t count, uint32_t* wave_sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t inc = count;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)inc, off, 64);
        if (lane >= off) inc += o;
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    uint32_t base = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) base += w < wave ? wave_sum[w] : 0u;
    return base + inc - count;
}

// Lanes of this wave whose (valid) digit equals this lane's: of those that agree so
// far, those with this lane's value of the next bit.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool valid) {
    const uint64_t all = __ballot(valid);
    uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
    for (int b = 0; b < bits; ++b) {
        const uint32_t mine = (uint32_t)__builtin_amdgcn_sbfe((int)digit, b, 1);    // all ones or none
        const uint64_t one = __ballot(mine != 0);
        lo &= ~((uint32_t)one ^ mine);
        hi &= ~((uint32_t)(one >> 32) ^ mine);
    }
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Place of a lane's entry among its wave's entries of the same digit so far
// (`count`: this wave's counters), which it joins.
__device__ __forceinline__ uint32_t wave_rank(uint32_t* count, uint32_t digit, int bits, bool valid) {
    const int lane = threadIdx.x & 63;
    const uint64_t peers = same_digit(digit, bits, valid);
    const uint32_t rank = (uint32_t)__popcll(peers & ((uint64_t(1) << lane) - 1));
    const uint32_t base = valid ? count[digit] : 0u;
    // every lane has read the counter before the last of its peers moves it on
    wave_lds_sync();
    if (valid && (peers >> lane) == 1u) count[digit] = base + rank + 1u;
    wave_lds_sync();
    return base + rank;
}

// Zeroing, by workgroups that ride along in other launches.  Up to the sort's first
// scatter every row of a share is zeroed, those of tokens too, which are written later; then
// there is a flag byte for each row, and only those without a token are.  A thread takes one
// or two 16-byte pieces at a time, whatever row they belong to, so that what is in flight
// lies in a narrow, moving window of memory.  Zeroing 1.07 GB alone runs at 6.5 TB/s so; with
// four pieces a thread at 5.8, past the caches at 6.3 and 5.1, and by 512 workgroups that
// loop at 4.8 (247 MB, which the memory-side cache takes, at 8.0).  The flagged shares go past
// the caches, beside the rows that are gathered: 16384 tokens into 151000 x 2048 bf16 take 123 us
// so, 149 through them, and 143 where every row is zeroed and nothing is flagged; 127 with
// four pieces.
constexpr int kFillDepth = 2;     // pieces a thread looks up the flags of at a time
struct FillArgs {
    char* p;                      // 16-byte aligned
    int64_t pieces, groups;       // 16-byte pieces, and workgroups that share them
    const uint8_t* flags;         // null: every row; else rows are whole pieces,
    int64_t first;                // p is this piece of the gradient,
    uint32_t row, magic;          // a row this many, and magic: 2^32 / row, rounded up
    uint16_t* edge[2];            // what lies before the first border and past the last,
    int32_t edge_n[2];            // in 2-byte units (with the first share)
};

// The part of workgroup `g` of those that zero.
__device__ __forceinline__ void fill(const FillArgs& f, int64_t g) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int T = blockDim.x, tid = threadIdx.x;
    u32x4* p = reinterpret_cast<u32x4*>(f.p);
    if (!f.flags) {
        if (g == 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (tid < f.edge_n[k]) f.edge[k][tid] = 0;
        }
        for (int64_t i = g * T + tid; i < f.pieces; i += f.groups * T) p[i] = zero;
        return;
    }
    for (int64_t i0 = g * kFillDepth * T; i0 < f.pieces; i0 += f.groups * kFillDepth * T) {
        // the row of the workgroup's first piece, and the others' rows from there: the
        // quotient of n < row + kFillDepth T by row, exact while n (magic row - 2^32) < 2^32
        // (at most 2^12 2^11 here)
        const int64_t row0 = (f.first + i0) / f.row;
        const uint32_t rem = (uint32_t)(f.first + i0 - row0 * f.row);
        bool has[kFillDepth];
#pragma unroll
        for (int k = 0; k < kFillDepth; ++k) {
            const uint32_t n = i0 + k * T + tid < f.pieces ? rem + (uint32_t)(k * T + tid) : rem;
            const uint32_t r = f.row > (uint32_t)(kFillDepth * kSortThreads) ? (n >= f.row ? 1u : 0u)
                                                                             : __umulhi(n, f.magic);
            has[k] = f.flags[row0 + r] != 0;
        }
#pragma unroll
        for (int k = 0; k < kFillDepth; ++k) {
            const int64_t i = i0 + k * T + tid;
            if (i < f.pieces && !has[k]) put16<true>(p + i, zero);
        }
    }
}

// Digit counts of each block's entries: counts[block][digit].  The first pass
// also clears the flags.  A pass is bound by its latencies (tokens, LDS, counts), not by its
// bytes: 50021 tokens take 4.8 us to count and 6.2 to scatter by themselves, 16384 take 4.8
// and 5.3, and zeroing rides along almost for nothing (32 MB beside the former: 7 and 8.1 us;
// 8 MB beside the latter: 5.7 and 6.3; 148 MB of flagged rows: 26 us, 5.8 TB/s).
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortIn s, uint32_t* __restrict__ counts,
                                                             FillArgs f) {
    if ((int)blockIdx.x >= s.blocks) {
        fill(f, (int)blockIdx.x - s.blocks);
        return;
    }
    __shared__ uint32_t hist[kSortWaves][kMaxDigits];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nd = 1 << s.bits;
    for (int d = lane; d < nd; d += 64) hist[wave][d] = 0;
    wave_lds_sync();
    const int64_t i0 = (int64_t)blockIdx.x * s.per, i1 = min(s.n, i0 + s.per);
    // (uniform over the wave; one addition per digit and wave, since most of a
    // batch may share a digit)
    for (int64_t i = i0 + wave * 64; i < i1; i += kSortThreads) {
        const bool valid = i + lane < i1;
        const uint32_t d = valid ? (sort_key(s, i + lane) >> s.shift) & (uint32_t)(nd - 1) : 0u;
        wave_rank(hist[wave], d, s.bits, valid);
    }
    if (s.token_bytes && s.flags) {
        // (the flags' memory is 16-byte aligned and padded to 16)
        for (int64_t v = ((int64_t)blockIdx.x * kSortThreads + tid) * 16; v < s.vocab;
             v += (int64_t)s.blocks * kSortThreads * 16)
            *reinterpret_cast<u32x4*>(s.flags + v) = (u32x4){0u, 0u, 0u, 0u};
    }
    __syncthreads();
    if (tid < nd) {
        uint32_t c = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c += hist[w][tid];
        counts[(int64_t)blockIdx.x * nd + tid] = c;
    }
}

// Stable scatter of each block's entries to their sorted places: the entries of
// a digit go after those of smaller digits, then of earlier blocks, then of
// earlier waves (each wave owns a contiguous part of the block's range and
// walks it 64 entries at a time).  The first pass also sets the flags.
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(SortIn s,
                                                               const uint32_t* __restrict__ counts,
                                                               uint32_t* __restrict__ keys_out,
                                                               int32_t* __restrict__ pos_out,
                                                               FillArgs f) {
    if ((int)blockIdx.x >= s.blocks) {
        fill(f, (int)blockIdx.x - s.blocks);
        return;
    }
    __shared__ uint32_t next[kSortWaves][kMaxDigits];
    __shared__ uint32_t wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nd = 1 << s.bits;
    const int64_t i0 = (int64_t)blockIdx.x * s.per, i1 = min(s.n, i0 + s.per);
    const int64_t part = (s.per + kSortWaves - 1) / kSortWaves;
    const int64_t w0 = min(i1, i0 + wave * part), w1 = min(i1, w0 + part);
    for (int d = lane; d < nd; d += 64) next[wave][d] = 0;
    wave_lds_sync();
    // the wave's first entries stay in registers with their ranks; only where it has more
    // (above 131072 tokens) are those ranked again below
    uint32_t key0 = 0, at0 = 0;
    int32_t pos0 = 0;
    const bool valid0 = w0 + lane < w1;
    if (valid0) {
        key0 = sort_key(s, w0 + lane);
        pos0 = s.token_bytes ? (int32_t)(w0 + lane) : s.pos[w0 + lane];
    }
    // over all blocks: total of this thread's digit, and what earlier blocks hold of it
    uint32_t all = 0, before = 0;
    if (tid < nd) {
#pragma unroll 16
        for (int b = 0; b < s.blocks; ++b) {
            const uint32_t c = counts[(int64_t)b * nd + tid];
            all += c;
            before += b < (int)blockIdx.x ? c : 0u;
        }
    }
    if (w0 < w1) at0 = wave_rank(next[wave], (key0 >> s.shift) & (uint32_t)(nd - 1), s.bits, valid0);
    for (int64_t i = w0 + 64; i < w1; i += 64) {
        const bool valid = i + lane < w1;
        const uint32_t d = valid ? (sort_key(s, i + lane) >> s.shift) & (uint32_t)(nd - 1) : 0u;
        wave_rank(next[wave], d, s.bits, valid);
    }
    const uint32_t start = digit_prefix(all, wave_sum);     // (a barrier: all counts are in)
    if (tid < nd) {
        uint32_t at = start + before;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = next[w][tid];
            next[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
    auto place = [&](uint32_t at, uint32_t key, int32_t pos) {
        keys_out[at] = key;
        pos_out[at] = pos;
        if (s.token_bytes && s.flags && key < (uint32_t)s.vocab) s.flags[key] = 1;
    };
    const uint32_t d0 = (key0 >> s.shift) & (uint32_t)(nd - 1);
    if (w1 - w0 <= 64) {
        if (valid0) place(next[wave][d0] + at0, key0, pos0);
        return;
    }
    // (the loop is uniform over the wave; next[wave] is this wave's own)
    for (int64_t i = w0; i < w1; i += 64) {
        const bool valid = i + lane < w1;
        const uint32_t key = valid ? sort_key(s, i + lane) : 0u;
        const int32_t pos = valid ? (s.token_bytes ? (int32_t)(i + lane) : s.pos[i + lane]) : 0;
        const uint32_t at = wave_rank(next[wave], (key >> s.shift) & (uint32_t)(nd - 1), s.bits, valid);
        if (valid) place(at, key, pos);
    }
}

// The whole sort of at most 1024 * ROUNDS tokens by one workgroup: entries in
// registers, all passes through LDS.  Two passes of 9 bits: 6 us for 1024 tokens, 10.8 for 4096.
template <int ROUNDS>
__global__ __launch_bounds__(kSortThreads) void k_sort_lds(SortIn s, int passes,
                                                           uint32_t* __restrict__ keys_out,
                                                           int32_t* __restrict__ pos_out, FillArgs f) {
    if (blockIdx.x > 0) {
        fill(f, (int)blockIdx.x - 1);
        return;
    }
    __shared__ uint32_t keys[kSortThreads * ROUNDS];
    __shared__ uint16_t poss[kSortThreads * ROUNDS];
    __shared__ uint32_t next[kSortWaves][kMaxDigits];
    __shared__ uint32_t wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nd = 1 << s.bits, n = (int)s.n;
    uint32_t key[ROUNDS], at[ROUNDS];
    int pos[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = (wave * ROUNDS + r) * 64 + lane;
        key[r] = i < n ? sort_key(s, i) : 0u;
        pos[r] = i;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * s.bits;
        for (int d = lane; d < nd; d += 64) next[wave][d] = 0;
        wave_lds_sync();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            at[r] = wave_rank(next[wave], (key[r] >> shift) & (uint32_t)(nd - 1), s.bits,
                              (wave * ROUNDS + r) * 64 + lane < n);
        __syncthreads();
        uint32_t all = 0;
        if (tid < nd) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) all += next[w][tid];
        }
        uint32_t start = digit_prefix(all, wave_sum);
        if (tid < nd) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = next[w][tid];
                next[w][tid] = start;
                start += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if ((wave * ROUNDS + r) * 64 + lane < n) {
                const uint32_t to = next[wave][(key[r] >> shift) & (uint32_t)(nd - 1)] + at[r];
                keys[to] = key[r];
                poss[to] = (uint16_t)pos[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int i = (wave * ROUNDS + r) * 64 + lane;
            if (i < n) {
                key[r] = keys[i];
                pos[r] = poss[i];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = (wave * ROUNDS + r) * 64 + lane;
        if (i < n) {
            keys_out[i] = key[r];
            pos_out[i] = pos[r];
        }
    }
}

// --------------------------------------------------------------- sums --
struct SumArgs {
    const void* dout;
    void* grad;
    float* partials;              // [n_chunks][2][pitch]: head, tail
    uint32_t* tails;              // per chunk: the row whose run begins in it and goes on, or vocab
    uint8_t* through;             // per chunk: does the run it begins with go on through it all?
    const uint32_t* keys;
    const int32_t* pos;
    int64_t dout_stride, n, vocab, n_chunks;
    int64_t sum_blocks;           // workgroups before those that zero rows
    int64_t pitch;                // of a partial row: hidden rounded up to 8
    float scale;
    int32_t accumulate;
    int32_t hidden, chunk;
    int32_t lane_bits;            // lanes (log2) that take a row
};

constexpr int kSumDepth = 8;      // rows of dout in flight per thread
constexpr int kMaxChunk = 256;
constexpr int kSumEntries = 2048; // sorted entries a workgroup holds

// acc (scaled) into a unit of a row of the gradient, or added to it.
template <typename TG, int MODE>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, const Cols<MODE>& c, float* acc) {
    TG* g = static_cast<TG*>(a.grad) + (int64_t)key * a.hidden + c.at;
    if (a.accumulate) {
        float old[8];
        load_unit<TG, MODE == kAligned>(g, c.cnt, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(acc[e], a.scale, old[e]);
        if (MODE == kShifted && c.shared > 0) {
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (e >= c.shared) g[e] = (TG)acc[e];
            return;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= a.scale;
    }
    store_unit<TG, MODE == kAligned>(g, c.cnt, acc);
}

// acc += rows at[0 .. cnt) of dout (its columns c), in order, kSumDepth at a time.
template <typename TD, int MODE, typename AT>
__device__ __forceinline__ void add_rows(float* acc, const TD* dout, int64_t stride, const Cols<MODE>& c,
                                         const AT* at, int cnt) {
    for (int i = 0; i < cnt; i += kSumDepth) {
        float v[kSumDepth][8];
        // (loads past the last repeat it: no branch)
#pragma unroll
        for (int k = 0; k < kSumDepth; ++k)
            load_unit<TD, MODE == kAligned>(dout + (int64_t)at[min(i + k, cnt - 1)] * stride + c.at, c.cnt, v[k]);
#pragma unroll
        for (int k = 0; k < kSumDepth; ++k) {
            if (i + k >= cnt) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += v[k][e];
        }
    }
}

// Workgroups [0, sum_blocks): the chunks; the rest: rows without a token.  Reads the
// gathered rows and writes each row of the table once, 8 rows of dout in flight per thread.
// Bound by HBM where rows are 16-byte aligned (16384 tokens into 151000 x 2048 bf16, with half of
// the zeroing: 53 us, 7 TB/s); 50021 tokens into 32003 x 1001 fp32 take 37 us (94 MB read, 50
// written: 4 TB/s; rows of 4004 bytes at any address, so a store covers parts of lines).
template <typename TD, typename TG, int MODE>
__global__ __launch_bounds__(kThreads) void k_emb_sum(SumArgs a, FillArgs f) {
    __shared__ uint32_t s_key[kSumEntries];
    __shared__ int32_t s_pos[kSumEntries];
    if ((int64_t)blockIdx.x >= a.sum_blocks) {
        fill(f, (int64_t)blockIdx.x - a.sum_blocks);
        return;
    }
    const int lanes = 1 << a.lane_bits, per = kThreads >> a.lane_bits;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x >> a.lane_bits;
    const int64_t c = (int64_t)blockIdx.x * per + sub;
    const int64_t i0 = c * a.chunk;
    const int cnt = c < a.n_chunks ? (int)min<int64_t>(a.chunk, a.n - i0) : 0;
    uint32_t* key = s_key + sub * a.chunk;
    int32_t* pos = s_pos + sub * a.chunk;
    const uint32_t none = (uint32_t)a.vocab;
    // the neighbours' nearest keys (none: they do not continue)
    const uint32_t prev = cnt > 0 && i0 > 0 ? a.keys[i0 - 1] : none;
    const uint32_t next = cnt > 0 && i0 + cnt < a.n ? a.keys[i0 + cnt] : none;
    for (int i = lane; i < cnt; i += lanes) {
        key[i] = a.keys[i0 + i];
        pos[i] = a.pos[i0 + i];
    }
    __syncthreads();
    if (cnt == 0) return;
    const uint32_t first = key[0], last = key[cnt - 1];
    const bool from_before = prev == first, goes_on = next == last;
    if (lane == 0) {
        const bool through = from_before && goes_on && first == last;
        a.tails[c] = goes_on && !through ? last : none;     // (none where it is the row of no token, too)
        a.through[c] = through;
    }
    const TD* dout = static_cast<const TD*>(a.dout);
    // (entries of no row come last; a load past the others repeats the last of them,
    // so that no load sits behind a branch)
    int some = cnt;
    while (some > 0 && key[some - 1] == none) --some;
    for (int u = lane; u * 8 < a.hidden && some > 0; u += lanes) {
        const Cols<MODE> col(u, a.hidden);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        uint32_t cur = first;
        bool head = from_before;      // the current run began in an earlier chunk
        float* part = a.partials + c * 2 * a.pitch + col.at;
        for (int i = 0; i < some; i += kSumDepth) {
            float v[kSumDepth][8];
#pragma unroll
            for (int k = 0; k < kSumDepth; ++k)
                load_unit<TD, MODE == kAligned>(dout + (int64_t)pos[min(i + k, some - 1)] * a.dout_stride + col.at,
                                                col.cnt, v[k]);
#pragma unroll
            for (int k = 0; k < kSumDepth; ++k) {
                if (i + k >= some) break;
                const uint32_t kk = key[i + k];
                if (kk != cur) {
                    if (head) store_unit<float, MODE == kAligned>(part, 8, acc);
                    else write_row<TG, MODE>(a, cur, col, acc);
                    head = false;
                    cur = kk;
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += v[k][e];
            }
        }
        // (where entries of no row follow cur's run, `last` is theirs)
        if (head) store_unit<float, MODE == kAligned>(part, 8, acc);
        else if (goes_on && cur == last) store_unit<float, MODE == kAligned>(part + a.pitch, 8, acc);
        else write_row<TG, MODE>(a, cur, col, acc);
    }
}

// Runs that cross chunks: a workgroup looks at as many chunks as it has groups of
// threads; for each in which such a run begins (grid.y: column slabs) it adds the
// run's pieces: the tail of that chunk, then the heads of the following ones.  A group adds a
// run of up to kJoinShort pieces by itself; the groups share a longer one, each taking
// every kJoinWays-th piece in rising order, and add their sums in group order.  Mostly one launch's
// latency: 5 us where few runs cross, 7 for 50021 tokens.  Four pieces in flight: with eight
// a batch of which half is one row (65536 into 1000 x 256) takes 71 us instead of 43.
constexpr int kJoinWays = 8;
constexpr int kJoinChunks = kJoinWays;
constexpr int kJoinShort = 8;
constexpr int kJoinLanes = kThreads / kJoinWays;    // column units of a slab

template <typename TG, int MODE>
__global__ __launch_bounds__(kThreads) void k_emb_join(SumArgs a) {
    __shared__ float part[kJoinWays][kJoinLanes][8];
    __shared__ int s_pieces[kJoinChunks];
    __shared__ uint32_t s_row[kJoinChunks];
    const int64_t c0 = (int64_t)blockIdx.x * kJoinChunks;
    for (int j = threadIdx.x >> 6; j < kJoinChunks; j += kThreads / 64) {      // (a wave each)
        const int64_t c = c0 + j;
        const int l = threadIdx.x & 63;
        const uint32_t row = c < a.n_chunks ? a.tails[c] : (uint32_t)a.vocab;
        int pieces = 0;
        if (row != (uint32_t)a.vocab) {
            // the chunk the run ends in: the first after c that it does not go
            // through, 1024 of them looked at per step
            for (int64_t base = (c + 1) & ~int64_t(15);; base += 1024) {
                const int64_t i0 = base + 16 * l;
                u32x4 w = {0u, 0u, 0u, 0u};
                if (i0 < a.n_chunks) w = *reinterpret_cast<const u32x4*>(a.through + i0);
                int stop = 16;
#pragma unroll
                for (int k = 15; k >= 0; --k) {
                    const bool on = ((w[k >> 2] >> (8 * (k & 3))) & 0xffu) != 0 && i0 + k < a.n_chunks;
                    if (i0 + k > c && !on) stop = k;
                }
                const uint64_t any = __ballot(stop < 16);
                if (any) {
                    const int at = __builtin_ctzll(any);
                    pieces = (int)(base + 16 * at + __shfl(stop, at, 64) - c) + 1;
                    break;
                }
            }
        }
        if (l == 0) {
            s_pieces[j] = pieces;
            s_row[j] = row;
        }
    }
    __syncthreads();
    const int way = threadIdx.x / kJoinLanes, lane = threadIdx.x % kJoinLanes;
    const int u = (int)blockIdx.y * kJoinLanes + lane;
    const bool mine = u * 8 < a.hidden;
    const Cols<MODE> col(mine ? u : 0, a.hidden);
    // piece p of the run that begins in chunk c
    auto add_pieces = [&](float* acc, int64_t c, int p0, int step, int pieces) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int p = p0; p < pieces; p += step) {
            float v[8];
            load_unit<float, MODE == kAligned>(a.partials + ((c + p) * 2 + (p == 0 ? 1 : 0)) * a.pitch + col.at, 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
    };
    float acc[8];
    const int own = s_pieces[way];
    if (own > 0 && own <= kJoinShort && mine) {
        add_pieces(acc, c0 + way, 0, 1, own);
        write_row<TG, MODE>(a, s_row[way], col, acc);
    }
    for (int j = 0; j < kJoinChunks; ++j) {
        if (s_pieces[j] <= kJoinShort) continue;
        const int64_t c = c0 + j;
        if (mine) add_pieces(acc, c, way, kJoinWays, s_pieces[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) part[way][lane][e] = acc[e];
        __syncthreads();
        if (way == 0 && mine) {
            for (int w = 1; w < kJoinWays; ++w) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += part[w][lane][e];
            }
            write_row<TG, MODE>(a, s_row[j], col, acc);
        }
        __syncthreads();
    }
}

// Few tokens: one launch.  A workgroup owns `rows` rows of the table and up to 64
// column units (grid.y: slabs of them); it lists the positions of the tokens of its rows,
// by row and then in token order, and then writes every row: zeros, or the sum
// of its list, which `ways` groups of threads share (contiguous parts, added in
// group order).  512 tokens into 1000 x 256 fp32: 6.4 to 7.4 us, of which a bare launch is 2.3.
constexpr int kDirectTokens = 1024;
constexpr int kDirectRows = 32;
constexpr int kDirectLanes = 64;

struct DirectArgs {
    SortIn in;
    SumArgs sum;
    int32_t rows;
};

template <typename TD, typename TG, int MODE>
__global__ __launch_bounds__(kThreads) void k_emb_direct(DirectArgs d) {
    constexpr int W = kThreads / 64;
    __shared__ int s_row[kDirectTokens];        // table rows (local) of the listed tokens,
    __shared__ uint16_t s_tok[kDirectTokens];   // and their positions, in token order
    __shared__ uint16_t s_pos[kDirectTokens];   // positions by row
    __shared__ int s_count[W * kDirectTokens / kThreads], s_start[kDirectRows + 1];
    __shared__ float part[W][kDirectLanes][8];
    const SumArgs& a = d.sum;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t r0 = (int64_t)blockIdx.x * d.rows;
    const int rows = (int)min<int64_t>(d.rows, a.vocab - r0);
    const int n = (int)d.in.n;
    // token k * kThreads + tid is this thread's k-th
    constexpr int K = kDirectTokens / kThreads;
    int row[K], before[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = k * kThreads + tid;
        const int64_t r = i < n ? (int64_t)sort_key(d.in, i) - r0 : -1;
        row[k] = r >= 0 && r < rows ? (int)r : -1;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint64_t m = __ballot(row[k] >= 0);
        if (lane == 0) s_count[k * W + wave] = __popcll(m);
        before[k] = __popcll(m & ((uint64_t(1) << lane) - 1));
    }
    __syncthreads();
    int listed = 0;
#pragma unroll
    for (int c = 0; c < K * W; ++c) {
#pragma unroll
        for (int k = 0; k < K; ++k) before[k] += c < k * W + wave ? s_count[c] : 0;
        listed += s_count[c];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (row[k] < 0) continue;
        s_row[before[k]] = row[k];
        s_tok[before[k]] = (uint16_t)(k * kThreads + tid);
    }
    __syncthreads();
    // where each row's list begins: entries of smaller rows (a wave counts a row)
    for (int r = wave; r <= rows; r += W) {
        int before = 0;
        for (int i = lane; i < listed; i += 64) before += s_row[i] < r;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off, 64);
        if (lane == 0) s_start[r] = before;
    }
    __syncthreads();
    for (int r = wave; r < rows; r += W) {
        int at = s_start[r];
        if (at == s_start[r + 1]) continue;
        for (int i = 0; i < listed; i += 64) {
            const bool hit = i + lane < listed && s_row[i + lane] == r;
            const uint64_t m = __ballot(hit);
            if (hit) s_pos[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = s_tok[i + lane];
            at += __popcll(m);
        }
    }
    __syncthreads();
    const int lanes = 1 << a.lane_bits, groups = kThreads >> a.lane_bits;
    const int gl = tid & (lanes - 1), group = tid >> a.lane_bits;
    const int u = (int)blockIdx.y * kDirectLanes + gl;
    const bool mine = u * 8 < a.hidden;
    const Cols<MODE> col(mine ? u : 0, a.hidden);
    const TD* dout = static_cast<const TD*>(a.dout);
    // lists of up to 16 tokens, and none: a group a row
    for (int r = group; r < rows; r += groups) {
        const int b = s_start[r], cnt = s_start[r + 1] - b;
        if (cnt > 16 || !mine) continue;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        add_rows<TD, MODE>(acc, dout, a.dout_stride, col, s_pos + b, cnt);
        if (cnt > 0 || !a.accumulate) write_row<TG, MODE>(a, (uint32_t)(r0 + r), col, acc);
    }
    // longer ones: all groups (at most W of them) share a row
    const int ways = min(groups, W);
    for (int r = 0; r < rows; ++r) {
        const int b = s_start[r], cnt = s_start[r + 1] - b;
        if (cnt <= 16) continue;
        const int each = (cnt + ways - 1) / ways;
        const int p0 = min(cnt, group * each), p1 = min(cnt, p0 + each);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        if (group < ways) {
            if (mine) add_rows<TD, MODE>(acc, dout, a.dout_stride, col, s_pos + b + p0, p1 - p0);
#pragma unroll
            for (int e = 0; e < 8; ++e) part[group][gl][e] = acc[e];
        }
        __syncthreads();
        if (group == 0 && mine) {
            for (int w = 1; w < ways; ++w) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += part[w][gl][e];
            }
            write_row<TG, MODE>(a, (uint32_t)(r0 + r), col, acc);
        }
        __syncthreads();
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int64_t per16(int32_t dtype) { return dtype == MA_PARAM_BF16 ? 8 : 4; }

// log2 of the threads that share a row of `units` column units, within [least, most].
int lane_bits_for(int64_t units, int least, int most) {
    int b = least;
    while (b < most && (int64_t(1) << b) < units) ++b;
    return b;
}

}  // namespace

// Up to this many tokens one workgroup sorts: its two passes take 10.8 us at 4096
// tokens (6 at 2048), the four launches over many workgroups 22.
static constexpr int64_t kLdsSortTokens = 4096;

// Bytes that each of the first two of several sort launches zeroes, before the flags are
// there.  (32 MB instead: 65536 tokens into 151000 x 2048 187 us instead of 184, since more rows of
// tokens are written twice.)
static constexpr int64_t kFillBlind = int64_t(8) << 20;
static constexpr int64_t kFillAll = int64_t(1) << 50;

// Few tokens into a table of few rows: no sort.  (Each workgroup reads all tokens, so a
// large table pays for that many times over: 1024 tokens into 151000 x 2048 bf16 took
// 170 us so, against 115 us sorted.  512 tokens into 1000 x 256 take 6.5 us on the
// GPU so, and three launches of 6 + 7 + 5 us sorted.)
static bool direct(int64_t n_tokens, int64_t vocab, int64_t hidden) {
    return n_tokens <= kDirectTokens && vocab * ceil_div(ceil_div(hidden, 8), kDirectLanes) <= 16384;
}

EmbPlan embedding_plan(int64_t n_tokens, int64_t vocab, int64_t hidden) {
    EmbPlan p;
    if (n_tokens == 0 || direct(n_tokens, vocab, hidden)) return p;
    int nbits = 1;
    while ((int64_t(1) << nbits) <= vocab) ++nbits;       // keys 0 .. vocab
    p.passes = (nbits + 9) / 10;
    p.bits = (nbits + p.passes - 1) / p.passes;
    p.per = std::max<int64_t>(kSortThreads, round_up(ceil_div(n_tokens, 128), kSortThreads));
    p.blocks = ceil_div(n_tokens, p.per);
    // Chunks of up to 64 entries, so many that each CU gets the same number of
    // workgroups, or longer ones where that number would pass 4 (a run through very many
    // chunks is joined by few threads); of 16 entries at least, since a chunk may leave two
    // partial rows.  (Against chunks for 256 K threads, 16 to 24 entries here: 16384 tokens
    // into 151000 x 2048 bf16 142 -> 130 us, 65536 into 1000 x 256 34 -> 31, 50021 into
    // 32003 x 1001 76 -> 74.5.  Always 64: 524288 tokens into 32000 x 1024, half of them
    // one row, 380 -> 469.)
    p.lane_bits = lane_bits_for(ceil_div(hidden, 8), 3, 8);
    const int64_t per = kThreads >> p.lane_bits;
    const int64_t most = std::min<int64_t>(kMaxChunk, kSumEntries / per);
    const int64_t rounds = std::min<int64_t>(4, ceil_div(n_tokens, per * kCus * 64));
    p.chunk = std::min(most, std::max<int64_t>(16, ceil_div(n_tokens, per * kCus * rounds)));
    p.n_chunks = ceil_div(n_tokens, p.chunk);
    p.pitch = round_up(hidden, 8);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    if (n_tokens > kLdsSortTokens) p.flags = take((size_t)vocab);
    const int bufs = n_tokens <= kLdsSortTokens ? 1 : 2;
    for (int k = 0; k < bufs; ++k) {
        p.keys[k] = take((size_t)n_tokens * 4);
        p.pos[k] = take((size_t)n_tokens * 4);
    }
    if (n_tokens > kLdsSortTokens) p.counts = take((size_t)p.blocks * ((size_t)1 << p.bits) * 4);
    p.tails = take((size_t)p.n_chunks * 4);
    p.through = take((size_t)p.n_chunks);
    p.partials = take((size_t)p.n_chunks * 2 * (size_t)p.pitch * 4);
    p.total = off;
    return p;
}

int launch_embedding_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t hidden,
                            int64_t table_stride, const void* tokens, int32_t token_bytes,
                            int64_t n_tokens, float scale, void* out, int32_t out_dtype,
                            int64_t out_stride, void* stream) {
    if (n_tokens == 0) return (int)hipSuccess;
    const bool al = aligned16(table) && aligned16(out) && hidden % 8 == 0 &&
                    table_stride % per16(table_dtype) == 0 && out_stride % per16(out_dtype) == 0;
    const bool nt = streams_past_caches(n_tokens * hidden, out_dtype);
    const int lb = lane_bits_for(ceil_div(hidden, 8), 0, 8);
    const int64_t rows = (int64_t)(kThreads >> lb) * kLookRows;
    // (a launch's threads along one axis stay below 2^32)
    const int64_t blocks = ceil_div(n_tokens, rows), wide = std::min<int64_t>(blocks, 65536);
    const dim3 grid((unsigned)wide, (unsigned)ceil_div(blocks, wide));
#define GO(TI, TO, TOK, MODE, NT)                                                               \
    hipLaunchKernelGGL((k_emb_lookup<TI, TO, TOK, MODE, NT>), grid, dim3(kThreads), 0,             \
                       (hipStream_t)stream, static_cast<const TI*>(table), table_stride, vocab,  \
                       static_cast<const TOK*>(tokens), n_tokens, scale, static_cast<TO*>(out),   \
                       out_stride, (int)hidden, lb)
#define GO_AL(TI, TO, TOK)                                                                      \
    do {                                                                                        \
        if (al && nt) GO(TI, TO, TOK, kAligned, true);                                          \
        else if (al) GO(TI, TO, TOK, kAligned, false);                                          \
        else if (hidden >= 8) GO(TI, TO, TOK, kShifted, false);                                 \
        else GO(TI, TO, TOK, kTiny, false);                                                     \
    } while (0)
#define GO_TOK(TI, TO)                                                                          \
    do {                                                                                        \
        if (token_bytes == 8) GO_AL(TI, TO, int64_t);                                           \
        else GO_AL(TI, TO, int32_t);                                                            \
    } while (0)
    const bool ti = table_dtype == MA_PARAM_BF16, to = out_dtype == MA_PARAM_BF16;
    if (ti && to) GO_TOK(__bf16, __bf16);
    else if (ti) GO_TOK(__bf16, float);
    else if (to) GO_TOK(float, __bf16);
    else GO_TOK(float, float);
#undef GO_TOK
#undef GO_AL
#undef GO
    return (int)hipGetLastError();
}

namespace {

using Mode0 = std::integral_constant<int, kAligned>;
using Mode1 = std::integral_constant<int, kShifted>;
using Mode2 = std::integral_constant<int, kTiny>;

// Calls f(TD{}, TG{}, mode) with the call's types and its rows' mode.
template <typename F>
void by_types(bool dout_bf16, bool grad_bf16, bool al, int64_t hidden, F f) {
    auto with = [&](auto td, auto tg) {
        if (al) f(td, tg, Mode0{});
        else if (hidden >= 8) f(td, tg, Mode1{});
        else f(td, tg, Mode2{});
    };
    if (dout_bf16 && grad_bf16) with(__bf16{}, __bf16{});
    else if (dout_bf16) with(__bf16{}, float{});
    else if (grad_bf16) with(float{}, __bf16{});
    else with(float{}, float{});
}

// share(bytes, flags, T): the next part of the zeroing, for a launch of workgroups of T
// threads to carry.
template <typename F>
int launch_sort(const EmbGradArgs& g, const EmbPlan& p, SortIn s, int& at, F share, hipStream_t st) {
    auto keys = [&](int k) { return reinterpret_cast<uint32_t*>(g.ws + p.keys[k]); };
    auto pos = [&](int k) { return reinterpret_cast<int32_t*>(g.ws + p.pos[k]); };
    if (g.n_tokens <= kLdsSortTokens) {
        at = 0;
        const FillArgs f = share(kFillAll, nullptr, kSortThreads);
        const dim3 grid((unsigned)(1 + f.groups));
        if (g.n_tokens <= kSortThreads)
            hipLaunchKernelGGL((k_sort_lds<1>), grid, dim3(kSortThreads), 0, st, s, p.passes, keys(0), pos(0), f);
        else if (g.n_tokens <= 2 * kSortThreads)
            hipLaunchKernelGGL((k_sort_lds<2>), grid, dim3(kSortThreads), 0, st, s, p.passes, keys(0), pos(0), f);
        else
            hipLaunchKernelGGL((k_sort_lds<4>), grid, dim3(kSortThreads), 0, st, s, p.passes, keys(0), pos(0), f);
        return (int)hipGetLastError();
    }
    uint32_t* counts = reinterpret_cast<uint32_t*>(g.ws + p.counts);
    // with flags: a quarter of what the first two launches leave; without: each the same
    const int64_t bytes = g.vocab * g.hidden * (g.grad_dtype == MA_PARAM_BF16 ? 2 : 4);
    const int64_t early = s.flags ? kFillBlind : bytes / (2 * p.passes) + 4096;
    const int64_t later = s.flags ? std::max<int64_t>(0, bytes - 2 * kFillBlind) / 4 + 4096 : early;
    for (int k = 0; k < p.passes; ++k) {
        s.token_bytes = k == 0 ? g.token_bytes : 0;
        s.shift = k * p.bits;
        if (k > 0) {
            s.keys = keys((k - 1) & 1);
            s.pos = pos((k - 1) & 1);
        }
        FillArgs f = share(k == 0 ? early : later, k == 0 ? nullptr : s.flags, kSortThreads);
        hipLaunchKernelGGL(k_sort_count, dim3((unsigned)(p.blocks + f.groups)), dim3(kSortThreads), 0, st, s,
                           counts, f);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
        f = share(k == 0 ? early : later, k == 0 ? nullptr : s.flags, kSortThreads);
        hipLaunchKernelGGL(k_sort_scatter, dim3((unsigned)(p.blocks + f.groups)), dim3(kSortThreads), 0, st, s,
                           counts, keys(k & 1), pos(k & 1), f);
        e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
    }
    at = (p.passes - 1) & 1;
    return (int)hipSuccess;
}

}  // namespace

int launch_embedding_grad(const EmbGradArgs& g, const EmbPlan& p, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (g.n_tokens == 0 && g.accumulate) return (int)hipSuccess;
    const bool al = aligned16(g.dout) && aligned16(g.grad) && g.hidden % 8 == 0 &&
                    g.dout_stride % per16(g.dout_dtype) == 0;
    const bool bd = g.dout_dtype == MA_PARAM_BF16, bg = g.grad_dtype == MA_PARAM_BF16;
    const int64_t units = ceil_div(g.hidden, 8);
    SumArgs a{};
    a.dout = g.dout;
    a.grad = g.grad;
    a.dout_stride = g.dout_stride;
    a.n = g.n_tokens;
    a.vocab = g.vocab;
    a.hidden = (int)g.hidden;
    a.chunk = (int)p.chunk;
    a.n_chunks = p.n_chunks;
    a.pitch = p.pitch;
    a.scale = g.scale;
    a.accumulate = g.accumulate;
    SortIn s{};
    s.tokens = g.tokens;
    s.n = g.n_tokens;
    s.vocab = g.vocab;
    s.pad = g.padding_token;
    s.bits = p.bits;
    s.per = p.per;
    s.blocks = (int)p.blocks;
    s.token_bytes = g.token_bytes;
    if (g.n_tokens > 0 && direct(g.n_tokens, g.vocab, g.hidden)) {
        DirectArgs d{};
        d.in = s;
        a.lane_bits = lane_bits_for(units, 0, 6);
        d.sum = a;
        const unsigned slabs = (unsigned)ceil_div(units, kDirectLanes);
        // about four workgroups per CU, of at most kDirectRows rows
        d.rows = (int)std::min<int64_t>(kDirectRows, std::max<int64_t>(1, ceil_div(g.vocab * slabs, 4 * kCus)));
        const dim3 grid((unsigned)ceil_div(g.vocab, d.rows), slabs);
        by_types(bd, bg, al, g.hidden, [&](auto td, auto tg, auto w) {
            hipLaunchKernelGGL((k_emb_direct<decltype(td), decltype(tg), decltype(w)::value>), grid,
                               dim3(kThreads), 0, st, d);
        });
        return (int)hipGetLastError();
    }
    const uintptr_t first = reinterpret_cast<uintptr_t>(g.grad);
    const uintptr_t last = first + (uintptr_t)(g.vocab * g.hidden * (bg ? 2 : 4));
    // (whole lines, and every share of whole lines: a share that began 16 bytes off them
    // took 32.7 us instead of 25.3 for 148 MB)
    const uintptr_t from = std::min(last, (first + 127) & ~(uintptr_t)127), to = std::max(from, last & ~(uintptr_t)15);
    const int64_t row_bytes = g.hidden * (bg ? 2 : 4);
    int64_t shared = 0;           // pieces that launches have taken
    bool edges = false;           // and whether one has taken the edges (a gradient of a few
                                  // bytes has no piece; later shares run beside the sums)
    auto share = [&](int64_t bytes, const uint8_t* flags, int threads) {
        FillArgs f{};
        if (g.accumulate) return f;
        const int64_t left = (int64_t)((to - from) / 16) - shared;
        f.pieces = std::min(left, round_up(bytes / 16, 256));
        f.p = reinterpret_cast<char*>(from) + shared * 16;
        f.first = (int64_t)(from - first) / 16 + shared;
        f.flags = flags;
        f.row = (uint32_t)(row_bytes / 16);
        f.magic = flags ? (uint32_t)(((uint64_t(1) << 32) + f.row - 1) / f.row) : 0;
        const int64_t each = (flags ? kFillDepth : 1) * threads;
        f.groups = std::min<int64_t>(ceil_div(f.pieces, each), (int64_t(1) << 31) / threads);
        if (!edges && !flags) {
            edges = true;
            f.groups = std::max<int64_t>(f.groups, 1);
            f.edge[0] = reinterpret_cast<uint16_t*>(first);
            f.edge_n[0] = (int)((from - first) / 2);
            f.edge[1] = reinterpret_cast<uint16_t*>(to);
            f.edge_n[1] = (int)((last - to) / 2);
        }
        shared += f.pieces;
        return f;
    };
    if (g.n_tokens == 0) {
        const FillArgs f = share(kFillAll, nullptr, kSortThreads);
        s.blocks = 0;
        hipLaunchKernelGGL(k_sort_count, dim3((unsigned)f.groups), dim3(kSortThreads), 0, st, s, nullptr, f);
        return (int)hipGetLastError();
    }
    // (Rows of odd bytes share pieces: all are zeroed in the sort's launches.  32003 x 1001
    // fp32, a third of them with tokens: 74.5 us, and 78 to 83 by pieces cut where rows with and
    // without a token meet; 151000 x 1001 bf16, a third too: 116, and 110 row by row.)
    const bool whole_pieces = first % 16 == 0 && row_bytes % 16 == 0 && row_bytes > 16;
    if (whole_pieces) s.flags = reinterpret_cast<uint8_t*>(g.ws + p.flags);
    int at = 0;
    const int err = launch_sort(g, p, s, at, share, st);
    if (err != (int)hipSuccess) return err;
    a.keys = reinterpret_cast<const uint32_t*>(g.ws + p.keys[at]);
    a.pos = reinterpret_cast<const int32_t*>(g.ws + p.pos[at]);
    a.partials = reinterpret_cast<float*>(g.ws + p.partials);
    a.tails = reinterpret_cast<uint32_t*>(g.ws + p.tails);
    a.through = reinterpret_cast<uint8_t*>(g.ws + p.through);
    a.lane_bits = p.lane_bits;
    a.sum_blocks = ceil_div(a.n_chunks, kThreads >> a.lane_bits);
    const FillArgs rest = share(kFillAll, s.flags, kThreads);
    const dim3 grid((unsigned)(a.sum_blocks + rest.groups));
    by_types(bd, bg, al, g.hidden, [&](auto td, auto tg, auto w) {
        hipLaunchKernelGGL((k_emb_sum<decltype(td), decltype(tg), decltype(w)::value>), grid,
                           dim3(kThreads), 0, st, a, rest);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_chunks < 2) return (int)e;
    const dim3 jgrid((unsigned)ceil_div(a.n_chunks, kJoinChunks), (unsigned)ceil_div(units, kJoinLanes));
    by_types(bd, bg, al, g.hidden, [&](auto, auto tg, auto w) {
        hipLaunchKernelGGL((k_emb_join<decltype(tg), decltype(w)::value>), jgrid, dim3(kThreads), 0, st, a);
    });
    return (int)hipGetLastError();
}

}  // namespace ma
