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
// further workgroups of the chunk launch.  No atomic touches a sum, so reruns
// are bitwise equal.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "grads_device.h"
#include "grads_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------- lookup --
// A row of the output is taken by `lanes` threads (a power of two), each of
// which moves its column units of kLookRows rows at a time, so that many
// gathered rows are in flight per thread.
constexpr int kLookRows = 4;

template <typename TI, typename TO, typename TOK, int V>
__global__ __launch_bounds__(kThreads) void k_emb_lookup(const TI* __restrict__ table,
                                                         int64_t table_stride, int64_t vocab,
                                                         const TOK* __restrict__ tokens,
                                                         int64_t n, float scale,
                                                         TO* __restrict__ out, int64_t out_stride,
                                                         int units, int lane_bits) {
    const int lanes = 1 << lane_bits, per = kThreads >> lane_bits;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x >> lane_bits;
    const int64_t t0 = (int64_t)blockIdx.x * per * kLookRows + sub;
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
    for (int u = lane; u < units; u += lanes) {
        float v[kLookRows][V];
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            if (row[r] >= 0) {
                load_v<TI, V>(table + row[r] * table_stride + (int64_t)u * V, v[r]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[r][e] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            const int64_t t = t0 + (int64_t)r * per;
            if (t >= n) continue;
            if (row[r] >= 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[r][e] *= scale;
            }
            store_v<TO, V>(out + t * out_stride + (int64_t)u * V, v[r]);
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
constexpr int kSortWaves = kThreads / 64;

// Where a pass reads its keys and positions: the tokens themselves (pass 0) or
// the previous pass's output.
struct SortIn {
    const void* tokens;
    const uint32_t* keys;
    const int32_t* pos;
    int64_t n, vocab, pad;
    int32_t token_bytes;    // 4, 8; 0: keys and pos
    int32_t shift, bits;
    int64_t per;            // entries per block
};

__device__ __forceinline__ uint32_t sort_key(const SortIn& s, int64_t i) {
    if (s.token_bytes == 8) return token_key((const int64_t*)s.tokens, i, s.vocab, s.pad);
    if (s.token_bytes == 4) return token_key((const int32_t*)s.tokens, i, s.vocab, s.pad);
    return s.keys[i];
}

// Digit counts of each block's entries: counts[block][digit].
__global__ __launch_bounds__(kThreads) void k_sort_count(SortIn s, uint32_t* __restrict__ counts) {
    __shared__ uint32_t hist[kMaxDigits];
    const int nd = 1 << s.bits;
    for (int d = threadIdx.x; d < nd; d += kThreads) hist[d] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * s.per, i1 = min(s.n, i0 + s.per);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads)
        atomicAdd(&hist[(sort_key(s, i) >> s.shift) & (nd - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < nd; d += kThreads)
        counts[(int64_t)blockIdx.x * nd + d] = hist[d];
}

// Exclusive prefix of val[0 .. nd) into val, by one block.
__device__ __forceinline__ void block_prefix(uint32_t* val, int nd, uint32_t* wave_sum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nt = (int)blockDim.x;
    const int per = (nd + nt - 1) / nt;
    uint32_t sum = 0;
    for (int k = 0; k < per; ++k) {
        const int d = tid * per + k;
        if (d < nd) sum += val[d];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)inc, off, 64);
        if (lane >= off) inc += o;
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    uint32_t base = inc - sum;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    for (int k = 0; k < per; ++k) {
        const int d = tid * per + k;
        if (d < nd) {
            const uint32_t c = val[d];
            val[d] = base;
            base += c;
        }
    }
    __syncthreads();
}

// Lanes of this wave whose (valid) digit equals this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool valid) {
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((digit >> b) & 1u);
        m &= ((digit >> b) & 1u) ? one : ~one;
    }
    return m;
}

// Stable scatter of each block's entries to their sorted places: the entries of
// a digit go after those of smaller digits, then of earlier blocks, then of
// earlier waves (each wave owns a contiguous part of the block's range and
// walks it 64 entries at a time).
__global__ __launch_bounds__(kThreads) void k_sort_scatter(SortIn s,
                                                           const uint32_t* __restrict__ counts,
                                                           uint32_t* __restrict__ keys_out,
                                                           int32_t* __restrict__ pos_out) {
    __shared__ uint32_t total[kMaxDigits];
    __shared__ uint32_t next[kSortWaves][kMaxDigits];
    __shared__ uint32_t wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nd = 1 << s.bits;
    const int64_t i0 = (int64_t)blockIdx.x * s.per, i1 = min(s.n, i0 + s.per);
    const int64_t part = (s.per + kSortWaves - 1) / kSortWaves;
    const int64_t w0 = min(i1, i0 + wave * part), w1 = min(i1, w0 + part);
    for (int d = lane; d < nd; d += 64) next[wave][d] = 0;
    __syncthreads();
    for (int64_t i = w0 + lane; i < w1; i += 64)
        atomicAdd(&next[wave][(sort_key(s, i) >> s.shift) & (nd - 1)], 1u);
    // over all blocks: totals per digit, and what earlier blocks hold of it
    uint32_t before[kMaxDigits / kThreads];
#pragma unroll
    for (int k = 0; k < kMaxDigits / kThreads; ++k) {
        before[k] = 0;
        const int d = k * kThreads + tid;
        if (d >= nd) continue;
        uint32_t all = 0;
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const uint32_t c = counts[(int64_t)b * nd + d];
            all += c;
            if (b < (int)blockIdx.x) before[k] += c;
        }
        total[d] = all;
    }
    __syncthreads();
    block_prefix(total, nd, wave_sum);
#pragma unroll
    for (int k = 0; k < kMaxDigits / kThreads; ++k) {
        const int d = k * kThreads + tid;
        if (d >= nd) continue;
        uint32_t at = total[d] + before[k];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = next[w][d];
            next[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
    // (the loop is uniform over the wave; `next` is this wave's own)
    for (int64_t i = w0; i < w1; i += 64) {
        const bool valid = i + lane < w1;
        const uint32_t key = valid ? sort_key(s, i + lane) : 0u;
        const int32_t pos = valid ? (s.token_bytes ? (int32_t)(i + lane) : s.pos[i + lane]) : 0;
        const uint32_t digit = (key >> s.shift) & (uint32_t)(nd - 1);
        const uint64_t peers = same_digit(digit, s.bits, valid);
        const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
        if (valid) {
            const uint32_t at = next[wave][digit] + (uint32_t)rank;
            keys_out[at] = key;
            pos_out[at] = pos;
        }
        // every lane has read its digit's place before the last peer moves it on
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (valid && (peers >> lane) == 1u) next[wave][digit] += (uint32_t)rank + 1u;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// --------------------------------------------------------------- sums --
struct SumArgs {
    const void* dout;
    void* grad;
    float* partials;              // [n_chunks][2][hidden]: head, tail
    const uint32_t* keys;
    const int32_t* pos;
    int64_t dout_stride, n, vocab, hidden, chunk, n_chunks;
    int64_t sum_blocks;           // workgroups before those that zero rows
    float scale;
    int32_t accumulate;
    int32_t units, lane_bits;     // column units of a row, and lanes (log2) that take them
};

constexpr int kFillRows = 32;     // rows a zeroing workgroup looks at
constexpr int kSumDepth = 8;      // rows of dout in flight per thread

// First sorted entry whose key is at least `key`.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t key) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <typename TG, int V>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, int64_t col, float* acc) {
    TG* g = static_cast<TG*>(a.grad) + (int64_t)key * a.hidden + col;
    float old[V];
    if (a.accumulate) load_v<TG, V>(g, old);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = a.accumulate ? fmaf(acc[e], a.scale, old[e]) : acc[e] * a.scale;
    store_v<TG, V>(g, acc);
}

// Workgroups [0, sum_blocks): the chunks; the rest: rows without a token.
template <typename TD, typename TG, int V>
__global__ __launch_bounds__(kThreads) void k_emb_sum(SumArgs a) {
    if ((int64_t)blockIdx.x >= a.sum_blocks) {
        __shared__ int empty[kFillRows];
        const int64_t r0 = ((int64_t)blockIdx.x - a.sum_blocks) * kFillRows;
        if (threadIdx.x < kFillRows) {
            const int64_t r = r0 + threadIdx.x;
            int e = 0;
            if (r < a.vocab) {
                const int64_t at = lower_bound(a.keys, a.n, (uint32_t)r);
                e = at >= a.n || a.keys[at] != (uint32_t)r;
            }
            empty[threadIdx.x] = e;
        }
        __syncthreads();
        const float zero[V] = {};
        for (int r = 0; r < kFillRows; ++r) {
            if (!empty[r]) continue;
            TG* g = static_cast<TG*>(a.grad) + (r0 + r) * a.hidden;
            for (int u = threadIdx.x; u < a.units; u += kThreads) store_v<TG, V>(g + (int64_t)u * V, zero);
        }
        return;
    }
    const int lanes = 1 << a.lane_bits, per = kThreads >> a.lane_bits;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x >> a.lane_bits;
    const int64_t c = (int64_t)blockIdx.x * per + sub;
    if (c >= a.n_chunks) return;
    const int64_t i0 = c * a.chunk, i1 = min(a.n, i0 + a.chunk);
    const uint32_t first = a.keys[i0], last = a.keys[i1 - 1];
    const uint32_t none = (uint32_t)a.vocab;
    const bool from_before = i0 > 0 && a.keys[i0 - 1] == first;
    const bool goes_on = i1 < a.n && a.keys[i1] == last;
    const TD* dout = static_cast<const TD*>(a.dout);
    for (int u = lane; u < a.units; u += lanes) {
        const int64_t col = (int64_t)u * V;
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        uint32_t cur = first;
        bool head = from_before;      // the current run began in an earlier chunk
        for (int64_t i = i0; i < i1; i += kSumDepth) {
            uint32_t key[kSumDepth];
            float v[kSumDepth][V];
#pragma unroll
            for (int k = 0; k < kSumDepth; ++k) {
                key[k] = i + k < i1 ? a.keys[i + k] : none;
                if (key[k] != none)
                    load_v<TD, V>(dout + (int64_t)a.pos[i + k] * a.dout_stride + col, v[k]);
            }
#pragma unroll
            for (int k = 0; k < kSumDepth; ++k) {
                if (i + k >= i1) break;
                if (key[k] != cur) {
                    // (a run of no row never comes first and then ends)
                    if (head) store_v<float, V>(a.partials + (c * 2) * a.hidden + col, acc);
                    else write_row<TG, V>(a, cur, col, acc);
                    head = false;
                    cur = key[k];
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = 0.f;
                }
                if (key[k] != none) {
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] += v[k][e];
                }
            }
        }
        if (cur == none) continue;
        if (head) store_v<float, V>(a.partials + (c * 2) * a.hidden + col, acc);
        else if (goes_on) store_v<float, V>(a.partials + (c * 2 + 1) * a.hidden + col, acc);
        else write_row<TG, V>(a, cur, col, acc);
    }
}

// Runs that cross chunks: the workgroups of the chunk in which such a run
// begins (grid.y: column slabs) add its pieces: the tail of that chunk, then
// the heads of the following ones.  kJoinWays threads share a column, each
// taking every kJoinWays-th piece in rising order; their sums are added in
// thread order.
constexpr int kJoinWays = 16;
constexpr int kJoinCols = kThreads / kJoinWays;    // column units of a slab

template <typename TG, int V>
__global__ __launch_bounds__(kThreads) void k_emb_join(SumArgs a) {
    __shared__ float part[kJoinWays][kJoinCols][V];
    const int64_t c = blockIdx.x;
    const int64_t i0 = c * a.chunk, i1 = min(a.n, i0 + a.chunk);
    const uint32_t key = a.keys[i1 - 1];
    if (key == (uint32_t)a.vocab || i1 >= a.n || a.keys[i1] != key) return;
    if (i0 > 0 && a.keys[i0] == key && a.keys[i0 - 1] == key) return;   // began earlier
    const int64_t end = lower_bound(a.keys, a.n, key + 1u);             // one past the run
    const int64_t pieces = (end - 1) / a.chunk - c + 1;
    const int way = threadIdx.x / kJoinCols, lane = threadIdx.x % kJoinCols;
    const int u = (int)blockIdx.y * kJoinCols + lane;
    const int64_t col = (int64_t)u * V;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    if (u < a.units) {
#pragma unroll 4
        for (int64_t p = way; p < pieces; p += kJoinWays) {
            float v[V];
            load_v<float, V>(a.partials + ((c + p) * 2 + (p == 0 ? 1 : 0)) * a.hidden + col, v);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) part[way][lane][e] = acc[e];
    __syncthreads();
    if (way != 0 || u >= a.units) return;
    for (int w = 1; w < kJoinWays; ++w) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += part[w][lane][e];
    }
    write_row<TG, V>(a, key, col, acc);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int64_t per16(int32_t dtype) { return dtype == MA_PARAM_BF16 ? 8 : 4; }

// log2 of the threads that share a row of `units` column units.
int lane_bits_for(int64_t units) {
    int b = 0;
    while ((1 << b) < kThreads && (int64_t(1) << b) < units) ++b;
    return b;
}

}  // namespace

EmbPlan embedding_plan(int64_t n_tokens, int64_t vocab, int64_t hidden) {
    EmbPlan p;
    if (n_tokens == 0) return p;
    int nbits = 1;
    while ((int64_t(1) << nbits) <= vocab) ++nbits;       // keys 0 .. vocab
    p.passes = (nbits + 9) / 10;
    p.bits = (nbits + p.passes - 1) / p.passes;
    p.per = std::max<int64_t>(1024, round_up(ceil_div(n_tokens, 128), 256));
    p.blocks = ceil_div(n_tokens, p.per);
    p.chunk = std::min<int64_t>(256, std::max<int64_t>(32, round_up(ceil_div(n_tokens, 2048), 8)));
    p.n_chunks = ceil_div(n_tokens, p.chunk);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        p.keys[k] = take((size_t)n_tokens * 4);
        p.pos[k] = take((size_t)n_tokens * 4);
    }
    p.counts = take((size_t)p.blocks * ((size_t)1 << p.bits) * 4);
    p.partials = take((size_t)p.n_chunks * 2 * (size_t)hidden * 4);
    p.total = off;
    return p;
}

int launch_embedding_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t hidden,
                            int64_t table_stride, const void* tokens, int32_t token_bytes,
                            int64_t n_tokens, float scale, void* out, int32_t out_dtype,
                            int64_t out_stride, void* stream) {
    if (n_tokens == 0) return (int)hipSuccess;
    const bool vec = aligned16(table) && aligned16(out) && hidden % 8 == 0 &&
                     table_stride % per16(table_dtype) == 0 && out_stride % per16(out_dtype) == 0;
    const int64_t units = vec ? hidden / 8 : hidden;
    const int lb = lane_bits_for(units);
    const int64_t rows = (int64_t)(kThreads >> lb) * kLookRows;
    const dim3 grid((unsigned)ceil_div(n_tokens, rows));
#define GO(TI, TO, TOK, V)                                                                      \
    hipLaunchKernelGGL((k_emb_lookup<TI, TO, TOK, V>), grid, dim3(kThreads), 0,                  \
                       (hipStream_t)stream, static_cast<const TI*>(table), table_stride, vocab,  \
                       static_cast<const TOK*>(tokens), n_tokens, scale, static_cast<TO*>(out),   \
                       out_stride, (int)units, lb)
#define GO_V(TI, TO, TOK)                                                                       \
    do {                                                                                        \
        if (vec) GO(TI, TO, TOK, 8);                                                            \
        else GO(TI, TO, TOK, 1);                                                                \
    } while (0)
#define GO_TOK(TI, TO)                                                                          \
    do {                                                                                        \
        if (token_bytes == 8) GO_V(TI, TO, int64_t);                                            \
        else GO_V(TI, TO, int32_t);                                                             \
    } while (0)
    const bool ti = table_dtype == MA_PARAM_BF16, to = out_dtype == MA_PARAM_BF16;
    if (ti && to) GO_TOK(__bf16, __bf16);
    else if (ti) GO_TOK(__bf16, float);
    else if (to) GO_TOK(float, __bf16);
    else GO_TOK(float, float);
#undef GO_TOK
#undef GO_V
#undef GO
    return (int)hipGetLastError();
}

int launch_embedding_grad(const EmbGradArgs& g, const EmbPlan& p, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    SumArgs a{};
    a.dout = g.dout;
    a.grad = g.grad;
    a.dout_stride = g.dout_stride;
    a.n = g.n_tokens;
    a.vocab = g.vocab;
    a.hidden = g.hidden;
    a.chunk = p.chunk;
    a.n_chunks = p.n_chunks;
    a.scale = g.scale;
    a.accumulate = g.accumulate;
    if (g.n_tokens > 0) {
        SortIn s{};
        s.tokens = g.tokens;
        s.n = g.n_tokens;
        s.vocab = g.vocab;
        s.pad = g.padding_token;
        s.bits = p.bits;
        s.per = p.per;
        uint32_t* counts = reinterpret_cast<uint32_t*>(g.ws + p.counts);
        for (int k = 0; k < p.passes; ++k) {
            s.token_bytes = k == 0 ? g.token_bytes : 0;
            s.shift = k * p.bits;
            if (k > 0) {
                s.keys = reinterpret_cast<const uint32_t*>(g.ws + p.keys[(k - 1) & 1]);
                s.pos = reinterpret_cast<const int32_t*>(g.ws + p.pos[(k - 1) & 1]);
            }
            hipLaunchKernelGGL(k_sort_count, dim3((unsigned)p.blocks), dim3(kThreads), 0, st, s,
                               counts);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return (int)e;
            hipLaunchKernelGGL(k_sort_scatter, dim3((unsigned)p.blocks), dim3(kThreads), 0, st, s,
                               counts, reinterpret_cast<uint32_t*>(g.ws + p.keys[k & 1]),
                               reinterpret_cast<int32_t*>(g.ws + p.pos[k & 1]));
            e = hipGetLastError();
            if (e != hipSuccess) return (int)e;
        }
        const int at = (p.passes - 1) & 1;
        a.keys = reinterpret_cast<const uint32_t*>(g.ws + p.keys[at]);
        a.pos = reinterpret_cast<const int32_t*>(g.ws + p.pos[at]);
        a.partials = reinterpret_cast<float*>(g.ws + p.partials);
    } else if (g.accumulate) {
        return (int)hipSuccess;
    }
    const bool vec = aligned16(g.dout) && aligned16(g.grad) && g.hidden % 8 == 0 &&
                     g.dout_stride % per16(g.dout_dtype) == 0;
    const int64_t units = vec ? g.hidden / 8 : g.hidden;
    a.units = (int)units;
    a.lane_bits = lane_bits_for(units);
    a.sum_blocks = ceil_div(a.n_chunks, kThreads >> a.lane_bits);
    const int64_t fill = g.accumulate ? 0 : ceil_div(g.vocab, kFillRows);
    const bool bd = g.dout_dtype == MA_PARAM_BF16, bg = g.grad_dtype == MA_PARAM_BF16;
    const dim3 grid((unsigned)(a.sum_blocks + fill));
#define GO(TD, TG)                                                                              \
    do {                                                                                        \
        if (vec) hipLaunchKernelGGL((k_emb_sum<TD, TG, 8>), grid, dim3(kThreads), 0, st, a);    \
        else hipLaunchKernelGGL((k_emb_sum<TD, TG, 1>), grid, dim3(kThreads), 0, st, a);        \
    } while (0)
    if (bd && bg) GO(__bf16, __bf16);
    else if (bd) GO(__bf16, float);
    else if (bg) GO(float, __bf16);
    else GO(float, float);
#undef GO
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_chunks < 2) return (int)e;
    const dim3 jgrid((unsigned)a.n_chunks, (unsigned)ceil_div(units, kJoinCols));
#define GO(TG)                                                                                  \
    do {                                                                                        \
        if (vec) hipLaunchKernelGGL((k_emb_join<TG, 8>), jgrid, dim3(kThreads), 0, st, a);      \
        else hipLaunchKernelGGL((k_emb_join<TG, 1>), jgrid, dim3(kThreads), 0, st, a);          \
    } while (0)
    if (bg) GO(__bf16);
    else GO(float);
#undef GO
    return (int)hipGetLastError();
}

}  // namespace ma
