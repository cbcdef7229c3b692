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
// each, which add up to it (but for bits below 2^-133, which no bf16 has), and enters as
// three products, side by side on the small tiles, part after part on the large ones.
// Sums are float32.
//
// LDS layout of a stage operand of W columns: token row t at t * 2 W bytes,
// its 16-byte chunk c (8 columns) at slot c ^ ((t & 3) << 2), so that the four
// rows of 64 bytes that half a wave reads together lie in distinct banks.  Counted per LDS
// access: no conflict cycle in the kernel of the large products, 0.34 in the other, which
// also writes its stages there.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads_device.h"
#include "grads_internal.h"
#include "lds_copy.h"

namespace ma {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kTile = 128;                       // output tile side
constexpr int kRow = 2 * kTile;                  // LDS bytes of a token row
constexpr int kRegion = kLgStage * kRow;         // LDS bytes of an operand's stage
constexpr int kAhead = 2;                        // stages loaded ahead into registers

__device__ __forceinline__ u32x2 lds_tr8(const char* p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
    return __builtin_bit_cast(u32x2, v);
}

// Which tile and token slice a workgroup takes.  Consecutive workgroups go to
// the XCDs in turn; each XCD gets a contiguous range of the work list, in which
// tiles that share operand columns are neighbours.
struct Work {
    int tn, tk, slice;
};
__device__ __forceinline__ Work work_of(uint32_t id, uint32_t total, uint32_t tiles_n, uint32_t tiles_k) {
    const uint32_t q = total / kXcds, r = total % kXcds;
    const uint32_t xcd = id % kXcds, local = id / kXcds;
    const uint32_t i = xcd * q + min(xcd, r) + local;
    const uint32_t tiles = tiles_n * tiles_k, slice = i / tiles, t = i - slice * tiles;
    // bands of four tile rows, walked column by column
    const uint32_t band = t / (4 * tiles_k), in = t - band * 4 * tiles_k;
    const uint32_t rows = min(4u, tiles_n - band * 4), tk = in / rows;
    return {(int)(band * 4 + in - tk * rows), (int)tk, (int)slice};
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
// (each takes the next 8 bits of the significand, cut, so none can overflow), exactly
// from |x| = 2^-110 up; below that the bits under 2^-133, bf16's smallest step, are cut
// off: by less than 2^-133, towards zero.  An infinity or NaN is all in the first part.
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

// A buffer of `bytes` from p on: loads past it give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0,
                                             (int)min<int64_t>(bytes, 0x7fffffff), 0x00020000);
}

// One 32 x 32 accumulator block into rows of `ld` elements: register r of lane l
// holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32, so a store covers two row
// pieces of 32 columns.  `rows` and `cols` from the block's origin exist (WHOLE:
// all 32).
template <typename T, bool WHOLE, bool ADD>
__device__ __forceinline__ void store_block(const f32x16& v, T* p, int64_t ld, int64_t rows,
                                            int64_t cols, int lane) {
    const int r0 = 4 * (lane >> 5), c = lane & 31;
    if (!WHOLE && c >= cols) return;
    T* q = p + r0 * ld + c;
    if (ADD) {
        float old[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int d = 8 * (r >> 2) + (r & 3);
            old[r] = WHOLE || r0 + d < rows ? (float)q[d * ld] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int d = 8 * (r >> 2) + (r & 3);
            if (WHOLE || r0 + d < rows) q[d * ld] = (T)(old[r] + v[r]);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int d = 8 * (r >> 2) + (r & 3);
            if (WHOLE || r0 + d < rows) q[d * ld] = (T)v[r];
        }
    }
}

// A wave's NI x NJ blocks (rows first) from output row `row`, column `col` on: partial
// sums, or the gradient, written or added to.
template <typename TG, int NI, int NJ, typename ACC>
__device__ __forceinline__ void store_wave(ACC acc, float* part, TG* grad, int accumulate,
                                           int64_t row, int64_t col, int64_t n_out, int64_t n_in,
                                           int lane) {
    const int64_t rows = n_out - row, cols = n_in - col, o = row * n_in + col;
    auto each = [&](auto whole, auto add, auto* base) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                store_block<std::remove_pointer_t<decltype(base)>, decltype(whole)::value, decltype(add)::value>(
                    acc(i, j), base + o + i * 32 * n_in + j * 32, n_in, rows - i * 32, cols - j * 32, lane);
    };
    auto by_size = [&](auto add, auto* base) {
        if (rows >= NI * 32 && cols >= NJ * 32) each(std::true_type{}, add, base);
        else each(std::false_type{}, add, base);
    };
    if (part) by_size(std::false_type{}, part);
    else if (accumulate) by_size(std::true_type{}, grad);
    else by_size(std::false_type{}, grad);
}

// 8 values of a row as they lie in memory (T's 16 or 32 bytes), from any element's
// address p on.  Where fewer than 8 are left in the row, the load begins `back` elements
// earlier and the values are shifted down; what comes in above them is of no
// matter.  No branch: the load stays in flight (the shift waits for it, so it
// belongs where the values are used).
template <typename T>
__device__ __forceinline__ void load_raw8(const T* p, int back, u32x4* w) {
    if constexpr (sizeof(T) == 4) {
        w[0] = *reinterpret_cast<const u32x4u4*>(p - back);
        w[1] = *(reinterpret_cast<const u32x4u4*>(p - back) + 1);
    } else {
        w[0] = *reinterpret_cast<const u32x4u2*>(p - back);
    }
}
template <typename T>
__device__ __forceinline__ void shift_raw8(int back, u32x4* w) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int b = 4; b > 0; b /= 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t up = e + b < 8 ? w[(e + b) >> 2][(e + b) & 3] : 0u;
                w[e >> 2][e & 3] = (back & b) ? up : w[e >> 2][e & 3];
            }
        }
    } else {
        uint64_t lo = (uint64_t)w[0][1] << 32 | w[0][0], hi = (uint64_t)w[0][3] << 32 | w[0][2];
        lo = (back & 4) ? hi : lo;
        const int n = 16 * (back & 3);
        lo = lo >> n | hi << 1 << (63 - n);          // (hi << 64 - n, also for n = 0)
        hi >>= n;
        w[0] = (u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
}

// The kernel for any type, stride and size: 128 x 128 tiles, four waves of 64
// x 64, two LDS stages, operands staged through registers, two stages ahead (three or
// four were no faster).  AL: rows of dY in 16-byte pieces, and a slice's operands within 2 GB
// of their start.  A small call is bound by the number of its tiles, so the token axis is
// cut, and then by a stage's latency and by the partial sums: 16001 tokens x 256 outputs x
// 1024 inputs in bf16 (16 tiles, 28 slices) take 21.6 us, and 5.9 more to join; two groups of
// waves sharing a workgroup's tile (half the partial sums) took 27.7 us instead of 26.2 for
// both.  77 tokens x 256 x 256 in float32, four tiles of three stages: 10 us.
template <typename TD, bool AL, typename TG>
__global__ __launch_bounds__(kThreads, 2) void k_linear_grad(LgArgs a, int tiles_n,
                                                          int tiles_k, int slices, int per) {
    constexpr int NP = sizeof(TD) == 4 ? 3 : 1;         // bf16 parts of dY
    constexpr int kStageBytes = (NP + 1) * kRegion;
    __shared__ __attribute__((aligned(1024))) char ring[2 * kStageBytes];
    const Work wk = work_of(blockIdx.x, gridDim.x, tiles_n, tiles_k);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t n0 = (int64_t)wk.tn * kTile, k0 = (int64_t)wk.tk * kTile;
    const int64_t t0 = (int64_t)wk.slice * per * kLgStage;
    const int64_t t1 = min<int64_t>(a.n_tokens, t0 + (int64_t)per * kLgStage);
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

    // a stage's share of this thread: 16 values of dY (bf16, or float) and 16 codes
    constexpr int ND = (int)sizeof(TD);
    struct Regs {
        u32x4 d[ND], c;
        uint32_t e;
        bool live;           // !AL: the row is this thread's own
    };
    // Loads are issued in stage order.  AL: buffer loads at running offsets, so that
    // what lies past the slice's last token arrives as zeros without a branch
    // (which would end the load's flight); what lies past a row's last column is
    // another row's, and ends in outputs that do not exist.
    const int64_t ld = a.dy_stride;
    const int64_t es = (int64_t)sizeof(TD);
    const char* bd = static_cast<const char*>(a.dy) + (t0 * ld + n0) * es;
    const int8_t* bc = a.codes + t0 * cp + k0;
    const uint8_t* be = a.exps + t0 * ep + (k0 >> 5);
    int64_t rows = t1 - t0;                               // left from the next load's first token on
    const auto rd = buffer(bd, ((rows - 1) * ld + a.n_out - n0) * es);
    const auto rc = buffer(bc, rows * cp - k0);
    const auto re = buffer(be, rows * ep - (k0 >> 5));
    uint32_t vd = (uint32_t)((srow * ld + scol) * es), vc = (uint32_t)(srow * cp + scol);
    uint32_t ve = (uint32_t)(srow * ep + (scol >> 5));
    const uint32_t sd = (uint32_t)(kLgStage * ld * es), sc = (uint32_t)(kLgStage * cp), se = (uint32_t)(kLgStage * ep);
    // !AL: how far back the two chunks of 8 columns begin so as to end with the row, a
    // column of codes that exists, and where the slice's last stage begins (for loads past it)
    const bool n8 = a.n_out >= 8;
    int back[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) back[h] = (int)max<int64_t>(0, n0 + scol + 8 * h + 8 - a.n_out);
    const int xcol = (int)min<int64_t>(scol, cp - 16 - k0);
    const char* last_d = bd;
    const int8_t* last_c = bc;
    const uint8_t* last_e = be;
    auto load = [&](Regs& v) {
        if constexpr (AL) {
#pragma unroll
            for (int q = 0; q < ND; ++q)
                v.d[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rd, vd + q * 16, 0, 0));
            v.c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, vc, 0, 0));
            v.e = __builtin_amdgcn_raw_buffer_load_b8(re, ve, 0, 0);
            vd += sd;
            vc += sc;
            ve += se;
        } else {
            // any alignment, stride and size: one of the slice's rows in any case
            // (`put` clears it if it is not this thread's own)
            const int64_t row = max<int64_t>(0, min<int64_t>(srow, rows - 1));
            const char* rowd = rows > 0 ? bd : last_d;
            const TD* d = reinterpret_cast<const TD*>(rowd) + row * ld + scol;
            const int8_t* c = (rows > 0 ? bc : last_c) + row * cp + xcol;
            const uint8_t* e = (rows > 0 ? be : last_e) + row * ep + (xcol >> 5);
            if (n8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) load_raw8<TD>(d + 8 * h, back[h], v.d + h * ND / 2);
            } else {
                // rows of fewer than 8 columns: the only ones this tile's first chunk has
#pragma unroll
                for (int q = 0; q < ND; ++q) v.d[q] = (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
                for (int k = 0; k < 7; ++k) {
                    if (scol + k >= a.n_out) break;
                    if constexpr (sizeof(TD) == 4) v.d[k >> 2][k & 3] = __float_as_uint(d[k]);
                    else v.d[0][k >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, d[k]) << (16 * (k & 1));
                }
            }
            v.c = *reinterpret_cast<const u32x4*>(c);
            v.e = *e;
            v.live = srow < rows;
            if (rows > kLgStage) {
                last_d = bd + kLgStage * ld * es;
                last_c = bc + kLgStage * cp;
                last_e = be + kLgStage * ep;
            }
            rows -= kLgStage;
            bd += kLgStage * ld * es;
            bc += kLgStage * cp;
            be += kLgStage * ep;
        }
    };
    auto put = [&](Regs& v, char* buf) {
        if constexpr (!AL) {
            if (n8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) shift_raw8<TD>(min(back[h], 7), v.d + h * ND / 2);
            }
#pragma unroll
            for (int q = 0; q < ND; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) v.d[q][e] = v.live ? v.d[q][e] : 0u;
            v.e = v.live ? v.e : 0u;
        }
        if constexpr (NP == 1) {
            *reinterpret_cast<u32x4*>(buf + s0) = v.d[0];
            *reinterpret_cast<u32x4*>(buf + s1) = v.d[1];
        } else {
            uint32_t w[NP][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t h0, m0, l0, h1, m1, l1;
                split3(__uint_as_float(v.d[e / 2][2 * (e & 1)]), h0, m0, l0);
                split3(__uint_as_float(v.d[e / 2][2 * (e & 1) + 1]), h1, m1, l1);
                w[0][e] = high_halves(h0, h1);
                w[1][e] = high_halves(m0, m1);
                w[2][e] = high_halves(l0, l1);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                *reinterpret_cast<u32x4*>(buf + p * kRegion + s0) = (u32x4){w[p][0], w[p][1], w[p][2], w[p][3]};
                *reinterpret_cast<u32x4*>(buf + p * kRegion + s1) = (u32x4){w[p][4], w[p][5], w[p][6], w[p][7]};
            }
        }
        u32x4 lo, hi;
        held16(v.c, act_scale(v.e), lo, hi);
        *reinterpret_cast<u32x4*>(buf + NP * kRegion + s0) = lo;
        *reinterpret_cast<u32x4*>(buf + NP * kRegion + s1) = hi;
    };
    auto frag = [&](const char* p) {
        const u32x2 lo = lds_tr8(p), hi = lds_tr8(p + 4 * kRow);
        return __builtin_bit_cast(bf16x8, (u32x4){lo[0], lo[1], hi[0], hi[1]});
    };
    struct Frags {
        bf16x8 a[NP][2], b[2];
    };
    auto read = [&](Frags& f, const char* buf, int kg) {
#pragma unroll
        for (int j = 0; j < 2; ++j) f.b[j] = frag(buf + NP * kRegion + fb[j] + kg * 16 * kRow);
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) f.a[p][i] = frag(buf + p * kRegion + fa[i] + kg * 16 * kRow);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int p = NP - 1; p >= 0; --p)            // smallest part first
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[p][i], f.b[j], acc[i][j], 0, 0, 0);
    };

    // Stage s in two halves of 16 tokens.  While the first is multiplied, the
    // second's fragments are read and stage s + 1 goes from its registers into the other
    // LDS buffer (last read in stage s - 1, before that stage's barrier), the
    // load kAhead stages on taking its place (past the slice it loads zeros);
    // while the second is multiplied, the next stage's first fragments are read.
    const int stages = t1 > t0 ? (int)((t1 - t0 + kLgStage - 1) / kLgStage) : 0;
    Regs reg[kAhead];
    Frags f0, f1;
    auto step = [&](Regs& next, int s) {
        char* cur = ring + (s & 1) * kStageBytes;
        char* nxt = ring + ((s + 1) & 1) * kStageBytes;
        read(f1, cur, 1);
        put(next, nxt);
        load(next);
        multiply(f0);
        __syncthreads();
        read(f0, nxt, 0);
        multiply(f1);
    };
    if (stages > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load(reg[k]);
        put(reg[0], ring);
        load(reg[0]);
        __syncthreads();
        read(f0, ring, 0);
        // (in whole rounds of kAhead: stages past the last are zeros)
#pragma unroll 1
        for (int s = 0; s < stages; s += kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) step(reg[(k + 1) % kAhead], s + k);
        }
    }

    store_wave<TG, 2, 2>([&](int i, int j) -> const f32x16& { return acc[i][j]; },
                         slices > 1 ? a.partials + wk.slice * a.n_out * a.n_in : nullptr,
                         static_cast<TG*>(a.grad), a.accumulate, n0 + wm * 64, k0 + wn * 64, a.n_out,
                         a.n_in, lane);
}

// ---------------------------------------------------------------------------
// Large products: 256 x 256 tiles, eight waves, operands copied from global
// memory straight into LDS.
//
// Codes turned into bf16 inside the GEMM would be turned again by every tile
// row, so a first launch (k_lg_expand) turns X once into bf16 in the workspace,
// in the order the GEMM reads it: per 32 tokens, per 32 features, a 2 KB block
// of 32 feature rows of 32 tokens each, 16-byte chunk c (8 tokens) of row k at
// slot c ^ ((k >> 2) & 3).  A stage of a tile (32 tokens by 256 features) is
// then 16 KB in one piece, and a fragment (8 tokens of a feature) one 16-byte
// LDS read, at twice the rate of the transposing read that dY's fragments need.
// The wave tile is 128 features by 64 outputs, so four of a wave's six fragments
// per step are such reads.  Both expanded axes are padded with zeros (tokens to 32,
// features to 256).
//
// A ring of five stages (16 KB of dY, 16 KB of X each) is filled four stages
// ahead by buffer loads that write LDS; two waves per SIMD cover each other's
// waits.  Rows of dY past the last token and stages past the slice's end lie outside the
// buffer's extent, and arrive as zeros.
//
// 32768 tokens x 8192 outputs x 2048 inputs: k_lg_expand 35 us (84 MB read, 134 written: 6.3 TB/s), the products
// 792 to 880 us: 1.25 to 1.39 PFLOP/s, against 1.39 of the library's bf16 product of three
// 8192 x 8192 matrices and 920 to 935 us for the library's product of this shape from a
// bf16 X.  Bound by the matrix cores and the clock they leave.
// ---------------------------------------------------------------------------
constexpr int kBigTile = 256;
constexpr int kBigThreads = 512;
constexpr int kBigRegion = 16384;               // one operand's part of a stage
constexpr int kBigStage = 2 * kBigRegion;
constexpr int kBigStages = 5;
constexpr int kBigRow = 512;                    // LDS bytes of a token row of dY

__global__ __launch_bounds__(kThreads) void k_lg_expand(const int8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ exps,
                                                        char* __restrict__ out, int64_t n_tokens,
                                                        int64_t stages, int64_t cp, int64_t ep,
                                                        int64_t blocks_k) {
    __shared__ __attribute__((aligned(16))) char buf[kBigRegion];
    const int tid = threadIdx.x, oct = tid >> 6, f = (tid & 63) * 4;
    const int64_t k = (int64_t)blockIdx.x * kBigTile + f;
    for (int64_t s = blockIdx.y; s < stages; s += gridDim.y) {
        const int64_t t0 = s * kLgStage + oct * 8;
        uint32_t w[8], e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            w[r] = 0u;
            e[r] = 0u;
            if (t0 + r < n_tokens && k < cp) {
                w[r] = *reinterpret_cast<const uint32_t*>(codes + (t0 + r) * cp + k);
                e[r] = exps[(t0 + r) * ep + (k >> 5)];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4 v;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = pack_bf16(act_value(w[2 * q], c, act_scale(e[2 * q])),
                                 act_value(w[2 * q + 1], c, act_scale(e[2 * q + 1])));
            const int row = f + c;
            const int slot = oct ^ (((row & 31) >> 2) & 3);
            *reinterpret_cast<u32x4*>(buf + row * 64 + slot * 16) = v;
        }
        __syncthreads();
        char* o = out + (s * blocks_k + (int64_t)blockIdx.x * 8) * 2048;
#pragma unroll
        for (int i = 0; i < kBigRegion / (kThreads * 16); ++i) {
            const int at = (i * kThreads + tid) * 16;
            *reinterpret_cast<u32x4*>(o + at) = *reinterpret_cast<const u32x4*>(buf + at);
        }
        __syncthreads();
    }
}

// Rows of a dY that cannot be copied in aligned 16-byte pieces, into ones that can
// (stride n8, n_out rounded up to 8; the columns between are zeros).  16384 tokens x 2001
// outputs x 2048 inputs take 172 us with this copy, 220 on k_linear_grad's loads of odd rows.
__global__ __launch_bounds__(kThreads) void k_lg_align(const __bf16* __restrict__ dy, int64_t stride,
                                                       int64_t n_tokens, int64_t n_out,
                                                       __bf16* __restrict__ out, int64_t n8) {
    const int64_t col = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (col >= n8) return;
    const int cnt = (int)min<int64_t>(8, n_out - col);
    for (int64_t t = blockIdx.y; t < n_tokens; t += gridDim.y) {
        float v[8];
        load_unit<__bf16, false>(dy + t * stride + col, cnt, v);
        store_unit<__bf16, true>(out + t * n8 + col, 8, v);
    }
}

// The three bf16 parts of a float32 dY, as three matrices of `rows` token rows (whole stages;
// those past the last token are zeros) and n8 columns.  The product then runs over the three as
// over one token axis, and begins X again with each.  Bound by HBM: 8192 x 4096 in 51 us
// (335 MB, 6.6 TB/s), 32768 x 8192 in 520 (2.7 GB, 5.2).  With it, products by 256 x 256 tiles take
// 243 us instead of 309 by k_linear_grad's (8192 tokens x 4096 x 1024), 189 instead of 265
// (2048 x 8192 x 2048) and 2830 instead of 4120 (32768 x 8192 x 2048: 1.17 PFLOP/s of the
// three products' 3.3 TFLOP in all, 1.36 in the product itself).
template <bool AL>
__global__ __launch_bounds__(kThreads) void k_lg_split(const float* __restrict__ dy, int64_t stride,
                                                       int64_t n_tokens, int64_t n_out,
                                                       __bf16* __restrict__ out, int64_t rows, int64_t n8) {
    const int64_t col = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (col >= n8) return;
    const int cnt = (int)min<int64_t>(8, n_out - col);
    for (int64_t t = blockIdx.y; t < rows; t += gridDim.y) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (t < n_tokens) load_unit<float, AL>(dy + t * stride + col, cnt, v);
        uint32_t part[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3(v[e], part[0][e], part[1][e], part[2][e]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = high_halves(part[p][2 * i], part[p][2 * i + 1]);
            *reinterpret_cast<u32x4*>(out + (p * rows + t) * n8 + col) = w;
        }
    }
}

// s_waitcnt vmcnt(n) alone, n = 8 or 12.
__device__ __forceinline__ void wait_vm8() { __builtin_amdgcn_s_waitcnt(0x0F78); }
__device__ __forceinline__ void wait_vm12() { __builtin_amdgcn_s_waitcnt(0x0F7C); }

// Workgroup barrier that orders this wave's LDS reads around it without
// waiting for outstanding copies into LDS.
__device__ __forceinline__ void stage_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    __builtin_amdgcn_sched_barrier(0);
}

struct BigArgs {
    const char* dy;
    const char* xt;            // the expanded X
    void* grad;
    float* partials;
    int64_t n_tokens, n_out, n_in, dy_stride, dy_cols, blocks_k;     // dy_cols: n_out, or with padding
    int64_t xt_stages;         // stages of X: those of dY, or a third where dY is in parts
    int32_t tiles_n, tiles_k, slices, per;
    int32_t accumulate;
};

// This wave's copies of one stage: two 1 KB pieces of dY (two token rows each)
// and two of X.
struct BigCopy {
    const char* dy;            // this tile's columns of the stage's first token
    const char* xt;            // the stage's 16 KB of X
    int64_t dy_bytes;          // extent from dy to the end of the last row
    int64_t dy_step, xt_step;  // bytes from stage to stage
    int64_t left;              // stages not copied yet
    int64_t xt_left, xt_all;   // stages of X until it begins again, and all of them
    uint32_t voff_d[2], voff_x[2];
    uint32_t wbase;

    __device__ __forceinline__ void piece(uint32_t buf, int i) const {
        if (i < 2) dma16(make_rsrc(dy, left > 0 ? dy_bytes : 0), buf + wbase + i * 1024, voff_d[i]);
        else
            dma16(make_rsrc(xt, left > 0 ? kBigRegion : 0),
                  buf + kBigRegion + wbase + (i - 2) * 1024, voff_x[i - 2]);
    }
    __device__ __forceinline__ void next() {
        dy += dy_step;
        xt += xt_step;
        dy_bytes -= dy_step;
        --left;
        if (--xt_left == 0) {
            xt -= xt_all * xt_step;
            xt_left = xt_all;
        }
    }
};

template <typename TG>
__global__ __launch_bounds__(kBigThreads) void k_linear_grad_big(BigArgs a) {
    __shared__ __attribute__((aligned(1024))) char ring[kBigStages * kBigStage];
    const Work wk = work_of(blockIdx.x, gridDim.x, a.tiles_n, a.tiles_k);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 3, wx = wave >> 2;         // 64 outputs, 128 features each
    const int64_t n0 = (int64_t)wk.tn * kBigTile, k0 = (int64_t)wk.tk * kBigTile;
    const int64_t st0 = (int64_t)wk.slice * a.per;   // first stage of the slice
    const int64_t all = (a.n_tokens + kLgStage - 1) / kLgStage;
    const int nk = (int)min<int64_t>(a.per, all - st0);

    BigCopy cp;
    cp.dy = a.dy + (st0 * kLgStage * a.dy_stride + n0) * 2;
    cp.dy_bytes = ((a.n_tokens - st0 * kLgStage - 1) * a.dy_stride + a.dy_cols - n0) * 2;
    cp.dy_step = kLgStage * a.dy_stride * 2;
    const int64_t xt0 = st0 % a.xt_stages;
    cp.xt = a.xt + (xt0 * a.blocks_k + k0 / 32) * 2048;
    cp.xt_all = a.xt_stages;
    cp.xt_left = a.xt_stages - xt0;
    cp.xt_step = a.blocks_k * 2048;
    cp.left = nk;
    cp.wbase = (uint32_t)wave * 2048u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 4 * wave + 2 * i + (lane >> 5);
        const int chunk = (lane & 31) ^ ((row & 3) << 2);
        cp.voff_d[i] = (uint32_t)row * (uint32_t)(a.dy_stride * 2) + (uint32_t)chunk * 16u;
        cp.voff_x[i] = (uint32_t)(wave * 2048 + i * 1024 + lane * 16);
    }
    uint32_t fx[2], fd[2];
    {
        const int r32 = lane & 31, sw = (r32 >> 2) & 3, half = lane >> 5;
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
            fx[kg] = (uint32_t)(kBigRegion + (wx * 128 + r32) * 64 + (((2 * kg + half) ^ sw) << 4));
        const int g = lane >> 4, j = lane & 15, tsw = (j >> 2) & 3;
        const int row = 8 * (g >> 1) + (j >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int chunk = (((wn * 2 + i) ^ tsw) << 2) + 2 * (g & 1) + ((j & 3) >> 1);
            fd[i] = (uint32_t)(row * kBigRow + (chunk << 4) + 8 * (j & 1));
        }
    }
    auto frag_x = [&](const char* buf, int kg, int i) {
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(buf + fx[kg] + i * 2048));
    };
    auto frag_d = [&](const char* buf, int kg, int j) {
        const char* p = buf + fd[j] + kg * 16 * kBigRow;
        const u32x2 lo = lds_tr8(p), hi = lds_tr8(p + 4 * kBigRow);
        return __builtin_bit_cast(bf16x8, (u32x4){lo[0], lo[1], hi[0], hi[1]});
    };

    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const uint32_t lring = lds_addr(ring);
#pragma unroll
    for (int st = 0; st < kBigStages - 1; ++st) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp.piece(lring + st * kBigStage, i);
        cp.next();
    }
    // every wave always has the copies of four stages in flight (past the
    // slice's end they are empty), so the counts below hold for every stage
    wait_vm12();
    stage_barrier();
    bf16x8 xa[4], da[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) xa[i] = frag_x(ring, 0, i);
#pragma unroll
    for (int j = 0; j < 2; ++j) da[j] = frag_d(ring, 0, j);

    int slot = 0;
#pragma unroll 1
    for (int s = 0; s < nk; ++s) {
        const int nslot = slot == kBigStages - 1 ? 0 : slot + 1;
        const int tslot = slot == 0 ? kBigStages - 1 : slot - 1;    // stage s + 4
        const char* cur = ring + slot * kBigStage;
        const char* nxt = ring + nslot * kBigStage;
        const uint32_t tgt = lring + tslot * kBigStage;
        bf16x8 xb[4], db[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(da[0], xa[i], acc[i][0], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            xb[i] = frag_x(cur, 1, i);
            __builtin_amdgcn_sched_barrier(0);
            acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(da[1], xa[i], acc[i][1], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (i < 2) db[i] = frag_d(cur, 1, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        // stage s + 1 has landed once only those of the two after it are in flight; past
        // the barrier every wave has read stage s - 1 to its end
        wait_vm8();
        stage_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(db[0], xb[i], acc[i][0], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            cp.piece(tgt, i);
            __builtin_amdgcn_sched_barrier(0);
            acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(db[1], xb[i], acc[i][1], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            xa[i] = frag_x(nxt, 0, i);
            __builtin_amdgcn_sched_barrier(0);
            if (i < 2) da[i] = frag_d(nxt, 0, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        cp.next();
        slot = nslot;
    }

    // (the empty copies past the end)
    __builtin_amdgcn_s_waitcnt(0x0F70);
    store_wave<TG, 2, 4>([&](int j, int i) -> const f32x16& { return acc[i][j]; },
                         a.slices > 1 ? a.partials + wk.slice * a.n_out * a.n_in : nullptr,
                         static_cast<TG*>(a.grad), a.accumulate, n0 + wn * 64, k0 + wx * 128, a.n_out,
                         a.n_in, lane);
}

// The slices' partial sums, added in slice order.  AL: both arrays in whole,
// 16-byte aligned units of 8.  28 slices of 256 x 1024: 5.9 us, 29 MB out of the caches
// at 5 TB/s.
template <typename TG, bool AL>
__global__ __launch_bounds__(kThreads) void k_linear_join(const float* __restrict__ partials,
                                                          TG* __restrict__ grad, int64_t n,
                                                          int64_t slices, int accumulate) {
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (i >= n) return;
    const int cnt = (int)min<int64_t>(8, n - i);
    float acc[8];
    load_unit<float, AL>(partials + i, cnt, acc);
#pragma unroll 4
    for (int64_t s = 1; s < slices; ++s) {
        float v[8];
        load_unit<float, AL>(partials + s * n + i, cnt, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[e];
    }
    if (accumulate) {
        float old[8];
        load_unit<TG, AL>(grad + i, cnt, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += old[e];
    }
    store_unit<TG, AL>(grad + i, cnt, acc);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// What the kernel and the number of slices are chosen by: a model of a call's time
// in microseconds, fitted to sweeps of both kernels over 1 to 64 slices, 1024 to 32768
// tokens and 256 to 8192 outputs and inputs (its choice is within about 10 % of the best swept).
// stage: a workgroup's time per stage where 1, 2 or 3 of them share a CU (0: they
// do not fit); idle: how much less of it there is where nearly no CU is busy.
struct Model {
    double stage[3];
    double idle;
    double fixed;              // a workgroup's prologue and epilogue
};
constexpr Model kBigModel = {{0.66, 0.0, 0.0}, 0.14, 4.0};
constexpr Model kSmallBf16 = {{0.48, 0.60, 0.78}, 0.0, 4.7};
constexpr Model kSmallOdd = {{0.55, 0.75, 1.10}, 0.0, 4.7};      // bf16 rows at any address
constexpr Model kSmallFp32 = {{1.37, 2.10, 0.0}, 0.0, 5.0};
constexpr double kLaunchUs = 3.0;
constexpr double kPartialsPerUs = 7.5e5;   // partial sums written and read back
constexpr double kExpandPerUs = 1.7e6;     // codes expanded to bf16
constexpr double kAlignPerUs = 1.2e6;      // values of dY copied into aligned rows
constexpr double kSplitPerUs = 5.5e5;      // float32 values of dY cut into three parts

double modelled(const Model& m, int64_t groups, int64_t per, int64_t slices, double elems) {
    int most = 1;
    while (most < 3 && m.stage[most] > 0.0) ++most;
    const int64_t rounds = ceil_div(groups, kCus * most);
    const int64_t share = std::min<int64_t>(most, ceil_div(groups, kCus));
    const double busy = groups < kCus ? (double)groups / kCus : 1.0;
    return rounds * (per * (m.stage[share - 1] - m.idle * (1.0 - busy)) + m.fixed) +
           (slices > 1 ? kLaunchUs + slices * elems / kPartialsPerUs : 0.0);
}

}  // namespace

bool linear_grad_big_rows(const void* dy, int64_t n_out, int64_t stride) {
    return aligned16(dy) && n_out % 8 == 0 && stride % 8 == 0 && stride >= n_out &&
           stride <= (int64_t(1) << 24);
}

LgPlan linear_grad_plan(int64_t n_tokens, int64_t n_out, int64_t n_in, int32_t dy_dtype,
                        bool big_rows) {
    const int64_t stages = ceil_div(n_tokens, kLgStage);
    const double elems = (double)n_out * (double)n_in;
    const bool bf16 = dy_dtype == MA_PARAM_BF16;
    LgPlan best;
    double least = -1.0;
    for (int big = 0; big < 2; ++big) {
        // (below 512 outputs the expansion of X costs more than it saves)
        if (big && !(n_out >= 512 && n_in >= 256 && n_tokens >= 512)) continue;
        const int64_t tile = big ? kBigTile : kTile;
        const Model& m = big ? kBigModel : !bf16 ? kSmallFp32 : big_rows ? kSmallBf16 : kSmallOdd;
        LgPlan p;
        p.big = big != 0;
        p.tiles_n = ceil_div(n_out, tile);
        p.tiles_k = ceil_div(n_in, tile);
        const int64_t tiles = p.tiles_n * p.tiles_k;
        p.align = big && bf16 && !big_rows;
        p.split = big && !bf16;
        const int64_t run = p.split ? 3 * stages : stages;
        double expand = 0.0;
        if (p.big) expand += kLaunchUs + (double)n_tokens * (double)round_up(n_in, kBigTile) / kExpandPerUs;
        if (p.align) expand += kLaunchUs + (double)n_tokens * (double)n_out / kAlignPerUs;
        if (p.split) expand += kLaunchUs + (double)n_tokens * (double)n_out / kSplitPerUs;
        // (where the tiles are many, slices only even out the last round, for partial sums of
        // the gradient's size each: no more than 8 workgroups per CU come of them)
        const int64_t most = std::min<int64_t>({64, std::max<int64_t>(1, run / 4), ceil_div(8 * kCus, tiles)});
        for (int64_t n = 1; n <= most; ++n) {
            p.per = std::max<int64_t>(1, ceil_div(run, n));
            p.slices = std::max<int64_t>(1, ceil_div(run, p.per));
            const double t = expand + modelled(m, tiles * p.slices, p.per, p.slices, elems);
            if (least < 0.0 || t < least) {
                least = t;
                best = p;
            }
        }
    }
    best.total = best.slices > 1 ? (size_t)round_up(best.slices * n_out * n_in * 4, 256) : 0;
    if (best.big) {
        best.xt_off = best.total;
        best.total += (size_t)(stages * kLgStage) * (size_t)round_up(n_in, kBigTile) * 2;
    }
    if (best.align) {
        best.dy_off = best.total;
        best.total += (size_t)round_up(n_tokens * round_up(n_out, 8) * 2, 256);
    }
    if (best.split) {
        best.dy_off = best.total;
        best.total += (size_t)(3 * stages * kLgStage) * (size_t)round_up(n_out, 8) * 2;
    }
    return best;
}

namespace {

int launch_big(const LgArgs& a, const LgPlan& p, hipStream_t st) {
    const int64_t stages = ceil_div(a.n_tokens, kLgStage);
    char* xt = reinterpret_cast<char*>(a.partials) + p.xt_off;
    BigArgs b{};
    b.dy = static_cast<const char*>(a.dy);
    b.xt = xt;
    b.grad = a.grad;
    b.partials = a.partials;
    b.n_tokens = a.n_tokens;
    b.n_out = a.n_out;
    b.n_in = a.n_in;
    b.dy_stride = a.dy_stride;
    b.dy_cols = a.n_out;
    b.xt_stages = stages;
    if (p.align) {
        __bf16* rows = reinterpret_cast<__bf16*>(reinterpret_cast<char*>(a.partials) + p.dy_off);
        const int64_t n8 = round_up(a.n_out, 8);
        const dim3 agrid((unsigned)ceil_div(n8 / 8, kThreads), (unsigned)std::min<int64_t>(a.n_tokens, 4096));
        hipLaunchKernelGGL(k_lg_align, agrid, dim3(kThreads), 0, st, static_cast<const __bf16*>(a.dy),
                           a.dy_stride, a.n_tokens, a.n_out, rows, n8);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
        b.dy = reinterpret_cast<const char*>(rows);
        b.dy_stride = b.dy_cols = n8;
    } else if (p.split) {
        __bf16* rows = reinterpret_cast<__bf16*>(reinterpret_cast<char*>(a.partials) + p.dy_off);
        const int64_t n8 = round_up(a.n_out, 8), r = stages * kLgStage;
        const dim3 sgrid((unsigned)ceil_div(n8 / 8, kThreads), (unsigned)std::min<int64_t>(r, 4096));
        const float* dy = static_cast<const float*>(a.dy);
        if (aligned16(dy) && a.n_out % 8 == 0 && a.dy_stride % 4 == 0)
            hipLaunchKernelGGL((k_lg_split<true>), sgrid, dim3(kThreads), 0, st, dy, a.dy_stride, a.n_tokens,
                               a.n_out, rows, r, n8);
        else
            hipLaunchKernelGGL((k_lg_split<false>), sgrid, dim3(kThreads), 0, st, dy, a.dy_stride, a.n_tokens,
                               a.n_out, rows, r, n8);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
        b.dy = reinterpret_cast<const char*>(rows);
        b.dy_stride = b.dy_cols = n8;
        b.n_tokens = 3 * r;
    }
    b.blocks_k = round_up(a.n_in, kBigTile) / 32;
    b.tiles_n = (int)p.tiles_n;
    b.tiles_k = (int)p.tiles_k;
    b.slices = (int)p.slices;
    b.per = (int)p.per;
    b.accumulate = a.accumulate;
    const dim3 egrid((unsigned)p.tiles_k, (unsigned)std::min<int64_t>(stages, 65535));
    hipLaunchKernelGGL(k_lg_expand, egrid, dim3(kThreads), 0, st, a.codes, a.exps, xt, a.n_tokens,
                       stages, act_code_pitch(a.n_in), act_exp_pitch(a.n_in), b.blocks_k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_k * p.slices));
    if (a.grad_dtype == MA_PARAM_BF16)
        hipLaunchKernelGGL((k_linear_grad_big<__bf16>), grid, dim3(kBigThreads), 0, st, b);
    else
        hipLaunchKernelGGL((k_linear_grad_big<float>), grid, dim3(kBigThreads), 0, st, b);
    return (int)hipGetLastError();
}

template <typename TD, bool AL>
int launch_small_as(const LgArgs& a, const LgPlan& p, hipStream_t st) {
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_k * p.slices));
    if (a.grad_dtype == MA_PARAM_BF16)
        hipLaunchKernelGGL((k_linear_grad<TD, AL, __bf16>), grid, dim3(kThreads), 0, st, a,
                           (int)p.tiles_n, (int)p.tiles_k, (int)p.slices, (int)p.per);
    else
        hipLaunchKernelGGL((k_linear_grad<TD, AL, float>), grid, dim3(kThreads), 0, st, a,
                           (int)p.tiles_n, (int)p.tiles_k, (int)p.slices, (int)p.per);
    return (int)hipGetLastError();
}

int launch_small(const LgArgs& a, const LgPlan& p, hipStream_t st) {
    const bool bf16 = a.dy_dtype == MA_PARAM_BF16;
    const bool al = aligned16(a.dy) && a.n_out % 8 == 0 && a.dy_stride % (bf16 ? 8 : 4) == 0 &&
                    a.dy_stride >= a.n_out &&
                    p.per * kLgStage * std::max(a.dy_stride * (bf16 ? 2 : 4), act_code_pitch(a.n_in)) <
                        (int64_t(1) << 31);
    if (bf16) return al ? launch_small_as<__bf16, true>(a, p, st) : launch_small_as<__bf16, false>(a, p, st);
    return al ? launch_small_as<float, true>(a, p, st) : launch_small_as<float, false>(a, p, st);
}

template <typename TG, bool AL>
void launch_join(const LgArgs& a, const LgPlan& p, hipStream_t st) {
    const int64_t n = a.n_out * a.n_in;
    hipLaunchKernelGGL((k_linear_join<TG, AL>), dim3((unsigned)ceil_div(ceil_div(n, 8), kThreads)),
                       dim3(kThreads), 0, st, a.partials, static_cast<TG*>(a.grad), n, p.slices,
                       a.accumulate);
}

}  // namespace

int launch_linear_grad(const LgArgs& a, const LgPlan& p, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    const int e = p.big ? launch_big(a, p, st) : launch_small(a, p, st);
    if (e != (int)hipSuccess || p.slices == 1) return e;
    const bool al = a.n_out * a.n_in % 8 == 0 && aligned16(a.grad);
    if (a.grad_dtype == MA_PARAM_BF16) {
        if (al) launch_join<__bf16, true>(a, p, st); else launch_join<__bf16, false>(a, p, st);
    } else {
        if (al) launch_join<float, true>(a, p, st); else launch_join<float, false>(a, p, st);
    }
    return (int)hipGetLastError();
}

}  // namespace ma
