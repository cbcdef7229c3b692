// The gradients of the keys and values: a workgroup takes 32 key rows a wave of one key head
// and walks the queries of the heads that share it, recomputing the scores S = Q K^T and P =
// 2^(S - lse), with dP = dout V^T and dS = P (dP - delta) summing dv^T += dout^T P and dk^T +=
// Q^T dS: four products a tile.
//
// 20011 tokens of 7 sequences, 16 / 4 heads of 128, bf16, in 575 to 605 us (502 GFLOP, 0.83 to 0.87
// PFLOP/s) and 41 to join two pieces: matrix instructions on 55 % of a SIMD's cycles, vector ones on 33, LDS reads
// on 42 % of the CU's.  All 256 registers are taken: constant LDS slots, two
// tiles a turn as in the other walks, spill.
//
// Heads of 256 in bfloat16 spill 16 registers, most of them fragments of K or V that are read back inside the
// loop over tiles, and each of those reads waits for every copy into LDS too, so the next tile's are not
// under way during this one: 10011 tokens of 4 sequences, 8 / 1 heads, take 807 us, 0.36 PFLOP/s.

#include <hip/hip_runtime.h>

#include "attention_tile.h"

namespace ma {
namespace {

// Whether a workgroup's rows of V stay in LDS instead of registers, which then fit two waves.
template <typename T, int DP>
constexpr bool kStage = sizeof(T) == 2 && DP == 128;

template <typename T, int DP, int WAVES>
__global__ __launch_bounds__(64 * WAVES * kHalves<DP>, (kPer<T, DP>)) void k_attention_dkv(AttnArgs a, AttnGrid grid) {
    constexpr int BLOCK = 32 * WAVES, QT = 32, RING = 2, HALVES = kHalves<DP>, DW = DP / HALVES, ALL = WAVES * HALVES;
    using QTile = Tile<T, DP, QT, 64 * ALL>;
    using VTile = Tile<T, DP, BLOCK, 64 * ALL>;
    // with dk and dv of 128 columns in registers there is room for two operands, not four
    // (20011 tokens, 16 / 4 heads of 128: 1061 us a backward against 1145 with spills and 1135
    // without reading ahead; of 256: 1110 against 1437 and 1236; of 64, four: 628 against 649)
    constexpr int AHEAD = DP >= 128 ? 2 : kAhead<T>;
    constexpr bool STAGE = kStage<T, DP>;
    __shared__ __attribute__((aligned(1024))) char lds[RING][2][QTile::kBytes];
    __shared__ __attribute__((aligned(1024))) char vlds[STAGE ? VTile::kBytes : 16];
    __shared__ __attribute__((aligned(256))) float stat[RING][ALL][2 * QT];
    __shared__ Exchange<HALVES == 2 ? ALL : 0> exchange;
    const Job j = job_of<true, BLOCK>(a, grid);        // (its head is a key head)
    if (!j.any) return;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave % HALVES;
    const int group = a.heads / a.kv_heads;
    const int key = j.row0 + 32 * (wave / HALVES) + (lane & 31);
    const Rows<T> kx = rows_of<T>(a.k, j.head, j.k_at, j.k_len, a.cols);
    const Rows<T> vx = rows_of<T>(a.v, j.head, j.k_at, j.k_len, a.cols);
    // (of two waves one forms the scores, the other dout v)
    Frag<T> kf[DP / 16], vf[HALVES == 1 && !STAGE ? DP / 16 : 1];
    load_row<T, DP / 16>(half == 0 ? kx : vx, key, 0, kf);
    if constexpr (STAGE) {
        const typename VTile::Copy copy_v(vx);
        copy_v(vlds, vx, j.row0);
    } else if constexpr (HALVES == 1) {
        load_row<T, DP / 16>(vx, key, 0, vf);
    }
    f32x16 dk[DW / 32], dv[DW / 32];
#pragma unroll
    for (int b = 0; b < DW / 32; ++b) dk[b] = dv[b] = zero16();
    const float k = a.scale * kLog2e;
    // the first tile with a query that sees this workgroup's first key
    const int off = j.k_len - j.q_len;
    const int first = a.causal ? max(0, j.row0 - off) / QT : 0;
    const int per = max(0, (j.q_len + QT - 1) / QT - first);
    const Share sh(per * group, j.piece, grid.pieces);
    const typename QTile::Copy copy_q(rows_of<T>(a.q, 0, 0, 0, a.cols)), copy_d(rows_of<T>(a.dout, 0, 0, 0, a.cols));
    // the next tile to copy: its number, its head of the group, and which of the head's it is
    int next = sh.first, nhead = per ? sh.first / per : 0, ntile = sh.first - nhead * per, ahead = 0;
    auto fetch = [&]() {
        const bool in = next < sh.last;          // (past the last tile the copies are empty)
        const int head = j.head * group + (in ? nhead : 0), q0 = in ? (first + ntile) * QT : j.q_len;
        copy_q(lds[ahead][0], rows_of<T>(a.q, head, j.q_at, j.q_len, a.cols), q0);
        copy_d(lds[ahead][1], rows_of<T>(a.dout, head, j.q_at, j.q_len, a.cols), q0);
        const float* s = a.stats + ((int64_t)head * a.n_queries + j.q_at + q0) * 2;
        dma4(make_rsrc(s, (int64_t)(j.q_len - q0) * 8), lds_addr(stat[ahead][wave]), lane * 4u);
        ahead ^= 1;
        ++next;
        if (++ntile == per) {
            ntile = 0;
            ++nhead;
        }
    };
    int slot = 0;
    auto tile = [&](int n, auto part) {
        copies_barrier<0>();
        fetch();
        const char* qt = lds[slot][0];
        const char* dt = lds[slot][1];
        const float* sd = stat[slot][wave];
        slot ^= 1;
        f32x16 s = zero16(), p = zero16();
        constexpr int ND = DP / 16;
        if constexpr (HALVES == 1) {
            struct Two {
                Frag<T> a, v;
            };
            read_ahead<2 * ND, AHEAD>(
                [&](int i) {
                    Two f;
                    f.a = QTile::rows(i < ND ? qt : dt, 0, i % ND);
                    if constexpr (STAGE) {
                        if (i >= ND) f.v = VTile::rows(vlds, 32 * wave, i % ND);
                    }
                    return f;
                },
                [&](int i, const Two& f) {
                    if (i < ND) s = mma(f.a, kf[i], s);
                    else if constexpr (STAGE) p = mma(f.a, f.v, p);
                    else p = mma(f.a, vf[i - ND], p);
                });
        } else {
            const char* mine = half == 0 ? qt : dt;
            read_ahead<ND, AHEAD>([&](int d) { return QTile::rows(mine, 0, d); },
                                      [&](int d, const Frag<T>& f) { s = mma(f, kf[d], s); });
            p = exchange(s);
            if (half == 1) {
                const f32x16 t = s;
                s = p;
                p = t;
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            // lse and delta of four queries
            const f32x4 x = *reinterpret_cast<const f32x4*>(sd + 16 * g + 8 * h);
            const f32x4 y = *reinterpret_cast<const f32x4*>(sd + 16 * g + 8 * h + 4);
            const float l4[4] = {x[0], x[2], y[0], y[2]}, d4[4] = {x[1], x[3], y[1], y[3]};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * g + e;
                s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], k, -l4[e]));
                p[i] = s[i] * (p[i] - d4[e]);
            }
        }
        if constexpr (decltype(part)::value) {
            // the first query of the tile that sees this lane's key
            const int from = key - off - (first + n) * QT;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool in = result_row(i, h) >= from;
                s[i] = in ? s[i] : 0.f;
                p[i] = in ? p[i] : 0.f;
            }
        }
        constexpr int NB = DW / 32;
        const Frag<T> fs[2] = {frag_of<T>(s, 0), frag_of<T>(s, 1)}, fp[2] = {frag_of<T>(p, 0), frag_of<T>(p, 1)};
        read_ahead<4 * NB, AHEAD>(
            [&](int i) { return QTile::cols(i < 2 * NB ? dt : qt, 16 * (i / NB % 2), half * DW + 32 * (i % NB)); },
            [&](int i, const Frag<T>& f) {
                if (i < 2 * NB) dv[i % NB] = mma(f, fs[i / NB], dv[i % NB]);
                else dk[i % NB] = mma(f, fp[i / NB - 2], dk[i % NB]);
            });
    };
    if (sh.first < sh.last) {
        // of a head's tiles the first `partial` hold queries that do not see every key of the
        // workgroup
        const int partial = a.causal ? max(0, (j.row0 + BLOCK - 1 - off + QT - 1) / QT - first) : 0;
        int n = ntile;
        fetch();
        for (int t = sh.first; t < sh.last;) {
            const int stop = min(per, n + sh.last - t);
            t += stop - n;
            for (; n < min(stop, partial); ++n) tile(n, std::true_type{});
            for (; n < stop; ++n) tile(n, std::false_type{});
            n = 0;
        }
    }
    if (key >= j.k_len) return;
    const int64_t row = (int64_t)j.k_at + key;
    if (grid.pieces > 1) {
        store_row<float, DW / 32>(part_row(a.parts, j.piece, a.kv_heads, j.head, a.n_keys, row, a.dim), a.dim, half * DW,
                                  dk, a.scale, a.dim % 4 == 0);
        store_row<float, DW / 32>(part_row(a.parts, grid.pieces + j.piece, a.kv_heads, j.head, a.n_keys, row, a.dim),
                                  a.dim, half * DW, dv, 1.f, a.dim % 4 == 0);
    } else {
        store_row<T, DW / 32>(row_of<T>(a.dk, j.head, row), a.dim, half * DW, dk, a.scale, a.wide);
        store_row<T, DW / 32>(row_of<T>(a.dv, j.head, row), a.dim, half * DW, dv, 1.f, a.wide);
    }
}

}  // namespace

int launch_attention_dkv(const AttnArgs& a, const AttnSplit& sp, void* stream) {
    const AttnGrid grid = grid_of(a.n_keys, a.n_seqs, a.kv_heads, sp.rows, sp.pieces);
    return by_kind(a, sp.rows, [&](auto t, auto dp, auto wv) {
        constexpr int DP = decltype(dp)::value, WAVES = decltype(wv)::value;
        // (float32 and 256 features: workgroups of 64 or 32 rows; else 128 or 64)
        if constexpr (sizeof(t) == 4 && kHalves<DP> == 2 ? WAVES <= 2 : WAVES >= 2)
            hipLaunchKernelGGL((k_attention_dkv<decltype(t), DP, WAVES>),
                               dim3((unsigned)grid.slots * a.kv_heads * grid.pieces), dim3(64 * WAVES * kHalves<DP>), 0,
                               (hipStream_t)stream, a, grid);
    });
}

}  // namespace ma
