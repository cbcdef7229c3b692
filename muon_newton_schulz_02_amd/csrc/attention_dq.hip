// The gradient of the queries: a workgroup takes 32 query rows a wave of one head and walks
// the keys, recomputing the scores S^T = K Q^T and P^T = 2^(S^T - lse), with dP^T = V dout^T
// and dS^T = P^T (dP^T - delta) summing dq^T += K^T dS^T: three products a tile.
//
// Bound as the forward pass is: 20011 tokens of 7 sequences, 16 / 4 heads of 128, bf16, in 385 us (376
// GFLOP, 0.98 PFLOP/s), matrix instructions on 58 % of a SIMD's cycles, vector ones on 39.

#include <hip/hip_runtime.h>

#include "attention_tile.h"

namespace ma {
namespace {

// The copies of tile t + RING - 1 are under way while tile t is worked on.
template <typename T, int DP>
constexpr int kRing = DP * (int)sizeof(T) <= 256 ? 3 : 2;
template <typename T, int DP, int WAVES>
__global__ __launch_bounds__(64 * WAVES * kHalves<DP>, (kPer<T, DP>)) void k_attention_dq(AttnArgs a, AttnGrid grid) {
    constexpr int BLOCK = 32 * WAVES, KV = 32, RING = kRing<T, DP>, HALVES = kHalves<DP>, DW = DP / HALVES;
    using KT = Tile<T, DP, KV, 64 * WAVES * HALVES>;
    constexpr int kTileCopies = 2 * KT::kCopies;
    __shared__ __attribute__((aligned(1024))) char lds[RING][2][KT::kBytes];
    __shared__ Exchange<HALVES == 2 ? 2 * WAVES : 0> exchange;
    const Job j = job_of<false, BLOCK>(a, grid);
    if (!j.any) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
    const int half = __builtin_amdgcn_readfirstlane(wave % HALVES);
    const int kvh = j.head / (a.heads / a.kv_heads);
    const Rows<T> kx = rows_of<T>(a.k, kvh, j.k_at, j.k_len, a.cols);
    const Rows<T> vx = rows_of<T>(a.v, kvh, j.k_at, j.k_len, a.cols);
    const Rows<T> qx = rows_of<T>(a.q, j.head, j.q_at, j.q_len, a.cols);
    const Rows<T> dx = rows_of<T>(a.dout, j.head, j.q_at, j.q_len, a.cols);
    const int q = j.row0 + 32 * (wave / HALVES) + (lane & 31);
    // (of two waves one forms the scores, the other dout v)
    Frag<T> qf[DP / 16], df[HALVES == 1 ? DP / 16 : 1];
    load_row<T, DP / 16>(half == 0 ? qx : dx, q, 0, qf);
    if constexpr (HALVES == 1) load_row<T, DP / 16>(dx, q, 0, df);
    const float* st = a.stats + ((int64_t)j.head * a.n_queries + j.q_at + q) * 2;
    const float ls = q < j.q_len ? st[0] : kInf, delta = q < j.q_len ? st[1] : 0.f;

    f32x16 dq[DW / 32];
#pragma unroll
    for (int b = 0; b < DW / 32; ++b) dq[b] = zero16();
    const float k = a.scale * kLog2e;
    const int end = min(j.row0 + BLOCK, j.q_len) - 1;
    const Share sh(max(0, seen(a, j, end) + KV - 1) / KV, j.piece, grid.pieces);
    const int sees = seen(a, j, q);
    const typename KT::Copy copy_k(kx), copy_v(vx);
    int ahead = 0;
    // (past the last tile the copies are empty)
    auto fetch = [&](int t) {
        const int row = t < sh.last ? t * KV : j.k_len;
        copy_k(lds[ahead][0], kx, row);
        copy_v(lds[ahead][1], vx, row);
        ahead = ahead == RING - 1 ? 0 : ahead + 1;
    };
    auto tile = [&](int t, auto slot, auto part) {
        constexpr int AT = decltype(slot)::value;
        copies_barrier<(RING - 2) * kTileCopies>();
        fetch(t + RING - 1);
        const char* kt = lds[AT][0];
        const char* vt = lds[AT][1];
        f32x16 s = zero16(), p = zero16();
        constexpr int ND = DP / 16, NB = DW / 32;
        if constexpr (HALVES == 1) {
            read_ahead<2 * ND, kAhead<T>>([&](int i) { return KT::rows(i < ND ? kt : vt, 0, i % ND); },
                                          [&](int i, const Frag<T>& f) {
                                              if (i < ND) s = mma(f, qf[i], s);
                                              else p = mma(f, df[i - ND], p);
                                          });
        } else {
            const char* mine = half == 0 ? kt : vt;
            read_ahead<ND, kAhead<T>>([&](int d) { return KT::rows(mine, 0, d); },
                                      [&](int d, const Frag<T>& f) { s = mma(f, qf[d], s); });
            p = exchange(s);
            if (half == 1) {
                const f32x16 t = s;
                s = p;
                p = t;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(s[i], k, -ls)) * (p[i] - delta);
        if constexpr (decltype(part)::value) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = t * KV + result_row(i, h) < sees ? p[i] : 0.f;
        }
        const Frag<T> fp[2] = {frag_of<T>(p, 0), frag_of<T>(p, 1)};
        read_ahead<2 * NB, kAhead<T>>([&](int i) { return KT::cols(kt, 16 * (i / NB), half * DW + 32 * (i % NB)); },
                                      [&](int i, const Frag<T>& f) { dq[i % NB] = mma(f, fp[i / NB], dq[i % NB]); });
    };
    if (sh.first < sh.last) {
        for (int i = 0; i < RING - 1; ++i) fetch(sh.first + i);
        // tiles that every row of the workgroup sees whole, and the others
        const int whole = min(max(seen(a, j, j.row0), 0) / KV, sh.last);
        // (the ring's slots as constants, as in the forward pass)
        int t = sh.first;
        for (; t + RING <= whole; t += RING) {
            tile(t, Int<0>{}, std::false_type{});
            tile(t + 1, Int<1>{}, std::false_type{});
            if constexpr (RING == 3) tile(t + 2, Int<2>{}, std::false_type{});
        }
        for (; t < sh.last; t += RING) {
            tile(t, Int<0>{}, std::true_type{});
            if (t + 1 < sh.last) tile(t + 1, Int<1>{}, std::true_type{});
            if constexpr (RING == 3)
                if (t + 2 < sh.last) tile(t + 2, Int<2>{}, std::true_type{});
        }
    }
    if (q >= j.q_len) return;
    const int64_t row = (int64_t)j.q_at + q;
    if (grid.pieces > 1)
        store_row<float, DW / 32>(part_row(a.parts, j.piece, a.heads, j.head, a.n_queries, row, a.dim), a.dim,
                                  half * DW, dq, a.scale, a.dim % 4 == 0);
    else
        store_row<T, DW / 32>(row_of<T>(a.dq, j.head, row), a.dim, half * DW, dq, a.scale, a.wide);
}

}  // namespace

int launch_attention_dq(const AttnArgs& a, const AttnSplit& sp, void* stream) {
    const AttnGrid grid = grid_of(a.n_queries, a.n_seqs, a.heads, sp.rows, sp.pieces);
    return by_kind(a, sp.rows, [&](auto t, auto dp, auto wv) {
        constexpr int DP = decltype(dp)::value, WAVES = decltype(wv)::value;
        if constexpr (WAVES * kHalves<DP> == 4 || WAVES * kHalves<DP> == 2)
            hipLaunchKernelGGL((k_attention_dq<decltype(t), DP, WAVES>),
                               dim3((unsigned)grid.slots * a.heads * grid.pieces), dim3(64 * WAVES * kHalves<DP>), 0,
                               (hipStream_t)stream, a, grid);
    });
}

}  // namespace ma
