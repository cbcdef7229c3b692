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

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// Buffer resource: base address, stride 0, extent in bytes (accesses past it
// read zero), raw format.
__device__ __forceinline__ u32x4 make_rsrc(const void* base, int64_t bytes) {
    const uint64_t a = (uint64_t)base;
    u32x4 r;
    r.x = (uint32_t)a;
    r.y = (uint32_t)(a >> 32) & 0xffffu;
    r.z = bytes <= 0 ? 0u : bytes > 0x7fffffffLL ? 0x7fffffffu : (uint32_t)bytes;
    r.w = 0x00020000u;
    return r;
}

// 16 bytes per lane from global memory straight into LDS: lane t of the wave
// writes bytes [lds + 16 t, lds + 16 t + 16).  The kernel orders these copies
// itself, with explicit vmcnt waits and barriers.
__device__ __forceinline__ void dma16(u32x4 rsrc, uint32_t lds, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory");
}

// All of this wave's copies have landed, and every wave's LDS reads before are done.
__device__ __forceinline__ void copies_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0F70);          // vmcnt(0)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    __builtin_amdgcn_sched_barrier(0);
}

// One head of a packed array, as the rows of one sequence.
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

    // Where this thread's copy i comes from: its row of the tile and first column.
    struct From {
        int row, col;
    };
    __device__ static __forceinline__ From from(int i) {
        const int s = i * NT + (int)threadIdx.x, row = s / kChunks;
        return {row, ((s % kChunks) ^ turn(row)) * (16 / (int)sizeof(T))};
    }

    // Copies rows [row0, row0 + ROWS) of x into `lds`; rows past x.len and columns past x.dim
    // become zeros.  AL: rows and dim are whole 16-byte chunks, and the copies go straight into
    // LDS (they have landed after copies_barrier); extents within a tile stay below 2^31.
    template <bool AL>
    __device__ static __forceinline__ void copy(char* lds, const Rows<T>& x, int row0) {
        const int left = min(x.len - row0, ROWS);
        const T* base = x.p + (int64_t)row0 * x.stride;
        if constexpr (AL) {
            const u32x4 rsrc =
                make_rsrc(base, left > 0 ? ((int64_t)(left - 1) * x.stride + x.dim) * (int64_t)sizeof(T) : 0);
            const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024u;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const From f = from(i);
                const uint32_t at = (uint32_t)f.row * (uint32_t)(x.stride * sizeof(T)) + (uint32_t)(f.col * sizeof(T));
                dma16(rsrc, lds_addr(lds) + (uint32_t)(i * NT * 16) + wave,
                      f.col < x.dim && f.row < left ? at : 0x80000000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const From f = from(i);
                const T* p = base + (int64_t)f.row * x.stride + f.col;
                T v[16 / sizeof(T)];
#pragma unroll
                for (int e = 0; e < 16 / (int)sizeof(T); ++e)
                    v[e] = f.row < left && f.col + e < x.dim ? p[e] : (T)0.f;
                *reinterpret_cast<u32x4*>(lds + (i * NT + (int)threadIdx.x) * 16) =
                    __builtin_bit_cast(u32x4, v);
            }
        }
    }

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

// Straight operands of row `row` of x (zeros past its length and dim), from global memory.
template <typename T, int DP, bool AL>
__device__ __forceinline__ void load_row(const Rows<T>& x, int row, Frag<T>* f) {
    const int h = (threadIdx.x & 63) >> 5;
    const T* p = x.p + (int64_t)row * x.stride;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int col = 16 * s + 8 * h;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        if (row < x.len && col < x.dim) load_unit<T, AL>(p + col, x.dim - col, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[s][e] = (T)v[e];
    }
}

// Stores a wave's transposed results (columns of x by rows of 32 at a time) as row `row`:
// acc[b] element i is column 32 b + result_row(i, h).
template <typename T, int NB>
__device__ __forceinline__ void store_row(T* p, int dim, const f32x16* acc, float scale, bool wide) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = 32 * b + 8 * g + 4 * h;
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

// A value of lane ^ 32.
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

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

}  // namespace
}  // namespace ma
