// Device helpers shared by the gradient operators' kernels: element types,
// vector access, and the 8-bit form of activations.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace ma {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}

// A column unit of 8 elements.  AL: whole and 16-byte aligned; otherwise
// only the first `cnt` (at least 1) exist, at any element's address: whole units
// still move as 16-byte accesses (global memory takes them at any alignment), the
// row's last part element by element.  Kernels that keep several loads in flight
// avoid that branch (after which the compiler waits for what was loaded in it): they
// shift a row's last unit back to end with the row, over columns of its neighbour.
typedef unsigned int u32x4u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x4u4 __attribute__((ext_vector_type(4), aligned(4)));

// NT: past the caches, for streams larger than they are.
template <bool NT, typename W>
__device__ __forceinline__ u32x4 get16(const W* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, typename W>
__device__ __forceinline__ void put16(W* p, u32x4 w) {
    if constexpr (NT) __builtin_nontemporal_store(w, p);
    else *p = w;
}

template <typename T>
__device__ __forceinline__ void widen(const u32x4* w, float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e >> 2][e & 3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[0][e] << 16);
            v[2 * e + 1] = __uint_as_float(w[0][e] & 0xffff0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ void narrow(const float* v, u32x4* w) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2][e & 3] = __float_as_uint(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[0][e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    }
}

template <typename T, bool AL, bool NT = false>
__device__ __forceinline__ void load_unit(const T* p, int cnt, float* v) {
    using W = std::conditional_t<AL, u32x4, std::conditional_t<sizeof(T) == 4, u32x4u4, u32x4u2>>;
    if (AL || cnt >= 8) {
        u32x4 w[sizeof(T) / 2];
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) w[q] = get16<NT>(reinterpret_cast<const W*>(p) + q);
        widen<T>(w, v);
    } else {
        // (loads past cnt repeat the last element: without a branch around each, all
        // are in flight together)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = (float)p[min(e, cnt - 1)];
            v[e] = e < cnt ? x : 0.f;
        }
    }
}

template <typename T, bool AL, bool NT = false>
__device__ __forceinline__ void store_unit(T* p, int cnt, const float* v) {
    using W = std::conditional_t<AL, u32x4, std::conditional_t<sizeof(T) == 4, u32x4u4, u32x4u2>>;
    if (AL || cnt >= 8) {
        u32x4 w[sizeof(T) / 2];
        narrow<T>(v, w);
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) put16<NT>(reinterpret_cast<W*>(p) + q, w[q]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) p[e] = (T)v[e];
    }
}

// ------------------------------------------------- activations in 8 bits --
// A group of 32 features is held as codes q and one exponent byte b = e + 127:
// x stands for q 2^e.  With the group's largest magnitude m 2^k (1 <= m < 2),
// e = k - 6 makes the largest quotient 64 m, which rounds to at most 127 for
// 64 m < 127.5; above that e = k - 5.  The byte is kept within [1, 248], so the
// scale and its inverse are normal floats and 127 2^e is finite; quotients are
// exact (powers of two) and rounded once, to nearest even.

// Exponent byte of a group from the bits of its largest magnitude (as an
// unsigned integer: NaN above infinity above every finite value).
__device__ __forceinline__ uint32_t act_exp_byte(uint32_t top) {
    const int k = (int)(top >> 23);                              // biased exponent
    if (k == 255) return 255u;                                   // infinity or NaN
    const int b = k - 6 + ((top & 0x7fffffu) >= 0x7f0000u ? 1 : 0);
    return (uint32_t)min(max(b, 1), 248);
}

// 2^(b - 127); infinity for the NaN mark 255, so that code 0 times it is NaN.
__device__ __forceinline__ float act_scale(uint32_t b) { return __uint_as_float(b << 23); }
// 2^(127 - b) for b in [1, 248]; 0 for the NaN mark.
__device__ __forceinline__ float act_inv_scale(uint32_t b) {
    return b == 255u ? 0.f : __uint_as_float((254u - b) << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The codes of 8 values, lowest byte first.  Adding 1.5 2^23 to a quotient rounds
// it to an integer (nearest, ties to even: the sum's unit is 1) and leaves that
// in the low bits, so a product and rounding are one fma, and the low byte is the
// two's complement code.  Only at the largest exponent can a quotient round above
// 127 and has to be cut.
__device__ __forceinline__ u32x2 act_codes(const float* v, uint32_t b) {
    const float inv = act_inv_scale(b);
    float q[8];
    if (__builtin_expect(__any(b == 248u), 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = __builtin_amdgcn_fmed3f(v[e] * inv, -127.f, 127.f) + 12582912.f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = fmaf(v[e], inv, 12582912.f);
    }
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // v_perm_b32 picks bytes of {second, first} = 7..0
        const uint32_t a = __builtin_amdgcn_perm(__float_as_uint(q[4 * h + 1]), __float_as_uint(q[4 * h]), 0x0c0c0400u);
        const uint32_t c = __builtin_amdgcn_perm(__float_as_uint(q[4 * h + 3]), __float_as_uint(q[4 * h + 2]), 0x0c0c0400u);
        w[h] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    }
    // (a NaN's payload may end in any byte)
    if (b == 255u) w = (u32x2){0u, 0u};
    return w;
}

__device__ __forceinline__ float act_value(uint32_t w, int byte, float scale) {
    return (float)(int)(int8_t)(w >> (8 * byte)) * scale;
}

}  // namespace
}  // namespace ma
