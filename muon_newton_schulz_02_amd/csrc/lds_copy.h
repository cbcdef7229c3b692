// Copies from global memory straight into LDS, shared by every kernel that
// stages its operands so.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ma {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Buffer resource (gfx9 layout): base address, stride 0, extent in bytes (reads past it
// return zero) and the raw 32-bit-element format word.
__device__ __forceinline__ u32x4 make_rsrc(const void* base, int64_t bytes) {
    const uint64_t a = (uint64_t)base;
    u32x4 r;
    r.x = (uint32_t)a;
    r.y = (uint32_t)(a >> 32) & 0xffffu;
    r.z = bytes <= 0 ? 0u : bytes > 0x7fffffffLL ? 0x7fffffffu : (uint32_t)bytes;
    r.w = 0x00020000u;
    return r;
}

// LDS byte address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// 16 (or 4) bytes per lane into LDS: lane t of the wave writes bytes [lds + 16 t,
// lds + 16 t + 16).  Issued as inline assembly so the compiler's own wait-count insertion
// does not treat every later LDS read as dependent on it (it cannot tell the stage
// buffers apart); the kernel orders these copies itself with explicit vmcnt waits and
// barriers.  Nor does the compiler put in the wait state that has to lie between the write of
// m0 and the copy that reads it: s_nop 0 is that state.
__device__ __forceinline__ void dma16(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma16(u32x4 rsrc, uint32_t lds, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(u32x4 rsrc, uint32_t lds, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

}  // namespace
}  // namespace ma
