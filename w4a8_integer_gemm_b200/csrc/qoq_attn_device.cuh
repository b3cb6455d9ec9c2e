// qoq_attn_device.cuh -- device code the attention kernels share: waits,
// asynchronous copies, and the expansion of cached codes to FP16.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "qoq_attn_internal.h"
#include "qoq_ptx.cuh"

namespace qoq {

// Asynchronous copy of 16 bytes, or zeros without reading when not valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src)
{
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// wait_bounded() for waits of a microsecond: try_wait without a time hint
// suspends the thread in hardware and wakes it when the phase completes; the
// hint adds sleeps and clock reads between tries, which took half of the
// attention kernel's issue slots.  The clock is looked at every 64 tries.
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity, volatile int *abort, uint64_t budget_ns)
{
    uint64_t start = 0;
    for (uint32_t tries = 1; !mbar_try_wait(bar, parity); ++tries) {
        if (tries % 64) continue;
        if (*abort) return false;
        const uint64_t now = global_timer_ns();
        if (start == 0) start = now;
        if (now - start > budget_ns) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// Minimum and maximum that are NaN where an operand is.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// 32 bytes at once, 32-byte aligned.
__device__ __forceinline__ void st_global32(void *dst, uint4 a, uint4 b)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr)
{
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
    return x;
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 x)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Eight 4-bit codes -> fp16(s c + m), in order.  A nibble in bits 0-3 under
// the exponent of 1024 is 1024 + c, in bits 4-7 under that of 64 it is
// 64 + c (the mantissa's unit is 2^-4 there); so with a byte in both halves of
// a word one logic operation and one exact subtraction give its two codes,
// and one multiply-add rounds once.  par: (s, m).  The exponent patterns come
// in a register, e4 = 0x54006400, whose value the compiler does not know: a
// logic instruction has room for one constant, and with two it becomes two.
__device__ __forceinline__ uint4 expand4(uint32_t x, uint32_t par, uint32_t e4)
{
    const uint32_t s = __byte_perm(par, par, 0x1010), m = __byte_perm(par, par, 0x3232);
    const uint32_t a = sub_h2((__byte_perm(x, x, 0x0000) & 0x00F0000Fu) | e4, 0x54006400u);
    const uint32_t b = sub_h2((__byte_perm(x, x, 0x1111) & 0x00F0000Fu) | e4, 0x54006400u);
    const uint32_t c = sub_h2((__byte_perm(x, x, 0x2222) & 0x00F0000Fu) | e4, 0x54006400u);
    const uint32_t d = sub_h2((__byte_perm(x, x, 0x3333) & 0x00F0000Fu) | e4, 0x54006400u);
    return make_uint4(fma_h2(a, s, m), fma_h2(b, s, m), fma_h2(c, s, m), fma_h2(d, s, m));
}

// Eight 8-bit codes (x: channels 0-3, y: 4-7) -> fp16(s c + m), in order.
__device__ __forceinline__ uint4 expand8(uint32_t x, uint32_t y, uint32_t par, uint32_t e6)
{
    const uint32_t s = __byte_perm(par, par, 0x1010), m = __byte_perm(par, par, 0x3232);
    const uint32_t a = sub_h2(__byte_perm(x, e6, 0x5150), 0x64006400u);
    const uint32_t b = sub_h2(__byte_perm(x, e6, 0x5352), 0x64006400u);
    const uint32_t c = sub_h2(__byte_perm(y, e6, 0x5150), 0x64006400u);
    const uint32_t d = sub_h2(__byte_perm(y, e6, 0x5352), 0x64006400u);
    return make_uint4(fma_h2(a, s, m), fma_h2(b, s, m), fma_h2(c, s, m), fma_h2(d, s, m));
}

}  // namespace qoq
