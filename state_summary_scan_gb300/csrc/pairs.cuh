// pairs.cuh -- fp32 arithmetic on pairs (one issued instruction for two elements), and pairs of bf16.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace rmcp {

__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint64_t pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ void unpair(uint64_t p, uint32_t& x, uint32_t& y) { asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(p)); }
__device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// two bf16 in 32 bits, x in the lower half
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(uint64_t p) {
    uint32_t x, y;
    unpair(p, x, y);
    return pack2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ uint64_t widen2(uint32_t p) { return pair(p << 16, p & 0xffff0000u); }
// p as the sum of two bf16 pairs
__device__ __forceinline__ void split2(uint64_t p, uint32_t& hi, uint32_t& lo) {
    hi = pack2(p);
    lo = pack2(sub2(p, widen2(hi)));
}
// and of three, which hold the 24 bits of fp32
__device__ __forceinline__ void split2(uint64_t p, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack2(p);
    split2(sub2(p, widen2(hi)), mid, lo);
}

}  // namespace rmcp
