// Pieces of the paged attention kernels: mma.sync with bf16 or f16 operands,
// ldmatrix, conversions of e4m3 values, packed fp32, and the output's store.
//
// One new token's query heads of one key head are at most a few rows, and a
// byte of the cache takes part in 2 * rows operations: the tensor pipe idles
// whichever instruction feeds it, and the warp-wide form leaves every warp
// free to stream its own keys without waiting for another.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "attn_internal.cuh"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoRef = -3e38f;   // a softmax row's reference before its first finite logit

namespace mma {

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).  Lane (g, c) = (lane / 4, lane %
// 4) holds rows g, g + 8 and columns 2c, 2c + 1 of D; a0/a2 rows g, a1/a3 rows
// g + 8 of A at k = 2c.. (a0, a1) and 2c + 8.. (a2, a3); b0/b1 column g of B
// at k = 2c.. and 2c + 8...
template <bool kF16>
__device__ __forceinline__ void m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared-memory loads.  Volatile without a memory clobber: they stay between
// the barrier waits and the warp barriers around them (which have one), and
// the products may move among them.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t saddr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr));
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t saddr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr));
}

__device__ __forceinline__ uint4 lds128(uint32_t saddr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr));
    return v;
}

// The two e4m3 values in the low 16 bits, as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// Two f16 values to e4m3 (nearest, finite), in the low 16 bits.
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t two) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed pairs of fp32.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void upk(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The same, NaN if one of them is.
__device__ __forceinline__ float max3n(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Over an e4m3 cache a query row is held as q * 2^(to - e), with e this exponent
// of its largest value (2^e <= top < 2^(e+1)).  bf16 reaches 2^127; below 2^-100
// the row keeps less of its bits, which no logit in the range of fp32 shows.
__device__ __forceinline__ int query_exponent(float top) { return top > 0.f ? max(-100, min(127, ilogbf(top))) : 0; }

// What takes such a row's products with the keys as stored to powers of two:
// scale * 2^(e - to) * k_scale.  Kept finite and above 0, so that a product of 0
// and a masked one of -infinity stay what they are.
__device__ __forceinline__ float query_factor(float scale, int e_to, float k_scale) {
    return fmaxf(1e-37f, fminf(3e38f, scale * exp2f((float)e_to) * k_scale));
}

// Four consecutive channels of one head's output row; a row that sees no key is
// zero whatever its gate holds.
__device__ __forceinline__ void store4(const AttnIO& io, size_t at, float4 v, bool sees) {
    if (io.gate && sees) {
        const float4 g = *reinterpret_cast<const float4*>(io.gate + at);
        v.x /= 1.f + exp2_approx(-g.x * kLog2e);
        v.y /= 1.f + exp2_approx(-g.y * kLog2e);
        v.z /= 1.f + exp2_approx(-g.z * kLog2e);
        v.w /= 1.f + exp2_approx(-g.w * kLog2e);
    }
    if (io.o_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(io.o) + at) = v;
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(io.o) + at) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

}  // namespace mma
}  // namespace kda
