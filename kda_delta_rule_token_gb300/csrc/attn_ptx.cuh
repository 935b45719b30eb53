// Inline-PTX wrappers beyond ptx.cuh and tc.cuh that the attention kernels
// use, written from the PTX ISA: barrier tests, 5-D TMA loads, register
// splits, and kind::f16 MMAs with f16 or bf16 operands in either majorness.
// A file of its own: recorded profiles of the other kernels hold for exact
// versions of those two headers.
#pragma once

#include <stdint.h>

#include "ptx.cuh"
#include "tc.cuh"

namespace kda {
namespace ptx {

constexpr int kErrAttnWait = 1 << 5;   // beside the error-word bits of ptx.cuh

// Whether the phase with the given parity is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* m, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(m)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Tiled TMA load of a 5-D box (coordinates innermost first) into shared
// memory, completing its bytes on mbarrier m.
__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* m) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(smem_u32(dst)), "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(m))
        : "memory");
}

}  // namespace ptx

namespace tc {

// Shared-memory matrix descriptor: K-major, SWIZZLE_128B, 8-row atoms `eight` bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t eight) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(eight >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same of an MN-major operand: rows of 128 bytes (64 16-bit elements of
// MN) for consecutive K, 8-row atoms `eight` bytes apart along K, further
// blocks of 64 elements of MN `block` bytes on.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr, uint32_t block, uint32_t eight) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(eight >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor: kind::f16 with A and B both bf16 or both f16, D =
// f32, A K-major, B K-major or (b_mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_f16kind(int M, int N, bool bf16, bool b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands (A packed two per 32-bit column).
__device__ __forceinline__ void mma_ts_f16kind(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], both e4m3, K = 32 per instruction (the
// instruction descriptor is idesc_f16kind's for f16, whose type fields are 0).
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Registers of the calling warpgroup's threads (every warp of it calls).
template <int kRegs>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

}  // namespace tc
}  // namespace kda
