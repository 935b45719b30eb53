// RMS norm of every query and key head, rotary position, and the keys and
// values into their cache slots, in one pass over a step's new tokens.
//
//   y = x * rsqrt(mean(x^2) + eps) * gamma
//   (a, b) <- (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq
//
// The call moves each value once (reads (Hq + 2 Hkv) * 128 bf16 per token,
// writes as many in bf16 or e4m3) and computes a few operations per byte: it
// is bound by HBM at prompt sizes and by the launch at single tokens.
//
// Sixteen lanes hold one head of one token, eight consecutive channels each
// (16-byte loads and stores); the norm is a sum over sixteen lanes and the
// partner of a rotated channel lies eight values in another lane (or in the
// same one, when the pairs are interleaved).  The angles depend on token and
// channel only, so a CTA computes them once for its tokens: position *
// turn modulo 2^64 is the exact fraction of a full turn (integer arithmetic,
// no loss at far positions), its top 32 bits as a signed fraction of a half
// turn go to sincospif.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "attn_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadLanes = 16;
constexpr int kRowsPerPass = kThreads / kHeadLanes;
constexpr int kHalf = kHeadDim / 2;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
kda_attn_append_kernel(const AttnLayer l, const __grid_constant__ RopeTurns turns, const AttnAppendIO io,
                       int tokens_per_cta, int* err) {
    extern __shared__ float s_trig[];   // [tokens][cos of 64 pairs, sin of 64 pairs]
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tokens_per_cta;
    const int nt = min(tokens_per_cta, io.N - t0);
    const int half = l.rotary >> 1;
    for (int i = tid; i < nt * kHalf; i += kThreads) {
        const int t = i / kHalf, p = i % kHalf;
        if (p < half) {
            const uint64_t turn = (uint64_t)(long long)io.positions[t0 + t] * turns.turn[p];
            float s, c;
            sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
            s_trig[t * kHeadDim + p] = c;
            s_trig[t * kHeadDim + kHalf + p] = s;
        }
    }
    __syncthreads();

    const int heads = l.Hq + 2 * l.Hkv;
    const int lane = tid & (kHeadLanes - 1);
    const int d0 = lane * 8;
    const long long slots = (long long)l.num_pages << l.page_shift;
    const int rows = nt * heads;
    // All sixteen lanes of a head, and both heads of a warp, stay in the loop
    // together (the shuffles below name the whole warp).
    const int rounds = (rows + kRowsPerPass - 1) / kRowsPerPass;
    for (int i = 0; i < rounds; ++i) {
        const int r = i * kRowsPerPass + tid / kHeadLanes;
        const bool live = r < rows;
        const int t = live ? r / heads : 0, h = live ? r % heads : 0;
        const int tok = t0 + t;
        const int kind = h < l.Hq ? 0 : h < l.Hq + l.Hkv ? 1 : 2;   // q, k, v
        const int hh = kind == 0 ? h : kind == 1 ? h - l.Hq : h - l.Hq - l.Hkv;
        const uint16_t* src = (kind == 0 ? io.q + tok * io.q_stride : kind == 1 ? io.k + tok * io.k_stride
                                                                                 : io.v + tok * io.v_stride) +
                              (size_t)hh * kHeadDim + d0;
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(src), x);
        const float* gamma = kind == 0 ? l.q_gamma : kind == 1 ? l.k_gamma : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int m = 1; m < kHeadLanes; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (gamma) {
            const float rn = rsqrtf(ss * (1.0f / kHeadDim) + l.rms_eps);
            const float4 g0 = *reinterpret_cast<const float4*>(gamma + d0);
            const float4 g1 = *reinterpret_cast<const float4*>(gamma + d0 + 4);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * rn * g[e];
        }
        const float* trig = s_trig + t * kHeadDim;
        if (kInterleaved) {
            if (kind != 2 && d0 < l.rotary) {
                const float4 c = *reinterpret_cast<const float4*>(trig + d0 / 2);
                const float4 s = *reinterpret_cast<const float4*>(trig + kHalf + d0 / 2);
                const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = x[2 * e], b = x[2 * e + 1];
                    x[2 * e] = a * cs[e] - b * sn[e];
                    x[2 * e + 1] = b * cs[e] + a * sn[e];
                }
            }
        } else {
            // Channel d of the first half pairs with d + half: rotary / 16 lanes on.
            const int span = l.rotary / 16;
            const bool second = lane >= span;
            const int partner = (tid & 16) + ((second ? lane - span : lane + span) & 15);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
            if (kind != 2 && d0 < l.rotary) {
                const int p = second ? d0 - half : d0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 c = *reinterpret_cast<const float4*>(trig + p + 4 * q);
                    const float4 s = *reinterpret_cast<const float4*>(trig + kHalf + p + 4 * q);
                    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[4 * q + e] = x[4 * q + e] * cs[e] + (second ? y[4 * q + e] : -y[4 * q + e]) * sn[e];
                }
            }
        }
        if (!live) continue;
        if (kind == 0) {
            *reinterpret_cast<uint4*>(io.q_out + ((size_t)tok * l.Hq + hh) * kHeadDim + d0) = pack8(x);
            continue;
        }
        const long long slot = io.slots[tok];
        if (slot < 0 || slot >= slots) {
            if (slot != -1 && lane == 0) atomicOr(err, kErrAttnIndex);
            continue;
        }
        const long long page = slot >> l.page_shift;
        const int row = (int)(slot & (l.page_size - 1));
        const size_t at = (((size_t)page * l.Hkv + hh) * l.page_size + row) * kHeadDim + d0;
        void* cache = kind == 1 ? l.k_cache : l.v_cache;
        if (kE4m3) {
            const float inv = 1.0f / (kind == 1 ? l.k_scale : l.v_scale)[hh];
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) =
                make_uint2(pack4_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                           pack4_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at) = pack8(x);
        }
    }
}

}  // namespace

cudaError_t launch_attn_append(const AttnLayer& l, const RopeTurns& turns, const AttnAppendIO& io,
                               const DeviceInfo& dev, int* err_word, cudaStream_t stream) {
    // One token per CTA while that leaves room on the SMs, else four, so that
    // the angles' latency is paid once per four tokens.
    const int per = io.N <= 8 * dev.sm_count ? 1 : 4;
    const int grid = (io.N + per - 1) / per;
    const size_t smem = (size_t)per * kHeadDim * sizeof(float);
    auto kernel = l.e4m3 ? (l.interleaved ? kda_attn_append_kernel<true, true> : kda_attn_append_kernel<true, false>)
                         : (l.interleaved ? kda_attn_append_kernel<false, true> : kda_attn_append_kernel<false, false>);
    kernel<<<grid, kThreads, smem, stream>>>(l, turns, io, per, err_word);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
