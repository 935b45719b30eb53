// RMS norm of every query and key head, rotary position, and the keys and
// values into their cache slots, in one pass over a step's new tokens.
//
//   y = x * rsqrt(mean(x^2) + eps) * gamma
//   (a, b) <- (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq
//
// The call moves each value once (reads (Hq + 2 Hkv) * 128 bf16 per token,
// writes as many in bf16 or e4m3) and computes a few operations per byte: it
// is bound by HBM at prompt sizes and by the launch at single tokens.  Measured:
// 16381 tokens of 32 + 8 + 8 heads in bf16, 403 MB: 78 us, 5.2 TB/s, 0.77 of the
// measured copy rate; one token 4 us.  What is left at prompt sizes is the
// latency of each half warp's chain position -> angles -> rows (the SMs issue
// 43 % of the time): fewer rows loaded ahead (two: 88 us), more CTAs per SM
// (four: 79 us) or more half warps per token (two: 89 us) were not faster.
//
// Sixteen lanes (a half warp) take one token, or a share of its heads, and go
// through them a row at a time, eight consecutive channels per lane (16-byte
// loads and stores), kBatch rows loaded ahead.  What depends on the token
// alone is made once: with C = gamma cos and S = -+ gamma' sin (gamma' the
// partner channel's), a row needs only x <- (x C + x' S) * rsqrt(...), one
// product and one sum per channel, the partner x' exchanged as loaded.  The
// angle is exact at any position: position * turn modulo 2^64 is the fraction of
// a full turn, and its top 32 bits give the quadrant and the rest of the angle,
// whose sine and cosine the Taylor series at 0 gives to fp32.  A token's heads are shared out among as many half warps (up to
// 16) as it takes to give every SM its threads: 1 for prompts, 16 for a step
// of few requests.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "attn_internal.cuh"
#include "attn_mma.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadLanes = 16;
constexpr int kBatch = 4;

using mma::f32x2;

// Eight bf16 values as four packed pairs of fp32.
__device__ __forceinline__ void unpack8(const uint4& u, f32x2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mma::pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const f32x2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        mma::upk(x[i], a, b);
        w[i] = mma::pack_bf16(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Cosine and sine of u / 2^32 of a full turn: the nearest quarter turn, and x
// within pi / 4 of it, where the series' first omitted terms (x^10 / 10!,
// x^11 / 11!) are below 2^-25.
__device__ __forceinline__ void cos_sin(uint32_t u, float& c, float& s) {
    const uint32_t quarter = (u + (1u << 29)) >> 30;
    const float x = (float)(int)(u - (quarter << 30)) * (float)(1.57079632679489661923 / (1 << 30));
    const float x2 = x * x;
    float sn = fmaf(x2, 1.f / 362880, -1.f / 5040);
    sn = fmaf(x2, sn, 1.f / 120);
    sn = fmaf(x2, sn, -1.f / 6);
    sn = fmaf(x2 * x, sn, x);
    float cs = fmaf(x2, 1.f / 40320, -1.f / 720);
    cs = fmaf(x2, cs, 1.f / 24);
    cs = fmaf(x2, cs, -0.5f);
    cs = fmaf(x2, cs, 1.f);
    const bool swap = quarter & 1;
    c = swap ? sn : cs;
    s = swap ? cs : sn;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

template <bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3)
kda_attn_append_kernel(const AttnLayer l, const __grid_constant__ RopeTurns turns, const AttnAppendIO io,
                       int share_shift, int* err) {
    __shared__ uint64_t s_turn[kHeadDim / 2];
    if (threadIdx.x < kHeadDim / 2) s_turn[threadIdx.x] = turns.turn[threadIdx.x];
    __syncthreads();
    const int lane = threadIdx.x & (kHeadLanes - 1);
    const long long job = (long long)blockIdx.x * (kThreads / kHeadLanes) + threadIdx.x / kHeadLanes;
    const int shares = 1 << share_shift, share = (int)(job & (shares - 1));
    const long long tok = job >> share_shift;
    if (tok >= io.N) return;
    // The two half warps of a warp go their own ways: shuffles name one of them.
    const uint32_t mask = 0xffffu << (threadIdx.x & 16);
    const int d0 = lane * 8, half = l.rotary >> 1;
    const bool turned = d0 < l.rotary;
    const int span = l.rotary >> 4;              // lanes of the first half of the rotated channels
    const bool second = lane >= span;            // channel d pairs with d - half, else with d + half
    const int partner = (second ? lane - span : lane + span) & 15;

    const int pos = io.positions[tok];
    const long long slot = io.slots[tok];
    float cs[8], sn[8];                          // of this lane's channels, sn with the sign of x'
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turned) {
#pragma unroll
        for (int e = 0; e < (kInterleaved ? 4 : 8); ++e) {
            const int p = kInterleaved ? d0 / 2 + e : (second ? d0 - half : d0) + e;
            float s, c;
            cos_sin((uint32_t)(((uint64_t)(long long)pos * s_turn[p]) >> 32), c, s);
            if (kInterleaved) {
                cs[2 * e] = cs[2 * e + 1] = c;
                sn[2 * e] = -s;
                sn[2 * e + 1] = s;
            } else {
                cs[e] = c;
                sn[e] = second ? s : -s;
            }
        }
    }

    // Heads first, first + shares, ... of q, k or v.
    auto rows = [&](const uint16_t* src, int first, int heads, const float* gamma, auto norm_rotate, auto&& store) {
        f32x2 C[4], S[4];
        if (norm_rotate) {
            float4 g0 = make_float4(1.f, 1.f, 1.f, 1.f), g1 = g0;
            if (gamma) {
                g0 = *reinterpret_cast<const float4*>(gamma + d0);
                g1 = *reinterpret_cast<const float4*>(gamma + d0 + 4);
            }
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = sn[e] * (kInterleaved ? g[e ^ 1] : __shfl_sync(mask, g[e], partner, 16));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                C[e] = mma::pk(cs[2 * e] * g[2 * e], cs[2 * e + 1] * g[2 * e + 1]);
                S[e] = mma::pk(t[2 * e], t[2 * e + 1]);
            }
        }
        for (int h0 = first; h0 < heads; h0 += kBatch * shares) {
            uint4 raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (h0 + i * shares < heads)
                    raw[i] = *reinterpret_cast<const uint4*>(src + (size_t)(h0 + i * shares) * kHeadDim + d0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int h = h0 + i * shares;
                if (h >= heads) break;
                f32x2 x[4];
                unpack8(raw[i], x);
                if (norm_rotate) {
                    float rn = 1.f;
                    if (gamma) {
                        f32x2 ss2 = mma::mul2(x[0], x[0]);
#pragma unroll
                        for (int e = 1; e < 4; ++e) ss2 = mma::fma2(x[e], x[e], ss2);
                        float a, b;
                        mma::upk(ss2, a, b);
                        float ss = a + b;
#pragma unroll
                        for (int m = 1; m < kHeadLanes; m <<= 1) ss += __shfl_xor_sync(mask, ss, m);
                        rn = rsqrtf(ss * (1.0f / kHeadDim) + l.rms_eps);
                    }
                    uint4 o = raw[i];   // the partners
                    if (kInterleaved) {
                        o = make_uint4(__byte_perm(o.x, 0, 0x1032), __byte_perm(o.y, 0, 0x1032),
                                       __byte_perm(o.z, 0, 0x1032), __byte_perm(o.w, 0, 0x1032));
                    } else {
                        o.x = __shfl_sync(mask, o.x, partner, 16);
                        o.y = __shfl_sync(mask, o.y, partner, 16);
                        o.z = __shfl_sync(mask, o.z, partner, 16);
                        o.w = __shfl_sync(mask, o.w, partner, 16);
                    }
                    // Channels that are not rotated have no partner: 0 * infinity is none of their business.
                    if (!turned) o = make_uint4(0u, 0u, 0u, 0u);
                    f32x2 y[4];
                    unpack8(o, y);
                    const f32x2 rn2 = mma::pk(rn, rn);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mma::mul2(mma::fma2(y[e], S[e], mma::mul2(x[e], C[e])), rn2);
                }
                store(h, x, raw[i]);
            }
        }
    };

    const int of_k = (share - l.Hq) & (shares - 1), of_v = (share - l.Hq - l.Hkv) & (shares - 1);
    rows(io.q + tok * io.q_stride, share, l.Hq, l.q_gamma, std::true_type(), [&](int h, const f32x2 (&x)[4], const uint4&) {
        *reinterpret_cast<uint4*>(io.q_out + ((size_t)tok * l.Hq + h) * kHeadDim + d0) = pack8(x);
    });

    if (slot < 0 || slot >= ((long long)l.num_pages << l.page_shift)) {
        if (slot != -1 && lane == 0) atomicOr(err, kErrAttnIndex);
        return;
    }
    const size_t at = ((size_t)(slot >> l.page_shift) * l.Hkv * l.page_size + (slot & (l.page_size - 1))) * kHeadDim + d0;
    const size_t head_pitch = (size_t)l.page_size * kHeadDim;
    auto quantised = [&](void* cache, const float* scale, int h, const f32x2 (&x)[4]) {
        const float inv = 1.0f / scale[h];
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) mma::upk(mma::mul2(x[e], mma::pk(inv, inv)), y[2 * e], y[2 * e + 1]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at + h * head_pitch) =
            make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
    };
    rows(io.k + tok * io.k_stride, of_k, l.Hkv, l.k_gamma, std::true_type(), [&](int h, const f32x2 (&x)[4], const uint4&) {
        if (kE4m3) quantised(l.k_cache, l.k_scale, h, x);
        else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(l.k_cache) + at + h * head_pitch) = pack8(x);
    });
    rows(io.v + tok * io.v_stride, of_v, l.Hkv, nullptr, std::false_type(), [&](int h, const f32x2 (&x)[4], const uint4& raw) {
        if (kE4m3) quantised(l.v_cache, l.v_scale, h, x);
        else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(l.v_cache) + at + h * head_pitch) = raw;
    });
}

}  // namespace

cudaError_t launch_attn_append(const AttnLayer& l, const RopeTurns& turns, const AttnAppendIO& io,
                               const DeviceInfo& dev, int* err_word, cudaStream_t stream) {
    // Half warps per token: as few as fill the SMs' threads, since each makes
    // the token's angles for itself.
    const long long full = (long long)dev.sm_count * 2048 / kHeadLanes;
    int shift = 0;
    while (shift < 4 && ((long long)io.N << shift) < full) ++shift;
    const int per = kThreads / kHeadLanes;
    const long long grid = (((long long)io.N << shift) + per - 1) / per;
    auto kernel = l.e4m3 ? (l.interleaved ? kda_attn_append_kernel<true, true> : kda_attn_append_kernel<true, false>)
                         : (l.interleaved ? kda_attn_append_kernel<false, true> : kda_attn_append_kernel<false, false>);
    kernel<<<(unsigned)grid, kThreads, 0, stream>>>(l, turns, io, shift, err_word);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
