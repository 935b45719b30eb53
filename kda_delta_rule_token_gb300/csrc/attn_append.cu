// RMS norm of every query and key head, rotary position, and the keys and
// values into their cache slots, in one pass over a step's new tokens.
//
//   y = x * rsqrt(mean(x^2) + eps) * gamma
//   (a, b) <- (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq
//
// The call moves each value once (reads (Hq + 2 Hkv) * 128 bf16 per token,
// writes as many in bf16 or e4m3) and computes a few operations per byte: it
// is bound by HBM at prompt sizes and by the launch at single tokens.  Measured:
// 16381 tokens of 32 + 8 + 8 heads in bf16, 403 MB: 68 us, 5.9 TB/s, 0.88 of the
// measured copy rate (131072 tokens: at that rate); one token 4 us.
//
// A unit is four heads of q, of k or of v of two tokens, one token to each half
// warp, eight consecutive channels per lane.  Warps take equal, contiguous
// ranges of units, however they cut a token's: every SM has all its warps from
// a step of 600 tokens on.  A prompt's ranges are six units, several times as
// many as are resident, dealt by the hardware as warps end (one long range per
// resident warp: 80 us, the SMs that are slower to reach the memory last; 12
// units 70 us, 4 units 74 us, where starting a range costs).  A lane copies its
// own 16 bytes of three units ahead into shared memory (cp.async), so that
// neither a token's angles nor the sums of a row hold up the loads (without
// copies ahead, a token or a power-of-two share of its heads per half warp: 80 us,
// 2000 tokens 29 us where they take 19 now).
//
// What depends on the token alone is made once a range: with C = gamma cos and
// S = -+ gamma' sin (gamma' the partner channel's), a row needs only
// x <- (x C + x' S) * rsqrt(...), one product and one sum per channel, the
// partner x' exchanged as loaded.  The angle is exact at any position: position *
// turn modulo 2^64 is the fraction of a full turn, and its top 32 bits give the
// quadrant and the rest of the angle, whose sine and cosine the Taylor series at
// 0 gives to fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "attn_internal.cuh"
#include "attn_mma.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kCtasPerSm = 6;
constexpr int kBatch = 4;                        // heads of a unit
constexpr int kDepth = 3;                        // units of a warp in flight or in use
constexpr int kWarpUnits = 6;                    // of a warp, where there are more than the resident ones' share

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

__device__ __forceinline__ void store_e4m3(uint8_t* to, const f32x2 (&x)[4], float inv) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) mma::upk(mma::mul2(x[e], mma::pk(inv, inv)), y[2 * e], y[2 * e + 1]);
    *reinterpret_cast<uint2*>(to) = make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
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

// A lane's own 16 bytes of a row, copied behind the computation.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(kLeft) : "memory"); }

// A unit of a pair of tokens: up to kBatch heads of q, k or v.
struct Units {
    int q, k, all;   // units of q, of k, of q, k and v
};

template <bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
kda_attn_append_kernel(const AttnLayer l, const __grid_constant__ RopeTurns turns, const AttnAppendIO io,
                       const Units units, long long total, int warps, int* err) {
    __shared__ uint4 s_rows[kDepth][kBatch][kThreads];
    __shared__ uint64_t s_turn[kHeadDim / 2];
    __shared__ float s_gamma[2][kHeadDim];
    __shared__ float4 s_angle[4][kThreads];      // a lane's channels': cosines, and sines with the sign of x'
    const int tid = threadIdx.x, lane = tid & 15, side = (tid >> 4) & 1;
    const int w = (int)blockIdx.x * (kThreads / 32) + (tid >> 5);
    // The warp's units, the same number for all to within one.
    const long long first = total * w / warps;
    const int left = w < warps ? (int)(total * (w + 1) / warps - first) : 0;
    const int d0 = lane * 8, half = l.rotary >> 1;

    // A place among the units, the copies' ahead of the computation's.
    struct Place {
        long long tok;   // of this half warp
        int unit;
    };
    Place at{2 * (first / units.all) + side, (int)(first % units.all)};
    Place ahead = at;
    int to_copy = left;
    auto copy = [&](int stage) {
        if (to_copy > 0 && ahead.tok < io.N) {
            const bool is_q = ahead.unit < units.q, is_v = ahead.unit >= units.q + units.k;
            const int h0 = (ahead.unit - (is_q ? 0 : is_v ? units.q + units.k : units.q)) * kBatch;
            const uint16_t* src = (is_q ? io.q + ahead.tok * io.q_stride : is_v ? io.v + ahead.tok * io.v_stride
                                                                                 : io.k + ahead.tok * io.k_stride) +
                                  (size_t)h0 * kHeadDim + d0;
            const int heads = (is_q ? l.Hq : l.Hkv) - h0;
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(&s_rows[stage][0][tid]);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i < heads) copy16(to + i * kThreads * 16, src + i * kHeadDim);
        }
        copies_commit();
        --to_copy;
        if (++ahead.unit == units.all) {
            ahead.unit = 0;
            ahead.tok += 2;
        }
    };
#pragma unroll
    for (int st = 0; st < kDepth; ++st) copy(st);

    for (int i = tid; i < kHeadDim / 2; i += kThreads) s_turn[i] = turns.turn[i];
    for (int i = tid; i < kHeadDim; i += kThreads) {
        s_gamma[0][i] = l.q_gamma ? l.q_gamma[i] : 1.f;
        s_gamma[1][i] = l.k_gamma ? l.k_gamma[i] : 1.f;
    }
    __syncthreads();

    const bool turned = d0 < l.rotary;
    const int span = l.rotary >> 4;              // lanes of the first half of the rotated channels
    const bool second = lane >= span;            // channel d pairs with d - half, else with d + half
    const int partner = (second ? lane - span : lane + span) & 15;
    const size_t head_pitch = (size_t)l.page_size * kHeadDim;

    int pos = 0;
    long long slot = -1;
    auto token = [&](long long tok, int& p, long long& sl) {
        p = tok < io.N ? io.positions[tok] : 0;
        sl = tok < io.N ? io.slots[tok] : -1;
    };
    if (left > 0) token(at.tok, pos, slot);

    bool live = false, stored = false;
    size_t to = 0;                               // of this lane's channels in the cache's first head
    int next_pos = 0;
    long long next_slot = -1;
    f32x2 C[4], S[4];                            // cosines and sines with the norm's weights
    int kind = -1;                               // that C and S are for: q, k
    for (int n = 0, stage = 0; n < left; ++n) {
        if (kind < 0) {   // a pair's first unit here
            live = at.tok < io.N;
            stored = slot >= 0 && slot < ((long long)l.num_pages << l.page_shift);
            if (!stored && slot != -1 && lane == 0) atomicOr(err, kErrAttnIndex);
            if (stored)
                to = ((size_t)(slot >> l.page_shift) * l.Hkv * l.page_size + (slot & (l.page_size - 1))) * kHeadDim + d0;
            const int p0 = pos;
            token(at.tok + 2, next_pos, next_slot);
            // Four angles per lane: its own (interleaved), or half of those that it shares with its partner.
            float c4[4] = {1.f, 1.f, 1.f, 1.f}, s4[4] = {0.f, 0.f, 0.f, 0.f};
            if (turned) {
                const int a0 = kInterleaved ? d0 / 2 : second ? d0 - half + 4 : d0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    cos_sin((uint32_t)(((uint64_t)(long long)p0 * s_turn[a0 + e]) >> 32), c4[e], s4[e]);
            }
            if (kInterleaved) {
                s_angle[0][tid] = make_float4(c4[0], c4[0], c4[1], c4[1]);
                s_angle[1][tid] = make_float4(c4[2], c4[2], c4[3], c4[3]);
                s_angle[2][tid] = make_float4(-s4[0], s4[0], -s4[1], s4[1]);
                s_angle[3][tid] = make_float4(-s4[2], s4[2], -s4[3], s4[3]);
            } else {
                float c[4], sn[4];   // the partner's
                const float sign = second ? 1.f : -1.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    c[e] = __shfl_sync(0xffffffffu, c4[e], partner, 16);
                    sn[e] = sign * __shfl_sync(0xffffffffu, s4[e], partner, 16);
                    s4[e] *= sign;
                    if (!turned) {
                        c[e] = 1.f;
                        sn[e] = 0.f;
                    }
                }
                s_angle[second][tid] = make_float4(c4[0], c4[1], c4[2], c4[3]);
                s_angle[!second][tid] = make_float4(c[0], c[1], c[2], c[3]);
                s_angle[2 + second][tid] = make_float4(s4[0], s4[1], s4[2], s4[3]);
                s_angle[3 - second][tid] = make_float4(sn[0], sn[1], sn[2], sn[3]);
            }
        }
        const bool is_q = at.unit < units.q, is_v = at.unit >= units.q + units.k;
        const int h0 = (at.unit - (is_q ? 0 : is_v ? units.q + units.k : units.q)) * kBatch;
        const int heads = (is_q ? l.Hq : l.Hkv) - h0;
        if (!is_v && kind != !is_q) {
            kind = !is_q;
            const float* gamma = s_gamma[kind];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 c = s_angle[x][tid], sn = s_angle[2 + x][tid];
                const float4 g = *reinterpret_cast<const float4*>(gamma + d0 + 4 * x);
                const float4 o = kInterleaved ? make_float4(g.y, g.x, g.w, g.z)
                                              : *reinterpret_cast<const float4*>(gamma + partner * 8 + 4 * x);
                C[2 * x] = mma::pk(c.x * g.x, c.y * g.y);
                C[2 * x + 1] = mma::pk(c.z * g.z, c.w * g.w);
                S[2 * x] = mma::pk(sn.x * o.x, sn.y * o.y);
                S[2 * x + 1] = mma::pk(sn.z * o.z, sn.w * o.w);
            }
        }
        kind = max(kind, 0);

        // Where the unit's rows go, and the distance between two.
        const bool to_cache = !is_q, writes = is_q ? live : stored;
        const size_t pitch = is_q ? kHeadDim : head_pitch;
        const size_t off = is_q ? ((size_t)at.tok * l.Hq + h0) * kHeadDim + d0 : to + h0 * head_pitch;
        void* dst = is_q ? static_cast<void*>(io.q_out) : is_v ? l.v_cache : l.k_cache;
        uint16_t* dst16 = static_cast<uint16_t*>(dst) + off;
        uint8_t* dst8 = static_cast<uint8_t*>(dst) + off;
        float inv[kBatch];
        if (kE4m3 && to_cache) {
            const float* scale = (is_v ? l.v_scale : l.k_scale) + h0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) inv[i] = i < heads ? 1.0f / scale[i] : 0.f;
        }
        const bool norm = (is_q ? l.q_gamma : l.k_gamma) != nullptr;

        // kRows rows from row i0 of the unit on.
        auto rows = [&](auto count, int i0) {
            constexpr int kRows = decltype(count)::value;
            uint4 raw[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) raw[i] = s_rows[stage][i0 + i][tid];
            if (is_v) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    if (kE4m3) {
                        f32x2 x[4];
                        unpack8(raw[i], x);
                        if (writes) store_e4m3(dst8 + (i0 + i) * pitch, x, kRows > 1 ? inv[i] : inv[0]);
                    } else if (writes) {
                        *reinterpret_cast<uint4*>(dst16 + (i0 + i) * pitch) = raw[i];
                    }
                }
                return;
            }
            float rn[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) rn[i] = 1.f;
            if (norm) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    f32x2 x[4];
                    unpack8(raw[i], x);
                    f32x2 ss2 = mma::mul2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) ss2 = mma::fma2(x[e], x[e], ss2);
                    float a, b;
                    mma::upk(ss2, a, b);
                    rn[i] = a + b;
                }
#pragma unroll
                for (int m = 1; m < 16; m <<= 1)
#pragma unroll
                    for (int i = 0; i < kRows; ++i) rn[i] += __shfl_xor_sync(0xffffffffu, rn[i], m);
#pragma unroll
                for (int i = 0; i < kRows; ++i) rn[i] = rsqrtf(rn[i] * (1.0f / kHeadDim) + l.rms_eps);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                uint4 o = raw[i];   // the partners
                if (kInterleaved) {
                    o = make_uint4(__byte_perm(o.x, 0, 0x1032), __byte_perm(o.y, 0, 0x1032),
                                   __byte_perm(o.z, 0, 0x1032), __byte_perm(o.w, 0, 0x1032));
                } else {
                    o.x = __shfl_sync(0xffffffffu, o.x, partner, 16);
                    o.y = __shfl_sync(0xffffffffu, o.y, partner, 16);
                    o.z = __shfl_sync(0xffffffffu, o.z, partner, 16);
                    o.w = __shfl_sync(0xffffffffu, o.w, partner, 16);
                }
                // Channels that are not rotated have no partner: 0 * infinity is none of their business.
                if (!turned) o = make_uint4(0u, 0u, 0u, 0u);
                f32x2 x[4], y[4];
                unpack8(raw[i], x);
                unpack8(o, y);
                const f32x2 rn2 = mma::pk(rn[i], rn[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = mma::mul2(mma::fma2(y[e], S[e], mma::mul2(x[e], C[e])), rn2);
                if (kE4m3 && to_cache) {
                    if (writes) store_e4m3(dst8 + (i0 + i) * pitch, x, kRows > 1 ? inv[i] : inv[0]);
                } else if (writes) {
                    *reinterpret_cast<uint4*>(dst16 + (i0 + i) * pitch) = pack8(x);
                }
            }
        };
        copies_wait<kDepth - 1>();
        if (heads >= kBatch) {
            rows(std::integral_constant<int, kBatch>(), 0);
        } else {
#pragma unroll 1
            for (int i = 0; i < heads; ++i) {
                rows(std::integral_constant<int, 1>(), i);
                if (kE4m3) {
                    inv[0] = inv[1];
                    inv[1] = inv[2];
                }
            }
        }
        copy(stage);
        if (++stage == kDepth) stage = 0;
        if (++at.unit == units.all) {
            at.unit = 0;
            at.tok += 2;
            pos = next_pos;
            slot = next_slot;
            kind = -1;
        }
    }
    copies_wait<0>();
}

}  // namespace

cudaError_t launch_attn_append(const AttnLayer& l, const RopeTurns& turns, const AttnAppendIO& io,
                               const DeviceInfo& dev, int* err_word, cudaStream_t stream) {
    const int q = (l.Hq + kBatch - 1) / kBatch, kv = (l.Hkv + kBatch - 1) / kBatch;
    const Units units{q, kv, q + 2 * kv};
    const long long total = ((long long)io.N + 1) / 2 * units.all;
    const long long most = (long long)dev.sm_count * kCtasPerSm * (kThreads / 32);
    // As many warps as are resident, or more where each still has kWarpUnits.
    const int warps = (int)(total < most ? total : total / kWarpUnits > most ? total / kWarpUnits : most);
    const int grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    auto kernel = l.e4m3 ? (l.interleaved ? kda_attn_append_kernel<true, true> : kda_attn_append_kernel<true, false>)
                         : (l.interleaved ? kda_attn_append_kernel<false, true> : kda_attn_append_kernel<false, false>);
    kernel<<<grid, kThreads, 0, stream>>>(l, turns, io, units, total, warps, err_word);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
