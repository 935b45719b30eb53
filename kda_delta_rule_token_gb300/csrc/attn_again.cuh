// Rows of the attention kernels once more, where a value that they do not see
// got into them.
//
// The products of a tile of keys take in all of its values, with weight 0 for keys
// that a row does not see, and 0 times NaN or infinity is NaN.  Values past a
// request's end are cleared; those of later tokens of the same chunk are not,
// since other rows of the tile see them.  So who wrote NaN or an infinity for a row
// that has a token goes over its rows after its work: where an unseen key of a
// row's tiles holds one, the channels that have it are added again in fp32, key by
// key, from the keys that the row sees, a lane per row.  Rare, and slow: one to five
// microseconds per key (a NaN in the 4000th token of an 8191-token prompt 13 ms, in
// its last but one 38 ms, in the last but one of 5 tokens behind 4091 keys 5 ms).
// Calls without such values pay for the look at the results only.
#pragma once

#include "attn_internal.cuh"
#include "attn_mma.cuh"

namespace kda {

// The first element of a key's row in the caches; -1 for a page outside them, whose rows are zeros.
template <typename Args>
__device__ __forceinline__ long long cached_row(const Args& a, int b, int h, int key) {
    const int page = a.io.block_table[(size_t)b * a.io.max_pages + (key >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) return -1;
    return (((((long long)page * a.Hkv + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * kHeadDim);
}

__device__ __forceinline__ float4 four_bf16(const uint2& w) {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

// Four channels of a cache as fp32, from element `at` on.
template <bool kE4m3>
__device__ __forceinline__ float4 cached4(const void* cache, long long at) {
    if (!kE4m3) return four_bf16(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(cache) + at));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + at);
    const uint32_t lo = mma::e4m3x2_f16x2(w), hi = mma::e4m3x2_f16x2(w >> 16);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(x.x, x.y, y.x, y.y);
}

// 0, or NaN if one of the four is NaN or infinite.
__device__ __forceinline__ float spoiled4(const float4& x) {
    return fmaf(x.x, 0.f, fmaf(x.y, 0.f, fmaf(x.z, 0.f, x.w * 0.f)));
}

// Up to 32 rows of request b and key head h, one per lane (live: it has one, its
// head of q at `head`), whose tiles hold keys [from, to) and which see the first
// `sees`: put(channel, v, ref, sum) for four channels at a time that have to be
// replaced, with the weighted values, their reference and the weights' sum.  The
// warp calls as a whole.
template <bool kE4m3, typename Args, typename Put>
__device__ __forceinline__ void rows_again(const Args& a, int b, int h, bool live, size_t head, int from, int to, int sees,
                                           Put&& put) {
    const int lane = threadIdx.x & 31;
    const int least = __reduce_min_sync(0xffffffffu, live ? max(from, sees) : to);
    const int most = __reduce_max_sync(0xffffffffu, live ? min(to, sees) : from);
    float z = 0.f;
#pragma unroll 2
    for (int key = least; key < to; ++key) {
        const long long at = cached_row(a, b, h, key);
        if (at >= 0) z += spoiled4(cached4<kE4m3>(a.v_cache, at + 4 * lane));
    }
    const float factor = a.scale * (kE4m3 ? a.k_scale[h] : 1.f);
    const uint16_t* q = a.io.q + (live ? head * kHeadDim : 0);
#pragma unroll 1
    for (uint32_t groups = __ballot_sync(0xffffffffu, z != 0.f); groups; groups &= groups - 1) {
        const int channel = 4 * (__ffs((int)groups) - 1);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float ref = kNoRef, sum = 0.f, unseen = 0.f;
#pragma unroll 1
        for (int key = from; key < to; ++key) {
            const long long at = cached_row(a, b, h, key);
            const float4 x = at >= 0 ? cached4<kE4m3>(a.v_cache, at + channel) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (key >= sees) unseen += spoiled4(x);
            if (key >= most) continue;
            float dot = 0.f;
            if (at >= 0) {
#pragma unroll 4
                for (int c = 0; c < kHeadDim; c += 4) {
                    const float4 k = cached4<kE4m3>(a.k_cache, at + c), w = four_bf16(*reinterpret_cast<const uint2*>(q + c));
                    dot = fmaf(w.x * factor, k.x, fmaf(w.y * factor, k.y, fmaf(w.z * factor, k.z, fmaf(w.w * factor, k.w, dot))));
                }
            }
            if (key < sees) {
                const float now = fmaxf(ref, dot), f = mma::exp2_approx(ref - now), p = mma::exp2_approx(dot - now);
                ref = now;
                sum = fmaf(sum, f, p);
                v.x = fmaf(p, x.x, v.x * f);
                v.y = fmaf(p, x.y, v.y * f);
                v.z = fmaf(p, x.z, v.z * f);
                v.w = fmaf(p, x.w, v.w * f);
            }
        }
        if (live && unseen != 0.f) put(channel, v, ref, sum);
    }
}

}  // namespace kda
