// Paged softmax attention, one warp per query row and head: the online
// softmax with a running maximum and sum, 4 channels per lane.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_fp16.h>

#include "attn_internal.cuh"

namespace kda {
namespace {

template <bool kE4m3>
__device__ __forceinline__ float4 load4(const void* cache, size_t at) {
    if (kE4m3) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + at);
        const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffff), __NV_E4M3));
        const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3));
        return make_float4(__low2float(lo), __high2float(lo), __low2float(hi), __high2float(hi));
    }
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(cache) + at);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

template <bool kE4m3>
__global__ void __launch_bounds__(256) kda_attn_rows_kernel(const AttnLayer l, const AttnIO io, int* err) {
    const int lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (job >= (long long)io.N * l.Hq) return;
    const int tok = (int)(job / l.Hq), h = (int)(job % l.Hq), kvh = h / l.G;
    int b = tok, seen_to;   // keys [0, seen_to) are seen
    const int bound = io.max_pages << l.page_shift;
    if (io.cu_new) {
        int lo = 0, hi = io.B;   // first b with cu_new[b + 1] > tok
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (io.cu_new[mid + 1] > tok) hi = mid; else lo = mid + 1;
        }
        if (lo >= io.B || io.cu_new[lo] > tok) return;
        b = lo;
        const int kv = min(max(io.kv_lens[b], 0), bound);
        seen_to = max(0, kv - (io.cu_new[b + 1] - tok) + 1);
    } else {
        seen_to = min(max(io.kv_lens[b], 0), bound);
    }
    const uint2 qu = *reinterpret_cast<const uint2*>(io.q + (size_t)job * kHeadDim + lane * 4);
    const float ks = kE4m3 ? l.k_scale[kvh] : 1.f, vs = kE4m3 ? l.v_scale[kvh] : 1.f;
    const float sc = l.softmax_scale * ks;
    const float q0 = __uint_as_float(qu.x << 16) * sc, q1 = __uint_as_float(qu.x & 0xffff0000u) * sc,
                q2 = __uint_as_float(qu.y << 16) * sc, q3 = __uint_as_float(qu.y & 0xffff0000u) * sc;
    float m = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < seen_to; ++j) {
        const int page = io.block_table[(size_t)b * io.max_pages + (j >> l.page_shift)];
        const bool in = page >= 0 && page < l.num_pages;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (in) {
            const size_t at = (((size_t)page * l.Hkv + kvh) * l.page_size + (j & (l.page_size - 1))) * kHeadDim + lane * 4;
            k = load4<kE4m3>(l.k_cache, at);
            v = load4<kE4m3>(l.v_cache, at);
        } else if (lane == 0) {
            atomicOr(err, kErrAttnIndex);
        }
        float s = q0 * k.x + q1 * k.y + q2 * k.z + q3 * k.w;
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float mn = fmaxf(m, s);
        const float a = __expf(m - mn), p = __expf(s - mn);
        sum = sum * a + p;
        acc.x = acc.x * a + p * v.x;
        acc.y = acc.y * a + p * v.y;
        acc.z = acc.z * a + p * v.z;
        acc.w = acc.w * a + p * v.w;
        m = mn;
    }
    const float inv = seen_to > 0 ? vs / sum : 0.f;
    float out[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    const size_t at = (size_t)job * kHeadDim + lane * 4;
    for (int e = 0; e < 4; ++e) {
        if (io.gate) out[e] *= 1.f / (1.f + __expf(-io.gate[at + e]));
        if (io.o_f32) static_cast<float*>(io.o)[at + e] = out[e];
        else static_cast<__nv_bfloat16*>(io.o)[at + e] = __float2bfloat16_rn(out[e]);
    }
    if (io.lse && lane == 0) io.lse[job] = seen_to > 0 ? m + logf(sum) : -INFINITY;
}

cudaError_t launch_rows(const AttnLayer& l, const AttnIO& io, int* err_word, cudaStream_t stream) {
    const long long jobs = (long long)io.N * l.Hq;
    const unsigned grid = (unsigned)((jobs + 7) / 8);
    auto kernel = l.e4m3 ? kda_attn_rows_kernel<true> : kda_attn_rows_kernel<false>;
    kernel<<<grid, 256, 0, stream>>>(l, io, err_word);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnLayer& l, const AttnIO& io, const DeviceInfo&, int* err_word,
                                cudaStream_t stream) {
    return launch_rows(l, io, err_word, stream);
}

}  // namespace kda
