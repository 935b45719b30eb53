// One warp's tile of up to 16 query rows against tiles of keys in shared memory:
// 16 keys in bf16, 32 in e4m3, 4 KiB of keys and 4 KiB of values behind them as TMA
// lays them out (128-byte swizzle).  Every row sees every key of a tile that it is
// given.  The arithmetic is that of the few-row kernel (attn_decode.cu): mma.sync
// products, fp32 sums, a running reference that is raised only when a logit passes
// it by more than kLimit powers of two, bf16 weights as the sum of two bf16 parts,
// e4m3 keys and values as f16 and the queries scaled by a power of two per row.
#pragma once

#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "ptx.cuh"

namespace kda {

constexpr uint32_t kRowTileBytes = 4096;   // keys (or values) of a tile

template <bool kE4m3>
struct RowTile {
    static constexpr int kKeys = kE4m3 ? 32 : 16;
    static constexpr int kNT = kKeys / 8;       // 8-key column tiles of the logits
    static constexpr float kOffset = kE4m3 ? 10.f : 0.f;
    static constexpr float kLimit = kE4m3 ? 15.f : 8.f;

    uint32_t qf[8][4];    // A fragments of the queries
    float fac[2];         // logit -> power of two
    float acc[16][4], ref[2], sum[2];

    // The words of a query row (128 bf16) that a lane's fragments are made of, zero for
    // no row.  e4m3: in the order in which the keys are read, step s takes channels 16 c
    // + 4 s + {0, 1 | 2, 3} of the lower half, then of the upper.
    static __device__ __forceinline__ void load(const uint16_t* q, bool live, uint32_t (&raw)[16]) {
        const int c = threadIdx.x & 3;
        if (!kE4m3) {
#pragma unroll
            for (int s = 0; s < 16; ++s) raw[s] = live ? *reinterpret_cast<const uint32_t*>(q + 8 * s + 2 * c) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (live) v = *reinterpret_cast<const uint4*>(q + (i >> 1) * 64 + 16 * c + (i & 1) * 8);
                raw[4 * i] = v.x; raw[4 * i + 1] = v.y;
                raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
            }
        }
    }

    // Rows g and g + 8 of the tile (g = lane / 4); scale: softmax scale * log2(e).
    __device__ __forceinline__ void begin(const uint32_t (&raw)[2][16], float scale, float k_scale) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t (&w)[16] = raw[half];
            fac[half] = scale;
            float up = 1.f;
            if (kE4m3) {
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = mma::query_exponent(top);
                up = exp2f((float)(14 - e));
                fac[half] = mma::query_factor(scale, e - 14, k_scale);
            }
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t v = w[2 * s + x];
                    qf[s][half + 2 * x] = !kE4m3 ? v : mma::pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
                }
        }
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
        ref[0] = ref[1] = kNoRef;
        sum[0] = sum[1] = 0.f;
    }

    // A tile, of which the first `valid` keys count.
    __device__ __forceinline__ void add(uint8_t* stage, int valid) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        const uint32_t ks = ptx::smem_u32(stage), vs = ks + kRowTileBytes;
        if (valid < kKeys) {
            // Values past the end may be anything, NaN too: their weight is 0, make them 0.
            for (int i = lane; i < (int)kRowTileBytes / 16; i += 32) {
                const int row = kE4m3 ? i >> 3 : (i >> 3) & 15;
                if (row >= valid) *reinterpret_cast<uint4*>(stage + kRowTileBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
        }

        // Logits: rows = query rows, columns = keys.
        float sc[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        if (!kE4m3) {
            const int key = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
            for (int st = 0; st < 8; ++st) {
                const int ch = 2 * st + odd;   // 16-byte chunk of the key's row
                uint32_t b[4];
                mma::ldmatrix4(b, ks + (ch >> 3) * 2048 + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                mma::m16n8k16<false>(sc[0], qf[st], b[0], b[1]);
                mma::m16n8k16<false>(sc[1], qf[st], b[2], b[3]);
            }
        } else {
            // Column n of a tile is key 4 (n % 2) + n / 2 of its eight, so that the two rows
            // that a quarter warp reads lie in different banks.
            const int kr = ((g & 1) << 2) | (g >> 1);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const uint32_t rowp = ks + (n * 8 + kr) * 128;
                const uint4 lo = mma::lds128(rowp + ((c ^ kr) << 4)), hi = mma::lds128(rowp + (((c + 4) ^ kr) << 4));
                const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int st = 0; st < 8; ++st)
                    mma::m16n8k16<true>(sc[n], qf[st], mma::e4m3x2_f16x2(w[st]), mma::e4m3x2_f16x2(w[st] >> 16));
            }
        }
        if (valid < kKeys) {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (n * 8 + (kE4m3 ? c + 4 * e : 2 * c + e) >= valid) sc[n][e] = sc[n][e + 2] = -INFINITY;
        }

        // Softmax weights against the row's reference; a row is looked at as a whole only
        // when one of its logits passes it.
        float top[2];
        bool raise = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float m = fmaxf(sc[0][2 * half], sc[0][2 * half + 1]);
#pragma unroll
            for (int n = 1; n < kNT; ++n) m = mma::max3(m, sc[n][2 * half], sc[n][2 * half + 1]);
            top[half] = m * fac[half];
            raise |= top[half] > ref[half] + kLimit;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float m = top[half];
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                if (m > ref[half] + kLimit) {
                    const float to_ref = m - kOffset;
                    const float f = mma::exp2_approx(ref[half] - to_ref);
                    ref[half] = to_ref;
                    sum[half] *= f;
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        acc[n][2 * half] *= f;
                        acc[n][2 * half + 1] *= f;
                    }
                }
            }
        }
        uint32_t hi[kNT][2], lo[kNT][2];   // A fragments of the weights, rows g and g + 8
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const float p0 = mma::exp2_approx(fmaf(sc[n][2 * half], fac[half], -ref[half]));
                const float p1 = mma::exp2_approx(fmaf(sc[n][2 * half + 1], fac[half], -ref[half]));
                sum[half] += p0 + p1;
                if (kE4m3) {
                    hi[n][half] = mma::pack_f16(p0, p1);
                } else {
                    const uint32_t p = mma::pack_bf16(p0, p1);
                    hi[n][half] = p;
                    lo[n][half] = mma::pack_bf16(p0 - __uint_as_float(p << 16), p1 - __uint_as_float(p & 0xffff0000u));
                }
            }

        // Weighted values.
        if (!kE4m3) {
            const int key = (lane & 7) + (((lane >> 3) & 1) << 3), odd = lane >> 4;
            const uint32_t ah[4] = {hi[0][0], hi[0][1], hi[1][0], hi[1][1]}, al[4] = {lo[0][0], lo[0][1], lo[1][0], lo[1][1]};
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                uint32_t b[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = 2 * (j + i) + odd;
                    mma::ldmatrix4_trans(b[i], vs + (ch >> 3) * 2048 + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma::m16n8k16<false>(acc[2 * (j + i)], ah, b[i][0], b[i][1]);
                    mma::m16n8k16<false>(acc[2 * (j + i) + 1], ah, b[i][2], b[i][3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma::m16n8k16<false>(acc[2 * (j + i)], al, b[i][0], b[i][1]);
                    mma::m16n8k16<false>(acc[2 * (j + i) + 1], al, b[i][2], b[i][3]);
                }
            }
        } else {
            // Rows of the transposed 8 x 8 loads in the weights' key order; a 16-bit column holds
            // channels 2 n and 2 n + 1 of its chunk, which are split into two column tiles.
            const int i = lane & 7, kr = ((i & 1) << 2) | (i >> 1);
            const int key8 = ((lane >> 3) & 1) << 3, odd = lane >> 4;
#pragma unroll
            for (int k2 = 0; k2 < kKeys / 16; ++k2) {
                const uint32_t ap[4] = {hi[2 * k2][0], hi[2 * k2][1], hi[2 * k2 + 1][0], hi[2 * k2 + 1][1]};
                const uint32_t rowp = vs + (k2 * 16 + key8 + kr) * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b[4];
                    mma::ldmatrix4_trans(b, rowp + (((2 * j + odd) ^ kr) << 4));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {   // chunk 2 j + x
                        const uint32_t y0 = __byte_perm(b[2 * x], 0, 0x3120), y1 = __byte_perm(b[2 * x + 1], 0, 0x3120);
                        mma::m16n8k16<true>(acc[4 * j + 2 * x], ap, mma::e4m3x2_f16x2(y0), mma::e4m3x2_f16x2(y1));
                        mma::m16n8k16<true>(acc[4 * j + 2 * x + 1], ap, mma::e4m3x2_f16x2(y0 >> 16), mma::e4m3x2_f16x2(y1 >> 16));
                    }
                }
            }
        }
    }

    // The sums of all of a row's keys, in every lane of the row.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
        }
    }

    // Row g + 8 half, times f, to 128 floats at `to`.
    __device__ __forceinline__ void store(int half, float f, float* to) const {
        const int c = threadIdx.x & 3;
        if (!kE4m3) {
#pragma unroll
            for (int n = 0; n < 16; ++n)
                *reinterpret_cast<float2*>(to + 8 * n + 2 * c) = make_float2(acc[n][2 * half] * f, acc[n][2 * half + 1] * f);
        } else {
#pragma unroll
            for (int n = 0; n < 16; n += 2)
                *reinterpret_cast<float4*>(to + 8 * n + 4 * c) =
                    make_float4(acc[n][2 * half] * f, acc[n + 1][2 * half] * f, acc[n][2 * half + 1] * f, acc[n + 1][2 * half + 1] * f);
        }
    }
};

}  // namespace kda
