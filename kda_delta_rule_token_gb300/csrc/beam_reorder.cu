// States and convolution windows of the sequences that others go on from.
//
// Bytes move and nothing else happens: bound by HBM, one read of every sequence
// that goes on elsewhere and one write of every one that is replaced.  In place every CTA lists the
// sequences that move, and the CTAs take 32 KiB chunks of these in turn, all loads before the first
// store.  The sequences that go on from the same one take the same chunk at about the same time, so that all
// but one read of it come from L2.
//
// Measured (calls in a row): 64 sequences of 32 heads, of which a third move, 83 MB that L2
// keeps in part, 9.2 us; 256 of 64 heads in bf16, an eighth of which move, 153 MB, 23.5 us, 6.5 TB/s;
// 256 of 64 heads into other buffers, 1,021 MB, 148 us.  A CTA for each 64 KiB of all sequences, most of which
// find that theirs stays: 14.1, 36.0 and 150.  In place a CTA takes several chunks: 12 CTAs per SM, of which
// four run at once (24: 10.7 and 23.6 us, but half of 256 sequences of 64 heads, 1,149 MB, 168 instead of
// 172; four: 8.8, 24.2 and 182).  Into other buffers, where as a rule all sequences move, a chunk each
// and no list.
#include "beam_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;
constexpr int kCopy = kThreads * kLoads * 16;
constexpr int kCtasPerSm = 4;          // at once
constexpr int kInPlaceCtas = 12;       // per SM, in place
constexpr int kMany = 2048;            // sequences that are listed at a time

__global__ void __launch_bounds__(kThreads, kCtasPerSm) kda_beam_reorder_kernel(const BeamReorderIO io, int chunks0, int chunks, int* err) {
    __shared__ int2 s_moves[kMany];   // sequence, and the one that it goes on from
    __shared__ int s_warp[kThreads / 32];
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto copy = [&](int b, int from, int chunk) {
        const bool conv = chunk >= chunks0;
        if (conv) chunk -= chunks0;
        const long long bytes = conv ? io.bytes[1] : io.bytes[0], at = (long long)chunk * kCopy;
        const uint4* src = reinterpret_cast<const uint4*>((conv ? io.src[1] : io.src[0]) + from * bytes + at);
        uint4* dst = reinterpret_cast<uint4*>((conv ? io.dst[1] : io.dst[0]) + b * bytes + at);
        const int vecs = (int)((bytes - at < kCopy ? bytes - at : kCopy) / 16);
        uint4 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i * kThreads + tid < vecs) v[i] = src[i * kThreads + tid];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i * kThreads + tid < vecs) dst[i * kThreads + tid] = v[i];
    };
    if (!io.in_place) {
        for (long long c = blockIdx.x; c < (long long)io.B * chunks; c += gridDim.x) {
            const int chunk = (int)(c / io.B), b = (int)(c - (long long)chunk * io.B), from = io.rows[b];
            if ((unsigned)from < (unsigned)io.B) copy(b, from, chunk);
            else if (from != -1 && chunk == 0 && tid == 0) atomicOr(err, kErrRows);
        }
        return;
    }
    for (int b0 = 0; b0 < io.B; b0 += kMany) {
        const int many = min(kMany, io.B - b0);
        int n = 0;
        for (int i = 0; i < many; i += kThreads) {
            const int b = b0 + i + tid, from = i + tid < many ? io.rows[b] : -1;
            bool moves = from != -1 && from != b;
            // A sequence that moves away may be gone before it is read.
            if (moves && ((unsigned)from >= (unsigned)io.B || io.rows[from] != from)) {
                if (blockIdx.x == 0) atomicOr(err, kErrRows);
                moves = false;
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, moves);
            __syncthreads();   // s_warp, and the list before, have been read
            if (lane == 0) s_warp[warp] = __popc(mask);
            __syncthreads();
            int at = n + __popc(mask & ((1u << lane) - 1));
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) at += s_warp[w];
                n += s_warp[w];
            }
            if (moves) s_moves[at] = make_int2(b, from);
        }
        __syncthreads();
        for (long long c = blockIdx.x; c < (long long)n * chunks; c += gridDim.x) {
            const int chunk = (int)(c / n);
            const int2 m = s_moves[(int)(c - (long long)chunk * n)];
            copy(m.x, m.y, chunk);
        }
    }
}

}  // namespace

cudaError_t launch_beam_reorder(const BeamReorderIO& io, const DeviceInfo& dev, int* err_word, cudaStream_t stream) {
    const long long chunks0 = (io.bytes[0] + kCopy - 1) / kCopy, chunks1 = (io.bytes[1] + kCopy - 1) / kCopy;
    if (chunks0 + chunks1 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const long long most = (chunks0 + chunks1) * io.B;
    const long long ctas = io.in_place ? (long long)dev.sm_count * kInPlaceCtas : 0x7fffffffLL;
    return launch_behind(kda_beam_reorder_kernel, dim3((unsigned)(most < ctas ? most : ctas)), kThreads, 0, stream, io, (int)chunks0,
                         (int)(chunks0 + chunks1), err_word);
}

}  // namespace kda
