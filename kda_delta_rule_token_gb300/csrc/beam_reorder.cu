// States and convolution windows of the sequences that others go on from.
//
// Bytes move and nothing else happens: bound by HBM, one read of every sequence
// that goes on elsewhere and one write of every one that is replaced.  A CTA
// copies 64 KiB of one sequence, all loads before the first store (16 KiB: 64 sequences
// of 32 heads, of which a third move, 21 us instead of 14, whose 83 MB take 12 at the
// copy rate; 32 KiB 15).  The sequences of a batch that go on from the same one
// take the same chunk at about the same time, so that all but one read of it come from
// L2: 256 sequences of 64 heads with bf16 states into other buffers, 1,021 MB, 151 us.
#include "beam_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 16;
constexpr int kCopy = kThreads * kLoads * 16;

__global__ void __launch_bounds__(kThreads) kda_beam_reorder_kernel(const BeamReorderIO io, int chunks0, int* err) {
    const int b = (int)(blockIdx.x % (unsigned)io.B);
    int chunk = (int)(blockIdx.x / (unsigned)io.B);
    ptx::griddep_wait();
    const int from = io.rows[b];
    if (from == -1 || (io.in_place && from == b)) return;
    // In place, a sequence that moves away may be gone before it is read.
    if ((unsigned)from >= (unsigned)io.B || (io.in_place && io.rows[from] != from)) {
        if (chunk == 0 && threadIdx.x == 0) atomicOr(err, kErrRows);
        return;
    }
    const int which = chunk >= chunks0;
    if (which) chunk -= chunks0;
    const long long bytes = io.bytes[which], at = (long long)chunk * kCopy;
    const uint4* src = reinterpret_cast<const uint4*>(io.src[which] + from * bytes + at);
    uint4* dst = reinterpret_cast<uint4*>(io.dst[which] + b * bytes + at);
    const int vecs = (int)((bytes - at < kCopy ? bytes - at : kCopy) / 16);
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * kThreads + (int)threadIdx.x < vecs) v[i] = src[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * kThreads + (int)threadIdx.x < vecs) dst[i * kThreads + threadIdx.x] = v[i];
}

}  // namespace

cudaError_t launch_beam_reorder(const BeamReorderIO& io, const DeviceInfo&, int* err_word, cudaStream_t stream) {
    const long long chunks0 = (io.bytes[0] + kCopy - 1) / kCopy, chunks1 = (io.bytes[1] + kCopy - 1) / kCopy;
    const long long grid = (chunks0 + chunks1) * io.B;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_behind(kda_beam_reorder_kernel, dim3((unsigned)grid), kThreads, 0, stream, io, (int)chunks0, err_word);
}

}  // namespace kda
