// Pages of the cache when requests take over one another: shared, released, and
// the last, partly full one copied.
//
// Request b goes on from request rows[b].  Of a request that goes on c times,
// every full page has c - 1 further holders, and c - 1 copies of its last page
// are wanted if that is partly full; a request that does not go on lets go of its
// pages, and those that nobody holds any more are free.  What moves is the table
// (8 bytes an entry), 8 bytes for each page whose holders change, and the copies'
// rows.  The bookkeeping is bound by the latency of two steps: the
// table's new entries follow from the old ones alone, but which page a copy gets
// from how many pages are released before it.
//
//  * kda_attn_fork_kernel: 32 columns of the table per CTA.  Every CTA counts the
//    requests' children by itself.  The first of the CTAs of some columns walks
//    over the requests that end, a warp for each column, their entries brought
//    to shared memory together: equal pages among 32 requests are found by one match, taken off the
//    count by one atomic, and the last holder's lane notes the page if nobody is
//    left.  A column is one warp's, in the order of the requests, so what is noted
//    does not depend on scheduling.
//  * put_pages: puts the columns' freed pages on the stack one after another and hands the
//    stack's end out to the copies.  The CTAs of tables of up to 256 columns are a cluster
//    and meet at its barrier in between (a launch less: 2.5 us of the host's time, the GPU's is the
//    same); wider ones take a second, dependent launch.
//
// kda_attn_copy_pages_kernel copies rows, bound by HBM or by its launch.
//
// Four requests of 1,100 tokens: 6.9 us, and 1.6 for one layer's copies; 256 of 8,000
// in pages of 128, a quarter of which ends: 16.2 us (the chain of loads and the
// atomics of one column after another) and 4.4 (16 MB).  The host's calls take 8 and 4 us.
#include <atomic>

#include "attn_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 32;            // columns of the table per CTA
constexpr int kColsPerWarp = kCols / kWarps;
constexpr int kMostCluster = 8;      // CTAs that may meet in one launch

// Workspace: pages that each column frees, requests that want a copy, in order,
// their number and that of the pages on the stack (which info may come to stand in the
// place of), the columns' freed pages.
struct Space {
    int* freed;      // [max_pages]
    int* wanting;    // [B]
    int* wants;      // [4]
    int* pages;      // [max_pages][B]
};
__host__ __device__ __forceinline__ Space space_of(void* ws, int B, int max_pages) {
    int* p = static_cast<int*>(ws);
    return Space{p, p + max_pages, p + max_pages + B, p + (size_t)max_pages + B + 4};
}

__device__ __forceinline__ int length_of(const AttnForkIO& io, int b, int shift) {
    return min(max(io.kv_lens[b], 0), io.max_pages << shift);
}

// The columns' freed pages onto the stack, one column after another, and its end to the copies; by the CTAs of the columns.
__device__ __forceinline__ void put_pages(const AttnForkIO& io, int shift, int num_pages, int* err) {
    __shared__ int s_before[kWarps], s_all[kWarps];
    const Space ws = space_of(io.workspace, io.B, io.max_pages);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col0 = blockIdx.x * kCols;
    // Pages freed by the columns before this CTA's, and by all.
    int before = 0, all = 0;
    for (int c = tid; c < io.max_pages; c += kThreads) {
        const int n = ws.freed[c];
        all += n;
        if (c < col0) before += n;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) {
        s_before[warp] = before;
        s_all[warp] = all;
    }
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < kWarps; ++w) {
        before += s_before[w];
        all += s_all[w];
    }
    const int wants = ws.wants[0], count = ws.wants[1];

    // Copy `nth` gets the page.
    auto give = [&](int nth, int page) {
        const int b = ws.wanting[nth], r = io.rows[b], len = length_of(io, r, shift), col = len >> shift;
        const int from = io.block_table[(size_t)r * io.max_pages + col];
        if ((unsigned)page >= (unsigned)num_pages || (unsigned)from >= (unsigned)num_pages) atomicOr(err, kErrAttnIndex);
        io.new_table[(size_t)b * io.max_pages + col] = page;
        io.copy_src[b] = from;
        io.copy_dst[b] = page;
        io.copy_rows[b] = len & ((1 << shift) - 1);
    };

    // This CTA's columns, a warp for each in turn: freed page k goes onto the stack, and to copy all - 1 - k.
    int mine = col0 + lane < io.max_pages ? ws.freed[col0 + lane] : 0, upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
    }
    for (int c = warp; c < kCols; c += kWarps) {
        const int n = __shfl_sync(0xffffffffu, mine, c), from = before + __shfl_sync(0xffffffffu, upto, c) - n;
        for (int i = lane; i < n; i += 32) {
            const int page = ws.pages[(size_t)(col0 + c) * io.B + i], k = from + i;
            io.page_refs[page] = 0;
            const bool taken = all - 1 - k < wants;
            if (count + k < io.free_capacity) io.free_pages[count + k] = page;
            else if (!taken) atomicOr(err, kErrAttnIndex);   // lost
            if (taken) give(all - 1 - k, page);
        }
    }
    if (blockIdx.x) return;
    // Copies beyond the freed pages get those that were free before; the last may get none.
    for (int nth = all + tid; nth < wants; nth += kThreads)
        if (nth - all < count) give(nth, io.free_pages[count - 1 - (nth - all)]);
    // These hold nothing: each by a warp.
    const int served = (int)min((long long)wants, (long long)all + count);
    for (int nth = served + warp; nth < wants; nth += kWarps) {
        const int b = ws.wanting[nth], r = io.rows[b], whole = length_of(io, r, shift) >> shift;
        for (int c = lane; c < whole; c += 32) {
            const int page = io.block_table[(size_t)r * io.max_pages + c];
            if ((unsigned)page < (unsigned)num_pages) atomicSub(&io.page_refs[page], 1);
        }
        if (lane == 0) io.new_lens[b] = 0;
    }
    if (tid == 0) {
        io.info[0] = all;
        io.info[1] = served;
        io.info[2] = (int)min((long long)count + all - served, (long long)io.free_capacity);
        io.info[3] = wants - served;
    }
}

// kAll: the grid's x is a cluster, and what the columns free is put away here too.
template <bool kAll>
__global__ void __launch_bounds__(kThreads) kda_attn_fork_kernel(const AttnForkIO io, int shift, int num_pages, int* err) {
    extern __shared__ int s_dyn[];
    int* s_children = s_dyn;             // [B] requests that go on from request b
    int* s_first = s_dyn + io.B;         // [B] the first of them
    __shared__ int s_tile[kThreads][kCols + 1];
    __shared__ int s_ended[kThreads];
    __shared__ int s_warp[kWarps];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const Space ws = space_of(io.workspace, io.B, io.max_pages);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col0 = blockIdx.x * kCols, part_mask = (1 << shift) - 1;
    for (int b = tid; b < io.B; b += kThreads) {
        s_children[b] = 0;
        s_first[b] = 0x7fffffff;
    }
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < io.B; b += kThreads) {
        const int r = io.rows[b];
        if ((unsigned)r < (unsigned)io.B) {
            atomicAdd(&s_children[r], 1);
            atomicMin(&s_first[r], b);
        } else {
            bad |= r != -1;
        }
    }
    __syncthreads();

    if (blockIdx.x == 0 && blockIdx.y == (kAll ? 0 : gridDim.y - 1)) {
        if (bad) atomicOr(err, kErrAttnIndex);
        // Lengths, and the requests that want a copy, in their order.
        const int per = (io.B + kThreads - 1) / kThreads, b0 = min(io.B, tid * per), b1 = min(io.B, b0 + per);
        auto wants = [&](int b) {
            const int r = io.rows[b];
            return (unsigned)r < (unsigned)io.B && s_first[r] != b && (length_of(io, r, shift) & part_mask);
        };
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int r = io.rows[b];
            io.new_lens[b] = (unsigned)r < (unsigned)io.B ? length_of(io, r, shift) : 0;
            io.copy_src[b] = io.copy_dst[b] = -1;
            io.copy_rows[b] = 0;
            mine += wants(b);
        }
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        if (lane == 31) s_warp[warp] = upto;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) upto += s_warp[w];
            all += s_warp[w];
        }
        int at = upto - mine;
        for (int b = b0; b < b1; ++b)
            if (wants(b)) ws.wanting[at++] = b;
        if (tid == 0) {
            ws.wants[0] = all;
            ws.wants[1] = min(max(io.free_count[0], 0), io.free_capacity);
        }
    }

    // New rows: the pages of the one that the request goes on from, but for a copy of its own.
    for (int b = blockIdx.y * kWarps + warp; b < io.B; b += gridDim.y * kWarps) {
        const int r = io.rows[b], col = col0 + lane;
        if ((unsigned)r >= (unsigned)io.B) continue;
        const int len = length_of(io, r, shift), whole = len >> shift;
        const bool first = s_first[r] == b;
        if (col >= (first ? (len + part_mask) >> shift : whole)) continue;
        const int page = io.block_table[(size_t)r * io.max_pages + col];
        io.new_table[(size_t)b * io.max_pages + col] = page;
        if (first && s_children[r] > 1 && col < whole) {
            if ((unsigned)page < (unsigned)num_pages) atomicAdd(&io.page_refs[page], s_children[r] - 1);
            else atomicOr(err, kErrAttnIndex);
        }
    }
    if (blockIdx.y) return;

    // Requests that end let go of their pages.
    int freed[kColsPerWarp];
#pragma unroll
    for (int c = 0; c < kColsPerWarp; ++c) freed[c] = 0;
    for (int base = 0; base < io.B; base += kThreads) {
        const int own = base + tid;
        const bool ends = own < io.B && s_children[own] == 0 && length_of(io, own, shift) > col0 << shift;
        const uint32_t mask = __ballot_sync(0xffffffffu, ends);
        __syncthreads();   // the tile and the list before are read
        if (lane == 0) s_warp[warp] = __popc(mask);
        __syncthreads();
        int at = __popc(mask & ((1u << lane) - 1)), ended = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s_warp[w];
            ended += s_warp[w];
        }
        if (ends) s_ended[at] = own;
        __syncthreads();
#pragma unroll 8
        for (int i = warp; i < ended; i += kWarps) {
            const int b = s_ended[i], col = col0 + lane;
            int page = -1;
            if (col < (length_of(io, b, shift) + part_mask) >> shift) {
                page = io.block_table[(size_t)b * io.max_pages + col];
                if ((unsigned)page >= (unsigned)num_pages) {   // nobody's page
                    atomicOr(err, kErrAttnIndex);
                    page = -1;
                }
            }
            s_tile[i][lane] = page;
        }
        __syncthreads();
        for (int i = 0; i < ended; i += 32) {
            int page[kColsPerWarp], left[kColsPerWarp];
#pragma unroll
            for (int c = 0; c < kColsPerWarp; ++c) {
                page[c] = i + lane < ended ? s_tile[i + lane][warp * kColsPerWarp + c] : -1;
                const uint32_t same = __match_any_sync(0xffffffffu, page[c]);
                const int count = __popc(same);
                left[c] = 0;
                if (page[c] >= 0 && lane == 31 - __clz(same)) {
                    const int had = atomicSub(&io.page_refs[page[c]], count);
                    if (had < 0 || had - count < -1) atomicOr(err, kErrAttnIndex);   // more let go of it than held it
                    left[c] = had >= 0 ? had - count : 0;
                }
            }
#pragma unroll
            for (int c = 0; c < kColsPerWarp; ++c) {
                const uint32_t gone = __ballot_sync(0xffffffffu, left[c] < 0);
                if (left[c] < 0)
                    ws.pages[(size_t)(col0 + warp * kColsPerWarp + c) * io.B + freed[c] + __popc(gone & ((1u << lane) - 1))] = page[c];
                freed[c] += __popc(gone);
            }
        }
    }
    if (lane == 0)
#pragma unroll
        for (int c = 0; c < kColsPerWarp; ++c)
            if (col0 + warp * kColsPerWarp + c < io.max_pages) ws.freed[col0 + warp * kColsPerWarp + c] = freed[c];
    if (kAll) {
        __threadfence();
        __syncthreads();
        ptx::cluster_sync();
        put_pages(io, shift, num_pages, err);
    }
}

__global__ void __launch_bounds__(kThreads) kda_attn_fork_pages_kernel(const AttnForkIO io, int shift, int num_pages, int* err) {
    ptx::griddep_wait();
    put_pages(io, shift, num_pages, err);
}

// rows x 128 values of one head's keys or values, from page src to page dst.
__global__ void __launch_bounds__(128) kda_attn_copy_pages_kernel(const AttnCopyIO io, const AttnLayer l, int* err) {
    ptx::griddep_wait();
    const int i = blockIdx.x, src = io.src[i], dst = io.dst[i];
    if (src == -1) return;
    if ((unsigned)src >= (unsigned)l.num_pages || (unsigned)dst >= (unsigned)l.num_pages) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(err, kErrAttnIndex);
        return;
    }
    const int rows = min(max(io.rows[i], 0), l.page_size);
    const int vecs = rows * (kHeadDim / 16) * (l.e4m3 ? 1 : 2);
    const size_t page = (size_t)l.page_size * (kHeadDim / 16) * (l.e4m3 ? 1 : 2);
    for (int part = blockIdx.y; part < 2 * l.Hkv; part += gridDim.y) {
        uint4* cache = static_cast<uint4*>(part & 1 ? l.v_cache : l.k_cache);
        const uint4* from = cache + ((size_t)src * l.Hkv + (part >> 1)) * page;
        uint4* to = cache + ((size_t)dst * l.Hkv + (part >> 1)) * page;
        constexpr int kLoads = 8;
        for (int v = threadIdx.x; v < vecs; v += 128 * kLoads) {
            uint4 w[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                if (v + 128 * k < vecs) w[k] = from[v + 128 * k];
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                if (v + 128 * k < vecs) to[v + 128 * k] = w[k];
        }
    }
}

std::atomic<bool> g_attr_done[64];

}  // namespace

size_t attn_fork_workspace_bytes(int B, int max_pages) {
    return ((size_t)max_pages + B + 4 + (size_t)max_pages * B) * sizeof(int);
}

cudaError_t launch_attn_fork(const AttnLayer& l, const AttnForkIO& io, const DeviceInfo& dev, int* err_word,
                             cudaStream_t stream) {
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kda_attn_fork_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, KDA_ATTN_MAX_PLAN_REQUESTS * 8);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kda_attn_fork_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, KDA_ATTN_MAX_PLAN_REQUESTS * 8);
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    const unsigned cols = (unsigned)((io.max_pages + kCols - 1) / kCols);
    // CTAs over the requests' rows until every SM has one.
    int over = (int)((dev.sm_count + cols - 1) / cols);
    const int most = (io.B + kWarps - 1) / kWarps;
    if (over > most) over = most;
    const dim3 grid(cols, (unsigned)over);
    if (cols <= (unsigned)kMostCluster)
        return launch_clusters_behind(kda_attn_fork_kernel<true>, grid, (int)cols, kThreads, (size_t)io.B * 8, stream, io, l.page_shift, l.num_pages,
                                      err_word);
    const cudaError_t e = launch_behind(kda_attn_fork_kernel<false>, grid, kThreads, (size_t)io.B * 8, stream, io, l.page_shift, l.num_pages, err_word);
    if (e != cudaSuccess) return e;
    return launch_behind(kda_attn_fork_pages_kernel, dim3(cols), kThreads, 0, stream, io, l.page_shift, l.num_pages, err_word);
}

cudaError_t launch_attn_copy_pages(const AttnLayer& l, const AttnCopyIO& io, int* err_word, cudaStream_t stream) {
    const unsigned parts = l.Hkv < 32768 ? 2u * l.Hkv : 65535u;
    return launch_behind(kda_attn_copy_pages_kernel, dim3((unsigned)io.n, parts), 128, 0, stream, io, l, err_word);
}

}  // namespace kda
