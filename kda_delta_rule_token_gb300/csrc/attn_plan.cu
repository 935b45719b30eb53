// Planning of a serving step on the device: page allocation, block-table
// entries, token positions and cache slots from the requests' lengths.
//
// Two prefix sums over the requests decide everything: E[b], the packed rows
// up to and with request b, and U[b], the pages needed by the fitting requests
// up to and with b.  Request b is admitted if it fits and needs no page or
// U[b] <= free; the i-th page taken overall is free_pages[free - 1 - i], so a
// token's page follows from U alone and no page is handed out by an atomic:
// the plan is the same in every run.
//
// Few bytes move (12 per token out, 8 per request in): the call is bound by
// the latency of its chain load -> scan -> load -> scan -> search -> store and
// by the launch.  Each CTA therefore repeats both scans by itself (the lengths
// come from L2) and then writes its own range of tokens, finding each token's
// request by a binary search over E in shared memory; CTAs never wait for one
// another, and one launch does it all: 4.3 us for 64 requests, 4.6 us for 256
// with 82,000 new tokens.
#include <atomic>

#include "attn_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
__device__ __forceinline__ long long block_exclusive(long long v, long long* s_warp, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        if (lane < kWarps) s_warp[lane] = w;
    }
    __syncthreads();
    const long long before = warp ? s_warp[warp - 1] : 0;
    *total = s_warp[kWarps - 1];
    __syncthreads();   // s_warp may be used again
    return before + x - v;
}

__device__ __forceinline__ int saturated(long long x) { return x > 0x7fffffffLL ? 0x7fffffff : (int)x; }

__global__ void __launch_bounds__(kThreads) kda_attn_plan_kernel(const AttnPlanIO io, int shift) {
    extern __shared__ int s_dyn[];
    int* s_end = s_dyn;          // [B] E[b], saturated
    int* s_page = s_dyn + io.B;  // [B] pages taken before request b, or -1 if it is not admitted
    __shared__ long long s_warp[kWarps];
    __shared__ int s_taken, s_refused;
    const int tid = threadIdx.x, P1 = (1 << shift) - 1;
    if (tid == 0) s_taken = s_refused = 0;

    // Requests [b0, b1) belong to this thread in both scans.
    const int per = (io.B + kThreads - 1) / kThreads;
    const int b0 = min(io.B, tid * per), b1 = min(io.B, b0 + per);
    const long long free_count = min(max(io.free_count[0], 0), io.free_capacity);
    long long rows = 0, total_rows, total_need;
    for (int b = b0; b < b1; ++b) rows += max(io.new_lens[b], 0);
    const long long rows0 = block_exclusive(rows, s_warp, &total_rows);

    // Pages that request b needs, -1 if it does not fit; `end` is E[b].
    auto need_of = [&](int b, long long end) -> long long {
        const long long c = io.cache_lens[b], n = io.new_lens[b];
        const long long after = (c + n + P1) >> shift;
        if (c < 0 || n < 0 || after > io.max_pages || end > io.N) return -1;
        return after - ((c + P1) >> shift);
    };
    long long end = rows0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        end += max(io.new_lens[b], 0);
        pages += max(need_of(b, end), 0LL);
    }
    const long long pages0 = block_exclusive(pages, s_warp, &total_need);
    end = rows0;
    long long upto = pages0;
    int taken = 0, refused = 0;
    const bool writes = blockIdx.x == 0;
    for (int b = b0; b < b1; ++b) {
        end += max(io.new_lens[b], 0);
        const long long need = need_of(b, end);
        upto += max(need, 0LL);
        const bool ok = need == 0 || (need > 0 && upto <= free_count);
        s_end[b] = saturated(end);
        s_page[b] = !ok ? -1 : need ? (int)(upto - need) : 0;   // with need == 0 the prefix may pass 2^31
        if (ok && need > 0) taken = (int)upto;
        refused += !ok;
        if (writes) {
            io.cu_new[b + 1] = saturated(end);
            io.kv_lens[b] = ok ? io.cache_lens[b] + io.new_lens[b] : 0;
        }
    }
    if (taken) atomicMax(&s_taken, taken);
    if (refused) atomicAdd(&s_refused, refused);
    __syncthreads();
    if (writes && tid == 0) {
        io.cu_new[0] = 0;
        io.info[0] = saturated(total_rows);
        io.info[1] = s_taken;
        io.info[2] = (int)free_count - s_taken;
        io.info[3] = s_refused;
    }

    const int used = (int)(total_rows < io.N ? total_rows : io.N);
    for (int t = blockIdx.x * kThreads + tid; t < io.N; t += gridDim.x * kThreads) {
        if (t >= used) {
            io.positions[t] = 0;
            io.slots[t] = -1;
            continue;
        }
        // The first request whose rows end past t.
        int lo = 0, hi = io.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > t) hi = mid; else lo = mid + 1;
        }
        const int b = lo;
        const int first = b ? s_end[b - 1] : 0;
        const int c = io.cache_lens[b];
        const long long pos = (long long)c + (t - first);
        io.positions[t] = (int)pos;
        long long slot = -1;
        if (s_page[b] >= 0) {
            const int p = (int)(pos >> shift), row = (int)pos & P1;
            const int fresh = p - ((c + P1) >> shift);   // < 0: a page the request holds already
            int* entry = io.block_table + (size_t)b * io.max_pages + p;
            int page;
            if (fresh >= 0) {
                page = io.free_pages[free_count - 1 - (s_page[b] + fresh)];
                if (row == 0) *entry = page;
            } else {
                page = *entry;
            }
            // An id below 0 must not come out as -1, which leaves a token unstored
            // without a word: a slot that the append reports.
            slot = page < 0 ? -2 : ((long long)page << shift) + row;
        }
        io.slots[t] = slot;
    }
}

std::atomic<bool> g_attr_done[64];

}  // namespace

cudaError_t launch_attn_plan(const AttnLayer& l, const AttnPlanIO& io, const DeviceInfo& dev, cudaStream_t stream) {
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kda_attn_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   KDA_ATTN_MAX_PLAN_REQUESTS * 8);
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    const int want = (io.N + kThreads - 1) / kThreads;
    const int grid = want < 1 ? 1 : want < dev.sm_count ? want : dev.sm_count;
    kda_attn_plan_kernel<<<grid, kThreads, (size_t)io.B * 8, stream>>>(io, l.page_shift);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
