// Attention of one new token per request where groups of requests share a prefix.
//
//   o = (e^a o_p + e^b o_r) / (e^a + e^b)
//
// with o_p and a = lse of the request's row over the prefix, o_r and b over the
// keys that are its own.  A prefix's keys are read once for all of its
// requests, whose rows stand beside each other in the products: n requests of G
// heads per key head are n * G rows.  Up to 32 of them the cache's bytes are what
// counts, and the few-row kernel (attn_decode.cu) takes the prefixes together
// with the requests' own keys, as one list of work; more go to the prompts' tensor
// core kernel (attn_prefill.cu), without a causal edge.  Both leave fp32 results
// and their lse in the workspace; what joins them reads 1 KiB per row.
//
// What the groups look like is worked out by one CTA before (3 us beside which
// nothing runs): which requests are long enough to take part (those that are not
// attend to all of their keys by themselves), whose table has the prefix's
// pages, and how much of the prefix counts: whole pages, and whole tiles of the few-row
// kernel, so that no tile has keys of both kinds.
#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;

struct Space {
    uint8_t* few;       // the kernels' own
    uint8_t* many;
    int* prefix;        // [B]
    int* group_len;     // [B], of which the groups' are used
    int* group_row;
    float* o;           // [2 B][Hq][128]
    float* lse;         // [2 B][Hq]
    size_t bytes;
};

Space space_of(void* workspace, const AttnLayer& l, int B, const DeviceInfo& dev) {
    Space s;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    auto take = [&](size_t bytes) {
        uint8_t* p = at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    s.few = take(attn_decode_workspace_bytes(dev));
    s.many = take(attn_prefill_workspace_bytes(dev));
    s.prefix = reinterpret_cast<int*>(take((size_t)B * 4));
    s.group_len = reinterpret_cast<int*>(take((size_t)B * 4));
    s.group_row = reinterpret_cast<int*>(take((size_t)B * 4));
    s.o = reinterpret_cast<float*>(take((size_t)2 * B * l.Hq * kHeadDim * 4));
    s.lse = reinterpret_cast<float*>(take((size_t)2 * B * l.Hq * 4));
    s.bytes = (size_t)(at - static_cast<uint8_t*>(workspace));
    return s;
}

// Offsets that are not ascending within the requests are an error, and nothing is
// shared then; the results are the same.
__global__ void __launch_bounds__(kPlanThreads)
kda_attn_shared_plan_kernel(const AttnSharedIO io, int* prefix, int* group_len, int* group_row, int shift, int unit, int* err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;
    for (int g = tid; g < io.groups; g += kPlanThreads) {
        const int from = io.cu_groups[g], to = io.cu_groups[g + 1];
        bad |= from < 0 || to < from || to > io.B;
    }
    for (int b = tid; b < io.B; b += kPlanThreads) prefix[b] = 0;
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) atomicOr(err, kErrAttnIndex);
    const int most = io.max_pages << shift;
    for (int g = warp; g < io.groups; g += kPlanThreads / 32) {
        const int from = bad ? 0 : io.cu_groups[g], to = bad ? 0 : io.cu_groups[g + 1];
        const int len = min(max(io.prefix_lens[g], 0), most) / unit * unit;
        int members = 0, row = 0;
        if (len)
            for (int b = from; b < to; b += 32) {
                const uint32_t has = __ballot_sync(0xffffffffu, b + lane < to && min(io.kv_lens[b + lane], most) >= len);
                if (members == 0 && has) row = b + __ffs((int)has) - 1;
                members += __popc(has);
            }
        const bool share = members > 1;
        if (lane == 0) {
            group_len[g] = share ? len : 0;
            group_row[g] = row;
        }
        if (share)
            for (int b = from + lane; b < to; b += 32)
                if (min(io.kv_lens[b], most) >= len) prefix[b] = len;
    }
}

// A warp per row, four channels per lane.
__global__ void __launch_bounds__(256) kda_attn_shared_join_kernel(const AttnIO out, const float* o, const float* lse,
                                                                   const int* prefix, int Hq, long long rows) {
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const bool shares = prefix[row / Hq] > 0;
    const float a = shares ? lse[row] : -INFINITY, b = lse[rows + row];
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 x = shares ? *reinterpret_cast<const float4*>(o + row * kHeadDim + 4 * lane) : none;
    const float4 y = *reinterpret_cast<const float4*>(o + (rows + row) * kHeadDim + 4 * lane);
    // NaN where either is; -infinity where no key is seen: weights of 0.
    const float top = a != a || b != b ? a + b : fmaxf(a, b);
    const float u = top == -INFINITY ? 0.f : mma::exp2_approx((a - top) * kLog2e);
    const float v = top == -INFINITY ? 0.f : mma::exp2_approx((b - top) * kLog2e);
    const float sum = u + v, n = sum != 0.f ? 1.f / sum : 0.f;
    mma::store4(out, row * kHeadDim + 4 * lane,
                make_float4((x.x * u + y.x * v) * n, (x.y * u + y.y * v) * n, (x.z * u + y.z * v) * n, (x.w * u + y.w * v) * n),
                sum != 0.f);
    if (out.lse && lane == 0) out.lse[row] = sum != 0.f ? top + logf(sum) : -INFINITY;
}

}  // namespace

size_t attn_shared_workspace_bytes(const AttnLayer& l, int B, const DeviceInfo& dev) {
    return space_of(nullptr, l, B, dev).bytes;
}

cudaError_t launch_attn_shared(const AttnLayer& l, const AttnMaps& maps, const AttnSharedIO& io, const DeviceInfo& dev,
                               int* err_word, cudaStream_t stream) {
    const Space s = space_of(io.workspace, l, io.B, dev);
    const int tile = l.e4m3 ? 32 : 16;
    kda_attn_shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(io, s.prefix, s.group_len, s.group_row, l.page_shift,
                                                                 l.page_size > tile ? l.page_size : tile, err_word);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    AttnIO a{};
    a.N = io.B;
    a.cu_new = io.cu_groups;
    a.q = io.q;
    a.block_table = io.block_table;
    a.max_pages = io.max_pages;
    a.kv_lens = io.kv_lens;
    a.o = s.o;
    a.o_f32 = 1;
    a.lse = s.lse;
    a.drop = io.drop;
    a.groups = io.groups;
    a.singles = io.B;
    a.prefix = s.prefix;
    a.group_len = s.group_len;
    a.group_row = s.group_row;
    const bool many = io.groups && !attn_few_rows(io.B, l.G);   // else no group has more
    if (many) {
        a.B = io.groups;
        a.workspace = s.many;
        if ((e = launch_attn_many_rows_shared(l, maps, a, dev, err_word, stream)) != cudaSuccess) return e;
    }
    a.B = io.groups + io.B;
    a.workspace = s.few;
    if ((e = launch_attn_few_rows_shared(l, maps, a, dev, err_word, stream, many)) != cudaSuccess) return e;
    AttnIO out{};
    out.o = io.o;
    out.o_f32 = io.o_f32;
    out.lse = io.lse;
    out.gate = io.gate;
    const long long rows = (long long)io.B * l.Hq;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kda_attn_shared_join_kernel, out, (const float*)s.o, (const float*)s.lse, (const int*)s.prefix,
                           l.Hq, rows);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
