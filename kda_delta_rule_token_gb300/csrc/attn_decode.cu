// Attention of one new token, or of a few, per request over a paged cache.
//
//   o = softmax(scale * q K^T) V,   per request, query head and token
//
// The rows of a key head are its G query heads, times n for n new tokens
// (token i of them sees the keys up to its own); this file takes requests of
// one token, and of n * G <= 32 rows.  Every cached byte of a request is then
// read once for each key head and takes part in 2 n G operations, so the call
// is bound by HBM: 64 requests of up to 8192 keys, 8 key heads, bf16, 1.16 GB:
// 176 us, 0.98 of the measured copy rate; one request of 262139 keys 91 us,
// 0.88; 256 requests in e4m3, 1.16 GB, 190 us, 0.91.  From 17 rows on the
// products of a tile take as long as its copy: 32 requests of 5 tokens and 4
// heads, 295 MB, 74.5 us, 0.59; 128 of 4096 keys, 2.1 GB, 394 us, 0.81.  The kernel is built around keeping enough bytes
// in flight on every SM:
//
//  * Work is cut into units of one tile (16 keys in bf16, 32 in e4m3) per warp
//    of one request and key head, numbered request-major.  Each CTA takes an
//    equal, contiguous range of units, whatever the lengths are: it finds its
//    first request by a prefix sum over the lengths.  A request whose units lie
//    in several CTAs leaves one partial result (weighted sum, maximum, sum) per
//    CTA, joined in a fixed order by a second, dependent launch, so the result
//    does not depend on scheduling.
//  * Inside a CTA each warp streams its own tiles: lane 0 copies the tile's
//    pages of K and V (4 KiB each) with TMA into the warp's private ring,
//    running ahead across the ends of requests, and the warp consumes them by
//    itself.  No warp waits for another before the end of a request's part,
//    where the four partial results meet in shared memory; another CTA of the
//    SM streams meanwhile (eight warps in one CTA: 194 us where two CTAs of
//    four take 176).
//  * The rows are those of a 16-row mma.sync tile: a byte of the cache takes
//    part in at most 64 operations there, which the warp-wide instruction
//    covers without a wait between warps.  From 17 rows on two warps share a
//    tile's copy, each with its 16 rows (one warp with both halves: twice the
//    time); a request of fewer rows in the same call lets the two take tiles by
//    turns (128 requests of 4 tokens, 2.1 GB in bf16, 355 us; with the second
//    warp on empty rows 412; in e4m3 255 and 331); beyond 32 query heads of one token there are several passes.  The
//    softmax keeps a reference (not the exact maximum) per row and rescales
//    only when a logit passes it by more than kLimit powers of two: the result
//    is the same, the rescaling almost never runs.
//  * bf16: the weights enter the second product as the sum of two bf16 parts
//    (what is left is below 2^-16 of a weight; one part alone is off by up to
//    2^-8, as much as the rounding of the output, and the pipe is idle
//    anyway).  e4m3: keys, values and weights are f16 (keys and values exactly,
//    weights to 2^-11, kept within 2^15 of the row's reference), q is scaled by
//    a power of two per row.
#include <cudaTypedefs.h>

#include <atomic>

#include "attn_again.cuh"
#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "attn_tma.cuh"
#include "attn_ptx.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// By the warps that share a tile (row tiles).  One: two CTAs per SM, each warp
// with two stages.  Two: a tile takes twice the work, so three CTAs, which the
// registers allow without loading a request's rows ahead.
template <int kRowTiles>
constexpr int ctas_per_sm() { return kRowTiles == 1 ? 2 : 3; }
template <int kRowTiles>
constexpr int stages_per_warp() { return kRowTiles == 1 ? 2 : 1; }
constexpr int kMostCtasPerSm = 3;
constexpr uint32_t kTileBytes = 4096;            // keys (or values) of one warp tile
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kMergeBytes = kWarps * 16 * kHeadDim * 4;
constexpr int kJoinRows = 4;                     // CTAs of the join per request and head, over rows, at least
constexpr int kFewParts = 8;                     // parts of a row that one warp of the join takes
constexpr int kJoinCtas = 1024;                  // up to which CTAs per row are added
constexpr int kMaxRows = kAttnFewRows;           // rows of one pass

template <int kRowTiles>
struct Smem {
    uint8_t ring[kWarps * stages_per_warp<kRowTiles>() * kStageBytes];
    float merge[kMergeBytes / 4];
    float ref[2][kWarps * 16];
    float sum[2][kWarps * 16];
    uint64_t full[kWarps * stages_per_warp<kRowTiles>()];
    uint64_t empty[kWarps * stages_per_warp<kRowTiles>()];
    long long scan[kWarps];
    uint32_t zeros[kWarps];
    long long total, first_unit, left;
    int first_b;
    int dead;
    int spoiled;   // a row of several tokens came out as NaN or infinite
};

struct DecodeArgs {
    AttnIO io;
    int Hq, Hkv, G;
    int passes, rows;        // head groups of a key head, and query heads of a group
    int page_shift, num_pages;
    float scale;             // softmax scale * log2(e)
    const float* k_scale;
    const float* v_scale;
    const void* k_cache;
    const void* v_cache;
};

// What a CTA leaves for the join: the request and (virtual) head whose first
// part it holds and that goes on in the next CTAs, up to CTA last.  b < 0: none.
struct JoinDesc {
    int b, vh, last, slot;
    int tok0, n;
};

// Workspace: a descriptor per CTA, then two slots per CTA of partial results,
// rows x (128 weighted sums, then reference and sum).
constexpr int kSlotFloats = kMaxRows * (kHeadDim + 2);

__host__ __device__ constexpr size_t desc_bytes(int ctas) { return ((size_t)ctas * sizeof(JoinDesc) + 255) & ~size_t(255); }

__device__ __forceinline__ JoinDesc* descs(void* ws) { return static_cast<JoinDesc*>(ws); }
__device__ __forceinline__ float* slot_at(void* ws, int ctas, int slot) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + desc_bytes(ctas)) + (size_t)slot * kSlotFloats;
}

// Request b as this file sees it: its new tokens, its cached keys, and those
// that it is worked on with (0 where it has no rows here).
struct Request {
    int tok0, n, keys, len;
};

__device__ __forceinline__ Request request(const DecodeArgs& a, int b) {
    const int keys = attn_kv_len(a.io, b, a.page_shift);
    Request r{b, 1, keys, keys};
    if (a.io.cu_new) {
        attn_tokens(a.io, b, r.tok0, r.n);
        if (r.n == 0 || !attn_few_rows(r.n, a.G)) r.len = 0;
    }
    return r;
}

// Rows of a request without keys that one CTA writes; of longer ones (a prompt
// chunk that the plan refused) every CTA writes a share.  4096 tokens of 64 heads
// among 300 requests of 2: 172 us, 1186 with a CTA for each request.
constexpr int kOwnZeroRows = 256;
__device__ __forceinline__ bool all_zero_it(const DecodeArgs& a, const Request& r) {
    return r.keys == 0 && (long long)r.n * a.Hq > kOwnZeroRows;
}

// A position in the CTA's range.  The range also counts kPartCost units for
// each request and head before its first unit: what starting and ending one
// costs, as measured, so that ranges of many short requests are not longer
// than ranges of one long one.
struct Walk {
    long long left;   // units of the range not yet passed, this one included; none if <= 0
    int b, vh, u;     // request, virtual head, unit of it
    int len, units;   // of request b
    int tok0, n;
};

// Units of a request and head, and those with its cost.
template <int kUnit>
__device__ __forceinline__ int units_of(int len) { return (int)(((long long)len + kUnit - 1) / kUnit); }

template <int kUnit>
__device__ __forceinline__ long long cost_of(int len, int part_cost) { return len ? units_of<kUnit>(len) + part_cost : 0; }

// To the next unit (of the next request with any, at the end of one).
template <int kUnit, int kPartCost>
__device__ __forceinline__ void step(const DecodeArgs& a, Walk& w) {
    --w.left;
    if (++w.u < w.units) return;
    w.u = 0;
    w.left -= kPartCost;
    if (++w.vh < a.Hkv * a.passes) return;
    w.vh = 0;
    if (w.left <= 0) return;
    do {
        const Request r = request(a, ++w.b);
        w.len = r.len;
        w.tok0 = r.tok0;
        w.n = r.n;
        w.units = units_of<kUnit>(w.len);
    } while (w.units == 0);
}

// The walk over a CTA's range of `left` units, from unit `first` of request b's heads on.
template <int kUnit, int kPartCost>
__device__ __forceinline__ Walk begin_walk(const DecodeArgs& a, long long left, int b, long long first) {
    Walk w;
    w.left = left;
    w.b = b;
    const Request r = request(a, b);
    w.len = r.len;
    w.tok0 = r.tok0;
    w.n = r.n;
    w.units = units_of<kUnit>(w.len);
    w.vh = (int)(first / (w.units + kPartCost));
    w.u = (int)(first % (w.units + kPartCost)) - kPartCost;
    if (w.u < 0) {
        w.left += w.u;
        w.u = 0;
    }
    return w;
}

// Puts right rows of several tokens (attn_again.cuh), a warp per request and head.
// Only CTAs that wrote NaN or an infinity for such a row come here, after their
// work (32 x 5 tokens without any 74.0 -> 74.6 us; looked for in the loop over tiles,
// by tile or by part: 77 to 84).
template <bool kE4m3, int kUnit, int kPartCost>
__device__ __noinline__ void mend_rows(const DecodeArgs& a, long long left, int first_b, long long first_unit) {
    const int warp = threadIdx.x >> 5, row = threadIdx.x & 31;
    Walk w = begin_walk<kUnit, kPartCost>(a, left, first_b, first_unit);
    for (int nth = 0; w.left > 0; ++nth) {
        const int u0 = w.u, u1 = (int)min((long long)w.units, u0 + w.left), h = w.vh;   // n > 1: one pass
        if (w.n > 1 && nth % kWarps == warp) {
            const size_t head = ((size_t)w.tok0 + row / a.G) * a.Hq + h * a.G + row % a.G;
            float* part = slot_at(a.io.workspace, gridDim.x, 2 * blockIdx.x + (nth == 0 ? 0 : 1));
            rows_again<kE4m3>(a, w.b, h, row < w.n * a.G, head, u0 * kUnit, (int)min((long long)w.len, (long long)u1 * kUnit),
                              w.len - w.n + 1 + row / a.G, [&](int channel, float4 v, float ref, float sum) {
                if (u0 == 0 && u1 == w.units) {
                    const float n = sum != 0.f ? (kE4m3 ? a.v_scale[h] : 1.f) / sum : 0.f;
                    mma::store4(a.io, head * kHeadDim + channel, make_float4(v.x * n, v.y * n, v.z * n, v.w * n), sum != 0.f);
                } else {
                    const float f = sum != 0.f ? mma::exp2_approx(ref - part[kMaxRows * kHeadDim + 2 * row]) : 0.f;
                    *reinterpret_cast<float4*>(part + row * kHeadDim + channel) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                }
            });
        }
        w.left -= u1 - u0 - 1;
        w.u = u1 - 1;
        step<kUnit, kPartCost>(a, w);
    }
}

template <bool kE4m3, int kRowTiles>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<kRowTiles>())
kda_attn_decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, int* err) {
    constexpr int kTile = kE4m3 ? 32 : 16;       // keys of a warp tile
    constexpr int kNT = kTile / 8;               // 8-key column tiles of the logits
    constexpr int kGroups = kWarps / kRowTiles;  // groups of warps that share a tile
    constexpr int kUnit = kGroups * kTile;       // keys of a unit
    constexpr int kPartCost = kRowTiles == 1 ? 1 : 3;   // units that a request and head costs beside its own
    constexpr int kDepth = stages_per_warp<kRowTiles>() * kRowTiles;  // stages of a group's ring
    constexpr float kOffset = kE4m3 ? 10.f : 0.f;
    constexpr float kLimit = kE4m3 ? 15.f : 8.f;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    auto& sm = *reinterpret_cast<Smem<kRowTiles>*>(sm_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int group = warp / kRowTiles, row_tile = warp % kRowTiles;
    const bool lead = row_tile == 0;             // the group's copying warp
    uint64_t* full = sm.full + group * kDepth;
    uint64_t* empty = sm.empty + group * kDepth; // the group's other warp has read the stage
    uint8_t* ring = sm.ring + group * kDepth * kStageBytes;

    ptx::griddep_launch_dependents();
    if (lane == 0 && lead)
        for (int s = 0; s < kDepth; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
    if (tid == 0) {
        sm.dead = sm.spoiled = 0;
        descs(a.io.workspace)[blockIdx.x].b = -1;
    }
    ptx::fence_mbar_init();

    // The CTA's range of units.
    const int heads = a.Hkv * a.passes;
    const int per = (a.io.B + kThreads - 1) / kThreads;
    const int b0 = min(a.io.B, tid * per), b1 = min(a.io.B, b0 + per);
    long long mine = 0;
    bool shares = false;   // there is a request whose zero rows all CTAs write
    for (int b = b0; b < b1; ++b) {
        const Request r = request(a, b);
        mine += cost_of<kUnit>(r.len, kPartCost);
        shares |= all_zero_it(a, r);
    }
    mine *= heads;
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 31) sm.scan[warp] = upto;
    shares = __syncthreads_or(shares);
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sm.scan[w];
        total += sm.scan[w];
    }
    const long long ctas = min((long long)gridDim.x, total);
    const bool works = blockIdx.x < ctas;
    const long long from = works ? total * blockIdx.x / ctas : 0, to = works ? total * (blockIdx.x + 1) / ctas : 0;
    if (works && upto - mine <= from && from < upto) {
        long long at = upto - mine;
        for (int b = b0;; ++b) {
            const long long n = cost_of<kUnit>(request(a, b).len, kPartCost) * heads;
            if (from < at + n) {
                sm.first_b = b;
                sm.first_unit = from - at;
                sm.left = to - from;
                break;
            }
            at += n;
        }
    }
    // Requests without keys: zero rows.
    auto zero_rows = [&](const Request& r, long long from, long long step) {
        const long long rows = (long long)r.n * a.Hq;
        for (long long i = from; i < rows * (kHeadDim / 4); i += step)
            mma::store4(a.io, (size_t)r.tok0 * a.Hq * kHeadDim + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f), false);
        if (a.io.lse)
            for (long long i = from; i < rows; i += step) a.io.lse[(size_t)r.tok0 * a.Hq + i] = -INFINITY;
    };
    for (int b = blockIdx.x; b < a.io.B; b += gridDim.x)
        if (attn_kv_len(a.io, b, a.page_shift) == 0) {
            const Request r = request(a, b);
            if (!all_zero_it(a, r)) zero_rows(r, tid, kThreads);
        }
    if (shares)
        for (int base = 0; base < a.io.B; base += kThreads) {
            const uint32_t found = __ballot_sync(0xffffffffu, base + tid < a.io.B && all_zero_it(a, request(a, base + tid)));
            if (lane == 0) sm.zeros[warp] = found;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w)
                for (uint32_t m = sm.zeros[w]; m; m &= m - 1)
                    zero_rows(request(a, base + 32 * w + __ffs((int)m) - 1), (long long)blockIdx.x * kThreads + tid,
                              (long long)gridDim.x * kThreads);
            __syncthreads();
        }
    __syncthreads();
    if (!works) {
        ptx::griddep_wait();
        return;
    }

    Walk cur = begin_walk<kUnit, kPartCost>(a, sm.left, sm.first_b, sm.first_unit);

    // Producer: lane 0 issues the warp's tiles; the page ids of the next tile
    // are loaded one issue ahead of their use.
    const int boxes = max(1, kTile >> a.page_shift), box_rows = kTile / boxes;
    const int page_mask = (1 << a.page_shift) - 1;
    Walk ahead = cur;
    int ids[kTile / 16];
    auto fetch_ids = [&]() {   // to the warp's next tile, if there is one
        while (ahead.left > 0 && (ahead.u * kGroups + group) * kTile >= ahead.len) step<kUnit, kPartCost>(a, ahead);
        if (ahead.left <= 0) return;
        const int key = (ahead.u * kGroups + group) * kTile;
        const int* t = a.io.block_table + (size_t)ahead.b * a.io.max_pages + (key >> a.page_shift);
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
            if (i < boxes) ids[i] = key + i * box_rows < ahead.len ? t[i] : ids[0];
    };
    int issued = 0;
    bool ok = true;
    auto issue = [&]() {   // the lead warp
        if (ahead.left <= 0) return;
        const int s = issued % kDepth;
        if (kRowTiles > 1 && issued >= kDepth)
            ok = ptx::mbar_wait_timed(&empty[s], (uint32_t)(issued / kDepth - 1) & 1u, &sm.dead);
        if (lane == 0 && ok && !(a.io.drop && group == 0 && issued == 0)) {
            uint8_t* st = ring + s * kStageBytes;
            const int row = (ahead.u * kGroups + group) * kTile & page_mask;
            const int h = ahead.vh / a.passes;
            ptx::mbar_arrive_expect_tx(&full[s], kStageBytes);
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i)
                if (i < boxes) {
                    const bool in = ids[i] >= 0 && ids[i] < a.num_pages;
                    if (!in) atomicOr(err, kErrAttnIndex);
                    // A page outside the cache: a box outside the tensor, which reads as zeros.
                    const int ph = (in ? ids[i] : a.num_pages) * a.Hkv + (in ? h : 0);
                    const uint32_t off = i * (kTileBytes / boxes);
                    ptx::tma_load_4d(st + off, &kmap, 0, row, 0, ph, &full[s]);
                    ptx::tma_load_4d(st + kTileBytes + off, &vmap, 0, row, 0, ph, &full[s]);
                }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
            sm.dead = 1;
            atomicOr(err, ptx::kErrAttnWait);
            return;
        }
        ++issued;
        step<kUnit, kPartCost>(a, ahead);
        fetch_ids();
    };
    if (lead) {
        fetch_ids();
        for (int s = 0; s < kDepth; ++s) issue();
    }

    // Row r of a request and head: query head r % G of token r / G (one pass),
    // or head row0 + r of the only token.
    struct Rows {
        int h, row0, n;
        size_t head0;
    };
    auto rows_of = [&](const Walk& w) {
        Rows x;
        x.h = w.vh / a.passes;
        x.row0 = w.vh % a.passes * a.rows;
        x.n = w.n > 1 ? w.n * a.G : min(a.rows, a.G - x.row0);
        x.head0 = (size_t)w.tok0 * a.Hq + x.h * a.G + x.row0;
        return x;
    };
    auto head_of = [&](const Walk& w, const Rows& x, int r) {
        return w.n > 1 ? x.head0 + (size_t)(r / a.G) * a.Hq + r % a.G : x.head0 + r;
    };
    // The query rows' words that this lane's A fragments are made of, loaded
    // before the partial results of the request before meet.  e4m3: channels in the
    // order in which the keys are read, step s takes 16 c + 4 s + {0, 1 | 2, 3}
    // of the lower half, then of the upper.
    uint32_t raw[2][16];
    auto load_rows = [&](const Walk& w) {
        const Rows x = rows_of(w);
        const int first = kRowTiles > 1 && x.n > 16 ? row_tile * 16 : 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = first + half * 8 + g;
            const uint16_t* q = a.io.q + head_of(w, x, r) * kHeadDim;
            if (!kE4m3) {
#pragma unroll
                for (int s = 0; s < 16; ++s)
                    raw[half][s] = r < x.n ? *reinterpret_cast<const uint32_t*>(q + 8 * s + 2 * c) : 0u;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < x.n) v = *reinterpret_cast<const uint4*>(q + (i >> 1) * 64 + 16 * c + (i & 1) * 8);
                    raw[half][4 * i] = v.x; raw[half][4 * i + 1] = v.y;
                    raw[half][4 * i + 2] = v.z; raw[half][4 * i + 3] = v.w;
                }
            }
        }
    };

    int used = 0, parity = 0;
    bool at_start = true;   // in the CTA's first request and head
    if (kRowTiles == 1 && cur.left > 0) load_rows(cur);
    while (cur.left > 0) {
        // One request and head (or the part of it in this CTA's range).
        if (kRowTiles > 1) load_rows(cur);
        const Rows rw = rows_of(cur);
        const int h = rw.h, nrows = rw.n;
        // The warps of a group share its tiles, each with rows of its own, or,
        // where one row tile holds them all, take them by turns.
        const bool turns = kRowTiles > 1 && nrows <= 16;
        const int first_row = turns ? 0 : row_tile * 16;
        const int u0 = cur.u, u1 = (int)min((long long)cur.units, u0 + cur.left);

        uint32_t qf[8][4];   // A fragments
        float fac[2];        // logit -> power of two
        int sees[2];         // keys that the row sees (all of them where there is one token)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = first_row + half * 8 + g;
            const uint32_t (&w)[16] = raw[half];
            fac[half] = a.scale;
            sees[half] = cur.n > 1 && r < nrows ? cur.len - cur.n + 1 + r / a.G : cur.len;
            float up = 1.f;
            if (kE4m3) {
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // q * 2^(14 - e) with 2^e <= top < 2^(e+1): exact in f16 down to 2^-28 of the row's largest.
                const int e = mma::query_exponent(top);
                up = exp2f((float)(14 - e));
                fac[half] = mma::query_factor(a.scale, e - 14, a.k_scale[h]);
            }
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t v = w[2 * s + x];
                    qf[s][half + 2 * x] = !kE4m3 ? v : mma::pack_f16(__uint_as_float(v << 16) * up,
                                                                       __uint_as_float(v & 0xffff0000u) * up);
                }
        }

        float acc[16][4], ref[2], sum[2];
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
        ref[0] = ref[1] = kNoRef;
        sum[0] = sum[1] = 0.f;

        for (int u = u0; u < u1 && ok; ++u) {
            const int key0 = (u * kGroups + group) * kTile;
            if (key0 >= cur.len) break;
            const int s = used % kDepth;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_timed(&full[s], (uint32_t)(used / kDepth) & 1u, &sm.dead));
            if (!ok) {
                sm.dead = 1;
                atomicOr(err, ptx::kErrAttnWait);
                break;
            }
            ++used;
            if (!turns || (u - u0) % kRowTiles == row_tile) {
                uint8_t* stage = ring + s * kStageBytes;
                const uint32_t ks = ptx::smem_u32(stage), vs = ks + kTileBytes;
                const int valid = cur.len - key0;   // keys of the tile, if below kTile
                if (valid < kTile) {
                    // Values past the request's end may be anything, NaN too: their
                    // weight is 0, make them 0 (every warp that reads them writes the same).
                    for (int i = lane; i < (int)kTileBytes / 16; i += 32) {
                        const int row = kE4m3 ? i >> 3 : (i >> 3) & 15;
                        if (row >= valid) *reinterpret_cast<uint4*>(stage + kTileBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }

                // Logits: rows = query heads, columns = keys.
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
                    // Column n of a tile is key 4 (n % 2) + n / 2 of its eight, so
                    // that the two rows that a quarter warp reads lie in different banks.
                    const int kr = ((g & 1) << 2) | (g >> 1);
    #pragma unroll
                    for (int n = 0; n < kNT; ++n) {
                        const uint32_t rowp = ks + (n * 8 + kr) * 128;
                        const uint4 lo = mma::lds128(rowp + ((c ^ kr) << 4)), hi = mma::lds128(rowp + (((c + 4) ^ kr) << 4));
                        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    #pragma unroll
                        for (int st = 0; st < 8; ++st) {
                            const uint32_t x0 = mma::e4m3x2_f16x2(w[st]), x1 = mma::e4m3x2_f16x2(w[st] >> 16);
                            mma::m16n8k16<true>(sc[n], qf[st], x0, x1);
                        }
                    }
                }
                if (valid - (cur.n - 1) < kTile) {
    #pragma unroll
                    for (int n = 0; n < kNT; ++n)
    #pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = key0 + n * 8 + (kE4m3 ? c + 4 * e : 2 * c + e);
                            if (k >= sees[0]) sc[n][e] = -INFINITY;
                            if (k >= sees[1]) sc[n][e + 2] = -INFINITY;
                        }
                }

                // Softmax weights against the row's reference.
                uint32_t hi[kNT][2], lo[kNT][2];   // A fragments of the weights, rows g and g + 8
                // A row is looked at as a whole only when one of its logits passes the reference.
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
                    uint32_t ah[4], al[4];
                    ah[0] = hi[0][0]; ah[1] = hi[0][1]; ah[2] = hi[1][0]; ah[3] = hi[1][1];
                    al[0] = lo[0][0]; al[1] = lo[0][1]; al[2] = lo[1][0]; al[3] = lo[1][1];
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
                    // Rows of the transposed 8 x 8 loads in the weights' key order; a
                    // 16-bit column holds channels 2 n and 2 n + 1 of its chunk, which
                    // are split into two column tiles.
                    const int i = lane & 7, kr = ((i & 1) << 2) | (i >> 1);
                    const int key8 = ((lane >> 3) & 1) << 3, odd = lane >> 4;
    #pragma unroll
                    for (int k2 = 0; k2 < kTile / 16; ++k2) {
                        uint32_t ap[4];
                        ap[0] = hi[2 * k2][0]; ap[1] = hi[2 * k2][1];
                        ap[2] = hi[2 * k2 + 1][0]; ap[3] = hi[2 * k2 + 1][1];
                        const uint32_t rowp = vs + (k2 * 16 + key8 + kr) * 128;
    #pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t b[4];
                            mma::ldmatrix4_trans(b, rowp + (((2 * j + odd) ^ kr) << 4));
    #pragma unroll
                            for (int x = 0; x < 2; ++x) {   // chunk 2 j + x
                                const uint32_t y0 = __byte_perm(b[2 * x], 0, 0x3120), y1 = __byte_perm(b[2 * x + 1], 0, 0x3120);
                                const uint32_t e0 = mma::e4m3x2_f16x2(y0), e1 = mma::e4m3x2_f16x2(y1);
                                const uint32_t o0 = mma::e4m3x2_f16x2(y0 >> 16), o1 = mma::e4m3x2_f16x2(y1 >> 16);
                                mma::m16n8k16<true>(acc[4 * j + 2 * x], ap, e0, e1);
                                mma::m16n8k16<true>(acc[4 * j + 2 * x + 1], ap, o0, o1);
                            }
                        }
                    }
                }
            }
            __syncwarp();   // every lane has read the stage: it may be filled again
            if (lead) issue();
            else if (lane == 0) ptx::mbar_arrive(&empty[s]);
        }
        Walk next = cur;
        next.left -= u1 - u0 - 1;
        next.u = u1 - 1;
        step<kUnit, kPartCost>(a, next);
        if (kRowTiles == 1 && next.left > 0) load_rows(next);

        // The warps' partial results meet.  The buffers of references and
        // sums alternate: a warp may be a request ahead of another's reading.
        float* s_ref = sm.ref[parity];
        float* s_sum = sm.sum[parity];
        parity ^= 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float l = sum[half];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (c == 0) {
                s_ref[warp * 16 + half * 8 + g] = ref[half];
                s_sum[warp * 16 + half * 8 + g] = l;
            }
        }
        if (__syncthreads_or(!ok)) {
            ok = false;
            break;
        }
        const int parts = turns ? kWarps : kGroups, rows = turns ? 16 : 16 * kRowTiles;   // partial results, rows of each
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = first_row + half * 8 + g;
            float top = kNoRef;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w < parts) top = fmaxf(top, s_ref[w * rows + r]);
            const float f = mma::exp2_approx(ref[half] - top);
            float* m = sm.merge + (warp * 16 + half * 8 + g) * kHeadDim;
            const int flip = (r & 3) << 3;
#pragma unroll
            for (int n = 0; n < 16; n += kE4m3 ? 2 : 1) {
                const float* x = acc[n];
                if (!kE4m3) {
                    *reinterpret_cast<float2*>(m + ((8 * n + 2 * c) ^ flip)) = make_float2(x[2 * half] * f, x[2 * half + 1] * f);
                } else {
                    const float* y = acc[n + 1];
                    *reinterpret_cast<float4*>(m + ((8 * n + 4 * c) ^ flip)) =
                        make_float4(x[2 * half] * f, y[2 * half] * f, x[2 * half + 1] * f, y[2 * half + 1] * f);
                }
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == cur.units;
        float* part = whole ? nullptr : slot_at(a.io.workspace, gridDim.x, 2 * blockIdx.x + (at_start ? 0 : 1));
        const float vscale = kE4m3 ? a.v_scale[h] : 1.f;
        for (int i = tid; i < nrows * (kHeadDim / 4); i += kThreads) {
            const int row = i / (kHeadDim / 4), col = i % (kHeadDim / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = kNoRef, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w < parts) {
                    const float4 x = *reinterpret_cast<const float4*>(sm.merge + (w * rows + row) * kHeadDim + (col ^ ((row & 3) << 3)));
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                    top = fmaxf(top, s_ref[w * rows + row]);
                }
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w < parts) l += s_sum[w * rows + row] * mma::exp2_approx(s_ref[w * rows + row] - top);
            if (kRowTiles > 1 && cur.n > 1 && !(fabsf(v.x + v.y + v.z + v.w) < INFINITY)) sm.spoiled = 1;
            if (whole) {
                const float n = l != 0.f ? vscale / l : 0.f;   // 0: the row sees no key (NaN is not 0: a NaN logit shows)
                const size_t at = head_of(cur, rw, row);
                mma::store4(a.io, at * kHeadDim + col, make_float4(v.x * n, v.y * n, v.z * n, v.w * n), l != 0.f);
                if (a.io.lse && col == 0) a.io.lse[at] = l != 0.f ? (top + log2f(l)) / kLog2e : -INFINITY;
            } else {
                *reinterpret_cast<float4*>(part + row * kHeadDim + col) = v;
                if (col == 0) {
                    part[kMaxRows * kHeadDim + 2 * row] = top;
                    part[kMaxRows * kHeadDim + 2 * row + 1] = l;
                }
            }
        }
        // The CTA that holds the first part of a request that goes on says up to where.
        if (tid == 0 && u0 == 0 && u1 < cur.units) {
            const long long last = to - 1 + (cur.units - u1);   // its last unit
            const int slot = 2 * (int)blockIdx.x + (at_start ? 0 : 1);
            // The CTA whose range [total i / ctas, total (i + 1) / ctas) holds it.
            descs(a.io.workspace)[blockIdx.x] =
                JoinDesc{cur.b, cur.vh, (int)(((last + 1) * ctas - 1) / total), slot, cur.tok0, cur.n};
        }
        cur = next;
        at_start = false;
    }
    if (!ok) {
        // Give-up path: the copies this warp issued complete (bounded waits) before its shared memory is released.
        for (int i = used; i < issued; ++i) ptx::mbar_wait_timed(&full[i % kDepth], (uint32_t)(i / kDepth) & 1u);
        __syncthreads();
    } else if (kRowTiles > 1) {   // (calls with more than a token to a request)
        __syncthreads();
        if (sm.spoiled) mend_rows<kE4m3, kUnit, kPartCost>(a, sm.left, sm.first_b, sm.first_unit);
    }
    ptx::griddep_wait();   // launched beside other kernels: ends after them
}

// Joins the parts of a request and head that lie in several CTAs: blockIdx.x
// the CTA that holds the first part (search: the blockIdx.x-th of those that
// hold one), blockIdx.y over query rows, four channels per lane.  Few parts: a
// warp per row.  Many: the eight warps share a row's.
__global__ void __launch_bounds__(256) kda_attn_join_kernel(const DecodeArgs a, int ctas, bool search) {
    __shared__ float4 s_acc[8][32];
    __shared__ float s_ref[8], s_sum[8];
    __shared__ uint32_t s_used[kJoinCtas / 32];
    ptx::griddep_wait();
    int first = (int)blockIdx.x;
    if (search) {
        for (int i = (int)threadIdx.x; i < kJoinCtas; i += 256) {
            const uint32_t used = __ballot_sync(0xffffffffu, i < ctas && descs(a.io.workspace)[i].b >= 0);
            if ((threadIdx.x & 31) == 0) s_used[i >> 5] = used;
        }
        __syncthreads();
        int before = first, word = 0;
        while (word < kJoinCtas / 32 && before >= __popc(s_used[word])) before -= __popc(s_used[word++]);
        if (word == kJoinCtas / 32) return;
        uint32_t used = s_used[word];
        while (before-- > 0) used &= used - 1;
        first = word * 32 + __ffs((int)used) - 1;
    }
    const JoinDesc d = descs(a.io.workspace)[first];
    if (d.b < 0) return;
    const int h = d.vh / a.passes, row0 = d.vh % a.passes * a.rows;
    const int rows = d.n > 1 ? d.n * a.G : min(a.rows, a.G - row0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = d.last - first + 1;

    float ref, sum;
    float4 acc;
    auto add = [&](float r, float l, float4 v) {
        const float to = fmaxf(ref, r);
        const float f = mma::exp2_approx(ref - to), e = mma::exp2_approx(r - to);
        ref = to;
        sum = sum * f + l * e;
        acc.x = acc.x * f + v.x * e;
        acc.y = acc.y * f + v.y * e;
        acc.z = acc.z * f + v.z * e;
        acc.w = acc.w * f + v.w * e;
    };
    auto add_parts = [&](int row, int from, int step) {
        ref = kNoRef;
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = from; i < parts; i += step) {
            const float* p = slot_at(a.io.workspace, ctas, i == 0 ? d.slot : 2 * (first + i));
            const float2 rl = *reinterpret_cast<const float2*>(p + kMaxRows * kHeadDim + 2 * row);
            add(rl.x, rl.y, *reinterpret_cast<const float4*>(p + row * kHeadDim + 4 * lane));
        }
    };
    auto finish = [&](int row) {
        const float n = sum != 0.f ? (a.v_scale ? a.v_scale[h] : 1.f) / sum : 0.f;
        const size_t head = ((size_t)d.tok0 + (d.n > 1 ? row / a.G : 0)) * a.Hq + h * a.G + (d.n > 1 ? row % a.G : row0 + row);
        mma::store4(a.io, head * kHeadDim + 4 * lane, make_float4(acc.x * n, acc.y * n, acc.z * n, acc.w * n), sum != 0.f);
        if (a.io.lse && lane == 0) a.io.lse[head] = sum != 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
    };
    if (parts <= kFewParts) {
        for (int row = blockIdx.y * 8 + warp; row < rows; row += gridDim.y * 8) {
            add_parts(row, 0, 1);
            finish(row);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        add_parts(row, warp, 8);
        s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_ref[warp] = ref;
            s_sum[warp] = sum;
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < 8; ++w) add(s_ref[w], s_sum[w], s_acc[w][lane]);
            finish(row);
        }
        __syncthreads();
    }
}

std::atomic<bool> g_attr_done[64];

template <bool kE4m3, int kRowTiles>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(kda_attn_decode_kernel<kE4m3, kRowTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Smem<kRowTiles>));
}

}  // namespace

bool attn_decode_maps(const AttnLayer& l, AttnMaps& maps) {
    const int tile = l.e4m3 ? 32 : 16;
    const int rows = l.page_size < tile ? l.page_size : tile;
    return make_cache_map(&maps.k_decode, l, l.k_cache, rows, l.e4m3 ? 1 : 2) &&
           make_cache_map(&maps.v_decode, l, l.v_cache, rows, l.e4m3 ? 1 : 2);
}

size_t attn_decode_workspace_bytes(const DeviceInfo& dev) {
    const int ctas = dev.sm_count * kMostCtasPerSm;
    return desc_bytes(ctas) + (size_t)ctas * 2 * kSlotFloats * sizeof(float);
}

cudaError_t launch_attn_few_rows(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev,
                                 int* err_word, cudaStream_t stream, bool beside) {
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        cudaError_t e = set_smem<false, 1>();
        if (e == cudaSuccess) e = set_smem<false, 2>();
        if (e == cudaSuccess) e = set_smem<true, 1>();
        if (e == cudaSuccess) e = set_smem<true, 2>();
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    DecodeArgs a{};
    a.io = io;
    a.Hq = l.Hq;
    a.Hkv = l.Hkv;
    a.G = l.G;
    a.passes = (l.G + kMaxRows - 1) / kMaxRows;
    a.rows = (l.G + a.passes - 1) / a.passes;
    a.page_shift = l.page_shift;
    a.num_pages = l.num_pages;
    a.scale = l.softmax_scale * kLog2e;
    a.k_scale = l.k_scale;
    a.v_scale = l.v_scale;
    a.k_cache = l.k_cache;
    a.v_cache = l.v_cache;
    // A call with a token per request has G rows at most; else any count up to 32 may occur.
    const int most_rows = io.cu_new && l.G < kMaxRows ? kMaxRows : a.rows;
    // Never more CTAs than the longest table allows units.
    const int tile = (most_rows <= 16 ? kWarps : kWarps / 2) * (l.e4m3 ? 32 : 16);
    const long long most = (long long)io.B * l.Hkv * a.passes * ((((long long)io.max_pages << l.page_shift) + tile - 1) / tile);
    const bool two = most_rows > 16;
    const int ctas = dev.sm_count * (two ? ctas_per_sm<2>() : ctas_per_sm<1>());
    const int grid = (int)(most < ctas ? most : ctas);
    auto kernel = l.e4m3 ? (two ? kda_attn_decode_kernel<true, 2> : kda_attn_decode_kernel<true, 1>)
                         : (two ? kda_attn_decode_kernel<false, 2> : kda_attn_decode_kernel<false, 1>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = two ? sizeof(Smem<2>) : sizeof(Smem<1>);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, maps.k_decode, maps.v_decode, err_word);
    count_launches(1);
    if (e != cudaSuccess || grid == 1) return e;   // one CTA leaves no parts
    // More than eight parts to a request and head, whose rows a CTA joins one
    // after another: CTAs for those that hold a first part only, and more of them
    // over the rows (one request of 30000 keys and 32 / 8 heads, 8 tokens: 65 -> 45 us,
    // 1 token: 40 both; eight requests, with up to eight parts each: 118 -> 120).
    const long long pairs = (long long)io.B * l.Hkv * a.passes;
    const bool search = pairs * kFewParts < grid && grid <= kJoinCtas;
    const int firsts = search ? (int)pairs : grid;
    int over_rows = search ? kJoinCtas / firsts : kJoinRows;
    if (over_rows > most_rows) over_rows = most_rows;
    cfg.gridDim = dim3((unsigned)firsts, (unsigned)over_rows);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kda_attn_join_kernel, a, grid, search);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
