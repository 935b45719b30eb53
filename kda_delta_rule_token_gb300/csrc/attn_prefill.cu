// Causal attention of prompt chunks over a paged cache, on tcgen05 tensor cores.
//
//   S = scale * Q K^T,  P = exp(S - ref),  O = P V / sum(P),   keys in tiles of 128
//
// A prompt token's head takes part in 4 * 128 operations per key: the call is
// bound by the tensor pipe (a 128 x 128 tile of S and of O take it 512 cycles
// each, its exponentials take the SM 512 as well).  Measured: 8192 tokens of 64
// heads in bf16, after a rest, 622 us, 1767 TFLOP/s of the tokens' own operations,
// 0.90 of the measured dense rate, and back to back 683 us, 1609 TFLOP/s, 0.92 of
// what a library product sustains (e4m3: 678 and 715 us); one key tile of two row
// tiles takes 2300 cycles of which the tensor pipe works 2048.
//
// The rows of one key head are (token, query head) pairs: floor(128 / G) tokens
// with their G heads fill one 128-row tile, so that all heads that share a key
// head share the keys' copies, and short chunks fill a tile as well.  One CTA
// works on a segment of two such tiles (consecutive tokens), X = 0 and 1, at a
// time:
//
//  * one warp copies K and V pages with TMA (128-byte swizzle, a box per page)
//    into two slots each;
//  * one thread issues the MMAs: S_X(j) = Q_X K_j^T into TMEM, and
//    O_X += P_X(j) V_j with P_X read from TMEM.  While the softmax of one
//    tile runs, the MMAs of the other one do.  What that thread executes
//    between two MMAs was what limited the kernel for long (see there);
//  * four warps per tile do the softmax, one thread per row: the row's 128
//    logits from TMEM, its maximum against a running reference, the
//    exponentials, and their bf16 roundings back into TMEM over S_X.  A row
//    rescales (its O in TMEM as well) only when a logit passes the reference
//    by more than kLimit powers of two, which after the first tile is rare.
//  * e4m3: S is made of the keys as they are, with Q (scaled by a power of two
//    per row) as the sum of two e4m3 parts, which hold bf16's eight bits: two
//    8-bit products take as long as one 16-bit one, and the keys need no
//    conversion.  Two further warps convert the values to f16, P is f16 within
//    2^15.  (Keys converted to f16 too, by a warpgroup of its own: 5 % longer, and
//    6 % on ragged chunks.)
//
// The loops of all these warps have to fit the SM's instruction cache together:
// where they do not (a converting loop written out for all of a thread's 16
// chunks is enough), the misses of all SMs fill the cache behind it, and every
// warp of an SM slows down two- and threefold for tens of microseconds at a
// time (ragged e4m3 chunks: hit rate 92 %, 83 % of that cache's peak).  So the
// converting loop is eight chunks long, and a key tile's MMAs are written once.
//
// TMEM: S_0, S_1 (128 columns each, P_X in the first 64), O_0, O_1.
//
// P is rounded to bf16 (half a step, 2^-8 of each weight, or f16's 2^-11 for
// e4m3) as the MMA's operand; the sum it is divided by is of the fp32 weights.
// (kShared with two bf16 parts, as the few-row kernels have, the second in the
// other half of S_X's columns: outputs 1.66e-3 of their norm off in bf16 instead of
// 2.2e-3, 32 prompts 136 us instead of 127, 64 samples 42 instead of 38, four documents
// over a bf16 cache 160 instead of 131.)
// e4m3: Q's two parts are exact for channels down to 2^-9 of the row's largest,
// below that off by up to 2^-17 of it, which is what a logit may be off by per
// unit of the keys' absolute sum; the products accumulate in fp32 (lse of 3000
// keys at logits of standard deviation 2: within 1e-5 of 64 bits).
//
// CTAs are persistent.  Segments are numbered with the longest of a request
// first and dealt to the CTAs back and forth, which evens out the causal
// triangle.  Where the busiest CTA would then be well above the average share
// (few segments, or long and short ones together), the keys are cut instead:
// each CTA takes an equal range of (segment, key tile) units and leaves partial
// results, joined in a fixed order by a dependent launch (128 tokens behind
// 32640 cached ones, 16 segments: 70 us).
//
// kShared: prefixes that groups of requests share (attn_shared.cu), whose single
// tokens all see all of it.  Segments are always cut into equal ranges then, found from
// the plan's sums without a schedule of its own, and the join is not this file's.
#include <atomic>
#include <type_traits>

#include "attn_again.cuh"
#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "attn_tma.cuh"
#include "attn_ptx.cuh"

namespace kda {
namespace {

constexpr int kRows = 128;                     // rows of a tile
constexpr int kKeys = 128;                     // keys of a tile
constexpr uint32_t kOperand = 32768;           // a 128 x 128 16-bit operand
constexpr uint32_t kBlock = 16384;             // Q: one 64-channel block of it; e4m3: a tile as copied
// K and V tiles: each eight keys are two swizzled 1024-byte atoms, channels 0-63 and 64-127.
constexpr uint32_t kAtom = 1024, kEight = 2 * kAtom;
constexpr uint32_t kOffQ = 0, kOffK = 2 * kOperand, kOffV = 4 * kOperand, kOffStage = 6 * kOperand;
// e4m3: K tiles as copied, half as large, and behind them the results on their way out; V tiles as copied.
template <bool kE4m3>
constexpr uint32_t kSlotK = kE4m3 ? kBlock : kOperand;
template <bool kE4m3>
constexpr uint32_t kOffOut = kE4m3 ? kOffK + 2 * kBlock : kOffStage;
constexpr int kScan = 128;                     // threads of the prefix sums
constexpr int kMaxCtas = 256;
constexpr int kJoinCost = 8;                   // key tiles that writing and joining partial results takes (11 us)
constexpr int kJoinCtas = 8;                   // CTAs of the join per SM (fewer leave its loads waiting, more cost calls without cut keys)
constexpr int kMostWeighed = 32;               // segments per CTA up to which their load is worked out

constexpr uint32_t kColS = 0, kColO = 256;     // TMEM columns, + 128 X

// Up to 2 * tokens consecutive new tokens of one request with one key head.
struct Segment {
    int b, h;
    int tok, m;              // packed row of the first token, number of tokens
    int first;               // keys that the first token sees (the i-th: first + i); may be <= 0
    int len;                 // keys of the request
    __device__ __forceinline__ int tokens_of(int x, int per) const { return x ? max(m - per, 0) : min(m, per); }
    // Key tiles of tile x (one, fully masked, where its rows see no key).
    __device__ __forceinline__ int tiles(int x, int per) const {
        const int t = tokens_of(x, per);
        if (t == 0) return 0;
        return max(1, (first + (x ? m : t) - 1 + kKeys - 1) / kKeys);
    }
    __device__ __forceinline__ int tiles_all(int per) const { return max(tiles(0, per), tiles(1, per)); }
};

// What a CTA does next: key tiles [j0, j0 + n) of a segment, cnt[x] of them for tile x.
struct Part {
    Segment s;
    int j0, n, cnt[2];       // n == 0: no more parts
    int slot;                // of the partial result, -1 if the part is the whole segment
    int last;                // the segment's first part, if it goes on: up to this CTA; else -1
};

struct Ctl {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], vraw;
    uint64_t qfull[2], sfull[2], pfull[2][2], ofull[2];   // pfull: by tile and half of its keys
    uint64_t cvfull[2], cvempty[2];                       // e4m3: values as copied
    uint64_t partfull[2], partempty[2];
    uint64_t drain;
    Part part[2];            // from the copying warp to the others
    uint32_t tmem;
    int dead;
    int busiest;
    int kissued, vissued, raws;   // copies issued (raws: of values whose request ends in the tile)
    int warp_sum[kScan / 32];
    int pre[kScan];          // pairs of token tiles before the requests of scan thread t
    int units[kScan];        // key tiles and costs before the segments of scan thread t
    int load[kMaxCtas];      // of each CTA, were the segments dealt whole
};

// Behind the operands: e4m3, two V tiles as copied; bf16, 16 KiB for either
// tile's results on their way out.
template <bool kE4m3>
constexpr uint32_t smem_bytes() { return kOffStage + 2 * kBlock + (uint32_t)sizeof(Ctl); }
static_assert(kOffStage + 2 * kBlock + sizeof(Ctl) <= 232448, "shared memory");

struct PrefillArgs {
    AttnIO io;
    int Hq, Hkv, G;
    int tokens;              // of a tile: 128 / G
    int all;                 // few-row requests and those without keys are taken too
    int part_cost;           // key tiles that starting and ending a segment costs beside its own: what deals
                             // ragged chunks best (bf16: 130 us at 3, 137 at 2; e4m3: 5.3 us of 1.5 us tiles)
    int page_shift, num_pages;
    float scale;             // softmax scale * log2(e)
    const float* k_scale;
    const float* v_scale;
    const void* k_cache;
    const void* v_cache;
};

struct Sched {
    int total;               // pairs of token tiles of all requests
    int per;                 // requests of a scan thread
    int segments;            // pairs * key heads (fewer than the query rows, whose memory bounds them)
    int chunk;               // segments of a scan thread
    bool split;
    int units, ctas;         // split: key tiles and costs of all segments, CTAs that share them
    long long all;           // groups: the same
};

struct PrefillJoin {
    int tok, m, h, last, slot, pad[3];   // m == 0: none
};

constexpr int kSlotFloats = 2 * kRows * (kHeadDim + 2);
__host__ __device__ constexpr size_t join_bytes(int ctas) { return ((size_t)ctas * sizeof(PrefillJoin) + 255) & ~size_t(255); }
__device__ __forceinline__ PrefillJoin* joins(void* ws) { return static_cast<PrefillJoin*>(ws); }
__device__ __forceinline__ float* slot_at(void* ws, int ctas, int slot) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + join_bytes(ctas)) + (size_t)slot * kSlotFloats;
}

// Pairs of token tiles of request b that this file works on.
__device__ __forceinline__ int pairs_of(const PrefillArgs& a, int b) {
    int tok0, n;
    attn_tokens(a.io, b, tok0, n);
    if (n == 0 || (!a.all && (attn_few_rows(n, a.G) || attn_kv_len(a.io, b, a.page_shift) == 0))) return 0;
    return (n + 2 * a.tokens - 1) / (2 * a.tokens);
}

__device__ __forceinline__ Segment find_segment(const PrefillArgs& a, const Ctl& ctl, const Sched& sc, int s) {
    const int pair = (int)((unsigned)s / (unsigned)a.Hkv);
    int lo = 0, hi = kScan - 1;   // the last scan thread with pre <= pair
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl.pre[mid] <= pair) lo = mid; else hi = mid - 1;
    }
    int at = ctl.pre[lo], b = lo * sc.per, n;
    while (at + (n = pairs_of(a, b)) <= pair && b + 1 < a.io.B) {
        at += n;
        ++b;
    }
    Segment g;
    g.b = b;
    g.h = s - pair * a.Hkv;
    int tok0, tokens;
    attn_tokens(a.io, b, tok0, tokens);
    const int i0 = (n - 1 - (pair - at)) * 2 * a.tokens;   // the longest first
    g.len = attn_kv_len(a.io, b, a.page_shift);
    g.tok = tok0 + i0;
    g.m = min(2 * a.tokens, tokens - i0);
    g.first = g.len - tokens + i0 + 1;
    return g;
}

// The segment after segment s - 1, which g holds: the next head of its pair, or the next pair.
__device__ __forceinline__ void next_segment(const PrefillArgs& a, const Ctl& ctl, const Sched& sc, int s, Segment& g) {
    if (g.h + 1 < a.Hkv) ++g.h;
    else if (s < sc.segments) g = find_segment(a, ctl, sc, s);
}

// Where a CTA is in its work (the copying warp's).
struct Cursor {
    int k;                   // whole segments: rounds dealt; cut: the next segment, -1 before the first
    int at;                  // cut: units before segment k
    bool begun;              // cut: a part was found
    Segment s;               // cut: segment k
    long long unit;          // groups: units passed (k: the group)
};

// The next part of this CTA; p.n = 0 past the last.
// kShared: groups of requests that share a prefix (AttnIO), which all of their tokens see.
template <bool kShared>
__device__ __forceinline__ void next_part(const PrefillArgs& a, const Ctl& ctl, const Sched& sc, Cursor& c, Part& p) {
    p.n = 0;
    if (kShared) {
        if ((int)blockIdx.x >= sc.ctas) return;
        const long long from = sc.all * blockIdx.x / sc.ctas, to = sc.all * (blockIdx.x + 1) / sc.ctas;
        if (c.k < 0) {
            // The last group whose segments begin at or before `from`; the warp's lanes look together.
            const int lane = threadIdx.x & 31;
            int lo = 0, n = a.io.B;
            while (n > 1) {
                const int step = (n + 31) >> 5;
                const uint32_t begun = __ballot_sync(0xffffffffu, lane * step < n && a.io.group_start[lo + min(lane * step, n)] <= from);
                const int k = 31 - __clz((int)begun);
                lo += k * step;
                n = min(step, n - k * step);
            }
            c.k = lo;
            c.unit = from;
        }
        while (c.unit < to) {
            while (a.io.group_start[c.k + 1] <= c.unit) ++c.k;
            const int g = c.k, len = a.io.group_len[g], tiles = (len + kKeys - 1) / kKeys, per = tiles + a.part_cost;
            const int segment = (int)((c.unit - a.io.group_start[g]) / per), pair = segment / a.Hkv;
            const long long at = a.io.group_start[g] + (long long)segment * per, end = min(at + per, to);
            const int j0 = max((int)(c.unit - at) - a.part_cost, 0), j1 = (int)(end - at) - a.part_cost;
            c.unit = end;
            if (j1 <= j0) continue;
            const int tok0 = a.io.cu_new[g], n = a.io.cu_new[g + 1] - tok0;
            p.s.b = a.io.group_row[g];
            p.s.h = segment - pair * a.Hkv;
            p.s.tok = tok0 + pair * 2 * a.tokens;
            p.s.m = min(2 * a.tokens, n - pair * 2 * a.tokens);
            p.s.first = p.s.len = len;
            p.j0 = j0;
            p.n = j1 - j0;
            for (int x = 0; x < 2; ++x) p.cnt[x] = p.s.tokens_of(x, a.tokens) ? p.n : 0;
            p.slot = j0 == 0 && j1 == tiles ? -1 : 2 * (int)blockIdx.x + (c.begun ? 1 : 0);
            p.last = -1;
            if ((threadIdx.x & 31) == 0) {   // (the copying warp calls this)
                int2* note = a.io.parts + (size_t)a.io.group_pairs[g] * a.Hkv + segment;
                const int slot = 2 * (int)blockIdx.x + (c.begun ? 1 : 0);
                if (j0 == 0) note->x = p.slot;
                if (j1 == tiles) note->y = slot;
            }
            c.begun = true;
            return;
        }
        return;
    }
    if (!sc.split) {
        for (;; ++c.k) {
            const long long base = (long long)c.k * gridDim.x;
            if (base >= sc.segments) return;
            const int s = (int)(base + ((c.k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x));
            if (s >= sc.segments) continue;
            p.s = find_segment(a, ctl, sc, s);
            break;
        }
        ++c.k;
        p.j0 = 0;
        p.n = p.s.tiles_all(a.tokens);
        p.cnt[0] = p.s.tiles(0, a.tokens);
        p.cnt[1] = p.s.tiles(1, a.tokens);
        p.slot = p.last = -1;
        return;
    }
    if ((int)blockIdx.x >= sc.ctas) return;
    const int from = (int)((long long)sc.units * blockIdx.x / sc.ctas), to = (int)((long long)sc.units * (blockIdx.x + 1) / sc.ctas);
    if (c.k < 0) {
        int lo = 0, hi = kScan - 1;   // the last scan thread whose segments begin at or before `from`
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ctl.units[mid] <= from) lo = mid; else hi = mid - 1;
        }
        c.k = lo * sc.chunk;
        c.at = ctl.units[lo];
        if (c.k < sc.segments) c.s = find_segment(a, ctl, sc, c.k);
    }
    while (c.k < sc.segments && c.at < to) {
        p.s = c.s;
        const int tiles = p.s.tiles_all(a.tokens), at = c.at;
        ++c.k;
        next_segment(a, ctl, sc, c.k, c.s);
        c.at += tiles + a.part_cost;
        // A segment's first part_cost units stand for its cost, the others for its tiles.
        const int j0 = max(from - at - a.part_cost, 0), j1 = min(to - at - a.part_cost, tiles);
        if (j1 <= j0) continue;
        p.j0 = j0;
        p.n = j1 - j0;
        for (int x = 0; x < 2; ++x) p.cnt[x] = min(max(p.s.tiles(x, a.tokens) - j0, 0), p.n);
        const bool whole = p.n == tiles;
        p.slot = whole ? -1 : 2 * (int)blockIdx.x + (c.begun ? 1 : 0);
        // The CTA whose range [units i / ctas, units (i + 1) / ctas) holds the segment's last unit.
        p.last = whole || j0 > 0 ? -1 : (int)(((long long)c.at * sc.ctas - 1) / sc.units);
        c.begun = true;
        return;
    }
}

__device__ __forceinline__ bool pwait(uint64_t* bar, uint32_t parity, int* dead, int* err) {
    if (ptx::mbar_wait_timed(bar, parity, dead)) return true;
    *(volatile int*)dead = 1;
    atomicOr(err, ptx::kErrAttnWait);
    return false;
}

// The next part, as the copying warp found it; false past the last (or if the CTA gave up).
__device__ __forceinline__ bool take_part(Ctl& ctl, int& np, Part& p, int* dead, int* err) {
    if (!__all_sync(0xffffffffu, pwait(&ctl.partfull[np & 1], (uint32_t)(np >> 1) & 1u, dead, err))) return false;
    p = ctl.part[np & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&ctl.partempty[np & 1]);
    ++np;
    return p.n > 0;
}

// Inclusive prefix of v over the first kScan threads; all threads of the CTA call it.
__device__ __forceinline__ int scan_inclusive(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    if (lane == 31 && warp < kScan / 32) s_warp[warp] = v;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kScan / 32; ++w) {
        if (w < warp) v += s_warp[w];
        all += s_warp[w];
    }
    *total = all;
    __syncthreads();
    return v;
}

constexpr int kWarpMma = 8, kWarpTma = 9, kWarpConvert = 10, kConvert = 64;   // e4m3: threads that convert
constexpr int kThreads = 384;
// Registers: the launch's share of each thread, and what the softmax
// warpgroups (0, 1) and the other one change to; the sum stays within the
// launch's (checked against the compiled kernel before its first launch).
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 80;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegsLaunch, "registers");

template <bool kE4m3, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
kda_attn_prefill_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int* err) {
    constexpr float kOffset = kE4m3 ? 10.f : 0.f;
    constexpr float kLimit = kE4m3 ? 15.f : 8.f;
    extern __shared__ __align__(1024) uint8_t sm[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(sm + kOffStage + 2 * kBlock);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* dead = &ctl.dead;

    ptx::griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ctl.kfull[i], 1);
            ptx::mbar_init(&ctl.vfull[i], kE4m3 ? kConvert : 1);
            ptx::mbar_init(&ctl.kempty[i], 1);
            ptx::mbar_init(&ctl.vempty[i], 1);
            ptx::mbar_init(&ctl.qfull[i], kRows);
            ptx::mbar_init(&ctl.sfull[i], 1);
            ptx::mbar_init(&ctl.pfull[i][0], kRows);
            ptx::mbar_init(&ctl.pfull[i][1], kRows);
            ptx::mbar_init(&ctl.ofull[i], 1);
            ptx::mbar_init(&ctl.cvfull[i], 1);
            ptx::mbar_init(&ctl.cvempty[i], kConvert);
            ptx::mbar_init(&ctl.partfull[i], 1);
            ptx::mbar_init(&ctl.partempty[i], kE4m3 ? 11 : 9);   // warps that take parts
        }
        ptx::mbar_init(&ctl.vraw, 1);
        ptx::mbar_init(&ctl.drain, 1);
        ptx::fence_mbar_init();
        ctl.dead = 0;
        ctl.busiest = 0;
        ctl.kissued = ctl.vissued = ctl.raws = 0;
        if (!kShared) joins(a.io.workspace)[blockIdx.x].m = 0;
    }
    Sched sc;
    if (kShared) {
        // The plan's sums, and what the work before the call wrote, are only sure to be seen behind this
        // kernel's own wait: that the few-row kernel before it has waited for the plan does not reach here.
        ptx::griddep_wait();
        sc.all = a.io.group_start[a.io.B];
        sc.ctas = (int)min((long long)gridDim.x, sc.all);
        if ((int)blockIdx.x >= sc.ctas) return;
        if (warp == kWarpMma) tc::alloc(&ctl.tmem, 512);
    } else {
        // Segments of all requests.
        sc.per = (a.io.B + kScan - 1) / kScan;
        long long sum_pairs = 0;
        if (tid < kScan)
            for (int b = min(a.io.B, tid * sc.per), end = min(a.io.B, b + sc.per); b < end; ++b) sum_pairs += pairs_of(a, b);
        const int mine = (int)min(sum_pairs, (long long)(0x7fffffff / kScan));
        const int upto = scan_inclusive(mine, ctl.warp_sum, &sc.total);
        if (sc.total == 0) return;   // every request has few rows
        if (sc.total > a.io.N) {
            // More pairs than tokens (or a share of them cut short, which memory has
            // no room for): the offsets claim rows more than once, and sums of so many
            // segments need not fit what follows.
            if (tid == 0 && blockIdx.x == 0) atomicOr(err, kErrAttnIndex);
            return;
        }
        if (warp == kWarpMma) tc::alloc(&ctl.tmem, 512);
        if (tid < kScan) ctl.pre[tid] = upto - mine;
        __syncthreads();
        sc.segments = sc.total * a.Hkv;
        sc.split = false;
        sc.units = sc.ctas = sc.chunk = 0;
        if (sc.segments > 0 && sc.segments <= kMostWeighed * (int)gridDim.x) {
            // The load of every CTA if whole segments are dealt, against equal
            // shares of key tiles, which cost up to two more parts per CTA and the join.
            for (int i = tid; i < kMaxCtas; i += blockDim.x) ctl.load[i] = 0;
            __syncthreads();
            const int n = sc.segments;
            sc.chunk = (sc.total + kScan - 1) / kScan * a.Hkv;   // whole pairs, so that the threads find theirs together
            long long sum = 0;
            if (tid < kScan && tid * sc.chunk < n) {
                int s = tid * sc.chunk;
                Segment g = find_segment(a, ctl, sc, s);
                int round = s / (int)gridDim.x, r = s - round * (int)gridDim.x;
                for (const int end = min(n, s + sc.chunk); s < end;) {
                    const int u = g.tiles_all(a.tokens) + a.part_cost;
                    sum += u;
                    atomicAdd(&ctl.load[(round & 1) ? gridDim.x - 1 - r : r], u);
                    if (++r == (int)gridDim.x) {
                        r = 0;
                        ++round;
                    }
                    next_segment(a, ctl, sc, ++s, g);
                }
            }
            const int u = (int)min(sum, (long long)(0x7fffffff / kScan));   // beyond that, shares are not worth cutting for
            const int to = scan_inclusive(u, ctl.warp_sum, &sc.units);
            if (tid < kScan) ctl.units[tid] = to - u;
            for (int i = tid; i < (int)gridDim.x; i += blockDim.x) atomicMax(&ctl.busiest, ctl.load[i]);
            const bool fits = !__syncthreads_or(tid < kScan && (long long)u != sum);
            sc.ctas = min((int)gridDim.x, sc.units);
            sc.split = fits && ctl.busiest > (sc.units + sc.ctas - 1) / sc.ctas + 2 * a.part_cost + kJoinCost;
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    constexpr uint32_t tm = 0;   // all 512 columns are this CTA's, so they start at 0
    if (tid == 0 && ctl.tmem != tm) {
        ctl.dead = 1;
        atomicOr(err, ptx::kErrAttnWait);
    }

    if (warp == kWarpTma) {
        // ---- copies
        tc::reg_dec<kRegsOther>();
        Part p;
        Cursor cur{kShared || sc.split ? -1 : 0, 0, false, {}, 0};
        const int rows = min(1 << a.page_shift, kKeys), boxes = kKeys / rows;   // rows of a box, pages of a tile
        const int is_v = lane >> 4;
        const int pg = lane & 15;
        int it = 0, raws = 0;
        for (int np = 0;; ++np) {
            next_part<kShared>(a, ctl, sc, cur, p);
            if (np >= 2 && !__all_sync(0xffffffffu, pwait(&ctl.partempty[np & 1], (uint32_t)((np >> 1) - 1) & 1u, dead, err)))
                break;
            if (lane == 0) {
                ctl.part[np & 1] = p;
                ptx::mbar_arrive(&ctl.partfull[np & 1]);
            }
            if (p.n == 0) break;
            const int* table = a.io.block_table + (size_t)p.s.b * a.io.max_pages;
            auto page_of = [&](int j) {
                const int key = j * kKeys + pg * rows;
                return pg < boxes && key < p.s.len ? table[key >> a.page_shift] : 0;
            };
            int id = page_of(p.j0);
            for (int j = p.j0; j < p.j0 + p.n; ++j, ++it) {
                const int s = it & 1;
                const uint32_t par = (uint32_t)((it >> 1) - 1) & 1u;
                const int valid = min(p.s.len - j * kKeys, kKeys);
                const int pages = (valid + rows - 1) / rows;
                const bool mine_box = pg < pages;
                const bool in = id >= 0 && id < a.num_pages;
                if (mine_box && !in) atomicOr(err, kErrAttnIndex);
                const int ph = (in ? id : a.num_pages) * a.Hkv + (in ? p.s.h : 0);
                const bool raw = !kE4m3 && valid < kKeys;   // values past the end have to be cleared
                const bool drop = a.io.drop && it == 0;
                bool ok = true;
                if (kE4m3) {
                    // Keys straight to the operand, values to a buffer that the converting warps empty.
                    if (it >= 2) ok = pwait(&ctl.kempty[s], par, dead, err);
                    if (ok && lane == 0 && !drop) ptx::mbar_arrive_expect_tx(&ctl.kfull[s], (uint32_t)(pages * rows * 128));
                    __syncwarp();
                    if (ok && mine_box && !is_v && !drop)
                        ptx::tma_load_4d(sm + kOffK + s * kBlock + pg * rows * 128, &kmap, 0, 0, 0, ph, &ctl.kfull[s]);
                    if (ok) ctl.kissued = it + 1;
                    if (ok && it >= 2) ok = pwait(&ctl.cvempty[s], par, dead, err);
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(&ctl.cvfull[s], (uint32_t)(pages * rows * 128));
                    __syncwarp();
                    if (ok && mine_box && is_v)
                        ptx::tma_load_4d(sm + kOffStage + s * kBlock + pg * rows * 128, &vmap, 0, 0, 0, ph, &ctl.cvfull[s]);
                    if (ok) ctl.vissued = it + 1;
                } else {
                    uint8_t* kd = sm + kOffK + s * kOperand + pg * rows * 256;
                    uint8_t* vd = sm + kOffV + s * kOperand + pg * rows * 256;
                    if (it >= 2) ok = pwait(&ctl.kempty[s], par, dead, err);
                    if (ok && lane == 0 && !drop) ptx::mbar_arrive_expect_tx(&ctl.kfull[s], (uint32_t)(pages * rows * 256));
                    __syncwarp();
                    if (ok && mine_box && !is_v && !drop) ptx::tma_load_5d(kd, &kmap, 0, 0, 0, 0, ph, &ctl.kfull[s]);
                    if (ok) ctl.kissued = it + 1;
                    if (ok && it >= 2) ok = pwait(&ctl.vempty[s], par, dead, err);
                    uint64_t* bar = raw ? &ctl.vraw : &ctl.vfull[s];
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(pages * rows * 256));
                    __syncwarp();
                    if (ok && mine_box && is_v) ptx::tma_load_5d(vd, &vmap, 0, 0, 0, 0, ph, bar);
                    if (ok && !raw) ctl.vissued = it + 1;
                    if (ok && raw) ctl.raws = raws + 1;
                }
                if (!__all_sync(0xffffffffu, ok)) goto copies_done;
                if (j + 1 < p.j0 + p.n) id = page_of(j + 1);
                if (raw) {
                    // The request ends in this tile: the values past it may be
                    // anything, NaN too, and weights of 0 do not silence NaN.
                    ok = pwait(&ctl.vraw, (uint32_t)raws & 1u, dead, err);
                    ++raws;
                    for (int i = lane; i < (kKeys - valid) * 16; i += 32) {
                        const int row = valid + (i >> 4), ch = i & 15;
                        *reinterpret_cast<uint4*>(sm + kOffV + s * kOperand + (row >> 3) * kEight + (ch >> 3) * kAtom + (row & 7) * 128 + (ch & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (!__all_sync(0xffffffffu, ok)) goto copies_done;
                    if (lane == 0) ptx::mbar_arrive(&ctl.vfull[s]);
                    ctl.vissued = it + 1;
                }
            }
        }
    copies_done:;
    } else if (warp == kWarpMma) {
        // ---- MMAs, issued by one thread.  It shares its scheduler with two
        // softmax warps, and the pipe holds only about two MMAs beyond the
        // one it works on, so every instruction between two MMAs counts:
        //  * the step of a key tile that both tiles go on from has all operands
        //    constants but the bases of its slots;
        //  * each barrier is tested before the batch of MMAs that precedes its
        //    use, and waited for only if it was not complete by then;
        //  * giving up leaves the loop from the waits, the MMAs carry no condition.
        // (With all operands worked out and conditions at each MMA the same
        // kernel ran 8191 tokens of 32 heads in 568 us, with conditions alone in
        // 442, like this in 333.)
        tc::reg_dec<kRegsOther>();
        Part p;
        int np = 0;
        constexpr uint32_t id_s = tc::idesc_f16kind(kRows, kKeys, !kE4m3, false);
        constexpr uint32_t id_o = tc::idesc_f16kind(kRows, kHeadDim, !kE4m3, true);
        const uint32_t base = ptx::smem_u32(sm);
        const uint64_t dq = tc::desc_sw128(base + kOffQ), dk = tc::desc_sw128(base + kOffK, kE4m3 ? kAtom : kEight);
        const uint64_t dv = tc::desc_sw128_mn(base + kOffV, kAtom, kEight);
        uint32_t qpar[2] = {0u, 0u}, ppar[2] = {0u, 0u};
        int it = 0;
        // S_x = Q_x K^T and four of the eight MMAs of O_x += P_x V.  e4m3: 32
        // channels of K with the two parts of those of Q, one after the other.
        auto mma_s = [&](int x, int slot) {
            const uint64_t k = tc::desc_add(dk, slot * kSlotK<kE4m3>);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t q = tc::desc_add(dq, x * kOperand + (i >> 2) * kBlock + (i & 3) * 32);
                if (kE4m3)
                    tc::mma_ss_e4m3(kColS + 128 * x, q, tc::desc_add(k, (i >> 1) * 32), id_s, i > 0);
                else
                    tc::mma_ss_bf16(kColS + 128 * x, q, tc::desc_add(k, (i >> 2) * kAtom + (i & 3) * 32), id_s, i > 0);
            }
            tc::commit(&ctl.sfull[x]);
        };
        auto mma_pv = [&](int x, int slot, int half, uint32_t add) {
            const uint64_t v = tc::desc_add(dv, slot * kOperand);
#pragma unroll
            for (int i = 4 * half; i < 4 * half + 4; ++i)
                tc::mma_ts_f16kind(kColO + 128 * x, kColS + 128 * x + 8 * i, tc::desc_add(v, i * 2 * kEight), id_o,
                                   i > 0 ? 1u : add);
        };
        // The rest of a wait whose barrier was tested before.
        auto need = [&](bool done, uint64_t* bar, uint32_t par) { return done || pwait(bar, par, dead, err); };
        // One key tile of both tiles, with another one after it for both.
        // `ready`: the test of P_0's first half, on return that of the next one's.
        auto full_step = [&](bool& ready, uint32_t add) -> bool {
            const int sl = it & 1;
            const uint32_t npar = (uint32_t)((it + 1) >> 1) & 1u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!need(ready, &ctl.pfull[x][0], ppar[x])) return false;
                tc::fence_after();
                bool t = ptx::mbar_test(&ctl.pfull[x][1], ppar[x]);
                mma_pv(x, sl, 0, add);
                if (!need(t, &ctl.pfull[x][1], ppar[x])) return false;
                tc::fence_after();
                uint64_t* kv = x ? &ctl.vfull[1 - sl] : &ctl.kfull[1 - sl];
                t = ptx::mbar_test(kv, npar);
                mma_pv(x, sl, 1, 1u);
                ppar[x] ^= 1u;
                if (x) tc::commit(&ctl.vempty[sl]);
                if (!need(t, kv, npar)) return false;
                ready = ptx::mbar_test(&ctl.pfull[1 - x][0], ppar[1 - x]);
                mma_s(x, 1 - sl);
            }
            tc::commit(&ctl.kempty[1 - sl]);
            return true;
        };
        // The same for any state of the two tiles.
        auto any_step = [&](int j) -> bool {
            const int sl = it & 1;
            const uint32_t npar = (uint32_t)((it + 1) >> 1) & 1u;
            for (int x = 0; x < 2; ++x) {
                if (j >= p.cnt[x]) continue;
                for (int half = 0; half < 2; ++half) {
                    if (!pwait(&ctl.pfull[x][half], ppar[x], dead, err)) return false;
                    tc::fence_after();
                    mma_pv(x, sl, half, half || j > 0);
                }
                ppar[x] ^= 1u;
                if (x || j >= p.cnt[1]) tc::commit(&ctl.vempty[sl]);
                if (j + 1 < p.cnt[x]) {
                    if (!pwait(&ctl.kfull[1 - sl], npar, dead, err)) return false;
                    mma_s(x, 1 - sl);
                } else {
                    tc::commit(&ctl.ofull[x]);
                }
            }
            if (j + 1 < p.n) {
                tc::commit(&ctl.kempty[1 - sl]);
                if (!pwait(&ctl.vfull[1 - sl], npar, dead, err)) return false;
            }
            return true;
        };
        auto part = [&]() -> bool {
            if (!pwait(&ctl.kfull[it & 1], (uint32_t)(it >> 1) & 1u, dead, err)) return false;
            for (int x = 0; x < 2; ++x) {
                if (p.cnt[x] <= 0) continue;
                if (!pwait(&ctl.qfull[x], qpar[x], dead, err)) return false;
                qpar[x] ^= 1u;
                tc::fence_after();
                mma_s(x, it & 1);
            }
            tc::commit(&ctl.kempty[it & 1]);
            if (!pwait(&ctl.vfull[it & 1], (uint32_t)(it >> 1) & 1u, dead, err)) return false;
            int j = 0;
            const int both = min(p.cnt[0], p.cnt[1]) - 1;   // steps that both tiles go on from
            bool ready = false;
#pragma unroll 1
            for (; j < both; ++j, ++it)
                if (!full_step(ready, j > 0)) return false;
#pragma unroll 1
            for (; j < p.n; ++j, ++it)
                if (!any_step(j)) return false;
            return true;
        };
        const bool issuer = tc::elect_one();
        bool ok = true;
        while (take_part(ctl, np, p, dead, err)) {
            if (issuer && ok) ok = part();
            __syncwarp();
        }
        if (issuer) tc::commit(&ctl.drain);   // completes once every MMA that it issued has
    } else if (kE4m3 && warp >= kWarpConvert) {
        // ---- e4m3 -> f16 of the values, two keys per thread
        tc::reg_dec<kRegsOther>();
        Part p;
        int np = 0;
        const int row0 = tid - 32 * kWarpConvert;
        int it = 0;
        bool ok = true;
        while (ok && take_part(ctl, np, p, dead, err))
            for (int j = p.j0; j < p.j0 + p.n; ++j, ++it) {
                const int s = it & 1;
                ok = pwait(&ctl.cvfull[s], (uint32_t)(it >> 1) & 1u, dead, err);
                if (ok && it >= 2) ok = pwait(&ctl.vempty[s], (uint32_t)((it >> 1) - 1) & 1u, dead, err);
                if (!ok) break;
#pragma unroll 1
                for (int row = row0; row < kKeys; row += kConvert) {
                    const bool live = j * kKeys + row < p.s.len;
                    const uint8_t* src = sm + kOffStage + s * kBlock + row * 128;
                    uint8_t* dst = sm + kOffV + s * kOperand + (row >> 3) * kEight + (row & 7) * 128;
#pragma unroll 8
                    for (int c = 0; c < 8; ++c) {
                        uint4 w = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
                        if (!live) w = make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                        uint32_t f[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[2 * i] = mma::e4m3x2_f16x2(u[i]);
                            f[2 * i + 1] = mma::e4m3x2_f16x2(u[i] >> 16);
                        }
                        uint8_t* d = dst + (c >> 2) * kAtom;
                        *reinterpret_cast<uint4*>(d + ((((2 * c) & 7) ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(d + ((((2 * c + 1) & 7) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&ctl.vfull[s]);
                ptx::mbar_arrive(&ctl.cvempty[s]);
            }
    } else if (warp < 8) {
        // ---- softmax, one thread per row of tile x
        tc::reg_inc<kRegsSoftmax>();
        Part p;
        int np = 0;
        const int x = warp >> 2, r = tid & (kRows - 1);
        const int i_row = r / a.G, g_row = r % a.G;
        const uint32_t ts = tc::taddr(tm, warp, kColS + 128 * x), to = tc::taddr(tm, warp, kColO + 128 * x);
        uint32_t spar = 0u, opar = 0u;
        bool ok = true;
        float spoiled = 0.f;   // NaN or infinite once a result of a row with a token was
        // The warp's 32 rows of Q_x, and of the results on their way out (rows
        // of kOut bytes), both swizzled as TMA would.
        constexpr int kOut = 128, kOutLanes = kOut / 16, kOutRows = 32 / kOutLanes;
        uint8_t* rows_q = sm + kOffQ + x * kOperand + (warp & 3) * 32 * 128;
        uint8_t* rows_o = sm + kOffOut<kE4m3> + warp * 32 * 128;
        auto place_q = [&](int row, int c) { return rows_q + (c >> 3) * kBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4); };
        auto place_o = [&](int row, int c) { return rows_o + row * 128 + ((c ^ (row & 7)) << 4); };
        // A part as this thread's row and the warp's rows see it.
        struct Rows {
            bool live;           // the row has a token
            uint32_t lives;      // the warp's rows that have
            size_t head;         // of the output, and of q
            float fac;           // logit -> power of two
        };
        auto head_of = [&](const Rows& w, int row) { return (size_t)__shfl_sync(0xffffffffu, (unsigned long long)w.head, row); };
        // Q rows into shared memory: the copies, two rows a round, and what
        // follows them.  The loops that run once per part stay rolled: their
        // instructions come from L2 each time.
        auto start_rows = [&](const Part& part) {
            Rows w;
            w.live = i_row < part.s.tokens_of(x, a.tokens);
            w.lives = __ballot_sync(0xffffffffu, w.live);
            w.head = ((size_t)part.s.tok + x * a.tokens + i_row) * a.Hq + part.s.h * a.G + g_row;
            w.fac = a.scale;
            if (part.cnt[x] > 0) {
#pragma unroll 2
                for (int i = 0; i < 16; ++i) {
                    const int row = 2 * i + (lane >> 4), c = lane & 15;
                    const size_t h = head_of(w, row);
                    ptx::cp_async16(place_q(row, c), a.io.q + h * kHeadDim + 8 * c, w.lives >> row & 1u);
                }
                ptx::cp_async_commit();
            }
            return w;
        };
        auto finish_rows = [&](const Part& part, Rows& w) {
            if (part.cnt[x] <= 0) return;
            ptx::cp_async_wait_all();
            __syncwarp();
            if (kE4m3) {
                // To two e4m3 parts, each lane its row: q * 2^(7 - e) with 2^e <= the
                // row's largest < 2^(e+1), rounded, and what that leaves of its eight
                // bits: exact for values down to 2^-9 of the row's largest, below
                // that off by up to 2^-17 of it.  Each 64 bytes of a row hold 32
                // channels' first parts, then their second.
                float top = 0.f;
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4*>(place_q(lane, c));
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = mma::max3(top, fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u)));
                }
                const int ex = mma::query_exponent(top);
                const float up = exp2f((float)(7 - ex));
                w.fac = mma::query_factor(a.scale, ex - 7, a.k_scale[part.s.h]);
                if (top == INFINITY) w.fac = __int_as_float(0x7fc00000);   // which e4m3 does not hold
#pragma unroll 1
                for (int c = 0; c < 16; c += 4) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = *reinterpret_cast<const uint4*>(place_q(lane, c + k));
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t f0 = mma::pack_f16(__uint_as_float(u[2 * e] << 16) * up, __uint_as_float(u[2 * e] & 0xffff0000u) * up);
                            const uint32_t f1 = mma::pack_f16(__uint_as_float(u[2 * e + 1] << 16) * up, __uint_as_float(u[2 * e + 1] & 0xffff0000u) * up);
                            const uint32_t h0 = mma::f16x2_e4m3x2(f0), h1 = mma::f16x2_e4m3x2(f1);
                            hi[2 * k + e] = h0 | h1 << 16;
                            lo[2 * k + e] = mma::f16x2_e4m3x2(mma::sub_f16x2(f0, mma::e4m3x2_f16x2(h0))) |
                                            mma::f16x2_e4m3x2(mma::sub_f16x2(f1, mma::e4m3x2_f16x2(h1))) << 16;
                        }
                    }
                    *reinterpret_cast<uint4*>(place_q(lane, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(place_q(lane, c + 1)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    *reinterpret_cast<uint4*>(place_q(lane, c + 2)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    *reinterpret_cast<uint4*>(place_q(lane, c + 3)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                }
            }
            ptx::fence_proxy_async_smem();
        };
        auto hand_over = [&](const Part& part) {   // Q_x, and S_x to be written
            tc::fence_before();
            if (part.cnt[x] > 0) ptx::mbar_arrive(&ctl.qfull[x]);
        };
        Rows w{};
        bool more = take_part(ctl, np, p, dead, err);
        if (more) {
            w = start_rows(p);
            finish_rows(p, w);
            hand_over(p);
        }
        while (more) {
            const bool live = w.live;
            const float fac = w.fac;
            float ref = kNoRef, sum = 0.f;
            const int cnt = p.cnt[x];
            if (cnt > 0) {
                // Keys that the row sees; rows without a token see all (their q is zero, nothing is stored).
                const int sees = kShared ? p.s.len : live ? p.s.first + x * a.tokens + i_row : 0x7fffffff;
                for (int j = p.j0; j < p.j0 + cnt; ++j) {
                    ok = pwait(&ctl.sfull[x], spar, dead, err);
                    spar ^= 1u;
                    tc::fence_after();
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, s[c]);
                    tc::wait_ld();
                    const int left = sees - j * kKeys;   // columns of the tile that the row sees
                    if (__any_sync(0xffffffffu, left < kKeys)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * c + e >= left) s[c][e] = 0xff800000u;   // -infinity
                    }
                    float m[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        m[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                        for (int e = 2; e < 32; e += 2) m[c] = mma::max3(m[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                    }
                    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * fac;
                    const bool raise = top > ref + kLimit;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float now = raise ? top - kOffset : ref;
                        const float f = mma::exp2_approx(ref - now);
                        ref = now;
                        sum *= f;
                        if (j > p.j0) {
                            // S_x(j) is complete, so P_x(j - 1) V is too: O_x is at rest.
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t o[16];
                                tc::ld16(to + 16 * c, o);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st16(to + 16 * c, o);
                            }
                        }
                    }
                    const mma::f32x2 fac2 = mma::pk(fac, fac), ref2 = mma::pk(-ref, -ref);
                    mma::f32x2 sum2[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float u, v;
                            mma::upk(mma::fma2(mma::pk(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), fac2, ref2), u, v);
                            u = mma::exp2_approx(u);
                            v = mma::exp2_approx(v);
                            sum2[e & 1] = mma::add2(sum2[e & 1], mma::pk(u, v));
                            pk[e] = kE4m3 ? mma::pack_f16(u, v) : mma::pack_bf16(u, v);
                        }
                        tc::st16(ts + 16 * c, pk);
                        if (c & 1) {
                            tc::wait_st();
                            tc::fence_before();
                            ptx::mbar_arrive(&ctl.pfull[x][c >> 1]);
                        }
                    }
                    float u, v;
                    mma::upk(mma::add2(sum2[0], sum2[1]), u, v);
                    sum += u + v;
                }
                if (!ok) break;
            }
            // The next part's Q rows come in under the last MMAs (Q_x is free
            // since the last logits), and its first logits are computed while
            // these results go out (S_x is free once O_x is complete).
            Part pn;
            Rows wn{};
            const bool more_n = take_part(ctl, np, pn, dead, err);
            if (more_n) {
                wn = start_rows(pn);
                finish_rows(pn, wn);
            }
            if (cnt > 0) {
                ok = pwait(&ctl.ofull[x], opar, dead, err);
                opar ^= 1u;
                tc::fence_after();
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            }
            if (more_n) hand_over(pn);
            // The rows' results, or this part's share of them, through shared
            // memory so that whole stretches of rows are stored together: in
            // bf16 where that is all there is to write, else in fp32.
            const bool whole = p.slot < 0;
            float* part = whole ? nullptr : slot_at(a.io.workspace, gridDim.x, p.slot);
            if (cnt > 0) {
                const float n = !whole ? 1.f : sum != 0.f ? (kE4m3 ? a.v_scale[p.s.h] : 1.f) / sum : 0.f;
                const bool plain = whole && !a.io.gate && !a.io.o_f32;
                const uint32_t seeing = __ballot_sync(0xffffffffu, sum != 0.f);   // rows that see a key
                const int step = plain ? kOut / 2 : kOut / 4;   // channels at a time
#pragma unroll 1
                for (int c0 = 0; c0 < kHeadDim; c0 += step) {
#pragma unroll 1
                    for (int c1 = 0; c1 < step; c1 += 32) {
                        uint32_t o[32];
                        tc::ld32(to + c0 + c1, o);
                        tc::wait_ld();
                        float z = 0.f;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) z = mma::max3n(z, fabsf(__uint_as_float(o[e])), fabsf(__uint_as_float(o[e + 1])));
                        if (!kShared && live) spoiled = mma::max3n(spoiled, z, z);
                        if (plain) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4*>(place_o(lane, (c1 + e) >> 3)) = make_uint4(
                                    mma::pack_bf16(__uint_as_float(o[e]) * n, __uint_as_float(o[e + 1]) * n),
                                    mma::pack_bf16(__uint_as_float(o[e + 2]) * n, __uint_as_float(o[e + 3]) * n),
                                    mma::pack_bf16(__uint_as_float(o[e + 4]) * n, __uint_as_float(o[e + 5]) * n),
                                    mma::pack_bf16(__uint_as_float(o[e + 6]) * n, __uint_as_float(o[e + 7]) * n));
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4*>(place_o(lane, (c1 + e) >> 2)) =
                                    make_float4(__uint_as_float(o[e]) * n, __uint_as_float(o[e + 1]) * n,
                                                __uint_as_float(o[e + 2]) * n, __uint_as_float(o[e + 3]) * n);
                        }
                    }
                    __syncwarp();
                    const int c = lane % kOutLanes, row0 = lane / kOutLanes;
                    if (plain) {
#pragma unroll 4
                        for (int row = row0; row < 32; row += kOutRows) {
                            const size_t h = head_of(w, row);
                            const uint4 v = *reinterpret_cast<const uint4*>(place_o(row, c));
                            if (w.lives >> row & 1u)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.io.o) + h * kHeadDim + c0 + 8 * c) = v;
                        }
                    } else {
#pragma unroll 4
                        for (int row = row0; row < 32; row += kOutRows) {
                            const size_t h = head_of(w, row);
                            const float4 v = *reinterpret_cast<const float4*>(place_o(row, c));
                            if (w.lives >> row & 1u) {
                                if (whole) mma::store4(a.io, h * kHeadDim + c0 + 4 * c, v, seeing >> row & 1u);
                                else *reinterpret_cast<float4*>(part + (size_t)(warp * 32 + row) * kHeadDim + c0 + 4 * c) = v;
                            }
                        }
                    }
                    __syncwarp();
                }
                tc::fence_before();
            }
            const size_t head = w.head;
            if (live && whole && a.io.lse) a.io.lse[head] = sum != 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
            if (live && !whole)
                *reinterpret_cast<float2*>(part + (size_t)2 * kRows * kHeadDim + 2 * (x * kRows + r)) = make_float2(ref, sum);
            if (tid == 0 && p.last >= 0)
                joins(a.io.workspace)[blockIdx.x] = PrefillJoin{p.s.tok, p.s.m, p.s.h, p.last, p.slot, {0, 0, 0}};
            p = pn;
            w = wn;
            more = more_n;
        }
        ptx::cp_async_wait_all();   // of a part that was given up
        if (!kShared && __any_sync(0xffffffffu, !(spoiled < INFINITY)) && __all_sync(0xffffffffu, *(volatile int*)dead == 0)) {
            // Values that they do not see may have got into this warp's rows (attn_again.cuh): its parts again.
            // (Looking at all results costs calls without such values 0.6 % of an 8191-token prompt's time, 0.8 % of the
            // ragged e4m3 chunks'; in the join kernel instead, what the join then carries cost calls with cut keys 3 %.)
            __syncwarp();
            Cursor cur{kShared || sc.split ? -1 : 0, 0, false, {}, 0};
            for (next_part<kShared>(a, ctl, sc, cur, p); p.n > 0; next_part<kShared>(a, ctl, sc, cur, p)) {
                const int i = x * a.tokens + i_row;
                const size_t head = ((size_t)p.s.tok + i) * a.Hq + p.s.h * a.G + g_row;
                float* part = slot_at(a.io.workspace, gridDim.x, max(p.slot, 0));
                if (p.cnt[x] > 0)
                    rows_again<kE4m3>(a, p.s.b, p.s.h, i_row < p.s.tokens_of(x, a.tokens), head, p.j0 * kKeys,
                                      min((p.j0 + p.cnt[x]) * kKeys, p.s.len), p.s.first + i,
                                      [&](int channel, float4 v, float ref, float sum) {
                        if (p.slot < 0) {
                            const float n = sum != 0.f ? (kE4m3 ? a.v_scale[p.s.h] : 1.f) / sum : 0.f;
                            mma::store4(a.io, head * kHeadDim + channel, make_float4(v.x * n, v.y * n, v.z * n, v.w * n), sum != 0.f);
                        } else {
                            const int at = x * kRows + r;
                            const float f = sum != 0.f ? mma::exp2_approx(ref - part[(size_t)2 * kRows * kHeadDim + 2 * at]) : 0.f;
                            *reinterpret_cast<float4*>(part + (size_t)at * kHeadDim + channel) =
                                make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                        }
                    });
            }
        }
    } else {
        tc::reg_dec<kRegsOther>();
    }

    tc::fence_before();
    if (__syncthreads_or(*(volatile int*)dead)) {
        // Give-up path: the MMAs and the copies this CTA issued complete
        // (bounded waits) before its TMEM and shared memory are released.
        if (tid == 32 * kWarpMma) ptx::mbar_wait_timed(&ctl.drain, 0);
        if (tid == 32 * kWarpTma) {
            for (int i = max(0, ctl.kissued - 2); i < ctl.kissued; ++i)
                ptx::mbar_wait_timed(&ctl.kfull[i & 1], (uint32_t)(i >> 1) & 1u);
            for (int i = max(0, ctl.vissued - 2); i < ctl.vissued; ++i)
                ptx::mbar_wait_timed(kE4m3 ? &ctl.cvfull[i & 1] : &ctl.vfull[i & 1], (uint32_t)(i >> 1) & 1u);
            if (ctl.raws) ptx::mbar_wait_timed(&ctl.vraw, (uint32_t)(ctl.raws - 1) & 1u);
        }
    }
    __syncthreads();
    if (warp == kWarpMma) tc::dealloc(tm, 512);
}

// Joins the parts of segments cut between CTAs, a warp per row, four channels
// per lane; the rows of all cut segments are shared out evenly.
__global__ void __launch_bounds__(256) kda_attn_prefill_join_kernel(const PrefillArgs a, int ctas) {
    __shared__ int s_end[kMaxCtas], s_warp[8];   // rows up to and with the segment that CTA i begins
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int end = tid < ctas ? joins(a.io.workspace)[tid].m * a.G : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += y;
    }
    if (lane == 31) s_warp[warp] = end;
    __syncthreads();
    int rows = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) end += s_warp[w];
        rows += s_warp[w];
    }
    s_end[tid] = end;
    __syncthreads();
    for (int at_row = blockIdx.x * 8 + warp; at_row < rows; at_row += gridDim.x * 8) {
        int lo = 0, hi = ctas - 1;   // the first CTA whose rows end past this one
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > at_row) hi = mid; else lo = mid + 1;
        }
        const PrefillJoin d = joins(a.io.workspace)[lo];
        const int row = at_row - (lo ? s_end[lo - 1] : 0);
        const int parts = d.last - lo + 1;
        const int i = row / a.G, g = row % a.G;
        const int at = i < a.tokens ? row : kRows + row - a.tokens * a.G;   // row of the pair of tiles
        float ref = kNoRef, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int q = 0; q < parts; ++q) {
            const float* s = slot_at(a.io.workspace, ctas, q == 0 ? d.slot : 2 * (lo + q));
            const float2 ls = *reinterpret_cast<const float2*>(s + (size_t)2 * kRows * kHeadDim + 2 * at);
            const float4 v = *reinterpret_cast<const float4*>(s + (size_t)at * kHeadDim + 4 * lane);
            // No key of this part is seen: the weighted sum was not written.  (A NaN sum goes in, and makes the row NaN.)
            if (ls.y == 0.f) continue;
            const float to = fmaxf(ref, ls.x);
            const float f = mma::exp2_approx(ref - to), e = mma::exp2_approx(ls.x - to);
            ref = to;
            sum = sum * f + ls.y * e;
            acc.x = acc.x * f + v.x * e;
            acc.y = acc.y * f + v.y * e;
            acc.z = acc.z * f + v.z * e;
            acc.w = acc.w * f + v.w * e;
        }
        const float n = sum != 0.f ? (a.v_scale ? a.v_scale[d.h] : 1.f) / sum : 0.f;
        const size_t head = ((size_t)d.tok + i) * a.Hq + d.h * a.G + g;
        mma::store4(a.io, head * kHeadDim + 4 * lane, make_float4(acc.x * n, acc.y * n, acc.z * n, acc.w * n), sum != 0.f);
        if (a.io.lse && lane == 0) a.io.lse[head] = sum != 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
    }
}

std::atomic<bool> g_attr_done[64];

template <bool kE4m3, bool kShared>
cudaError_t prepare_kernel() {
    cudaFuncAttributes f{};
    cudaError_t e = cudaFuncGetAttributes(&f, kda_attn_prefill_kernel<kE4m3, kShared>);
    if (e != cudaSuccess) return e;
    if (f.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;   // the splits would never be met
    return cudaFuncSetAttribute(kda_attn_prefill_kernel<kE4m3, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<kE4m3>());
}

}  // namespace

bool attn_prefill_maps(const AttnLayer& l, AttnMaps& maps) {
    const int rows = l.page_size < kKeys ? l.page_size : kKeys;
    if (l.e4m3)
        return make_cache_map(&maps.k_prefill, l, l.k_cache, rows, 1) && make_cache_map(&maps.v_prefill, l, l.v_cache, rows, 1);
    return make_cache_map_atoms(&maps.k_prefill, l, l.k_cache, rows) && make_cache_map_atoms(&maps.v_prefill, l, l.v_cache, rows);
}

int attn_many_rows_cost(const AttnLayer& l) { return l.e4m3 ? 4 : 3; }

float* attn_many_rows_slots(void* workspace, const DeviceInfo& dev) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + join_bytes(dev.sm_count));
}

size_t attn_prefill_workspace_bytes(const DeviceInfo& dev) {
    return join_bytes(dev.sm_count) + (size_t)dev.sm_count * 2 * kSlotFloats * sizeof(float);
}

namespace {
cudaError_t launch(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev, int* err_word,
                   cudaStream_t stream, bool all, bool shared) {
    if (dev.device < 0 || dev.device >= 64 || dev.sm_count > kMaxCtas) return cudaErrorInvalidDevice;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        cudaError_t e = prepare_kernel<false, false>();
        if (e == cudaSuccess) e = prepare_kernel<true, false>();
        if (e == cudaSuccess) e = prepare_kernel<false, true>();
        if (e == cudaSuccess) e = prepare_kernel<true, true>();
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    PrefillArgs a{};
    a.io = io;
    a.Hq = l.Hq;
    a.Hkv = l.Hkv;
    a.G = l.G;
    a.tokens = kRows / l.G;
    a.all = all;
    a.part_cost = attn_many_rows_cost(l);
    a.page_shift = l.page_shift;
    a.num_pages = l.num_pages;
    a.scale = l.softmax_scale * kLog2e;
    a.k_scale = l.k_scale;
    a.v_scale = l.v_scale;
    a.k_cache = l.k_cache;
    a.v_cache = l.v_cache;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = shared ? 1 : 0;
    const int grid = dev.sm_count;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = l.e4m3 ? smem_bytes<true>() : smem_bytes<false>();
    cfg.stream = stream;
    auto kernel = shared ? (l.e4m3 ? kda_attn_prefill_kernel<true, true> : kda_attn_prefill_kernel<false, true>)
                         : (l.e4m3 ? kda_attn_prefill_kernel<true, false> : kda_attn_prefill_kernel<false, false>);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, maps.k_prefill, maps.v_prefill, err_word);
    count_launches(1);
    if (e != cudaSuccess || shared) return e;
    cfg.gridDim = dim3((unsigned)grid * kJoinCtas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kda_attn_prefill_join_kernel, a, grid);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_many_rows(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev,
                                  int* err_word, cudaStream_t stream, bool all) {
    return launch(l, maps, io, dev, err_word, stream, all, false);
}

cudaError_t launch_attn_many_rows_shared(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io,
                                         const DeviceInfo& dev, int* err_word, cudaStream_t stream) {
    return launch(l, maps, io, dev, err_word, stream, false, true);
}

}  // namespace kda
