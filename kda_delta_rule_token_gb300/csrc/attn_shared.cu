// Attention of one new token per request where groups of requests share a prefix.
//
//   o = (e^a o_p + e^b o_r) / (e^a + e^b)
//
// with o_p and a = lse of the request's row over the prefix, o_r and b over the
// keys that are its own.  A prefix's keys are read once for all of its
// requests, whose rows stand beside each other in the products: n requests of G
// heads per key head are n * G rows.  Four launches:
//
//  * the plan, one CTA: which requests are long enough to take part (the others
//    attend to all of their keys by themselves), whose table has the prefix's pages, and
//    how much of the prefix counts: whole pages, and whole tiles of the next kernel, so
//    that no tile has keys of both kinds.  From these the work's prefix sums, which the
//    other kernels find their shares by.
//  * kda_attn_shared_few_kernel: the requests' own keys, and prefixes of few rows per
//    key head (16 in bf16; 32 in e4m3, and in calls that can have no more), 16 at a time.
//    Own keys are often few, so a warp works alone: all warps get equal ranges
//    of tiles, copied by TMA ahead of their use across the ends of requests, and no warp
//    waits for another.
//  * the prompts' tensor core kernel (attn_prefill.cu), without a causal edge: prefixes of
//    more rows, cut into equal ranges of key tiles for all SMs.  Its CTAs come as the few-row
//    kernel's end, and wait for all of it before they look at the plan.
//  * the join: a warp per row, or a CTA where rows are few.  What one warp (or CTA) had
//    of a row alone came to the workspace as a finished result, what several had as parts;
//    who had the first and the last one noted it.
//
// Measured (a kernel's share: what the call takes longer when it is launched twice): 32 prompts of up
// to 4,100 tokens with 1 to 30 requests each, 32 / 8 heads, bf16, 534 MB: 127 us, 0.62 of
// the copy rate (the few-row kernel 53 us and the tensor core kernel about 57, 5 TB/s each; plan
// 5, join 7).  64 requests behind 8,192 tokens, 65 MB: 38 us (plan 3, few-row kernel 9,
// tensor core kernel 15, join 7, whose 20 MB of parts come from L2; kda_attn_decode: 178 us); of
// the tensor core kernel's 15 its 3 or 4 key tiles take 6, the parts' way out 3 (6.4 TB/s).  256 requests of 64 heads
// behind four documents of up to 16,300 tokens in e4m3, 128 GFLOP: 135 us (plan 6, few-row kernel
// 17, tensor core kernel about 97, join 11).  What is left of each sum, 5, 2 and 4 us, the tensor core
// kernel waits for the last CTAs of the few-row kernel; that its own set-up comes before that wait
// changes nothing (127.2, 37.2 and 134.5 us).  The requests' own keys in the decode's kernel,
// where four warps share a request's tiles and meet at its end: 15 us slower.  Queries and
// requests brought near ahead of their use, more tiles per warp: no faster.  The join with
// several rows of a request per CTA, their places found once: 1 to 5 us slower.
#include <atomic>

#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "attn_ptx.cuh"
#include "attn_rows.cuh"
#include "attn_tma.cuh"
#include "launch.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024, kNear = 2048;
constexpr int kWarps = 4, kThreads = kWarps * 32, kCtasPerSm = 2;
constexpr int kStages = 3;                       // tiles that a warp has under way
constexpr uint32_t kStageBytes = 2 * kRowTileBytes;
constexpr int kRows = 16;                        // rows of a tile
constexpr int kCost = 2;                         // tiles that starting and ending a request and head costs beside its own
                                                 // (1, 4 and 6: within 1 %)
constexpr int kSlotFloats = kRows * (kHeadDim + 2);

// A request's own keys, or a group's prefix, as the few-row kernel sees it.
struct __align__(16) Item {
    long long table;     // place of its first page in the block table
    int len;             // keys, 0: nothing to do
    int q, out, n;       // first token of q and of the results, tokens
    int tiles;           // row tiles per key head
    int pad;
};

struct Args {
    AttnSharedIO io;
    int Hq, Hkv, G;
    int few_rows;        // rows of a group, at most, that the few-row kernel takes
    int tile_shift;      // keys of its tiles
    int page_shift, num_pages;
    int tokens;          // of a row tile of the tensor core kernel
    int many_cost;       // key tiles that a segment costs there
    float scale;         // softmax scale * log2(e)
    const float* k_scale;
    const float* v_scale;
    Item* items;             // [groups + B]
    long long* start;        // [groups + B + 1] units (tiles, and costs) before each, in the few-row kernel
    long long* many_start;   // [groups + 1] the same in the tensor core kernel
    int* many_pairs;         // [groups] pairs of its token tiles before each
    int2* few_parts;         // first part's slot (-1: finished) and last part's, of an item, key head and row tile
    int2* many_parts;        // [pairs][Hkv] the same of the tensor core kernel
    int* group_of;           // [B] the group that a request shares in, or -1
    int* group_len;          // [groups]
    int* group_row;          // [groups]
    float* slots;            // parts of the few-row kernel, two per warp
    const float* many_slots; // of the tensor core kernel, two per CTA
    void* decode;            // of kda_attn_decode's kernels
    float* o;                // [2 B][Hq][128] results over the prefix, then of own keys
    float* lse;              // [2 B][Hq]
    int warps;               // of the few-row kernel
    int many_ctas;
};

size_t carve(Args& a, AttnIO& many, void* workspace, const AttnLayer& l, int B, const DeviceInfo& dev) {
    uint8_t* at = static_cast<uint8_t*>(workspace);
    auto take = [&](size_t bytes) {
        uint8_t* p = at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    const size_t warps = (size_t)dev.sm_count * kCtasPerSm * kWarps, n = (size_t)2 * B;   // groups + B at most
    a.decode = take(attn_decode_workspace_bytes(dev));
    a.slots = reinterpret_cast<float*>(take(warps * 2 * kSlotFloats * 4));
    many.workspace = take(attn_prefill_workspace_bytes(dev));
    a.many_slots = attn_many_rows_slots(many.workspace, dev);
    a.items = reinterpret_cast<Item*>(take(n * sizeof(Item)));
    a.start = reinterpret_cast<long long*>(take((n + 1) * 8));
    a.many_start = reinterpret_cast<long long*>(take((size_t)(B + 1) * 8));
    a.many_pairs = reinterpret_cast<int*>(take((size_t)B * 4));
    a.few_parts = reinterpret_cast<int2*>(take((size_t)B * l.Hkv * (2 + (l.G + kRows - 1) / kRows) * 8));
    a.many_parts = reinterpret_cast<int2*>(take((size_t)B * l.Hkv * 8));
    a.group_of = reinterpret_cast<int*>(take((size_t)B * 4));
    a.group_len = reinterpret_cast<int*>(take((size_t)B * 4));
    a.group_row = reinterpret_cast<int*>(take((size_t)B * 4));
    a.o = reinterpret_cast<float*>(take(n * l.Hq * kHeadDim * 4));
    a.lse = reinterpret_cast<float*>(take(n * l.Hq * 4));
    return (size_t)(at - static_cast<uint8_t*>(workspace));
}

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
    long long w = lane < (int)(blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const long long before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    __syncthreads();   // s_warp may be used again
    return before + x - v;
}

// Offsets that are not ascending within the requests are an error, and nothing is
// shared then; the results are the same.
__global__ void __launch_bounds__(kPlanThreads) kda_attn_shared_plan_kernel(const Args a, int* err) {
    __shared__ long long s_warp[32];
    __shared__ int s_group[kNear], s_len[kNear];   // group_of and group_len, where they fit
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const AttnSharedIO& io = a.io;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const int shift = max(a.page_shift, a.tile_shift), most = io.max_pages << a.page_shift;
    int* group_of = io.B <= kNear ? s_group : a.group_of;
    int* group_len = io.B <= kNear ? s_len : a.group_len;   // (no more groups than requests)
    const int count = io.groups + io.B;
    const int per = (count + threads - 1) / threads, i0 = min(count, tid * per), i1 = min(count, i0 + per);
    bool bad = false;
    // What this thread's first item and this warp's first group need, on the way beside the offsets.
    const int kv0 = i0 < i1 && i0 >= io.groups ? io.kv_lens[i0 - io.groups] : 0;
    int from0 = 0, to0 = 0, len0 = 0;
    if (warp < io.groups) {
        from0 = io.cu_groups[warp];
        to0 = io.cu_groups[warp + 1];
        len0 = io.prefix_lens[warp];
    }
    for (int g = tid; g < io.groups; g += threads) bad |= bad_offsets(io.cu_groups, g, io.B);
    for (int b = tid; b < io.B; b += threads) group_of[b] = -1;
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) atomicOr(err, kErrAttnIndex);
    for (int g = warp; g < io.groups; g += threads / 32) {
        const bool near = g == warp;
        const int from = bad ? 0 : near ? from0 : io.cu_groups[g], to = bad ? 0 : near ? to0 : io.cu_groups[g + 1];
        const int len = min(max(near ? len0 : io.prefix_lens[g], 0), most) >> shift << shift;
        int members = 0, row = 0;
        uint32_t first32 = 0;   // who of the first 32 has so many keys
        if (len)
            for (int b = from; b < to; b += 32) {
                const uint32_t has = __ballot_sync(0xffffffffu, b + lane < to && min(io.kv_lens[b + lane], most) >= len);
                if (members == 0 && has) row = b + __ffs((int)has) - 1;
                if (b == from) first32 = has;
                members += __popc(has);
            }
        const bool share = members > 1;
        if (lane == 0) {
            group_len[g] = a.group_len[g] = share ? len : 0;
            a.group_row[g] = row;
        }
        if (share) {
            if (first32 >> lane & 1) group_of[from + lane] = g;
            for (int b = from + 32 + lane; b < to; b += 32)
                if (min(io.kv_lens[b], most) >= len) group_of[b] = g;
        }
    }
    __syncthreads();

    struct Cost {
        long long few, many;
        int pairs;
    };
    auto item_of = [&](int i, Cost& cost) {
        Item x;
        cost.many = 0;
        cost.pairs = 0;
        x.pad = 0;
        if (i < io.groups) {
            x.len = group_len[i];
            x.q = x.out = x.len ? io.cu_groups[i] : 0;
            x.n = x.len ? io.cu_groups[i + 1] - x.q : 0;
            x.table = (long long)a.group_row[i] * io.max_pages;
            if ((long long)x.n * a.G > a.few_rows) {
                cost.pairs = (x.n + 2 * a.tokens - 1) / (2 * a.tokens);
                cost.many = (long long)cost.pairs * a.Hkv * ((x.len + 127) / 128 + a.many_cost);
                x.len = 0;
            }
            x.tiles = (x.n * a.G + kRows - 1) / kRows;   // of groups with len: at most two
        } else {
            const int b = i - io.groups, g = group_of[b], before = g >= 0 ? group_len[g] : 0;
            a.group_of[b] = g;
            x.len = min(max(i == i0 ? kv0 : io.kv_lens[b], 0), most) - before;
            x.q = b;
            x.out = io.B + b;
            x.n = 1;
            x.table = (long long)b * io.max_pages + (before >> a.page_shift);
            x.tiles = (a.G + kRows - 1) / kRows;
        }
        cost.few = x.len ? (long long)(((x.len + (1 << a.tile_shift) - 1) >> a.tile_shift) + kCost) * a.Hkv * x.tiles : 0;
        return x;
    };
    Cost mine{0, 0, 0}, c{};
    Item x{};
    for (int i = i0; i < i1; ++i) {
        x = item_of(i, c);
        mine.few += c.few;
        mine.many += c.many;
        mine.pairs += c.pairs;
    }
    long long total, many_total, pairs_total;
    long long few = block_exclusive(mine.few, s_warp, &total);
    long long many = 0, pairs = 0;
    many_total = 0;
    if (__syncthreads_or(mine.many != 0)) {
        many = block_exclusive(mine.many, s_warp, &many_total);
        pairs = block_exclusive(mine.pairs, s_warp, &pairs_total);
    }
    for (int i = i0; i < i1; ++i) {
        if (per > 1) x = item_of(i, c);
        a.items[i] = x;
        a.start[i] = few;
        if (i < io.groups) {
            a.many_start[i] = many;
            a.many_pairs[i] = (int)pairs;
        }
        few += c.few;
        many += c.many;
        pairs += c.pairs;
    }
    if (tid == 0) {
        a.start[count] = total;
        a.many_start[io.groups] = many_total;
    }
}

// Where the notes on an item's parts begin.
__device__ __forceinline__ int2* parts_of(const Args& a, int i) {
    const size_t own = (size_t)(a.G + kRows - 1) / kRows * a.Hkv;
    return a.few_parts + (i < a.io.groups ? (size_t)i * 2 * a.Hkv : (size_t)a.io.groups * 2 * a.Hkv + (i - a.io.groups) * own);
}

// Whose units these are: the last i < count with start[i] <= unit, of those with any units.  A warp's lanes look together.
__device__ __forceinline__ int find_item(const long long* start, int count, long long unit) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = count;   // start[lo] <= unit < start[lo + n]
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lo + min(lane * step, n);
        const uint32_t below = __ballot_sync(0xffffffffu, lane * step < n && start[at] <= unit);
        const int k = 31 - __clz((int)below);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

struct Smem {
    uint8_t ring[kWarps * kStages * kStageBytes];
    uint64_t full[kWarps * kStages];
    int dead;
};

// A place in a warp's range of units.  The range also counts kCost units before each
// request's (or group's) and row tile's first.
struct Walk {
    long long left;      // units of the range not yet passed, this one included; none if <= 0
    int i, vh, u;        // item, (key head, row tile) of it, tile of keys
    int units;           // tiles of keys of item i
    Item x;
};

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
kda_attn_shared_few_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, int* err) {
    using Tile = RowTile<kE4m3>;
    constexpr int kKeys = Tile::kKeys;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(sm_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
    uint64_t* full = sm.full + warp * kStages;
    uint8_t* ring = sm.ring + warp * kStages * kStageBytes;
    if (lane == 0)
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s], 1);
    if (tid == 0) sm.dead = 0;
    ptx::fence_mbar_init();
    __syncthreads();
    ptx::griddep_wait();               // the plan
    ptx::griddep_launch_dependents();

    const int count = a.io.groups + a.io.B;
    const long long total = a.start[count];
    const long long warps = min((long long)a.warps, total);
    const int w = blockIdx.x * kWarps + warp;
    if (w >= warps) return;
    const long long from = total * w / warps, to = total * (w + 1) / warps;

    auto enter = [&](Walk& k, int i) {
        k.i = i;
        k.x = a.items[i];
        k.units = (k.x.len + kKeys - 1) / kKeys;
    };
    auto step = [&](Walk& k) {
        --k.left;
        if (++k.u < k.units) return;
        k.u = 0;
        k.left -= kCost;
        if (++k.vh < a.Hkv * k.x.tiles) return;
        k.vh = 0;
        if (k.left <= 0) return;
        do enter(k, k.i + 1);
        while (k.units == 0);
    };
    Walk cur;
    {
        int i = find_item(a.start, count, from);
        enter(cur, i);
        const long long in = from - a.start[i];
        const int per = cur.units + kCost;
        cur.vh = (int)(in / per);
        cur.u = (int)(in - (long long)cur.vh * per) - kCost;
        cur.left = to - from;
        if (cur.u < 0) {
            cur.left += cur.u;
            cur.u = 0;
        }
    }

    // Copies: lane 0 issues the warp's tiles; the page ids of the next tile are loaded one issue ahead.
    const int boxes = max(1, kKeys >> a.page_shift), box_rows = kKeys / boxes;
    const int page_mask = (1 << a.page_shift) - 1;
    Walk ahead = cur;
    int ids[kKeys / 16];
    auto fetch_ids = [&]() {
        if (ahead.left <= 0) return;
        const int key = ahead.u * kKeys;
        const int* t = a.io.block_table + ahead.x.table + (key >> a.page_shift);
#pragma unroll
        for (int i = 0; i < kKeys / 16; ++i)
            if (i < boxes) ids[i] = key + i * box_rows < ahead.x.len ? t[i] : ids[0];
    };
    int issued = 0;
    auto issue = [&]() {
        if (ahead.left <= 0) return;
        const int s = issued % kStages;
        if (lane == 0 && !(a.io.drop && warp == 0 && issued == 0)) {
            uint8_t* st = ring + s * kStageBytes;
            const int row = ahead.u * kKeys & page_mask, h = ahead.vh / ahead.x.tiles;
            ptx::mbar_arrive_expect_tx(&full[s], kStageBytes);
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
                if (i < boxes) {
                    const bool in = ids[i] >= 0 && ids[i] < a.num_pages;
                    if (!in) atomicOr(err, kErrAttnIndex);
                    // A page outside the cache: a box outside the tensor, which reads as zeros.
                    const int ph = (in ? ids[i] : a.num_pages) * a.Hkv + (in ? h : 0);
                    const uint32_t off = i * (kRowTileBytes / boxes);
                    ptx::tma_load_4d(st + off, &kmap, 0, row, 0, ph, &full[s]);
                    ptx::tma_load_4d(st + kRowTileBytes + off, &vmap, 0, row, 0, ph, &full[s]);
                }
        }
        __syncwarp();
        ++issued;
        step(ahead);
        fetch_ids();
    };
    fetch_ids();
    for (int s = 0; s < kStages; ++s) issue();

    // Row r of a row tile: query head R % G of token R / G, R = 16 * tile + r.
    uint32_t raw[2][16];
    auto load_rows = [&](const Walk& k) {
        const int h = k.vh / k.x.tiles, row0 = k.vh % k.x.tiles * kRows, rows = k.x.n * a.G;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int R = row0 + half * 8 + g, token = k.x.n > 1 ? R / a.G : 0;
            Tile::load(a.io.q + (((size_t)k.x.q + token) * a.Hq + h * a.G + R - token * a.G) * kHeadDim, R < rows, raw[half]);
        }
    };
    int used = 0;
    bool ok = true, first = true;
    if (cur.left > 0) load_rows(cur);
    while (cur.left > 0) {
        const int h = cur.vh / cur.x.tiles, row0 = cur.vh % cur.x.tiles * kRows, rows = cur.x.n * a.G;
        const int u0 = cur.u, u1 = (int)min((long long)cur.units, u0 + cur.left);
        Tile t;
        t.begin(raw, a.scale, kE4m3 ? a.k_scale[h] : 1.f);
        for (int u = u0; u < u1; ++u) {
            const int s = used % kStages;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_timed(&full[s], (uint32_t)(used / kStages) & 1u, &sm.dead));
            if (!ok) break;
            ++used;
            t.add(ring + s * kStageBytes, cur.x.len - u * kKeys);
            __syncwarp();   // every lane has read the stage: it may be filled again
            issue();
        }
        if (!ok) {
            sm.dead = 1;
            atomicOr(err, ptx::kErrAttnWait);
            break;
        }
        Walk next = cur;
        next.left -= u1 - u0 - 1;
        next.u = u1 - 1;
        step(next);
        if (next.left > 0) load_rows(next);
        t.finish();
        // Alone with the rows: their results.  Else a part of them.
        const bool whole = u0 == 0 && u1 == cur.units;
        const int slot = 2 * w + (first ? 0 : 1);
        float* part = a.slots + (size_t)slot * kSlotFloats;
        if (lane == 0) {
            int2* note = parts_of(a, cur.i) + cur.vh;
            if (u0 == 0) note->x = whole ? -1 : slot;
            if (u1 == cur.units) note->y = slot;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = half * 8 + g, R = row0 + r, token = cur.x.n > 1 ? R / a.G : 0;
            if (R >= rows) continue;
            const float l = t.sum[half];
            if (whole) {
                const size_t at = ((size_t)cur.x.out + token) * a.Hq + h * a.G + R - token * a.G;
                t.store(half, l != 0.f ? (kE4m3 ? a.v_scale[h] : 1.f) / l : 0.f, a.o + at * kHeadDim);
                if ((lane & 3) == 0) a.lse[at] = l != 0.f ? (t.ref[half] + log2f(l)) / kLog2e : -INFINITY;
            } else {
                t.store(half, 1.f, part + r * kHeadDim);
                if ((lane & 3) == 0) *reinterpret_cast<float2*>(part + kRows * kHeadDim + 2 * r) = make_float2(t.ref[half], l);
            }
        }
        cur = next;
        first = false;
    }
    // Gave up: the copies that this warp issued complete (bounded waits) before its shared memory is released.
    if (!ok)
        for (int i = used; i < issued; ++i) ptx::mbar_wait_timed(&full[i % kStages], (uint32_t)(i / kStages) & 1u);
}

// Rows of the join that get a CTA each, whose warps share the parts (64 samples, 2,048 rows of 20 parts: eight
// warps 37.9 us of the call, four and two 35.9; 8,192 rows and 16,384 of few parts, a warp each 122 and 131, four
// 126 and 144).
constexpr int kWideRows = 4096;
constexpr int kSplit = 4;

// kWide: a CTA per row, its warps taking parts in turn; else a warp per row.  Four
// channels per lane.
template <bool kWide>
__global__ void __launch_bounds__(256) kda_attn_shared_join_kernel(const __grid_constant__ Args a, const AttnIO out) {
    __shared__ float4 s_acc[kSplit][32];
    __shared__ float s_ref[kSplit], s_sum[kSplit];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = a.io.groups;
    const uint32_t rows = (uint32_t)a.io.B * a.Hq, row = kWide ? blockIdx.x : blockIdx.x * 8 + warp;
    if (row >= rows) return;
    const int b = (int)(row / (uint32_t)a.Hq), hq = (int)(row - (uint32_t)b * a.Hq), h = hq / a.G, head = hq - h * a.G;
    float ref = kNoRef, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float r, float l, const float4& v, float f) {
        if (l == 0.f) return;   // sees no key there (NaN is not 0: it goes in)
        const float to = fmaxf(ref, r), e = mma::exp2_approx(ref - to), d = mma::exp2_approx(r - to);
        ref = to;
        sum = sum * e + l * d;
        const float df = d * f;
        acc.x = acc.x * e + v.x * df;
        acc.y = acc.y * e + v.y * df;
        acc.z = acc.z * e + v.z * df;
        acc.w = acc.w * e + v.w * df;
    };
    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
    int nth = 0;   // parts so far: kWide, part p is warp p % kSplit's
    // Parts from the noted slots, two slots to a worker: the first part's, then the first slot of each worker
    // behind it up to the last one's.
    // A worker whose wait ran out left no note: what stands there instead is followed nowhere.
    auto add_parts = [&](int2 note, const float* slots, int workers, size_t slot_floats, size_t refs, int r, uint32_t at) {
        if (note.x < 0) {   // finished: its lse, and a sum of 1
            if (!kWide || (nth++ & (kSplit - 1)) == warp) {
                const float l = a.lse[at];
                add(l * kLog2e, l == -INFINITY ? 0.f : l == l ? 1.f : l, *reinterpret_cast<const float4*>(a.o + (size_t)at * kHeadDim + 4 * lane), 1.f);
            }
            return;
        }
        if ((unsigned)note.y >= 2u * workers) return;
        const int parts = (note.y >> 1) - (note.x >> 1) + 1;
#pragma unroll 4
        for (int p = kWide ? (warp - nth) & (kSplit - 1) : 0; p < parts; p += kWide ? kSplit : 1) {
            const float* s = slots + (size_t)(p ? (note.x & ~1) + 2 * p : note.x) * slot_floats;
            const float2 rl = *reinterpret_cast<const float2*>(s + refs + 2 * r);
            add(rl.x, rl.y, *reinterpret_cast<const float4*>(s + (size_t)r * kHeadDim + 4 * lane), vs);
        }
        nth += parts;
    };
    // Where the results are; a load that depends on another is under way before the parts are read.
    const int g = a.group_of[b], own = a.items[groups + b].len;
    const int2 own_note = parts_of(a, groups + b)[h * ((a.G + kRows - 1) / kRows) + head / kRows];   // (of no keys: not used)
    const bool many = g >= 0 && a.items[g].len == 0;
    int row_in = 0;
    int2 note = make_int2(0, 0);
    if (g >= 0) {
        const int i = b - a.io.cu_groups[g], tiles = a.items[g].tiles, before = a.many_pairs[g];
        if (!many) {
            const int R = i * a.G + head;
            note = parts_of(a, g)[h * tiles + R / kRows];
            row_in = R % kRows;
        } else {   // the tensor core kernel's: token tiles in pairs
            const int pair = i / (2 * a.tokens), in = i - pair * 2 * a.tokens, side = in >= a.tokens;
            note = a.many_parts[(size_t)(before + pair) * a.Hkv + h];
            row_in = side * 128 + (in - side * a.tokens) * a.G + head;
        }
    }
    if (own) add_parts(own_note, a.slots, a.warps, kSlotFloats, kRows * kHeadDim, head % kRows, rows + row);
    if (g >= 0)
        add_parts(note, many ? a.many_slots : a.slots, many ? a.many_ctas : a.warps, many ? 2 * 128 * (kHeadDim + 2) : kSlotFloats, (many ? 2 * 128 : kRows) * kHeadDim, row_in, row);
    if (kWide) {
        s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_ref[warp] = ref;
            s_sum[warp] = sum;
        }
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int w = 1; w < kSplit; ++w) add(s_ref[w], s_sum[w], s_acc[w][lane], 1.f);
    }
    const float n = sum != 0.f ? 1.f / sum : 0.f;
    mma::store4(out, (size_t)row * kHeadDim + 4 * lane, make_float4(acc.x * n, acc.y * n, acc.z * n, acc.w * n), sum != 0.f);
    if (out.lse && lane == 0) out.lse[row] = sum != 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
}

std::atomic<bool> g_attr_done[64];

}  // namespace

size_t attn_shared_workspace_bytes(const AttnLayer& l, int B, const DeviceInfo& dev) {
    Args a{};
    AttnIO many{};
    return carve(a, many, nullptr, l, B, dev);
}

cudaError_t launch_attn_shared(const AttnLayer& l, const AttnMaps& maps, const AttnSharedIO& io, const DeviceInfo& dev,
                               int* err_word, cudaStream_t stream) {
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    cudaError_t e;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kda_attn_shared_few_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kda_attn_shared_few_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    Args a{};
    AttnIO many{};
    carve(a, many, io.workspace, l, io.B, dev);
    // A block table too narrow for so many bytes of keys and values, were all of its pages full and nothing
    // shared: kda_attn_decode's kernels, whose two launches take less than four do (four requests of 600
    // tokens, 32 / 8 heads, 9.7 MB at most: 9.6 us and 13.5; 24 MB are 3.5 us of the copy rate).
    constexpr long long kSmall = 24LL << 20;
    if (!io.groups || ((long long)io.B * l.Hkv * io.max_pages << l.page_shift) * kHeadDim * (l.e4m3 ? 2 : 4) <= kSmall) {
        AttnIO d{};
        d.B = d.N = io.B;
        d.q = io.q;
        d.block_table = io.block_table;
        d.max_pages = io.max_pages;
        d.kv_lens = io.kv_lens;
        d.gate = io.gate;
        d.o = io.o;
        d.o_f32 = io.o_f32;
        d.lse = io.lse;
        d.workspace = a.decode;
        d.drop = io.drop;
        d.check_groups = io.groups;
        d.check_cu = io.cu_groups;
        return launch_attn_few_rows(l, maps, d, dev, err_word, stream, io.groups > 0);
    }
    a.io = io;
    a.Hq = l.Hq;
    a.Hkv = l.Hkv;
    a.G = l.G;
    // Groups of more rows than this go to the tensor core kernel.  17 to 32 rows are two row tiles in the few-row
    // kernel, which reads the keys for each: in e4m3, where the tensor core kernel converts them, still the
    // faster way (32 prompts of 4000 tokens with 8 requests, 4 heads on one: 105 us and 123; 16 of 8000 with two, 16
    // on one: 62 and 69), in bf16 not (132 and 143, the other way round; 74 and 103).  A call that can have none
    // of more than 32 leaves that kernel out, whose launch and set-up are as long as a short
    // prefix takes (8 requests behind 2000 tokens in bf16 17 us and 23, behind 8192 23 and 27, behind 60000 91 and 60).
    const bool has_many = io.groups && (long long)io.B * l.G > 2 * kRows;
    a.few_rows = has_many && !l.e4m3 ? kRows : 2 * kRows;
    a.tile_shift = l.e4m3 ? 5 : 4;
    a.page_shift = l.page_shift;
    a.num_pages = l.num_pages;
    a.tokens = 128 / l.G;
    a.many_cost = attn_many_rows_cost(l);
    a.scale = l.softmax_scale * kLog2e;
    a.k_scale = l.k_scale;
    a.v_scale = l.v_scale;
    const int grid = dev.sm_count * kCtasPerSm;
    a.warps = grid * kWarps;
    a.many_ctas = dev.sm_count;
    // A thread for each request and group, a warp for each group: no more meet than have something to do.
    int threads = 128;
    while (threads < kPlanThreads && (threads < io.B + io.groups || threads < 32LL * io.groups)) threads *= 2;
    if ((e = launch_behind(kda_attn_shared_plan_kernel, dim3(1), threads, 0, stream, a, err_word)) != cudaSuccess) return e;
    e = launch_behind(l.e4m3 ? kda_attn_shared_few_kernel<true> : kda_attn_shared_few_kernel<false>, dim3((unsigned)grid), kThreads, sizeof(Smem),
                      stream, a, maps.k_decode, maps.v_decode, err_word);
    if (e != cudaSuccess) return e;
    if (has_many) {
        many.B = io.groups;
        many.N = io.B;
        many.cu_new = io.cu_groups;
        many.q = io.q;
        many.block_table = io.block_table;
        many.max_pages = io.max_pages;
        many.o = a.o;
        many.o_f32 = 1;
        many.lse = a.lse;
        many.drop = io.drop;
        many.group_len = a.group_len;
        many.group_row = a.group_row;
        many.group_start = a.many_start;
        many.group_pairs = a.many_pairs;
        many.parts = a.many_parts;
        if ((e = launch_attn_many_rows_shared(l, maps, many, dev, err_word, stream)) != cudaSuccess) return e;
    }
    AttnIO out{};
    out.o = io.o;
    out.o_f32 = io.o_f32;
    out.lse = io.lse;
    out.gate = io.gate;
    const long long rows = (long long)io.B * l.Hq;
    const bool wide = rows <= kWideRows;
    return launch_behind(wide ? kda_attn_shared_join_kernel<true> : kda_attn_shared_join_kernel<false>, dim3((unsigned)(wide ? rows : (rows + 7) / 8)),
                         wide ? 32 * kSplit : 256, 0, stream, a, out);
}

}  // namespace kda
