// Causal attention of prompt chunks over a paged cache, on tcgen05 tensor cores.
//
//   S = scale * Q K^T,  P = exp(S - ref),  O = P V / sum(P),   keys in tiles of 128
//
// A prompt token's head takes part in 4 * 128 operations per key: the call is
// bound by the tensor pipe and, on a par with it, by the exponentials (a 128 x
// 128 tile of each takes the SM 512 cycles).
//
// The rows of one key head are (token, query head) pairs: floor(128 / G) tokens
// with their G heads fill one 128-row tile, so that all heads that share a key
// head share the keys' copies, and short chunks fill a tile as well.  One CTA
// works on a segment of two such tiles (consecutive tokens), X = 0 and 1, at a
// time:
//
//  * one warp copies K and V pages with TMA (128-byte swizzle, a box per page
//    and 64-channel block) into two slots each;
//  * one thread issues the MMAs: S_X(j) = Q_X K_j^T into TMEM, and
//    O_X += P_X(j) V_j with P_X read from TMEM.  While the softmax of one
//    tile runs, the MMAs of the other one do;
//  * four warps per tile do the softmax, one thread per row: the row's 128
//    logits from TMEM, its maximum against a running reference, the
//    exponentials, and their bf16 roundings back into TMEM over S_X.  A row
//    rescales (its O in TMEM as well) only when a logit passes the reference
//    by more than kLimit powers of two, which after the first tile is rare.
//  * e4m3: four further warps convert each copied tile to f16, Q is scaled
//    by a power of two per row, P is f16 within 2^15.
//
// TMEM: S_0, S_1 (128 columns each, P_X in the first 64), O_0, O_1.
//
// CTAs are persistent.  Segments are numbered with the longest of a request
// first and dealt to the CTAs back and forth, which evens out the causal
// triangle.  When there are fewer segments than CTAs and the longest is well
// above the average share, the keys are cut instead: each CTA takes an equal
// range of (segment, key tile) units and leaves partial results, joined in a
// fixed order by a dependent launch.
#include <atomic>
#include <type_traits>

#include "attn_internal.cuh"
#include "attn_mma.cuh"
#include "attn_tma.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int kRows = 128;                     // rows of a tile
constexpr int kKeys = 128;                     // keys of a tile
constexpr uint32_t kOperand = 32768;           // a 128 x 128 16-bit operand
constexpr uint32_t kBlock = 16384;             // one 64-channel block of it
constexpr uint32_t kOffQ = 0, kOffK = 2 * kOperand, kOffV = 4 * kOperand, kOffStage = 6 * kOperand;
constexpr int kScan = 256;                     // threads of the prefix sums
constexpr int kMaxCtas = 256;
constexpr int kSplitGain = 6;                  // key tiles that splitting has to save on the longest segment

constexpr uint32_t kColS = 0, kColO = 256;     // TMEM columns, + 128 X

struct Ctl {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], vraw;
    uint64_t qfull[2], sfull[2], pfull[2][2], ofull[2];   // pfull: by tile and half of its keys
    uint64_t ckfull, ckempty, cvfull, cvempty;   // e4m3 staging
    uint64_t drain;
    uint32_t tmem;
    int dead;
    int longest;
    int kissued, vissued;
    int warp_sum[8];
    int pre[kScan];          // tiles of tokens before the requests of scan thread t
    int seg_pre[kMaxCtas];   // split: units before segment s
};

template <bool kE4m3>
constexpr uint32_t smem_bytes() { return kOffStage + (kE4m3 ? 2 * kBlock : 0) + (uint32_t)sizeof(Ctl); }
static_assert(kOffStage + 2 * kBlock + sizeof(Ctl) <= 232448, "shared memory");

struct PrefillArgs {
    AttnIO io;
    int Hq, Hkv, G;
    int tokens;              // of a tile: 128 / G
    int page_shift, num_pages;
    float scale;             // softmax scale * log2(e)
    const float* k_scale;
    const float* v_scale;
};

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
    int j0, n, cnt[2];
    bool whole, first;       // the whole segment; the segment's first key tile is in it
    int slot;                // of the partial result, if not whole
};

struct Sched {
    int total;               // token tiles (pairs) of all requests
    int per;                 // requests of a scan thread
    long long segments;
    bool split;
    int units, ctas;         // split: key tiles of all segments, CTAs that share them
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
    if (n == 0 || attn_few_rows(n, a.G) || attn_kv_len(a.io, b, a.page_shift) == 0) return 0;
    return (n + 2 * a.tokens - 1) / (2 * a.tokens);
}

__device__ __forceinline__ Segment find_segment(const PrefillArgs& a, const Ctl& ctl, const Sched& sc, long long s) {
    const int pair = (int)(s / a.Hkv);
    int lo = 0, hi = kScan - 1;   // the last scan thread with pre <= pair
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl.pre[mid] <= pair) lo = mid; else hi = mid - 1;
    }
    int at = ctl.pre[lo], b = lo * sc.per, n;
    while (at + (n = pairs_of(a, b)) <= pair) {
        at += n;
        ++b;
    }
    Segment g;
    g.b = b;
    g.h = (int)(s % a.Hkv);
    int tok0, tokens;
    attn_tokens(a.io, b, tok0, tokens);
    const int i0 = (n - 1 - (pair - at)) * 2 * a.tokens;   // the longest first
    g.len = attn_kv_len(a.io, b, a.page_shift);
    g.tok = tok0 + i0;
    g.m = min(2 * a.tokens, tokens - i0);
    g.first = g.len - tokens + i0 + 1;
    return g;
}

// The k-th part of this CTA; false past the last.
__device__ __forceinline__ bool next_part(const PrefillArgs& a, const Ctl& ctl, const Sched& sc, int& k, Part& p) {
    if (!sc.split) {
        for (;; ++k) {
            const long long base = (long long)k * gridDim.x;
            if (base >= sc.segments) return false;
            const long long s = base + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (s >= sc.segments) continue;
            p.s = find_segment(a, ctl, sc, s);
            break;
        }
        ++k;
        p.j0 = 0;
        p.n = p.s.tiles_all(a.tokens);
        p.cnt[0] = p.s.tiles(0, a.tokens);
        p.cnt[1] = p.s.tiles(1, a.tokens);
        p.whole = p.first = true;
        return true;
    }
    if ((int)blockIdx.x >= sc.ctas) return false;
    const int from = (int)((long long)sc.units * blockIdx.x / sc.ctas), to = (int)((long long)sc.units * (blockIdx.x + 1) / sc.ctas);
    int s = k;
    if (k == 0)
        while (s + 1 < sc.segments && ctl.seg_pre[s + 1] <= from) ++s;
    if (s >= sc.segments || ctl.seg_pre[s] >= to) return false;
    p.s = find_segment(a, ctl, sc, s);
    const int all = p.s.tiles_all(a.tokens), at = ctl.seg_pre[s];
    p.j0 = max(from - at, 0);
    p.n = min(to - at, all) - p.j0;
    for (int x = 0; x < 2; ++x) p.cnt[x] = min(max(p.s.tiles(x, a.tokens) - p.j0, 0), p.n);
    p.whole = p.n == all;
    p.first = p.j0 == 0;
    p.slot = 2 * (int)blockIdx.x + (at <= from ? 0 : 1);
    k = s + 1;
    return true;
}

__device__ __forceinline__ bool pwait(uint64_t* bar, uint32_t parity, int* dead, int* err) {
    if (ptx::mbar_wait_timed(bar, parity, dead)) return true;
    *(volatile int*)dead = 1;
    atomicOr(err, ptx::kErrAttnWait);
    return false;
}

// Inclusive prefix of v over the first kScan threads; all of them call it.
__device__ __forceinline__ int scan_inclusive(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    if (lane == 31 && warp < 8) s_warp[warp] = v;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) v += s_warp[w];
        all += s_warp[w];
    }
    *total = all;
    __syncthreads();
    return v;
}

constexpr int kWarpMma = 8, kWarpTma = 9, kWarpConvert = 12;
template <bool kE4m3>
constexpr int threads_of() { return kE4m3 ? 512 : 384; }
// Registers: the launch's share of each thread, and what the softmax
// warpgroups (0, 1) and the other ones change to; the sum stays within the
// launch's (checked against the compiled kernel before its first launch).
template <bool kE4m3>
constexpr int regs_launch() { return kE4m3 ? 128 : 168; }
template <bool kE4m3>
constexpr int regs_softmax() { return kE4m3 ? 176 : 208; }
constexpr int kRegsOther = 80;
static_assert(256 * regs_softmax<false>() + 128 * kRegsOther <= 384 * regs_launch<false>(), "registers");
static_assert(256 * regs_softmax<true>() + 256 * kRegsOther <= 512 * regs_launch<true>(), "registers");

template <bool kE4m3>
__global__ void __launch_bounds__(threads_of<kE4m3>(), 1)
kda_attn_prefill_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int* err) {
    constexpr float kOffset = kE4m3 ? 10.f : 0.f;
    constexpr float kLimit = kE4m3 ? 15.f : 8.f;
    extern __shared__ __align__(1024) uint8_t sm[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(sm + kOffStage + (kE4m3 ? 2 * kBlock : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* dead = &ctl.dead;

    ptx::griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ctl.kfull[i], kE4m3 ? 128 : 1);
            ptx::mbar_init(&ctl.vfull[i], kE4m3 ? 128 : 1);
            ptx::mbar_init(&ctl.kempty[i], 1);
            ptx::mbar_init(&ctl.vempty[i], 1);
            ptx::mbar_init(&ctl.qfull[i], kRows);
            ptx::mbar_init(&ctl.sfull[i], 1);
            ptx::mbar_init(&ctl.pfull[i][0], kRows);
            ptx::mbar_init(&ctl.pfull[i][1], kRows);
            ptx::mbar_init(&ctl.ofull[i], 1);
        }
        ptx::mbar_init(&ctl.vraw, 1);
        ptx::mbar_init(&ctl.ckfull, 1);
        ptx::mbar_init(&ctl.cvfull, 1);
        ptx::mbar_init(&ctl.ckempty, 128);
        ptx::mbar_init(&ctl.cvempty, 128);
        ptx::mbar_init(&ctl.drain, 1);
        ptx::fence_mbar_init();
        ctl.dead = 0;
        ctl.longest = 0;
        ctl.kissued = ctl.vissued = 0;
        joins(a.io.workspace)[blockIdx.x].m = 0;
    }
    if (warp == kWarpMma) tc::alloc(&ctl.tmem, 512);

    // Segments of all requests.
    Sched sc;
    sc.per = (a.io.B + kScan - 1) / kScan;
    int mine = 0;
    if (tid < kScan)
        for (int b = min(a.io.B, tid * sc.per), end = min(a.io.B, b + sc.per); b < end; ++b) mine += pairs_of(a, b);
    const int upto = scan_inclusive(mine, ctl.warp_sum, &sc.total);
    if (tid < kScan) ctl.pre[tid] = upto - mine;
    __syncthreads();
    sc.segments = (long long)sc.total * a.Hkv;
    sc.split = false;
    sc.units = sc.ctas = 0;
    if (sc.segments < gridDim.x && sc.segments > 0) {   // and so at most kScan - 1
        int n = 0;
        if (tid < sc.segments) n = find_segment(a, ctl, sc, tid).tiles_all(a.tokens);
        if (n) atomicMax(&ctl.longest, n);
        const int u = scan_inclusive(n, ctl.warp_sum, &sc.units);
        if (tid < sc.segments) ctl.seg_pre[tid] = u - n;
        sc.ctas = min((int)gridDim.x, sc.units);
        sc.split = ctl.longest > (sc.units + sc.ctas - 1) / sc.ctas + kSplitGain;
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
        int k = 0;
        const int rows = min(1 << a.page_shift, kKeys), boxes = kKeys / rows;   // rows of a box, pages of a tile
        const int is_v = lane >> 4;
        const int pg = kE4m3 ? lane & 15 : (lane & 15) >> 1, block = kE4m3 ? 0 : lane & 1;
        int it = 0, raws = 0;
        while (next_part(a, ctl, sc, k, p)) {
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
                bool ok = true;
                if (kE4m3) {
                    // Staging: one buffer each, emptied by the converting warps.
                    if (it > 0) ok = pwait(&ctl.ckempty, (uint32_t)(it - 1) & 1u, dead, err);
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(&ctl.ckfull, (uint32_t)(pages * rows * 128));
                    __syncwarp();
                    if (ok && mine_box && !is_v)
                        ptx::tma_load_4d(sm + kOffStage + pg * rows * 128, &kmap, 0, 0, 0, ph, &ctl.ckfull);
                    if (ok) ctl.kissued = it + 1;
                    if (ok && it > 0) ok = pwait(&ctl.cvempty, (uint32_t)(it - 1) & 1u, dead, err);
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(&ctl.cvfull, (uint32_t)(pages * rows * 128));
                    __syncwarp();
                    if (ok && mine_box && is_v)
                        ptx::tma_load_4d(sm + kOffStage + kBlock + pg * rows * 128, &vmap, 0, 0, 0, ph, &ctl.cvfull);
                    if (ok) ctl.vissued = it + 1;
                } else {
                    uint8_t* kd = sm + kOffK + s * kOperand + block * kBlock + pg * rows * 128;
                    uint8_t* vd = sm + kOffV + s * kOperand + block * kBlock + pg * rows * 128;
                    if (it >= 2) ok = pwait(&ctl.kempty[s], par, dead, err);
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(&ctl.kfull[s], (uint32_t)(pages * rows * 256));
                    __syncwarp();
                    if (ok && mine_box && !is_v) ptx::tma_load_4d(kd, &kmap, 0, 0, block, ph, &ctl.kfull[s]);
                    if (ok) ctl.kissued = it + 1;
                    if (ok && it >= 2) ok = pwait(&ctl.vempty[s], par, dead, err);
                    uint64_t* bar = raw ? &ctl.vraw : &ctl.vfull[s];
                    if (ok && lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(pages * rows * 256));
                    __syncwarp();
                    if (ok && mine_box && is_v) ptx::tma_load_4d(vd, &vmap, 0, 0, block, ph, bar);
                    if (ok && !raw) ctl.vissued = it + 1;
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
                        *reinterpret_cast<uint4*>(sm + kOffV + s * kOperand + (ch >> 3) * kBlock + row * 128 + (ch & 7) * 16) =
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
        // ---- MMAs.  The warp runs the loop together and one lane issues.
        // The issuing lane shares its scheduler with two softmax warps, and
        // operands that have to be moved to uniform registers first made it
        // the slowest part of the loop (110 cycles per MMA, of which the
        // pipe needs 64): the slots' code is therefore written out for both
        // parities, with every operand a constant but the shared-memory base.
        tc::reg_dec<kRegsOther>();
        Part p;
        int k = 0;
        constexpr uint32_t id_s = tc::idesc_f16kind(kRows, kKeys, !kE4m3, false);
        constexpr uint32_t id_o = tc::idesc_f16kind(kRows, kHeadDim, !kE4m3, true);
        const uint32_t base = ptx::smem_u32(sm);
        const uint64_t dq = tc::desc_sw128(base + kOffQ), dk = tc::desc_sw128(base + kOffK);
        const uint64_t dv = tc::desc_sw128_mn(base + kOffV, kBlock);
        const bool issuer = tc::elect_one();
        uint32_t qpar = 0u, ppar = 0u;   // bit x: tile x
        int it = 0;
        bool ok = true;
        auto mma_s = [&](auto tile, auto slot) {   // S_x = Q_x K^T
            constexpr int x = decltype(tile)::value, sl = decltype(slot)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                tc::mma_ss_bf16(kColS + 128 * x, tc::desc_add(dq, x * kOperand + (i >> 2) * kBlock + (i & 3) * 32),
                                tc::desc_add(dk, sl * kOperand + (i >> 2) * kBlock + (i & 3) * 32), id_s, i > 0);
        };
        auto first_s = [&](auto tile, auto slot) {
            constexpr int x = decltype(tile)::value;
            if (p.cnt[x] <= 0) return;
            ok = ok && pwait(&ctl.qfull[x], (qpar >> x) & 1u, dead, err);
            qpar ^= 1u << x;
            tc::fence_after();
            if (issuer && ok) {
                mma_s(tile, slot);
                tc::commit(&ctl.sfull[x]);
            }
        };
        // O_x += P_x(j) V_j from this slot, S_x(j + 1) from the other one.
        auto tile_step = [&](auto tile, auto slot, int j) {
            constexpr int x = decltype(tile)::value, sl = decltype(slot)::value;
            if (j >= p.cnt[x]) return;
            const uint32_t par = (ppar >> x) & 1u;
            ppar ^= 1u << x;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                ok = ok && pwait(&ctl.pfull[x][half], par, dead, err);
                tc::fence_after();
                if (issuer && ok) {
#pragma unroll
                    for (int i = 4 * half; i < 4 * half + 4; ++i)
                        tc::mma_ts_f16kind(kColO + 128 * x, kColS + 128 * x + 8 * i,
                                           tc::desc_add(dv, sl * kOperand + i * 2048), id_o, i > 0 ? 1u : (uint32_t)(j > 0));
                }
            }
            if (issuer && ok) {
                if (x == 1 || j >= p.cnt[1]) tc::commit(&ctl.vempty[sl]);
                if (j + 1 < p.cnt[x]) {
                    mma_s(tile, std::integral_constant<int, 1 - sl>());
                    tc::commit(&ctl.sfull[x]);
                } else {
                    tc::commit(&ctl.ofull[x]);
                }
            }
        };
        auto both = [&](auto slot, int j) {
            constexpr int sl = decltype(slot)::value;
            // Normally there already: waited for while the pipe works on S_1(j).
            ok = ok && pwait(&ctl.vfull[sl], (uint32_t)(it >> 1) & 1u, dead, err);
            if (j + 1 < p.n) ok = ok && pwait(&ctl.kfull[1 - sl], (uint32_t)((it + 1) >> 1) & 1u, dead, err);
            tile_step(std::integral_constant<int, 0>(), slot, j);
            tile_step(std::integral_constant<int, 1>(), slot, j);
            if (j + 1 < p.n && issuer && ok) tc::commit(&ctl.kempty[1 - sl]);
        };
        using Slot0 = std::integral_constant<int, 0>;
        using Slot1 = std::integral_constant<int, 1>;
        while (ok && next_part(a, ctl, sc, k, p)) {
            ok = pwait(&ctl.kfull[it & 1], (uint32_t)(it >> 1) & 1u, dead, err);
            if (it & 1) {
                first_s(Slot0(), Slot1());
                first_s(Slot1(), Slot1());
            } else {
                first_s(Slot0(), Slot0());
                first_s(Slot1(), Slot0());
            }
            if (issuer && ok) tc::commit(&ctl.kempty[it & 1]);
            for (int j = 0; j < p.n && ok; ++j, ++it) {
                if (it & 1) both(Slot1(), j);
                else both(Slot0(), j);
            }
        }
        if (issuer) tc::commit(&ctl.drain);   // completes once every MMA that it issued has
    } else if (kE4m3 && warp >= kWarpConvert) {
        // ---- e4m3 -> f16, one key per thread
        tc::reg_dec<kRegsOther>();
        Part p;
        int k = 0;
        const int row = tid - 32 * kWarpConvert;
        int it = 0;
        bool ok = true;
        while (ok && next_part(a, ctl, sc, k, p))
            for (int j = p.j0; j < p.j0 + p.n && ok; ++j, ++it) {
                const int s = it & 1;
                const uint32_t par = (uint32_t)((it >> 1) - 1) & 1u;
                const bool live = j * kKeys + row < p.s.len;
#pragma unroll 1
                for (int v = 0; v < 2 && ok; ++v) {
                    ok = pwait(v ? &ctl.cvfull : &ctl.ckfull, (uint32_t)it & 1u, dead, err);
                    if (ok && it >= 2) ok = pwait(v ? &ctl.vempty[s] : &ctl.kempty[s], par, dead, err);
                    if (!ok) break;
                    const uint8_t* src = sm + kOffStage + v * kBlock + row * 128;
                    uint8_t* dst = sm + (v ? kOffV : kOffK) + s * kOperand + row * 128;
#pragma unroll
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
                        uint8_t* d = dst + (c >> 2) * kBlock;
                        *reinterpret_cast<uint4*>(d + ((((2 * c) & 7) ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(d + ((((2 * c + 1) & 7) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(v ? &ctl.vfull[s] : &ctl.kfull[s]);
                    ptx::mbar_arrive(v ? &ctl.cvempty : &ctl.ckempty);
                }
            }
    } else if (warp < 8) {
        // ---- softmax, one thread per row of tile x
        tc::reg_inc<regs_softmax<kE4m3>()>();
        Part p;
        int k = 0;
        const int x = warp >> 2, r = tid & (kRows - 1);
        const int i_row = r / a.G, g_row = r % a.G;
        const uint32_t ts = tc::taddr(tm, warp, kColS + 128 * x), to = tc::taddr(tm, warp, kColO + 128 * x);
        uint32_t spar = 0u, opar = 0u;
        bool ok = true;
        while (ok && next_part(a, ctl, sc, k, p)) {
            const int tokens = p.s.tokens_of(x, a.tokens);
            const int tok = p.s.tok + x * a.tokens + i_row;
            const bool live = i_row < tokens;
            const size_t head = (size_t)tok * a.Hq + p.s.h * a.G + g_row;
            float ref = kNoRef, sum = 0.f;
            const int cnt = p.cnt[x];
            if (cnt > 0) {
                // Q row into shared memory (swizzled as TMA would).
                float fac = a.scale;
                uint32_t w[64];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (live) v = *reinterpret_cast<const uint4*>(a.io.q + head * kHeadDim + 8 * c);
                    w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
                }
                if (kE4m3) {
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[c] << 16)), fabsf(__uint_as_float(w[c] & 0xffff0000u))));
                    // q * 2^(14 - e) with 2^e <= top < 2^(e+1): exact in f16 down to 2^-28 of the row's largest.
                    const int e = top > 0.f ? max(-100, min(100, ilogbf(top))) : 0;
                    const float up = exp2f((float)(14 - e));
                    fac = a.scale * a.k_scale[p.s.h] * exp2f((float)(e - 14));
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        w[c] = mma::pack_f16(__uint_as_float(w[c] << 16) * up, __uint_as_float(w[c] & 0xffff0000u) * up);
                }
                uint8_t* qd = sm + kOffQ + x * kOperand + r * 128;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    *reinterpret_cast<uint4*>(qd + (c >> 3) * kBlock + (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                ptx::fence_proxy_async_smem();
                tc::fence_before();
                ptx::mbar_arrive(&ctl.qfull[x]);

                // Keys that the row sees; rows without a token see all (their q is zero, nothing is stored).
                const int sees = live ? p.s.first + x * a.tokens + i_row : 0x7fffffff;
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
                ok = pwait(&ctl.ofull[x], opar, dead, err);
                opar ^= 1u;
                tc::fence_after();
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            }
            // The row's result, or its part of one.
            float* part = p.whole ? nullptr : slot_at(a.io.workspace, gridDim.x, p.slot) + (size_t)(x * kRows + r) * kHeadDim;
            if (cnt > 0) {
                const float n = !p.whole ? 1.f : sum > 0.f ? (kE4m3 ? a.v_scale[p.s.h] : 1.f) / sum : 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tc::ld32(to + 32 * c, o);
                    tc::wait_ld();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v = make_float4(__uint_as_float(o[e]) * n, __uint_as_float(o[e + 1]) * n,
                                                         __uint_as_float(o[e + 2]) * n, __uint_as_float(o[e + 3]) * n);
                            if (p.whole) mma::store4(a.io, head * kHeadDim + 32 * c + e, v);
                            else *reinterpret_cast<float4*>(part + 32 * c + e) = v;
                        }
                    }
                    __syncwarp();   // the warp reads TMEM together
                }
                tc::fence_before();
            }
            if (live && p.whole && a.io.lse) a.io.lse[head] = sum > 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
            if (live && !p.whole) {
                float* ls = slot_at(a.io.workspace, gridDim.x, p.slot) + (size_t)2 * kRows * kHeadDim + 2 * (x * kRows + r);
                ls[0] = ref;
                ls[1] = sum;
            }
            if (tid == 0 && !p.whole && p.first) {
                // The first part of a segment that goes on: up to the CTA that holds its last unit.
                const int s = k - 1;
                const long long last = ctl.seg_pre[s] + p.s.tiles_all(a.tokens) - 1;
                joins(a.io.workspace)[blockIdx.x] =
                    PrefillJoin{p.s.tok, p.s.m, p.s.h, (int)(((last + 1) * sc.ctas - 1) / sc.units), p.slot, {0, 0, 0}};
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
            if (kE4m3) {
                if (ctl.kissued) ptx::mbar_wait_timed(&ctl.ckfull, (uint32_t)(ctl.kissued - 1) & 1u);
                if (ctl.vissued) ptx::mbar_wait_timed(&ctl.cvfull, (uint32_t)(ctl.vissued - 1) & 1u);
            } else {
                for (int i = max(0, ctl.kissued - 2); i < ctl.kissued; ++i)
                    ptx::mbar_wait_timed(&ctl.kfull[i & 1], (uint32_t)(i >> 1) & 1u);
                for (int i = max(0, ctl.vissued - 2); i < ctl.vissued; ++i)
                    ptx::mbar_wait_timed(&ctl.vfull[i & 1], (uint32_t)(i >> 1) & 1u);
            }
        }
    }
    __syncthreads();
    if (warp == kWarpMma) tc::dealloc(tm, 512);
    ptx::griddep_wait();   // ends after the few-row kernels launched before it
}

// Joins the parts of segments cut between CTAs: blockIdx.x the CTA that holds
// the first part, a warp per row, four channels per lane.
__global__ void __launch_bounds__(256) kda_attn_prefill_join_kernel(const PrefillArgs a, int ctas) {
    ptx::griddep_wait();
    const PrefillJoin d = joins(a.io.workspace)[blockIdx.x];
    if (d.m == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = d.last - (int)blockIdx.x + 1;
    const int rows = d.m * a.G;
    for (int row = blockIdx.y * 8 + warp; row < rows; row += gridDim.y * 8) {
        const int i = row / a.G, g = row % a.G;
        const int at = i < a.tokens ? row : kRows + row - a.tokens * a.G;   // row of the pair of tiles
        float ref = kNoRef, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = 0; q < parts; ++q) {
            const float* s = slot_at(a.io.workspace, ctas, q == 0 ? d.slot : 2 * ((int)blockIdx.x + q));
            const float2 ls = *reinterpret_cast<const float2*>(s + (size_t)2 * kRows * kHeadDim + 2 * at);
            const float4 v = *reinterpret_cast<const float4*>(s + (size_t)at * kHeadDim + 4 * lane);
            if (!(ls.y > 0.f)) continue;   // no key of this part is seen: the weighted sum was not written
            const float to = fmaxf(ref, ls.x);
            const float f = mma::exp2_approx(ref - to), e = mma::exp2_approx(ls.x - to);
            ref = to;
            sum = sum * f + ls.y * e;
            acc.x = acc.x * f + v.x * e;
            acc.y = acc.y * f + v.y * e;
            acc.z = acc.z * f + v.z * e;
            acc.w = acc.w * f + v.w * e;
        }
        const float n = sum > 0.f ? (a.v_scale ? a.v_scale[d.h] : 1.f) / sum : 0.f;
        const size_t head = ((size_t)d.tok + i) * a.Hq + d.h * a.G + g;
        mma::store4(a.io, head * kHeadDim + 4 * lane, make_float4(acc.x * n, acc.y * n, acc.z * n, acc.w * n));
        if (a.io.lse && lane == 0) a.io.lse[head] = sum > 0.f ? (ref + log2f(sum)) / kLog2e : -INFINITY;
    }
}

std::atomic<bool> g_attr_done[64];

template <bool kE4m3>
cudaError_t prepare_kernel() {
    cudaFuncAttributes f{};
    cudaError_t e = cudaFuncGetAttributes(&f, kda_attn_prefill_kernel<kE4m3>);
    if (e != cudaSuccess) return e;
    if (f.numRegs < regs_launch<kE4m3>()) return cudaErrorLaunchOutOfResources;   // the splits would never be met
    return cudaFuncSetAttribute(kda_attn_prefill_kernel<kE4m3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<kE4m3>());
}

}  // namespace

bool attn_prefill_maps(const AttnLayer& l, AttnMaps& maps) {
    const int rows = l.page_size < kKeys ? l.page_size : kKeys;
    return make_cache_map(&maps.k_prefill, l, l.k_cache, rows, 1) && make_cache_map(&maps.v_prefill, l, l.v_cache, rows, 1);
}

size_t attn_prefill_workspace_bytes(const DeviceInfo& dev) {
    return join_bytes(dev.sm_count) + (size_t)dev.sm_count * 2 * kSlotFloats * sizeof(float);
}

cudaError_t launch_attn_many_rows(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev,
                                  int* err_word, cudaStream_t stream) {
    if (dev.device < 0 || dev.device >= 64 || dev.sm_count > kMaxCtas) return cudaErrorInvalidDevice;
    if (!g_attr_done[dev.device].load(std::memory_order_acquire)) {
        cudaError_t e = prepare_kernel<false>();
        if (e == cudaSuccess) e = prepare_kernel<true>();
        if (e != cudaSuccess) return e;
        g_attr_done[dev.device].store(true, std::memory_order_release);
    }
    PrefillArgs a{};
    a.io = io;
    a.Hq = l.Hq;
    a.Hkv = l.Hkv;
    a.G = l.G;
    a.tokens = kRows / l.G;
    a.page_shift = l.page_shift;
    a.num_pages = l.num_pages;
    a.scale = l.softmax_scale * kLog2e;
    a.k_scale = l.k_scale;
    a.v_scale = l.v_scale;
    // Both launches are programmatic: the first may start beside the few-row
    // kernels launched before it (it shares nothing with them but their
    // inputs, and waits for them before it ends), the join waits for the first.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int grid = dev.sm_count;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(l.e4m3 ? threads_of<true>() : threads_of<false>());
    cfg.dynamicSmemBytes = l.e4m3 ? smem_bytes<true>() : smem_bytes<false>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, l.e4m3 ? kda_attn_prefill_kernel<true> : kda_attn_prefill_kernel<false>,
                                       a, maps.k_prefill, maps.v_prefill, err_word);
    count_launches(1);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)grid, 16);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, kda_attn_prefill_join_kernel, a, grid);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
