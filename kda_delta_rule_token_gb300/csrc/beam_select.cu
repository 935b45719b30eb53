// The num best continuations of every group of beams.
//
//   score(k, v) = s_k + x_kv - lse_k,   lse_k = ln sum_v exp(x_kv)
//
// A row's scores have the order of its logits, so one pass over the logits
// finds both what a row can offer (its num largest logits) and what they are
// measured against (lse).  Every logit is read once; what is left is small:
// the call is bound by HBM, or by its two launches.
//
//  * kda_beam_rows_kernel: the tiles of all rows, 256 threads x 16 logits each, are
//    dealt in equal ranges to as many CTAs as run at once; what a CTA has of a row
//    is a segment.  The next tile's loads are under way.  A thread keeps the
//    largest of its logits and the sum of exp(x - ref), nothing else.  Every eight
//    tiles the CTA finds a bound that num of them reach and few others pass: 64 groups
//    of threads each have a largest logit, and the num-th of these is it.
//    The few threads whose largest logit reaches the bound are looked at again,
//    each by half a warp: logits that reach it join the list of candidates, the others
//    the sums anew.  Later logits have to pass the bound (T); the list's num best
//    stay at the end.
//  * kda_beam_join_kernel, a CTA per group: lse of every beam from its segments'
//    sums and lists, then the num best of the lists, by the same bound.
//
// Which of two beams' close candidates is the better one hangs on the last bits
// of their lse.  The largest terms decide these, and they are the candidates:
// they stay out of the fp32 sums (which carry what their additions lose along),
// and the join adds their exponentials to 2^-31 as whole numbers, in 64 bits, so
// in any order.  Scores are formed and compared in 64 bits and rounded once.
//
// Measured (both launches, inputs in HBM but for what L2 kept of them): 512 rows of
// 131072 logits in fp32, 268 MB, 53 us, of which the rows take 47 (5.7 TB/s, 0.84
// of the copy rate): looks at the largest logits, 3000 cycles each, which other CTAs of the SM
// cover in part.  128 rows of 131071 in bf16, 33 MB, 21 us: a look to a CTA's 8 tiles and the join.  Four rows of
// 32000, 7.5 us: two launches, and in the join a chain of loads, 64-bit arithmetic and instructions
// that no CTA before has fetched.  What runs once per segment or CTA is short for the same reason (the list
// ranked by loops written out 2 us more, the join with 16 candidates to a thread 1 us).  A look every four tiles 57 us; before that, the bound found bit
// by bit 65 instead of 62, threads looked at again by their own warps 59.7 instead of 57.6, by quarters of
// warps 60.7.  Tried earlier: copies of four tiles ahead by cp.async 62 us and 65, but 12.4 and 10 for
// the four rows; candidates taken out of every tile at once 69 to 73; two tiles'
// loads ahead in registers with three CTAs per SM 71.
#include <math.h>

#include "attn_mma.cuh"
#include "beam_internal.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;               // logits of a thread per tile
constexpr int kTile = kThreads * kPer;
constexpr int kSub = 8;                // tiles between two looks at the largest logits
static_assert(64 % kPer == 0 && kPer % 4 == 0, "four logits of a thread for each lane of half a warp");
constexpr int kList = 768;             // candidates that a CTA holds
constexpr int kThin = 256;             // more than these are brought down to num
static_assert(kThin + KDA_BEAM_MAX_NUM <= kList, "room for num candidates");
constexpr int kMostNum = KDA_BEAM_MAX_NUM;
constexpr int kJoinThreads = 1024;     // of the join, at most
constexpr int kJoinPer = 4;            // candidates of a group's segments that a thread of the join takes
constexpr int kJoinEntries = kJoinPer * kJoinThreads;
constexpr int kJoinList = 1280;
static_assert((kJoinPer + 1) * kMostNum <= kJoinList, "candidates that the join's bound leaves");
static_assert(KDA_BEAM_MAX_BEAMS * kMostNum <= kJoinEntries && KDA_BEAM_MAX_BEAMS <= kThreads, "a segment per beam");
constexpr float kRefMargin = 16.f;     // how far the largest logit may be from the reference of the sums

// What a segment leaves beside its candidates: the sum of exp(x - ref) over its other logits.
struct Part {
    float sum, more;   // and what the sum's additions lost
    float ref;         // -infinity: the sum is 0, or NaN
    float pad;
};

// A candidate: the logit in the order of unsigned numbers above, the complement of
// its token below, so that the larger of two is the better one.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 is 0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t order) {
    return __uint_as_float(order ^ ((order >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t candidate(float x, int token) {
    return (uint64_t)order_of(x) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float logit_of(uint64_t c) { return float_of((uint32_t)(c >> 32)); }
__device__ __forceinline__ int token_of(uint64_t c) { return (int)~(uint32_t)c; }

// exp(d): the exponent is off by 2^-24 and 2^-26 of itself, the product's rounding and log2 e's.
__device__ __forceinline__ float exp_of(float d) {
    return mma::exp2_approx(d * 1.44269502f);
}

__device__ __forceinline__ mma::f32x2 exp_of(mma::f32x2 d) {
    float a, b;
    mma::upk(mma::mul2(d, mma::pk(1.44269502f, 1.44269502f)), a, b);
    return mma::pk(mma::exp2_approx(a), mma::exp2_approx(b));
}

// 2^f, f in units of 2^-32, in units of 2^-31: the exponential's series in ln 2, whose
// eleventh term is below 2^-31, each product cut at 2^-32.
__device__ __forceinline__ uint32_t pow2_fixed(uint32_t f) {
    constexpr double c[11] = {0.69314718055994531, 0.24022650695910072, 0.055504108664821580, 0.0096181291076284772,
                              0.0013333558146428443, 1.5403530393381610e-4, 1.5252733804059841e-5, 1.3215486790144309e-6,
                              1.0178086009239700e-7, 7.0549116208011233e-9, 4.4455382718708116e-10};
    uint32_t p = 0;
#pragma unroll
    for (int k = 10; k >= 0; --k) p = (uint32_t)(c[k] * 4294967296.0) + __umulhi(p, f);
    return 0x80000000u + (__umulhi(p, f) >> 1);
}

// exp(x - top), x <= top, as m * 2^(i - 31); i < -40 stands for nothing.
struct Power {
    uint32_t m;
    int i;
};
__device__ __forceinline__ Power power_of(float x, float top) {
    // x - top exactly, and its product with log2 e to 2^-45 of it.
    constexpr float l1 = 1.44269502f, l2 = 1.92596299e-8f;
    const float d = x - top, back = d - x;
    const float low = (x - (d - back)) - (top + back);
    if (!(d > -40.f)) return Power{0, -64};
    const float t = d * l1;
    const float u = fmaf(d, l1, -t) + fmaf(d, l2, low * l1);
    const int i = __float2int_rd(t);
    const long long fixed = ((long long)i << 32) + __float2uint_rn((t - (float)i) * 4294967296.f) + __float2int_rn(u * 4294967296.f);
    return Power{pow2_fixed((uint32_t)fixed), (int)(fixed >> 32)};
}

// v * exp(x - top) in units of 2^-31, v finite.
__device__ __forceinline__ long long scaled(float v, const Power& p) {
    const uint32_t u = __float_as_uint(v);
    const int e = (int)(u >> 23 & 0xff);
    if (e == 0 || p.m == 0) return 0;
    const unsigned long long x = (unsigned long long)((u & 0x7fffff) | 0x800000) * p.m;   // below 2^56
    const int shift = e - 127 - 23 + p.i;
    const long long y = shift >= 0 ? (long long)(x << min(shift, 7)) : shift > -64 ? (long long)(x >> -shift) : 0;
    return u >> 31 ? -y : y;
}

// ln of x units of 2^-31, x > 0: log2 of the leading 32 bits in fp32, put right by what
// two to its power is off by, in units of 2^-40, times ln 2.
__device__ __forceinline__ double ln_fixed(unsigned long long x) {
    const int lead = __clzll((long long)x);
    const uint32_t m = (uint32_t)((x << lead) >> 32);
    const float y = fminf(fmaxf(log2f((float)m * 0x1p-31f), 0.f), 0x1.fffffep-1f);
    const uint32_t f = (uint32_t)(y * 4294967296.f), p = pow2_fixed(f);
    const float off = __fdividef((float)(int)(m - p), (float)p) * 1.44269504f;
    const long long log2 = ((long long)(63 - lead - 31) << 40) + ((long long)f << 8) + __float2int_rn(off * 0x1p40f);
    constexpr long long ln2 = 0x58b90bfbe8e7bcd6;   // units of 2^-63
    return (double)__mul64hi(log2 << 14, ln2) * 0x1p-53;
}

// Floating numbers in 64 bits without the unit of 64-bit arithmetic: x exactly (below 2^-126: 0).
__device__ __forceinline__ double widened(float x) {
    const uint32_t u = __float_as_uint(x), e = u >> 23 & 0xff;
    const uint32_t hi = (u & 0x80000000u) | (e == 0 ? 0 : e == 0xff ? 0x7ff00000u | (u & 0x7fffffu) >> 3 : ((u & 0x7fffffffu) >> 3) + 0x38000000u);
    return __hiloint2double((int)hi, e == 0 ? 0 : (int)(u << 29));
}

// A bound that num of the CTA's values reach, num from 1 to 64, and few others pass: of 64
// groups of `group` (4, 8 or 16) threads, the num-th largest of their largest values (0: fewer
// than num groups have one that is not 0).  *top: the largest of all.  Each group finds the place
// of its own, four threads each against sixteen others.  All threads call it; two barriers are in it.
constexpr int kGroups = 64, kGroup = kThreads / kGroups, kCounters = 4;
static_assert(kMostNum <= kGroups && kGroup == kCounters && kJoinThreads <= 16 * kGroups, "groups of the bound");
struct __align__(16) Groups {
    uint32_t best[kGroups];
    uint32_t bound, top;
};
__device__ __forceinline__ uint32_t group_bound(uint32_t best, int num, Groups& sm, uint32_t* top, int group = kGroup) {
    const int own = threadIdx.x / group, in = threadIdx.x % group, from = in % kCounters * (kGroups / kCounters);
    for (int d = 1; d < group; d *= 2) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
    if (in == 0) sm.best[own] = best;
    __syncthreads();
    int before = 0;   // of equal ones those of lower groups
#pragma unroll
    for (int j = 0; j < kGroups / kCounters; j += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(&sm.best[from + j]);
        before += (u.x >= best + (from + j >= own)) + (u.y >= best + (from + j + 1 >= own)) + (u.z >= best + (from + j + 2 >= own)) +
                  (u.w >= best + (from + j + 3 >= own));
    }
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    before += __shfl_xor_sync(0xffffffffu, before, 2);
    if (in == 0 && before == num - 1) sm.bound = best;
    if (in == 0 && before == 0) sm.top = best;
    __syncthreads();
    *top = sm.top;
    return sm.bound;
}

// 16 bytes of the logits.  (Behind the wait for the work that writes them, so an ordinary load; written out, as
// the compiler's own costs three registers more than a thread has.)
__device__ __forceinline__ uint4 load16(const uint4* from) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(from));
    return v;
}

// How the tiles are dealt: row r's are units [r * per_row, (r + 1) * per_row), CTA c
// has units [units * c / ctas, units * (c + 1) / ctas).  Segments are numbered
// r + c, which no two share.
struct Deal {
    int per_row, ctas;
    long long units;
    __host__ __device__ __forceinline__ long long first(long long cta) const { return units * cta / ctas; }
    __host__ __device__ __forceinline__ int cta_of(long long unit) const { return (int)(((unit + 1) * ctas - 1) / units); }
};

struct RowsArgs {
    BeamSelectIO io;
    Deal deal;
    Part* parts;         // [segments]
    uint64_t* lists;     // [segments][num]
    bool early;
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) kda_beam_rows_kernel(const RowsArgs a) {
    constexpr int kVec = kBf16 ? 8 : 4, kLoads = kPer / kVec, kBytes = kBf16 ? 2 : 4;
    __shared__ uint64_t s_list[kList], s_ranked[kList];
    __shared__ Groups s_group;
    __shared__ float2 s_sum[kThreads / 32];
    __shared__ int s_held, s_count[32], s_warp[kThreads / 32];
    __shared__ uint32_t s_mask[kThreads / 32];
    __shared__ uint16_t s_again[kThreads];
    // The join's CTAs may come now where SMs have room for them, else at the last segment's end: beside rows
    // they cost more than they save (64 rows of 50257 18.2 us instead of 13.0, 4 of 32000 7.7 instead of 8.2).
    ptx::griddep_wait();
    if (a.early) ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.io.num;
    const long long last = a.deal.first(blockIdx.x + 1LL);
    for (long long unit = a.deal.first(blockIdx.x), next; unit < last; unit = next) {
    const int row = (int)(unit / a.deal.per_row);
    const long long row0 = (long long)row * a.deal.per_row;
    next = min(row0 + a.deal.per_row, last);
    if (a.io.done && a.io.done[row]) continue;
    const bool alike = a.io.scores[row] == INFINITY;   // at which all finite logits give the same score

    // The row: logits before the first 16-byte boundary, whole vectors, logits behind them.
    const uint8_t* base = static_cast<const uint8_t*>(a.io.logits) + (long long)row * a.io.row_stride * kBytes;
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kBytes, a.io.vocab);
    const int vecs = (a.io.vocab - head) / kVec, tail = a.io.vocab - head - vecs * kVec;
    const int tiles = (vecs + kThreads * kLoads - 1) / (kThreads * kLoads);
    int begin = (int)(unit - row0), end = min((int)(next - row0), tiles);
    if (begin == 0 && head) begin = -1;                               // tile -1: the head, a logit per thread
    if (next - row0 == a.deal.per_row) end = tiles + (tail ? 1 : 0);  // tile `tiles`: the tail
    begin = min(begin, end);
    const uint4* body = reinterpret_cast<const uint4*>(base + (long long)head * kBytes);
    auto single = [&](int t) { return t < 0 || t >= tiles; };
    // Logit i of a tile, of thread `of`: its token, and whether there is one.
    auto token = [&](int t, int i, int of) {
        if (single(t)) return (t < 0 ? 0 : head + vecs * kVec) + of;
        return head + ((t * kLoads + i / kVec) * kThreads + of) * kVec + i % kVec;
    };
    auto there = [&](int t, int i, int of) {
        if (single(t)) return i == 0 && of < (t < 0 ? head : tail);
        return (t * kLoads + i / kVec) * kThreads + of < vecs;
    };
    auto put_right = [&](float x) { return alike && fabsf(x) < INFINITY ? 0.f : x; };
    auto logit_at = [&](int at) {
        return put_right(kBf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(base)[at] << 16)
                               : reinterpret_cast<const float*>(base)[at]);
    };
    if (tid == 0) s_held = 0;
    __syncthreads();

    uint4 raw[kLoads];
    auto load = [&](int t) {
        if (single(t)) {   // in the lowest bits of raw[0]
            if (there(t, 0, tid))
                raw[0].x = kBf16 ? reinterpret_cast<const uint16_t*>(base)[token(t, 0, tid)]
                                 : reinterpret_cast<const uint32_t*>(base)[token(t, 0, tid)];
            return;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (there(t, j * kVec, tid)) raw[j] = load16(body + (t * kLoads + j) * kThreads + tid);
    };
    float x[kPer];
    auto unpack = [&](int t) {
        if (single(t)) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = -INFINITY;
            if (there(t, 0, tid)) x[0] = put_right(__uint_as_float(kBf16 ? raw[0].x << 16 : raw[0].x));
            return;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                x[j * kVec + i] = __uint_as_float(!kBf16 ? w[i & 3] : i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
        if ((t + 1) * kLoads * kThreads > vecs)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (!there(t, i, tid)) x[i] = -INFINITY;
        if (alike)
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = put_right(x[i]);
    };

    // The reference is a logit of the segment; -infinity: there has been none above that, and the sum is 0 or NaN.
    float T = -INFINITY, ref = -INFINITY, sum = 0.f, low = 0.f;   // the sum and what its additions lost
    int held = 0;   // s_held, between the tiles of two looks
    auto add = [&](float v) {
        const float y = v - low, s = sum + y;
        low = (s - sum) - y;
        sum = s;
    };
    // The list's best n, in order; what leaves it joins the sums, in its order, so that they do not
    // depend on the one in which it was written.  All threads call it, behind a barrier.
    auto thin = [&]() {
        for (int i = tid; i < held; i += kThreads) {
            const uint64_t own = s_list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < held; ++j) rank += s_list[j] > own;
            s_ranked[rank] = own;
        }
        __syncthreads();
        for (int i = tid; i < held; i += kThreads) {
            const uint64_t c = s_ranked[i];
            if (i < n) s_list[i] = c;
            else add(exp_of(logit_of(c) - ref));
        }
        if (held >= n) T = fmaxf(T, logit_of(s_ranked[n - 1]));
        held = min(held, n);
        if (tid == 0) s_held = held;
        __syncthreads();
    };

    if (begin < end) load(begin);
    for (int t0 = begin, t1; t0 < end; t0 = t1) {
        t1 = end - t0 <= kSub + 2 ? end : t0 + kSub;   // (the head and the tail are no look of their own)
        const float sum0 = sum, low0 = low;
        float scale0 = 1.f, most;
        uint32_t bound, top;
        for (;;) {
            sum = sum0 * scale0;
            low = low0 * scale0;
            most = -INFINITY;
            for (int t = t0; t < t1; ++t) {
                unpack(t);
                if (t + 1 < end) load(t + 1);
                float m = mma::max3(mma::max3(x[0], x[1], x[2]), x[3], x[4]);
#pragma unroll
                for (int i = 5; i < kPer - 1; i += 2) m = mma::max3(m, x[i], x[i + 1]);
                m = fmaxf(m, x[kPer - 1]);
                m = fmaxf(m, -INFINITY);   // not NaN
                if (t == begin && ref == -INFINITY) {
                    const uint32_t w = __reduce_max_sync(0xffffffffu, order_of(m));
                    if (lane == 0) s_group.best[warp] = w;
                    __syncthreads();
                    const float first = float_of(__reduce_max_sync(0xffffffffu, s_group.best[lane & (kThreads / 32 - 1)]));
                    if (fabsf(first) < INFINITY) ref = first;
                    __syncthreads();
                }
                most = fmaxf(most, m);
                const float to = ref == -INFINITY ? 0.f : ref;
                mma::f32x2 part = mma::pk(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kPer; i += 2) part = mma::add2(part, exp_of(mma::add2(mma::pk(x[i], x[i + 1]), mma::pk(-to, -to))));
                float even, odd;
                mma::upk(part, even, odd);
                add(even + odd);
            }
            bound = group_bound(order_of(most), n, s_group, &top);
            const float now = float_of(top);
            if (fabsf(now) == INFINITY || (ref != -INFINITY && now - ref <= kRefMargin)) break;
            // The first logits above -infinity, or ones far above the reference: these tiles once more.
            if (ref != -INFINITY) scale0 *= expf(ref - now);
            ref = now;
            load(t0);
        }
        // Threads whose largest logit is a candidate, dealt to the half warps in turn: four of a thread's
        // logits for each lane.
        const float s0 = sum0 * scale0, l0 = low0 * scale0;
        const float least = float_of(max(bound, order_of(T) + 1));   // of a candidate: the bound, or above T
        const bool mine = most >= least;
        const uint32_t again = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) s_mask[warp] = again;
        __syncthreads();
        int total = 0, at = __popc(again & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int count = __popc(s_mask[w]);
            if (w < warp) at += count;
            total += count;
        }
        if (mine) {
            s_again[at] = (uint16_t)tid;
            sum = s0;
            low = l0;
        }
        __syncthreads();
        const int i_mine = 4 * (lane & 15) % kPer, turns = ((t1 - t0) * kPer + 63) / 64;
        for (int k = tid / 16; k < total * turns; k += kThreads / 16) {
            const int turn = k / total, thread = s_again[k - turn * total], t_mine = t0 + (turn * 64 + 4 * (lane & 15)) / kPer;
            const uint8_t* mine_at = base + (long long)token(t_mine, i_mine, 0) * kBytes;
            float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (t_mine < t1 && there(t_mine, i_mine, thread)) {
                if (single(t_mine)) {
                    v[0] = logit_at(token(t_mine, 0, thread));
                } else {
                    uint4 w;
                    if (kBf16) {
                        const uint2 two = *reinterpret_cast<const uint2*>(mine_at + thread * 16);
                        w = make_uint4(two.x << 16, two.x & 0xffff0000u, two.y << 16, two.y & 0xffff0000u);
                    } else {
                        w = *reinterpret_cast<const uint4*>(mine_at + thread * 16);
                    }
                    v[0] = put_right(__uint_as_float(w.x));
                    v[1] = put_right(__uint_as_float(w.y));
                    v[2] = put_right(__uint_as_float(w.z));
                    v[3] = put_right(__uint_as_float(w.w));
                }
            }
            float rest = 0.f;
            uint32_t in = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool is = v[i] >= least;
                in |= (uint32_t)is << i;
                rest += is ? 0.f : exp_of(v[i] - ref);
            }
            add(rest);
            for (; in; in &= in - 1) {
                const int i = __ffs((int)in) - 1, to = atomicAdd(&s_held, 1);
                const float x4 = i < 2 ? (i ? v[1] : v[0]) : (i == 2 ? v[2] : v[3]);
                if (to < kList) s_list[to] = candidate(x4, token(t_mine, i_mine + i, thread));
            }
        }
        __syncthreads();
        if (s_held > kList) {
            // Many logits are equal, or many of one thread pass all others.  The num-th largest above T by
            // its bits, and those that are equal to it in the order of their tokens.
            if (tid < 32) s_count[tid] = 0;
            __syncthreads();
            if (tid == 0) s_held = held;
            uint32_t nth = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t with = nth | 1u << bit;
                int count = 0;
                for (int t = t0; t < t1; ++t)
                    for (int i = 0; i < kPer; ++i)
                        if (there(t, i, tid)) {
                            const float v = logit_at(token(t, i, tid));
                            count += v > T && order_of(v) >= with;
                        }
                count = __reduce_add_sync(0xffffffffu, count);
                if (lane == 0) atomicAdd(&s_count[bit], count);
                __syncthreads();
                if (s_count[bit] >= n) nth = with;
            }
            __syncthreads();
            int above = 0;
            for (int t = t0; t < t1; ++t)
                for (int i = 0; i < kPer; ++i)
                    if (there(t, i, tid)) above += logit_at(token(t, i, tid)) > float_of(nth);
            above = __reduce_add_sync(0xffffffffu, above);
            if (lane == 0) s_warp[warp] = above;
            __syncthreads();
            int need = n;
            for (int w = 0; w < kThreads / 32; ++w) need -= s_warp[w];
            sum = s0;
            low = l0;
            for (int t = t0; t < t1; ++t)
                for (int j = 0; j < kPer; j += kVec) {
                    int equal = 0;
                    for (int i = j; i < j + kVec; ++i)
                        if (there(t, i, tid)) equal += logit_at(token(t, i, tid)) == float_of(nth);
                    int upto = equal;
                    for (int d = 1; d < 32; d <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, upto, d);
                        if (lane >= d) upto += y;
                    }
                    __syncthreads();
                    if (lane == 31) s_warp[warp] = upto;
                    __syncthreads();
                    int all = 0;
                    for (int w = 0; w < kThreads / 32; ++w) {
                        if (w == warp) upto += all;
                        all += s_warp[w];
                    }
                    int left = need - (upto - equal);   // of this thread's equal ones, the first that are wanted
                    float rest = 0.f;
                    for (int i = j; i < j + kVec; ++i) {
                        if (!there(t, i, tid)) continue;
                        const int at = token(t, i, tid);
                        const float v = logit_at(at);
                        if (v > float_of(nth) || (v == float_of(nth) && left-- > 0)) s_list[atomicAdd(&s_held, 1)] = candidate(v, at);
                        else rest += exp_of(v - ref);
                    }
                    add(rest);
                    need -= all;
                }
            __syncthreads();
        }
        held = s_held;   // (the next candidate is behind the next bound's barrier)
        T = fmaxf(T, float_of(bound));   // which num logits reach, all of them in the list
        if (held > kThin || t1 == end) thin();
    }
    if (next == last) ptx::griddep_launch_dependents();
    const int kept = held;
    const size_t segment = (size_t)row + blockIdx.x;

    // The threads' sums, with what the additions lose.
    float more = -low;
    auto join = [&](float s, float m) {
        const float t = sum + s, back = t - sum;
        more += m + ((sum - (t - back)) + (s - back));
        sum = t;
    };
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float s = __shfl_xor_sync(0xffffffffu, sum, d), m = __shfl_xor_sync(0xffffffffu, more, d);
        join(s, m);
    }
    if (lane == 0) s_sum[warp] = make_float2(sum, more);
    __syncthreads();
    if (tid == 0) {
        sum = more = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) join(s_sum[w].x, s_sum[w].y);
        a.parts[segment] = Part{sum, more, ref, 0.f};
    }
    for (int i = tid; i < n; i += kThreads) a.lists[segment * n + i] = i < kept ? s_list[i] : 0;
    __syncthreads();
    }
}

// A continuation: its score in the order of unsigned numbers (64-bit comparisons of
// floating numbers run at a sixty-fourth of the rate), and what decides between equal ones, the lower
// beam, the larger logit (whose score is the higher one by what 64 bits do not hold), the lower token:
// the beam's complement, the logit's order and the token's complement, 64 bits at most
// since beams * vocab is below 2^31.
struct __align__(16) Choice {
    uint64_t key, low;
};
constexpr uint64_t kLowestKey = 0x000fffffffffffffull;   // -infinity's
__device__ __forceinline__ uint64_t key_of(double score) {
    uint64_t u = (uint64_t)__double_as_longlong(score);
    if (u == 1ull << 63) u = 0;   // -0 is 0
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double score_of(uint64_t key) {
    return __longlong_as_double((long long)(key ^ ((key >> 63) ? 1ull << 63 : ~0ull)));
}
__device__ __forceinline__ bool better(const Choice& a, const Choice& b) {
    return (a.key > b.key) | ((a.key == b.key) & (a.low > b.low));   // no branch: loops over it are bound by its latency
}

struct JoinArgs {
    BeamSelectIO io;
    Deal deal;
    int most;            // segments of a row
    int rounds;          // candidates of a thread
    int beam_bits, token_bits;
    uint32_t per_segments, per_most;   // 2^31 over K * most and over most, rounded up: quotients of numbers below 2^12
    const Part* parts;
    const uint64_t* lists;
};

// (What runs once per CTA waits for its instructions: little of it is written out.)
template <int kMost>
__global__ void __launch_bounds__(kMost) kda_beam_join_kernel(const JoinArgs a) {
    __shared__ double s_from[KDA_BEAM_MAX_BEAMS];   // a score is (logit - most) + from
    __shared__ double s_most[KDA_BEAM_MAX_BEAMS];
    __shared__ int s_first[KDA_BEAM_MAX_BEAMS], s_segments[KDA_BEAM_MAX_BEAMS];
    __shared__ bool s_done[KDA_BEAM_MAX_BEAMS];     // at its end: its segments hold anything
    __shared__ Groups s_group;
    __shared__ Choice s_best[kMost], s_bound;
    __shared__ Choice s_list[kJoinList];
    __shared__ Choice s_sorted[kMostNum];
    __shared__ int s_held, s_beam[kMostNum];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = kMost;
    const int g = blockIdx.x, K = a.io.beams, n = a.io.num, S = a.most;
    const uint8_t* done = a.io.done ? a.io.done + (size_t)g * K : nullptr;
    const float* scores = a.io.scores + (size_t)g * K;
    const uint32_t beam_mask = (1u << a.beam_bits) - 1, token_mask = (1u << a.token_bits) - 1;
    auto low_of = [&](int beam, uint64_t c) {   // of candidate c
        return (uint64_t)(beam_mask - beam) << (32 + a.token_bits) | (c >> 32) << a.token_bits | ((uint32_t)c & token_mask);
    };
    auto beam_at = [&](uint64_t low) { return (int)(beam_mask - (uint32_t)(low >> (32 + a.token_bits))); };
    auto token_at = [&](uint64_t low) { return (int)(token_mask - ((uint32_t)low & token_mask)); };
    if (tid == 0) s_held = 0;
    if (tid < K) {
        const int k = tid;
        const long long row = (long long)g * K + k;
        const int from = a.deal.cta_of(row * a.deal.per_row), to = a.deal.cta_of((row + 1) * a.deal.per_row - 1);
        s_first[k] = (int)row + from;
        s_segments[k] = to - from + 1;
    }
    __syncthreads();
    ptx::griddep_wait();
    const bool ended = done && tid < K && done[tid];   // (under way beside the lists)

    // This thread's share of the segments' lists, taken as all first candidates, then all second ones,
    // ..., in turns by the groups of threads of the bound below: each group has some of every beam.
    const int segments = K * S;
    uint64_t own[kJoinPer];
    int beam_of[kJoinPer];
    {
        constexpr int group = kMost / kGroups;
        const int turn = tid % group * kGroups + tid / group;
#pragma unroll
        for (int j = 0; j < kJoinPer; ++j) {
            if (j >= a.rounds) break;
            const uint32_t i = j * threads + turn, nth = __umulhi(2 * i, a.per_segments), at = i - nth * segments;
            const int k = (int)__umulhi(2 * at, a.per_most), s = (int)at - k * S;
            beam_of[j] = k;
            own[j] = nth < (uint32_t)n && s < s_segments[k] ? a.lists[(size_t)(s_first[k] + s) * n + nth] : 0;
        }
    }

    if (tid < K) s_done[tid] = ended;
    __syncthreads();

    // The beams' sums of exp(x - most).  Where one is NaN, the beam has nothing to offer.
    for (int k = warp; k < K; k += threads / 32) {
        const int here = s_segments[k];
        if (s_done[k]) continue;
        const Part* p = a.parts + s_first[k];
        const uint64_t* l = a.lists + (size_t)s_first[k] * n;
        // Up to 32 parts and 64 candidates at once: one latency for all of them.
        const Part none{0.f, 0.f, -INFINITY, 0.f}, x0 = lane < here ? p[lane] : none;
        uint64_t head = lane < here ? l[lane * n] : 0;
        const uint64_t c0 = lane < here * n ? l[lane] : 0, c1 = lane + 32 < here * n ? l[lane + 32] : 0;
        for (int s = lane + 32; s < here; s += 32) head = max(head, l[s * n]);
        const uint32_t top = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32));
        const float most = top ? float_of(top) : -INFINITY;
        long long sum = 0;
        bool bad = !(most < INFINITY);
        auto add_candidate = [&](uint64_t c) {
            const Power e = power_of(c ? logit_of(c) : -INFINITY, most);
            sum += e.i > -32 ? e.m >> -e.i : 0u;
        };
        auto add_part = [&](const Part& x) {
            bad |= !(x.sum < INFINITY);
            if (x.ref != -INFINITY) {   // which is at most the segment's first candidate
                const Power e = power_of(x.ref, most);
                sum += scaled(x.sum, e) + scaled(x.more, e);
            }
        };
        add_candidate(c0);
        if (here * n > 32) add_candidate(c1);
        for (int i = lane + 64; i < here * n; i += 32) add_candidate(l[i]);
        add_part(x0);
        for (int s = lane + 32; s < here; s += 32) add_part(p[s]);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            s_most[k] = most;
            s_from[k] = bad || sum <= 0 ? -INFINITY : (double)scores[k] - ln_fixed((unsigned long long)sum);
        }
    }
    __syncthreads();

    // The continuations above -infinity; the last is that of a beam at its end.
    Choice mine[kJoinPer + 1];
    Choice best{0, 0};
#pragma unroll
    for (int j = 0; j <= kJoinPer; ++j) {
        if (j >= a.rounds && j < kJoinPer) continue;
        if (j < kJoinPer) {
            const int k = beam_of[j];
            const double score = (widened(logit_of(own[j])) - s_most[k]) + s_from[k];
            // Of NaN the key tells nothing.
            const bool number = ((uint64_t)__double_as_longlong(score) << 1) <= 0xffe0000000000000ull;
            const uint64_t key = key_of(score);
            mine[j] = Choice{own[j] && !s_done[k] && number && key > kLowestKey ? key : 0, low_of(k, own[j])};
        } else {
            mine[j] = Choice{0, 0};
            if (ended && scores[tid] > -INFINITY)
                mine[j] = Choice{key_of(scores[tid]), low_of(tid, candidate(0.f, a.io.end_token))};
        }
        if (better(mine[j], best)) best = mine[j];
    }
    // A bound that num of them reach, as in the rows' kernel; of equal scores all pass.
    uint32_t top;
    Choice bound{max((uint64_t)group_bound((uint32_t)(best.key >> 32), n, s_group, &top, kMost / kGroups) << 32, (uint64_t)1), 0};
    for (;;) {
        int count = 0;
#pragma unroll
        for (int j = 0; j <= kJoinPer; ++j)
            if (j < a.rounds || j == kJoinPer) count += !better(bound, mine[j]);
        int to = count ? atomicAdd(&s_held, count) : 0;
        const bool fits = to + count <= kJoinList;
        if (count && fits)
#pragma unroll
            for (int j = 0; j <= kJoinPer; ++j)
                if ((j < a.rounds || j == kJoinPer) && !better(bound, mine[j])) s_list[to++] = mine[j];
        if (!__syncthreads_or(!fits)) break;
        // Too many: the num-th best of the threads' best, which num threads at most reach.
        s_best[tid] = best;
        if (tid == 0) {
            s_held = 0;
            s_bound = Choice{1, 0};
        }
        __syncthreads();
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < threads; ++j) above += better(s_best[j], best);
        if (best.key && above == n - 1) s_bound = best;
        __syncthreads();
        bound = s_bound;
    }
    const int held = s_held, chosen = min(held, n);
    for (int i = tid; i < held; i += threads) {
        const Choice c = s_list[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < held; ++j) rank += better(s_list[j], c);
        if (rank < n) s_sorted[rank] = c;
    }
    __syncthreads();
    // Fewer than num above -infinity: the lowest others.
    if (warp == 0 && chosen < n) {
        int m = chosen;
        for (uint32_t at = 0; m < n; ++at) {
            const int beam = (int)(at / (uint32_t)a.io.vocab), token = (int)(at % (uint32_t)a.io.vocab);
            bool used = false;
            for (int i = lane; i < chosen; i += 32) used |= beam_at(s_sorted[i].low) == beam && token_at(s_sorted[i].low) == token;
            if (__any_sync(0xffffffffu, used)) continue;
            if (lane == 0) s_sorted[m] = Choice{kLowestKey, low_of(beam, candidate(0.f, token))};
            ++m;
        }
    }
    __syncthreads();
    if (tid < n) s_beam[tid] = beam_at(s_sorted[tid].low);
    __syncthreads();

    if (tid < n) {
        const int beam = s_beam[tid];
        int place = tid;
        if (a.io.keep) {
            // The first of its beam: the beam's place.  Others: the place that as many
            // free ones precede as others precede it.
            uint64_t kept = 0;   // places of beams that go on
            int others = 0;      // before this one
            bool first = true;
            for (int j = 0; j < n; ++j) {
                const int b = s_beam[j];
                const bool seen = kept >> b & 1;
                if (j < tid) {
                    others += seen;
                    first &= b != beam;
                }
                kept |= 1ull << b;
            }
            place = beam;
            if (!first) {
                place = 0;
                for (int left = others;; ++place) {
                    if (kept >> place & 1) continue;
                    if (left-- == 0) break;
                }
            }
        }
        const size_t out = (size_t)g * n + place;
        a.io.out_scores[out] = (float)score_of(s_sorted[tid].key);
        a.io.out_tokens[out] = token_at(s_sorted[tid].low);
        a.io.out_rows[out] = g * K + beam;
    }
}

// The deal, and the most segments of a row.  No CTA has less than a tile, and the
// join takes K * num candidates for each of a row's segments.  Fewer CTAs, each with
// a part of one row alone, if what they have more to read than all that fit costs less than
// the second segment does that these begin (256 rows of 8 tiles in bf16, 512 CTAs and 608: 14.5 us
// and 18; 400 rows of 13 tiles, as many CTAs and 608: 20.0 and 22.7; 512 rows of 32 tiles: 54.9 and 54.3).
constexpr int kCtasPerSm = 4;
constexpr int kSegmentCost = 5;        // tiles
Deal deal_of(int groups, int beams, int vocab, int num, const DeviceInfo& dev, int& most) {
    const long long rows = (long long)groups * beams;
    Deal d;
    d.per_row = (int)(((long long)vocab + kTile - 1) / kTile);   // (vocab may be 2^31 - 1)
    d.units = rows * d.per_row;
    long long ctas = (long long)kCtasPerSm * dev.sm_count;
    if (ctas > d.units) ctas = d.units;
    if (ctas >= rows) {
        const long long alone = ctas / rows * rows;
        if ((d.units + alone - 1) / alone < (d.units + ctas - 1) / ctas + kSegmentCost) ctas = alone;
    }
    for (;; ctas = ctas > 2 * rows ? ctas - rows : rows) {
        // Ranges of `least` units or one more: a row's units lie in so many of them at most.
        const long long least = d.units / ctas;
        most = ctas == rows ? 1 : (int)((d.per_row - 1 + least - 1) / least) + 1;
        if (most == 1 || (long long)beams * num * most <= kJoinEntries) break;
    }
    d.ctas = (int)ctas;
    return d;
}

size_t parts_bytes(size_t parts) { return (parts * sizeof(Part) + 255) & ~size_t(255); }
size_t parts_of(const BeamSelectIO& io, const Deal& d) { return (size_t)io.groups * io.beams + d.ctas; }

}  // namespace

size_t beam_select_workspace_bytes(int groups, int beams, int vocab, int num, const DeviceInfo& dev) {
    int most;
    const Deal d = deal_of(groups, beams, vocab, num, dev, most);
    const size_t parts = (size_t)groups * beams + d.ctas;
    return parts_bytes(parts) + parts * num * sizeof(uint64_t);
}

cudaError_t launch_beam_select(const BeamSelectIO& io, const DeviceInfo& dev, cudaStream_t stream) {
    int most;
    const Deal d = deal_of(io.groups, io.beams, io.vocab, io.num, dev, most);
    Part* p = static_cast<Part*>(io.workspace);
    uint64_t* lists = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(io.workspace) + parts_bytes(parts_of(io, d)));
    const RowsArgs r{io, d, p, lists, d.ctas <= dev.sm_count};
    const cudaError_t e = launch_behind(io.bf16 ? kda_beam_rows_kernel<true> : kda_beam_rows_kernel<false>, dim3((unsigned)d.ctas), kThreads, 0,
                                        stream, r);
    if (e != cudaSuccess) return e;
    const uint64_t segments = (uint64_t)io.beams * most;
    // Threads for all candidates, kJoinPer each at most.
    int threads = kThreads;
    while (threads < kJoinThreads && segments * io.num > (uint64_t)kJoinPer * threads) threads *= 2;
    auto bits = [](int n) {   // of numbers below n
        int b = 0;
        while (1LL << b < n) ++b;
        return b;
    };
    const JoinArgs j{io, d, most, (int)((segments * io.num + threads - 1) / threads), bits(io.beams), bits(io.vocab),
                     (uint32_t)(((1ull << 31) + segments - 1) / segments), (uint32_t)(((1ull << 31) + most - 1) / most), p, lists};
    auto join = threads == kThreads ? kda_beam_join_kernel<kThreads> : threads == 512 ? kda_beam_join_kernel<512> : kda_beam_join_kernel<kJoinThreads>;
    return launch_behind(join, dim3((unsigned)io.groups), threads, 0, stream, j);
}

}  // namespace kda
