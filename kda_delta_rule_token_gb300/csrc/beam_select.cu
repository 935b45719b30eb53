// The num best continuations of every group of beams.
//
//   score(k, v) = s_k + x_kv - lse_k,   lse_k = ln sum_v exp(x_kv)
//
// A row's scores have the order of its logits, so one pass over the logits
// finds both what a row can offer (its num largest logits) and what they are
// measured against (lse).  Every logit is read once; what is left is small:
// the call is bound by HBM, or by its two launches.
//
//  * kda_beam_rows_kernel: a CTA takes a segment of one row in tiles of 256
//    threads x 16 logits, the next tile's loads under way.  A logit that passes
//    the threshold T (the num-th largest that the CTA is sure of) joins the
//    list of candidates in shared memory, any other adds exp(x - ref) to its
//    thread's sum.  T rises when the list is full, and where one tile has more
//    candidates than the list holds: of the threads' largest logits the num-th
//    largest is a bound that at least num logits of the tile reach and at most
//    num threads pass.  After the first tile few logits pass.
//  * kda_beam_join_kernel, a CTA per group: lse of every beam from its segments'
//    sums, then the num best of the segments' lists, by the same bound over
//    the threads' best.
//
// Which of two beams' close candidates is the better one hangs on the last bits
// of their lse.  The largest terms decide these, and they are the candidates:
// they stay out of the fp32 sums, and their exponentials are taken and added in
// 64 bits.  Scores are formed and compared in 64 bits and rounded once.
#include <math.h>

#include "beam_internal.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;               // logits of a thread per tile
constexpr int kTile = kThreads * kPer;
constexpr int kList = 1536;            // candidates that a CTA holds
constexpr int kSoft = 512;             // above which they are thinned out after a tile
constexpr int kMostNum = KDA_BEAM_MAX_NUM;
static_assert(kSoft + kPer * kMostNum <= kList, "a raised threshold leaves at most kPer * num candidates of a tile");
constexpr int kJoinEntries = 8192 - KDA_BEAM_MAX_BEAMS;   // candidates of a group's segments that the join takes
constexpr int kJoinList = 2048;
static_assert((kJoinEntries + KDA_BEAM_MAX_BEAMS + kThreads - 1) / kThreads * kMostNum <= kJoinList, "candidates that the join's bound leaves");
constexpr int kJoinParts = 512;        // segments of a group's beams
constexpr float kRefMargin = 20.f;     // how far above the reference a logit of the sums may be

// What a segment leaves: the sum of exp(x - most) over it, and its candidates' number.
struct Part {
    double sum;
    float most;
    int count;
};

// A candidate: the logit in the order of unsigned numbers above, the complement of
// its token below, so that the larger of two is the better one.
__device__ __forceinline__ uint64_t candidate(float x, int token) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 is 0
    return (uint64_t)(u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u)) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float logit_of(uint64_t c) {
    const uint32_t u = (uint32_t)(c >> 32);
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int token_of(uint64_t c) { return (int)~(uint32_t)c; }

// exp(d), d <= kRefMargin: the product with log2 e to 2^-24 of itself.
__device__ __forceinline__ float exp_of(float d) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(d, 1.44269502f, d * 1.92596299e-8f)));
    return y;
}

struct RowsArgs {
    BeamSelectIO io;
    int segments;
    Part* parts;         // [rows][segments]
    uint64_t* lists;     // [rows][segments][num]
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) kda_beam_rows_kernel(const RowsArgs a) {
    constexpr int kVec = kBf16 ? 8 : 4, kLoads = kPer / kVec, kBytes = kBf16 ? 2 : 4;
    __shared__ uint64_t s_list[kList], s_best[kThreads];
    __shared__ uint64_t s_bound;
    __shared__ double s_sum[kThreads / 32];
    __shared__ int s_want[3], s_held;
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.io.num;
    const int row = blockIdx.x / a.segments, segment = blockIdx.x % a.segments;
    if (a.io.done && a.io.done[row]) return;
    const bool alike = a.io.scores[row] == INFINITY;   // at which all finite logits give the same score

    // The row: logits before the first 16-byte boundary, whole vectors, logits behind them.
    const uint8_t* base = static_cast<const uint8_t*>(a.io.logits) + (long long)row * a.io.row_stride * kBytes;
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kBytes, a.io.vocab);
    const int vecs = (a.io.vocab - head) / kVec, tail = a.io.vocab - head - vecs * kVec;
    const int tiles = (vecs + kThreads * kLoads - 1) / (kThreads * kLoads);
    int t = (int)((long long)tiles * segment / a.segments);
    int end = (int)((long long)tiles * (segment + 1) / a.segments);
    if (segment == 0 && head) t = -1;                      // tile -1: the head
    if (segment == a.segments - 1 && tail) end = tiles + 1;   // tile `tiles`: the tail
    const uint4* body = reinterpret_cast<const uint4*>(base + (long long)head * kBytes);

    if (tid == 0) {
        s_held = 0;
        s_want[0] = s_want[1] = s_want[2] = 0;
    }
    __syncthreads();

    uint4 raw[kLoads];
    auto load = [&](int tile) {
        if (tile < 0 || tile >= tiles) {   // a single logit in the lowest bits of raw[0]
            const int i = tile < 0 ? tid : head + vecs * kVec + tid;
            if (tid < (tile < 0 ? head : tail))
                raw[0].x = kBf16 ? reinterpret_cast<const uint16_t*>(base)[i] : reinterpret_cast<const uint32_t*>(base)[i];
            return;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int v = (tile * kLoads + j) * kThreads + tid;
            if (v < vecs) raw[j] = __ldcs(body + v);
        }
    };

    float T = -INFINITY, ref = -INFINITY, sum = 0.f, low = 0.f;   // the sum and what its additions lost
    auto add = [&](float x) {
        const float y = x - low, s = sum + y;
        low = (s - sum) - y;
        sum = s;
    };
    // A higher threshold; the sums stay within kRefMargin of their reference.
    auto raise = [&](float to) {
        T = fmaxf(T, to);
        if (ref == -INFINITY) {
            ref = T;
        } else if (T > ref + kRefMargin) {
            const float f = expf(ref - T);
            sum *= f;
            low *= f;
            ref = T;
        }
    };
    // The list's best n, in order; what leaves it joins the sums, in its order, so that they do not
    // depend on the one in which it was written.  All threads call it.
    auto thin = [&](int held) {
        uint64_t own[kList / kThreads];
        int rank[kList / kThreads];
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i) {
            rank[i] = -1;
            if (i * kThreads >= held) continue;
            if (i * kThreads + tid < held) {
                own[i] = s_list[i * kThreads + tid];
                rank[i] = 0;
                for (int j = 0; j < held; ++j) rank[i] += s_list[j] > own[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i)
            if (rank[i] >= 0) s_list[rank[i]] = own[i];
        if (tid == 0) s_held = min(held, n);
        __syncthreads();
        if (held >= n) raise(logit_of(s_list[n - 1]));
        for (int i = n + tid; i < held; i += kThreads) add(exp_of(logit_of(s_list[i]) - ref));
    };

    if (t < end) load(t);
    for (int turn = 0; t < end; ++t, turn = turn == 2 ? 0 : turn + 1) {
        float x[kPer];
        const bool single = t < 0 || t >= tiles;
        const int first = t < 0 ? 0 : t >= tiles ? head + vecs * kVec : head + t * kTile;
        const int at = first + tid * (single ? 1 : kVec);   // token of x[0]; of x[i]: at + i / kVec * kThreads * kVec + i % kVec
        if (single) {
            const bool in = tid < (t < 0 ? head : tail);
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = -INFINITY;
            if (in) x[0] = kBf16 ? __uint_as_float(raw[0].x << 16) : __uint_as_float(raw[0].x);
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const bool in = (t * kLoads + j) * kThreads + tid < vecs;
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float f = kBf16 ? __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) : __uint_as_float(w[i & 3]);
                    x[j * kVec + i] = in ? f : -INFINITY;
                }
            }
        }
        if (t + 1 < end) load(t + 1);
        if (alike) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (fabsf(x[i]) < INFINITY) x[i] = 0.f;
        }

        int want = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) want += x[i] > T;
        if (want) atomicAdd(&s_want[turn], want);
        __syncthreads();
        const int all = s_want[turn];
        if (tid == 0) s_want[turn ? turn - 1 : 2] = 0;   // the one after the next, which all have read
        if (all) {
            auto token = [&](int i) { return at + i / kVec * (kThreads * kVec) + i % kVec; };
            uint64_t bound = 0;
            if (s_held + all > kList) {
                // The num-th largest of the threads' best: at least num logits of the tile reach it.
                uint64_t best = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (x[i] > T) best = max(best, candidate(x[i], token(i)));
                s_best[tid] = best;
                if (tid == 0) s_bound = 0;
                __syncthreads();
                int above = 0;
#pragma unroll 8
                for (int j = 0; j < kThreads; ++j) above += s_best[j] > best;
                if (best && above == n - 1) s_bound = best;
                __syncthreads();
                bound = s_bound;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (x[i] > T) {
                    const uint64_t c = candidate(x[i], token(i));
                    if (c >= bound) {
                        s_list[atomicAdd(&s_held, 1)] = c;
                        x[i] = -INFINITY;
                    }
                }
            // Tokens behind this tile have to be above it to be better.
            if (bound) raise(logit_of(bound));
        }
        // Logits below the threshold: where there is none yet, they are all -infinity or NaN.
        const float to = ref == -INFINITY ? 0.f : ref;
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) part += exp_of(x[i] - to);
        add(part);
        if (all) {
            __syncthreads();
            if (s_held > kSoft) thin(s_held);
            __syncthreads();
        }
    }
    __syncthreads();
    thin(s_held);
    const int kept = s_held;

    // The segment's sum, measured from its largest candidate.
    double total = (double)sum - (double)low;
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) s_sum[warp] = total;
    __syncthreads();
    if (warp == 0) {
        const float most = kept ? logit_of(s_list[0]) : -INFINITY;
        total = lane < kThreads / 32 ? s_sum[lane] : 0.0;
        // Without a candidate above -infinity there is nothing to measure from: the sum is 0, or NaN.
        if (kept && ref != -INFINITY) total *= exp((double)ref - (double)most);
        for (int i = lane; i < kept; i += 32) total += exp((double)logit_of(s_list[i]) - (double)most);
#pragma unroll
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        if (lane == 0) a.parts[blockIdx.x] = Part{total, most, kept};
    }
    for (int i = tid; i < kept; i += kThreads) a.lists[(size_t)blockIdx.x * n + i] = s_list[i];
}

// A continuation: its score and beam * vocab + token.
struct Choice {
    double score;
    uint32_t at;
};
__device__ __forceinline__ bool better(const Choice& a, const Choice& b) {
    return a.score > b.score || (a.score == b.score && a.at < b.at);
}

struct JoinArgs {
    BeamSelectIO io;
    int segments;
    const Part* parts;
    const uint64_t* lists;
};

__global__ void __launch_bounds__(kThreads) kda_beam_join_kernel(const JoinArgs a) {
    __shared__ double s_most[KDA_BEAM_MAX_BEAMS], s_ln[KDA_BEAM_MAX_BEAMS], s_score[KDA_BEAM_MAX_BEAMS];
    __shared__ uint8_t s_done[KDA_BEAM_MAX_BEAMS];
    __shared__ Choice s_best[kThreads];
    __shared__ Choice s_list[kJoinList];
    __shared__ Choice s_sorted[kMostNum];
    __shared__ Choice s_bound;
    __shared__ int s_held, s_beam[kMostNum];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.x, K = a.io.beams, n = a.io.num, S = a.segments;
    for (int k = tid; k < K; k += kThreads) {
        s_score[k] = a.io.scores[(size_t)g * K + k];
        s_done[k] = a.io.done ? a.io.done[(size_t)g * K + k] : 0;
    }
    if (tid == 0) {
        s_held = 0;
        s_bound = Choice{-INFINITY, 0xffffffffu};
    }
    ptx::griddep_wait();
    __syncthreads();

    // The beams' sums: ln of the sum of exp(x - most).
    for (int k = warp; k < K; k += kThreads / 32) {
        if (s_done[k]) continue;
        const Part* p = a.parts + ((size_t)g * K + k) * S;
        float most = -INFINITY;
        for (int s = lane; s < S; s += 32) most = fmaxf(most, p[s].most);
#pragma unroll
        for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        double sum = 0.0;
        for (int s = lane; s < S; s += 32) {
            const Part x = p[s];
            // A segment of -infinities adds nothing (one with a NaN: NaN).
            sum += x.most == -INFINITY ? x.sum : x.sum * exp((double)x.most - (double)most);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) {
            s_most[k] = most;
            s_ln[k] = log(sum);
        }
    }
    __syncthreads();

    // The choice at place i of beam k's segments' lists, or a beam's end; false if there is none above -infinity.
    const int per_beam = S * n, entries = K * per_beam;
    auto entry = [&](int i, Choice& c) {
        if (i >= entries) {
            const int k = i - entries;
            c = Choice{s_score[k], (uint32_t)k * (uint32_t)a.io.vocab + (uint32_t)a.io.end_token};
            return s_done[k] && c.score > -INFINITY;
        }
        const int k = i / per_beam;
        if (s_done[k]) return false;
        const size_t part = ((size_t)g * K + k) * S + (i - k * per_beam) / n;
        if ((i - k * per_beam) % n >= a.parts[part].count) return false;
        const uint64_t x = a.lists[part * n + (i - k * per_beam) % n];
        // x - most is exact or rounded once; NaN is no choice.
        c = Choice{((double)logit_of(x) - s_most[k]) - s_ln[k] + s_score[k],
                   (uint32_t)k * (uint32_t)a.io.vocab + (uint32_t)token_of(x)};
        return c.score > -INFINITY;
    };

    // Of the threads' best, the num-th: no chosen one is below it.
    Choice best{-INFINITY, 0xffffffffu};
    bool any = false;
    for (int i = tid; i < entries + K; i += kThreads) {
        Choice c;
        if (entry(i, c) && (!any || better(c, best))) {
            best = c;
            any = true;
        }
    }
    s_best[tid] = best;
    __syncthreads();
    int above = 0;
    for (int j = 0; j < kThreads; ++j) above += better(s_best[j], best);
    if (any && above == n - 1) s_bound = best;
    __syncthreads();
    const Choice bound = s_bound;
    if (any && !better(bound, best))   // else none of this thread's reach it
        for (int i = tid; i < entries + K; i += kThreads) {
            Choice c;
            if (entry(i, c) && !better(bound, c)) s_list[atomicAdd(&s_held, 1)] = c;
        }
    __syncthreads();
    const int held = s_held, chosen = min(held, n);
    for (int i = tid; i < held; i += kThreads) {
        const Choice c = s_list[i];
        int rank = 0;
        for (int j = 0; j < held; ++j) rank += better(s_list[j], c);
        if (rank < n) s_sorted[rank] = c;
    }
    __syncthreads();
    // Fewer than num above -infinity: the lowest others.
    if (warp == 0 && chosen < n) {
        int m = chosen;
        for (uint32_t at = 0; m < n; ++at) {
            bool used = false;
            for (int i = lane; i < chosen; i += 32) used |= s_sorted[i].at == at;
            if (__any_sync(0xffffffffu, used)) continue;
            if (lane == 0) s_sorted[m] = Choice{-INFINITY, at};
            ++m;
        }
    }
    __syncthreads();
    if (tid < n) s_beam[tid] = (int)(s_sorted[tid].at / (uint32_t)a.io.vocab);
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
        a.io.out_scores[out] = (float)s_sorted[tid].score;
        a.io.out_tokens[out] = (int)(s_sorted[tid].at % (uint32_t)a.io.vocab);
        a.io.out_rows[out] = g * K + beam;
    }
}

// Segments per row: about four CTAs for every SM, none smaller than a tile, and no
// more lists than the join takes.
int segments_of(int groups, int beams, int vocab, int num, const DeviceInfo& dev) {
    const long long rows = (long long)groups * beams;
    long long s = (8LL * dev.sm_count + rows - 1) / rows;
    const long long tiles = (vocab + kTile - 1) / kTile;
    if (s > tiles) s = tiles;
    if (s > kJoinEntries / (beams * num)) s = kJoinEntries / (beams * num);
    if (s > kJoinParts / beams) s = kJoinParts / beams;
    return s < 1 ? 1 : (int)s;
}

size_t parts_bytes(size_t parts) { return (parts * sizeof(Part) + 255) & ~size_t(255); }

}  // namespace

size_t beam_select_workspace_bytes(int groups, int beams, int vocab, int num, const DeviceInfo& dev) {
    const size_t parts = (size_t)groups * beams * segments_of(groups, beams, vocab, num, dev);
    return parts_bytes(parts) + parts * num * sizeof(uint64_t);
}

cudaError_t launch_beam_select(const BeamSelectIO& io, const DeviceInfo& dev, cudaStream_t stream) {
    const int S = segments_of(io.groups, io.beams, io.vocab, io.num, dev);
    const size_t parts = (size_t)io.groups * io.beams * S;
    Part* p = static_cast<Part*>(io.workspace);
    uint64_t* lists = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(io.workspace) + parts_bytes(parts));
    const RowsArgs r{io, S, p, lists};
    if (io.bf16) kda_beam_rows_kernel<true><<<(unsigned)parts, kThreads, 0, stream>>>(r);
    else kda_beam_rows_kernel<false><<<(unsigned)parts, kThreads, 0, stream>>>(r);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const JoinArgs j{io, S, p, lists};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)io.groups);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kda_beam_join_kernel, j);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
