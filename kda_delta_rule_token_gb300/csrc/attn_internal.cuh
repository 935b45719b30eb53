// Internal declarations of the paged softmax-attention operators
// (include/kda_attn.h): what the host side hands to their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn.h"
#include "kda_internal.cuh"

namespace kda {

// Error-word bits of the attention context beside the bounded-wait ones of
// ptx.cuh: a page id or slot outside the cache was met (and not accessed), row
// offsets that claim rows more than once (and nothing was done), or a page that
// more requests let go of than held it.
constexpr int kErrAttnIndex = 1 << 16;

// One layer as its kernels see it.
struct AttnLayer {
    int Hq, Hkv, G;          // G = Hq / Hkv
    int page_size, page_shift;
    int e4m3;
    int rotary, interleaved;
    float rms_eps, softmax_scale;
    const float* q_gamma;    // may be null
    const float* k_gamma;    // may be null
    const float* k_scale;    // e4m3 only
    const float* v_scale;    // e4m3 only
    int num_pages;           // 0: no cache bound
    void* k_cache;
    void* v_cache;
};

// Tensor maps of the bound cache (attn_tma.cuh): boxes of the decode's warp
// tiles, and of whole pages for prompts.
struct AttnMaps {
    CUtensorMap k_decode, v_decode;
    CUtensorMap k_prefill, v_prefill;
};

// Rotation steps: pair i advances by turn[i] / 2^64 of a full turn per
// position, so position * turn[i] modulo 2^64 is the exact fraction of a turn.
struct RopeTurns {
    uint64_t turn[kHeadDim / 2];
};

struct AttnPlanIO {
    int B, N;
    const int* cache_lens;
    const int* new_lens;
    const int* free_pages;
    int free_capacity;
    const int* free_count;
    int* block_table;
    int max_pages;
    int* cu_new;
    int* kv_lens;
    int* positions;
    long long* slots;
    int* info;
};

struct AttnAppendIO {
    int N;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;
    const int* positions;
    const long long* slots;
    uint16_t* q_out;
};

struct AttnForkIO {
    int B;
    const int* rows;
    const int* kv_lens;
    const int* block_table;
    int max_pages;
    int* page_refs;
    int* free_pages;
    int free_capacity;
    const int* free_count;
    int* new_table;
    int* new_lens;
    int* copy_src;
    int* copy_dst;
    int* copy_rows;
    int* info;
    void* workspace;
};

struct AttnCopyIO {
    int n;
    const int* src;
    const int* dst;
    const int* rows;
};

struct AttnIO {
    int B, N;                // decode: N = B
    const int* cu_new;       // prefill; null for decode (one token each)
    const uint16_t* q;
    const int* block_table;
    int max_pages;
    const int* kv_lens;
    const float* gate;       // may be null
    void* o;
    int o_f32;
    float* lse;              // may be null
    void* workspace;
    // Test injection (KDA_FAULT_INJECT "attn_drop"): every CTA leaves out
    // its first copy of keys, so that a bounded wait runs out.
    int drop;
    // Groups of requests that share a prefix (attn_shared.cu; the many-row kernel alone):
    // B groups, whose members cu_new has, and whose single tokens see all of a prefix.
    const int* group_len;            // [B] keys of the prefix
    const int* group_row;            // [B] the block table's row that has its pages
    const long long* group_start;    // [B + 1] units of work before the group's, none for one that is not its own
    const int* group_pairs;          // [B] pairs of token tiles before the group's
    int2* parts;                     // [pairs][Hkv] (out) first part's slot, -1 if there is but one, and last part's
    // Offsets of groups that the few-row kernel's join looks over: kda_attn_decode_shared where it passes over them.
    int check_groups;
    const int* check_cu;             // [check_groups + 1]
};

// Whether group g's requests are none that there are, or out of order.
__device__ __forceinline__ bool bad_offsets(const int* cu, int g, int B) {
    return cu[g] < 0 || cu[g + 1] < cu[g] || cu[g + 1] > B;
}

struct AttnSharedIO {
    int B, groups;
    const int* cu_groups;
    const int* prefix_lens;
    const uint16_t* q;
    const int* block_table;
    int max_pages;
    const int* kv_lens;
    const float* gate;       // may be null
    void* o;
    int o_f32;
    float* lse;              // may be null
    void* workspace;
    int drop;
};

cudaError_t launch_attn_plan(const AttnLayer& l, const AttnPlanIO& io, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_attn_append(const AttnLayer& l, const RopeTurns& turns, const AttnAppendIO& io,
                               const DeviceInfo& dev, int* err_word, cudaStream_t stream);
size_t attn_fork_workspace_bytes(int B, int max_pages);
cudaError_t launch_attn_fork(const AttnLayer& l, const AttnForkIO& io, const DeviceInfo& dev, int* err_word,
                             cudaStream_t stream);
cudaError_t launch_attn_copy_pages(const AttnLayer& l, const AttnCopyIO& io, int* err_word, cudaStream_t stream);
// The bound cache's tensor maps; false if they cannot be encoded.
bool attn_decode_maps(const AttnLayer& l, AttnMaps& maps);
bool attn_prefill_maps(const AttnLayer& l, AttnMaps& maps);
// attn_decode.cu: every request of one token (cu_new null), or those of
// attn_few_rows (the others are left alone), and the zero rows of requests
// without keys.  attn_prefill.cu: the remaining requests of a call, or (`all`)
// all of them.
size_t attn_decode_workspace_bytes(const DeviceInfo& dev);
size_t attn_prefill_workspace_bytes(const DeviceInfo& dev);
// `beside`: the few-row kernel may start beside the launches before it, the
// many-row ones of the same call (it shares nothing with them but their inputs,
// and ends after them).
cudaError_t launch_attn_few_rows(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev,
                                 int* err_word, cudaStream_t stream, bool beside);
cudaError_t launch_attn_many_rows(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io, const DeviceInfo& dev,
                                  int* err_word, cudaStream_t stream, bool all);

// The prefixes of kda_attn_decode_shared in the many-row kernel: group g's segments of
// up to 2 * (128 / G) tokens and a key head, each of ceil(len / 128) + attn_many_rows_cost
// units, dealt in equal ranges to min(SMs, units) CTAs.  A segment that one CTA has
// whole goes to o and lse, others' parts to the slots, two of 256 rows per CTA: the
// first part's, then the first slot of each CTA behind it.
int attn_many_rows_cost(const AttnLayer& l);
float* attn_many_rows_slots(void* workspace, const DeviceInfo& dev);
cudaError_t launch_attn_many_rows_shared(const AttnLayer& l, const AttnMaps& maps, const AttnIO& io,
                                         const DeviceInfo& dev, int* err_word, cudaStream_t stream);
// All of kda_attn_decode_shared (attn_shared.cu).
size_t attn_shared_workspace_bytes(const AttnLayer& l, int B, const DeviceInfo& dev);
cudaError_t launch_attn_shared(const AttnLayer& l, const AttnMaps& maps, const AttnSharedIO& io, const DeviceInfo& dev,
                               int* err_word, cudaStream_t stream);

// Which of the two takes a request of n new tokens and G query heads per key
// head: up to 32 rows fit two 16-row warp tiles, whose kernel streams the
// cache at HBM rate; 128-row tensor-memory tiles pay from there on.
constexpr int kAttnFewRows = 32;
__host__ __device__ __forceinline__ bool attn_few_rows(int n, int G) {
    return n <= 1 || (long long)n * G <= kAttnFewRows;
}

// Whether a call of B requests and N tokens is left to the many-row kernel as
// a whole, which saves the two launches of the few-row one (6 us of a 512-token
// prompt's 25 us).  The host knows the requests' mean length only: from 512
// rows on, few-row requests among them are a small part of the work (on their
// own they run up to 1.5 times longer there in e4m3, the same in bf16).
inline bool attn_all_many(int B, int N, int G) { return B == 1 || (long long)N * G >= 512LL * B; }

#ifdef __CUDACC__
__device__ __forceinline__ int attn_kv_len(const AttnIO& io, int b, int page_shift) {
    return min(max(io.kv_lens[b], 0), io.max_pages << page_shift);
}

// Request b's rows of the packed inputs (offsets clamped to the N rows there are).
__device__ __forceinline__ void attn_tokens(const AttnIO& io, int b, int& tok0, int& n) {
    tok0 = min(max(io.cu_new[b], 0), io.N);
    n = max(min(max(io.cu_new[b + 1], 0), io.N) - tok0, 0);
}
#endif

}  // namespace kda
