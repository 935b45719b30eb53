/*
 * kda_attn.h -- C ABI of the paged softmax-attention operators that stand
 * beside the KDA token step (kda.h) in a hybrid model.
 *
 * A model that mixes KDA layers with softmax-attention layers keeps, for the
 * latter, the keys and values of every cached token.  This header serves one
 * such layer from a paged cache, for prompts and for single tokens:
 *
 *   kda_attn_plan     pages, block table, positions and cache slots of a step
 *                     from the requests' lengths (once per step, all layers)
 *   kda_attn_append   RMS norm of every q and k head, rotary position, k and v
 *                     into their cache slots
 *   kda_attn_decode   attention of one new token per request
 *   kda_attn_decode_shared  the same where groups of requests share a prefix,
 *                     whose keys are read once for all of them
 *   kda_attn_prefill  causal attention of a chunk of new tokens per request
 *   kda_attn_fork     pages shared, released and copied as requests take over
 *                     one another (beam search, samples of one prompt)
 *   kda_attn_copy_pages  those copies, in one layer's cache
 *
 * Heads are 128 wide (d).  Hq query heads share Hkv key/value heads, query
 * head h using key/value head h / (Hq / Hkv).
 *
 * The cache of one layer is two buffers, keys and values, each
 * [num_pages][Hkv][page_size][d], of bf16 or of e4m3 (with one fp32 scale per
 * key/value head: the value that a stored s stands for is s * scale).  A cache
 * slot is page * page_size + row.  Request b's key j lies in row
 * j % page_size of page block_table[b][j / page_size].
 *
 * Conventions are those of kda.h: device pointers unless said otherwise, work
 * on the caller's stream, no allocation and no synchronisation per call,
 * arguments checked on the host before any launch, one host thread per context
 * at a time, bounded waits, KDA_FAULT_INJECT (names "attn_plan",
 * "attn_append", "attn_decode", "attn_prefill", "attn_fork", "attn_copy_pages",
 * "attn_decode_shared"; "all" includes them; the name
 * "attn_drop", not part of "all", makes every CTA of the attention kernels leave
 * out its first copy of keys: the bounded waits on it run out and
 * kda_attn_sync_status reports KDA_ERR_TIMEOUT).
 *
 * What only the device knows (lengths, page ids, slots) is checked by the
 * kernels: nothing is read or written outside the buffers, and the cases that
 * are errors are noted in the context and reported by kda_attn_sync_status as
 * KDA_ERR_INVALID_ARG.
 */
#ifndef KDA_ATTN_H
#define KDA_ATTN_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kda_attn_ctx kda_attn_ctx;

/* Formats of the cached keys and values. */
enum { KDA_CACHE_BF16 = 0, KDA_CACHE_E4M3 = 1 };

/* Most requests of one kda_attn_plan or kda_attn_fork call. */
#define KDA_ATTN_MAX_PLAN_REQUESTS 16384

typedef struct kda_attn_config {
    int num_q_heads;       /* Hq >= 1 */
    int num_kv_heads;      /* Hkv >= 1, divides Hq; Hq / Hkv at most 128 */
    int head_dim;          /* d: 128 (others: KDA_ERR_UNSUPPORTED) */
    int page_size;         /* tokens of a page: 16, 32, 64 or 128 */
    int cache_type;        /* KDA_CACHE_BF16 or KDA_CACHE_E4M3 */
    int rotary_dim;        /* leading channels that are rotated: a multiple of 16, 0 to 128 */
    int rope_interleaved;  /* pairs (2i, 2i+1) if nonzero, else (i, i + rotary_dim / 2) */
    float rms_eps;         /* >= 0, finite */
    float softmax_scale;   /* > 0, finite */
} kda_attn_config;

/*
 * Create the context of one softmax-attention layer on the current device.
 *   inv_freq   HOST array of rotary_dim / 2 finite doubles: pair i turns by
 *              position * inv_freq[i] radians (copied; may be NULL when
 *              rotary_dim is 0).  The angle is reduced exactly: positions of
 *              31 bits keep full fp32 accuracy.
 *   q_gamma, k_gamma   [d] fp32 weights of the RMS norm, 16-byte aligned,
 *              borrowed; NULL: that side is not normalised
 *   k_scale, v_scale   [Hkv] fp32, positive, borrowed; required for
 *              KDA_CACHE_E4M3, ignored for KDA_CACHE_BF16
 */
KDA_API kda_status kda_attn_create(const kda_attn_config *cfg, const double *inv_freq,
                                   const float *q_gamma, const float *k_gamma,
                                   const float *k_scale, const float *v_scale, kda_attn_ctx **out);
KDA_API void kda_attn_destroy(kda_attn_ctx *ctx);

/*
 * Bind the layer's cache: two buffers of num_pages * Hkv * page_size * d
 * elements, 16-byte aligned, borrowed.  Rebinding replaces the previous
 * cache.  num_pages >= 1 and num_pages * Hkv below 2^31.  Launches nothing.
 */
KDA_API kda_status kda_attn_bind_cache(kda_attn_ctx *ctx, int num_pages, void *k_cache, void *v_cache);

/*
 * Plan one step of B requests.  Request b holds cache_lens[b] = c tokens and
 * brings new_lens[b] = n more; the N rows of the step's packed inputs are the
 * new tokens of request 0, 1, ....  With P = page_size it needs
 * ceil((c + n) / P) - ceil(c / P) new pages, taken from the END of the free
 * list in the order of requests and tokens: the i-th page taken is
 * free_pages[free_count - 1 - i].
 *
 * A request is admitted if c and n are not negative, its pages fit into
 * max_pages, its rows end within N, and the pages needed by it and the
 * fitting requests before it do not exceed free_count (a request that needs
 * none always meets this last condition).
 *
 *   cache_lens, new_lens  [B] int32 (in)
 *   free_pages  [free_capacity] int32 (in): a stack of unused page ids
 *   free_count  [1] int32 (in): its height (clamped to 0 .. free_capacity)
 *   block_table [B][max_pages] int32 (in, out): entries of the new pages of
 *               admitted requests are written, no other
 *   cu_new      [B + 1] int32 (out): row offsets, cu_new[0] = 0 (a negative n counts as 0)
 *   kv_lens     [B] int32 (out): c + n, or 0 for a request not admitted
 *   positions   [N] int32 (out): c + i for the i-th new token
 *   slots       [N] int64 (out): the token's cache slot, -1 for a request not admitted
 *               (a page id below 0, in the table or the free list, gives -2, which
 *               kda_attn_append reports)
 *   info        [4] int32 (out): new tokens of all requests (saturated at
 *               2^31 - 1), pages taken, pages left, requests not admitted
 * Rows past the last request's get position 0 and slot -1.  The first
 * free_count - info[1] pages of the list are still free: a caller that
 * carries on with count = info[2] needs no other bookkeeping.  No output may
 * alias an input other than block_table.  int32 arrays are 4-byte aligned,
 * slots 8-byte.  B == 0 or a null result is not launched: B == 0 is a no-op.
 * B above KDA_ATTN_MAX_PLAN_REQUESTS: KDA_ERR_UNSUPPORTED.
 */
KDA_API kda_status kda_attn_plan(kda_attn_ctx *ctx, int B, int N, const int32_t *cache_lens,
                                 const int32_t *new_lens, const int32_t *free_pages, int free_capacity,
                                 const int32_t *free_count, int32_t *block_table, int max_pages,
                                 int32_t *cu_new, int32_t *kv_lens, int32_t *positions, int64_t *slots,
                                 int32_t *info, void *stream);

/*
 * Norm, rotate and store the N new tokens of a step.  Per token and head, in
 * fp32: x <- x / sqrt(mean(x^2) + rms_eps) * gamma (q and k, where gamma was
 * given), then the rotation of q and k at the token's position; q is rounded
 * to bf16 once, k and v once to the cache's type (e4m3: x * (1 / scale),
 * clamped to +-448, to nearest even).
 *   q        [N][Hq][d] bf16, token stride q_stride elements (>= Hq * d, a multiple of 8)
 *   k, v     [N][Hkv][d] bf16, token strides k_stride, v_stride likewise
 *            (one fused projection's output serves all three); all 16-byte aligned
 *   positions [N] int32; slots [N] int64: -1 leaves that token's k and v
 *            unstored, any other value outside the cache is an error and stores nothing
 *   q_out    [N][Hq][d] bf16, dense; may be q itself when q is dense
 * Two tokens may not share a slot.  N == 0 is a no-op.
 */
KDA_API kda_status kda_attn_append(kda_attn_ctx *ctx, int N, const uint16_t *q, long long q_stride,
                                   const uint16_t *k, long long k_stride, const uint16_t *v,
                                   long long v_stride, const int32_t *positions, const int64_t *slots,
                                   uint16_t *q_out, void *stream);

/* Bytes of device workspace of kda_attn_fork. */
KDA_API size_t kda_attn_fork_workspace_bytes(const kda_attn_ctx *ctx, int B, int max_pages);

/*
 * Requests take over one another: request b goes on from the tokens of request
 * rows[b] (its own, or another's), for b = 0 .. B - 1; once per step, for all
 * layers.  With P = page_size and L = kv_lens[rows[b]]:
 *
 *   - new_table[b] gets the ceil(L / P) pages of rows[b]'s row and new_lens[b]
 *     gets L.  Full pages are shared by all requests that go on from rows[b].
 *   - A partly full last page stays with the first (lowest b) of these requests;
 *     every other one gets a page of its own, into which the rows that hold tokens
 *     are to be copied: copy_src[b], copy_dst[b], copy_rows[b] say from where,
 *     to where and how many, and kda_attn_copy_pages does it in every layer.
 *     copy_src[b] is -1 where nothing is to be copied.
 *   - A request that none goes on from lets go of its pages.  A page that nobody
 *     holds any more goes onto the free list's END: pages in the order of their
 *     place in the rows, pages of one place in the order of the requests (of the
 *     last one, where several let go of it).
 *   - The copies' pages come from the list's END, freed ones among them, in the
 *     order of the requests.  A request that finds none left is refused: new_lens[b]
 *     is 0 and it holds nothing.
 *
 *   rows        [B] int32 (in): 0 .. B - 1, or -1: request b is empty afterwards.  Any
 *               other value is an error and counts as -1.
 *   kv_lens     [B] int32 (in): tokens in the cache (clamped to 0 .. max_pages * P)
 *   block_table [B][max_pages] int32 (in); entries past a request's pages are not read
 *   page_refs   [num_pages of the bound cache] int32 (in, out): how many hold a page
 *               beside the first.  0 for a page that one request holds, and for a free
 *               one: all zero before the first fork, and kda_attn_plan has nothing to do
 *               with it.  Who holds a page outside of the block table (a prompt kept for
 *               later) adds 1.  A page is held at one and the same place of all rows that
 *               hold it, and a partly full one by one request.
 *   free_pages  [free_capacity] int32 (in, out), free_count [1] int32 (in): the stack, as
 *               for kda_attn_plan; entries from free_count on may be written.  free_count
 *               may be info + 2: a captured step carries on with what it left
 *   new_table   [B][max_pages] int32 (out), new_lens [B] int32 (out): not the old ones.
 *               Entries past a request's pages are not written.
 *   copy_src, copy_dst, copy_rows  [B] int32 (out)
 *   info        [4] int32 (out): pages freed, pages taken, pages left on the stack (carry
 *               on with free_count = info[2]), requests refused
 *   workspace   kda_attn_fork_workspace_bytes bytes, 16-byte aligned
 * int32 arrays are 4-byte aligned; no output may alias an input but those marked
 * (in, out), and info free_count.  A page id outside the cache is copied as it is and counted nowhere; it,
 * a page that more requests let go of than hold it, and a free list without room for
 * the freed pages that no copy takes (which are lost) are errors.  B == 0 is a no-op.  B above
 * KDA_ATTN_MAX_PLAN_REQUESTS: KDA_ERR_UNSUPPORTED.
 */
KDA_API kda_status kda_attn_fork(kda_attn_ctx *ctx, int B, const int32_t *rows, const int32_t *kv_lens,
                                 const int32_t *block_table, int max_pages, int32_t *page_refs,
                                 int32_t *free_pages, int free_capacity, const int32_t *free_count,
                                 int32_t *new_table, int32_t *new_lens, int32_t *copy_src, int32_t *copy_dst,
                                 int32_t *copy_rows, int32_t *info, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Copies the first rows[i] (clamped to 0 .. page_size) keys and values of page src[i],
 * all heads, to page dst[i], for i = 0 .. n - 1, in the bound cache.  src[i] == -1: nothing.
 * Any other page outside the cache is an error, and nothing is copied for that i.  No
 * destination may be a source, or a destination twice.  [n] int32 each, 4-byte
 * aligned.  n == 0 is a no-op.
 */
KDA_API kda_status kda_attn_copy_pages(kda_attn_ctx *ctx, int n, const int32_t *src, const int32_t *dst,
                                       const int32_t *rows, void *stream);

/* Bytes of device workspace that kda_attn_decode and kda_attn_prefill need,
 * whatever their sizes.  One workspace serves one call at a time. */
KDA_API size_t kda_attn_workspace_bytes(const kda_attn_ctx *ctx);

/*
 * Attention of one new token of each of B requests over its kv_lens[b] cached
 * keys (its own among them): o = softmax(softmax_scale * q K^T) V per head,
 * times sigmoid(gate_logit) where a gate is given.
 *   q           [B][Hq][d] bf16
 *   block_table [B][max_pages] int32; entries past a request's length are not read.
 *               A page id outside the cache reads as zeros and is an error.
 *   kv_lens     [B] int32 (clamped to 0 .. max_pages * page_size); 0: the
 *               request's o is zero, whatever its gate holds, and its lse -infinity
 *   gate_logit  [B][Hq][d] fp32, or NULL
 *   o           [B][Hq][d], bf16, or fp32 if o_f32 is nonzero (the input of kda_project_o)
 *   lse         [B][Hq] fp32 or NULL: ln of the sum of exp(softmax_scale * q.k);
 *               NaN where one of the row's logits is
 *   workspace   kda_attn_workspace_bytes bytes, 16-byte aligned
 * q, o and gate_logit 16-byte aligned, the others 4-byte.  What lies in the
 * cache past a request's length, or at keys that a row does not see, has no
 * effect on it, NaN and infinities among that.  A row that sees a NaN key is NaN;
 * one that sees a NaN or infinite value is NaN or infinite in that channel.
 * The result does not depend on the order in which parts of the work end.
 * B == 0 is a no-op.
 */
KDA_API kda_status kda_attn_decode(kda_attn_ctx *ctx, int B, const uint16_t *q, const int32_t *block_table,
                                   int max_pages, const int32_t *kv_lens, const float *gate_logit, void *o,
                                   int o_f32, float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* Bytes of device workspace of kda_attn_decode_shared for up to B requests. */
KDA_API size_t kda_attn_shared_workspace_bytes(const kda_attn_ctx *ctx, int B);

/*
 * kda_attn_decode where groups of requests have their first tokens in common
 * (beams, samples of one prompt: the block tables that kda_attn_fork makes).  Every
 * request's table row names all of its pages, as ever, and the results are
 * those of kda_attn_decode up to rounding; the groups say what need not be read more
 * than once.  What a group's rows per key head (requests * Hq / Hkv) decide is how the
 * softmax weights of its prefix are rounded: over a bf16 cache, in calls of more than 32 such
 * rows (B * Hq / Hkv), those of groups of more than 16 to bf16 once, as kda_attn_prefill
 * rounds them (2^-8 of each weight, o is off by up to that of the weighted sum of |v|);
 * all others as kda_attn_decode (2^-16, over an e4m3 cache 2^-11).
 *   groups      0 to B
 *   cu_groups   [groups + 1] int32, ascending from 0 or more to B or less: group g is
 *               requests cu_groups[g] to cu_groups[g + 1] - 1; requests of no group share
 *               nothing.  Other offsets are an error, and nothing is shared.
 *   prefix_lens [groups] int32: the first so many keys of the group's requests are the
 *               same keys.  The pages that they fill are read through the table row of any
 *               one request that has so many; a page that they fill in part counts as
 *               the request's own, and so do all keys of a request of fewer.
 *   workspace   kda_attn_shared_workspace_bytes bytes, 16-byte aligned
 * Otherwise as kda_attn_decode.  cu_groups and prefix_lens may be NULL if groups is 0.
 */
KDA_API kda_status kda_attn_decode_shared(kda_attn_ctx *ctx, int B, const uint16_t *q, const int32_t *block_table,
                                          int max_pages, const int32_t *kv_lens, int groups,
                                          const int32_t *cu_groups, const int32_t *prefix_lens,
                                          const float *gate_logit, void *o, int o_f32, float *lse,
                                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * Causal attention of the N packed new tokens of B requests, whose keys and
 * values are in the cache already (kda_attn_append): of request b's n =
 * cu_new[b + 1] - cu_new[b] tokens, the i-th sees keys 0 .. kv_lens[b] - n + i.
 * A row that sees no key gives o = 0, whatever its gate holds, and lse = -infinity.
 *   cu_new      [B + 1] int32, ascending; rows past cu_new[B] are not written.
 *               Offsets that claim rows more than once write some of them in no
 *               set order, or are an error and write none.
 *   q           [N][Hq][d] bf16;  gate_logit, o, lse: [N][Hq]... as for kda_attn_decode
 * Otherwise as kda_attn_decode.  B == 0 or N == 0 is a no-op.
 */
KDA_API kda_status kda_attn_prefill(kda_attn_ctx *ctx, int B, int N, const int32_t *cu_new, const uint16_t *q,
                                    const int32_t *block_table, int max_pages, const int32_t *kv_lens,
                                    const float *gate_logit, void *o, int o_f32, float *lse, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* As kda_sync_status: KDA_ERR_TIMEOUT if a bounded wait gave up,
 * KDA_ERR_INVALID_ARG if a kernel met a page id or slot outside the cache, row
 * offsets that are not ascending, or one of kda_attn_fork's errors. */
KDA_API kda_status kda_attn_sync_status(kda_attn_ctx *ctx, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H */
