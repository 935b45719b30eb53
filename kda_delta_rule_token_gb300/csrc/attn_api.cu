// Host side of the C ABI declared in include/kda_attn.h: argument
// validation, device checks, launch and error reporting of the paged
// softmax-attention operators.  No allocation happens on the per-call path;
// kda_attn_create allocates the 16-byte kernel error word.
//
// KDA_FAULT_INJECT, read once by kda_attn_create, replaces the launches of
// the entry points it names ("attn_plan", "attn_append", "attn_decode",
// "attn_prefill", or "all") by the error cudaErrorLaunchFailure.  The name
// "attn_drop" (not part of "all") instead makes every CTA of the attention
// kernels leave out its first copy of keys, so that a bounded wait inside the
// kernel runs out.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "attn_internal.cuh"

struct kda_attn_ctx {
    kda::AttnLayer layer;
    kda::AttnMaps maps;
    kda::RopeTurns turns;
    kda::DeviceInfo dev;
    int* err_word;
    unsigned inject;
};

namespace kda {
namespace {

constexpr unsigned kInjectPlan = 1u, kInjectAppend = 2u, kInjectDecode = 4u, kInjectPrefill = 8u, kInjectDrop = 16u;

unsigned parse_inject(const char* v) {
    unsigned m = 0u;
    for (const char* p = v; p && *p;) {
        const char* e = p;
        while (*e && *e != ',') ++e;
        const size_t n = (size_t)(e - p);
        auto is = [&](const char* w) { return std::strlen(w) == n && std::strncmp(p, w, n) == 0; };
        if (is("attn_plan")) m |= kInjectPlan;
        else if (is("attn_append")) m |= kInjectAppend;
        else if (is("attn_decode")) m |= kInjectDecode;
        else if (is("attn_prefill")) m |= kInjectPrefill;
        else if (is("attn_drop")) m |= kInjectDrop;
        else if (is("all")) m |= kInjectPlan | kInjectAppend | kInjectDecode | kInjectPrefill;
        p = *e ? e + 1 : e;
    }
    return m;
}

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

kda_status cuda_failed(const char* what, cudaError_t e) {
    set_error_text("%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return KDA_ERR_CUDA;
}

kda_status check_device(const kda_attn_ctx* ctx) {
    int cur = -1;
    const cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return cuda_failed("cudaGetDevice", e);
    if (cur != ctx->dev.device) {
        set_error_text("current device %d is not the context's device %d", cur, ctx->dev.device);
        return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

// The launch, or the injected failure in its place, as a status.
template <typename F>
kda_status launched(const kda_attn_ctx* ctx, unsigned what, const char* name, F&& launch) {
    if (const kda_status d = check_device(ctx); d != KDA_OK) return d;
    if (ctx->inject & what) {
        set_error_text("%s: %s (injected by KDA_FAULT_INJECT; nothing launched)", name,
                       cudaGetErrorName(cudaErrorLaunchFailure));
        return KDA_ERR_CUDA;
    }
    const cudaError_t e = launch();
    return e == cudaSuccess ? KDA_OK : cuda_failed(name, e);
}

kda_status need_cache(const kda_attn_ctx* ctx) {
    if (ctx->layer.num_pages > 0) return KDA_OK;
    set_error_text("no cache bound (kda_attn_bind_cache)");
    return KDA_ERR_INVALID_ARG;
}

// The two attention kernels' shares, the few-row one's first.
size_t workspace_bytes_of(const kda_attn_ctx* ctx) {
    return attn_decode_workspace_bytes(ctx->dev) + attn_prefill_workspace_bytes(ctx->dev);
}

// What kda_attn_decode and kda_attn_prefill check alike.
kda_status check_attend(const kda_attn_ctx* ctx, const AttnIO& io, size_t workspace_bytes) {
    if (!io.q || !io.block_table || io.max_pages < 1 || !io.kv_lens || !io.o || !io.workspace)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(io.q, 16) || !aligned(io.o, 16) || !aligned(io.gate, 16) || !aligned(io.workspace, 16) ||
        !aligned(io.block_table, 4) || !aligned(io.kv_lens, 4) || !aligned(io.lse, 4) || !aligned(io.cu_new, 4))
        return KDA_ERR_ALIGNMENT;
    if ((long long)io.max_pages * ctx->layer.page_size > 0x7fff0000LL) {   // tile ends stay within an int
        set_error_text("max_pages (%d) pages of %d tokens exceed 2^31 - 2^16 keys", io.max_pages, ctx->layer.page_size);
        return KDA_ERR_INVALID_ARG;
    }
    if (workspace_bytes < workspace_bytes_of(ctx)) {
        set_error_text("workspace of %zu bytes, %zu needed", workspace_bytes,
                       workspace_bytes_of(ctx));
        return KDA_ERR_INVALID_ARG;
    }
    return need_cache(ctx);
}

}  // namespace
}  // namespace kda

using kda::aligned;

extern "C" {

kda_status kda_attn_create(const kda_attn_config* cfg, const double* inv_freq, const float* q_gamma,
                           const float* k_gamma, const float* k_scale, const float* v_scale, kda_attn_ctx** out) {
    if (!out) return KDA_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg) return KDA_ERR_INVALID_ARG;
    if (cfg->num_q_heads < 1 || cfg->num_kv_heads < 1 || cfg->num_q_heads % cfg->num_kv_heads) {
        kda::set_error_text("num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)", cfg->num_q_heads,
                            cfg->num_kv_heads);
        return KDA_ERR_INVALID_ARG;
    }
    if (!(cfg->rms_eps >= 0.f) || !std::isfinite(cfg->rms_eps) || !(cfg->softmax_scale > 0.f) ||
        !std::isfinite(cfg->softmax_scale))
        return KDA_ERR_INVALID_ARG;
    if (cfg->cache_type != KDA_CACHE_BF16 && cfg->cache_type != KDA_CACHE_E4M3) return KDA_ERR_INVALID_ARG;
    if (cfg->rotary_dim < 0 || cfg->rotary_dim > kda::kHeadDim || cfg->rotary_dim % 16) {
        kda::set_error_text("rotary_dim (%d) must be a multiple of 16 from 0 to %d", cfg->rotary_dim, kda::kHeadDim);
        return KDA_ERR_INVALID_ARG;
    }
    if (cfg->rotary_dim && !inv_freq) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < cfg->rotary_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i])) return KDA_ERR_INVALID_ARG;
    const bool e4m3 = cfg->cache_type == KDA_CACHE_E4M3;
    if (e4m3 && (!k_scale || !v_scale)) {
        kda::set_error_text("an e4m3 cache needs k_scale and v_scale");
        return KDA_ERR_INVALID_ARG;
    }
    if (!aligned(q_gamma, 16) || !aligned(k_gamma, 16) || (e4m3 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return KDA_ERR_ALIGNMENT;
    int shift = 4;
    while (shift < 7 && (1 << shift) != cfg->page_size) ++shift;
    if (cfg->head_dim != kda::kHeadDim || (1 << shift) != cfg->page_size ||
        cfg->num_q_heads / cfg->num_kv_heads > 128) {
        kda::set_error_text("head_dim %d (128), page_size %d (16, 32, 64, 128), %d query heads per key head (at most 128)",
                            cfg->head_dim, cfg->page_size, cfg->num_q_heads / cfg->num_kv_heads);
        return KDA_ERR_UNSUPPORTED;
    }

    kda::DeviceInfo dev{};
    if (const kda_status s = kda::query_device(dev); s != KDA_OK) return s;
    kda_attn_ctx* c = new (std::nothrow) kda_attn_ctx{};
    if (!c) {
        kda::set_error_text("host allocation of the context failed");
        return KDA_ERR_INVALID_ARG;
    }
    kda::AttnLayer& l = c->layer;
    l.Hq = cfg->num_q_heads;
    l.Hkv = cfg->num_kv_heads;
    l.G = l.Hq / l.Hkv;
    l.page_size = cfg->page_size;
    l.page_shift = shift;
    l.e4m3 = e4m3;
    l.rotary = cfg->rotary_dim;
    l.interleaved = cfg->rope_interleaved != 0;
    l.rms_eps = cfg->rms_eps;
    l.softmax_scale = cfg->softmax_scale;
    l.q_gamma = q_gamma;
    l.k_gamma = k_gamma;
    l.k_scale = e4m3 ? k_scale : nullptr;
    l.v_scale = e4m3 ? v_scale : nullptr;
    for (int i = 0; i < cfg->rotary_dim / 2; ++i) {
        // Fraction of a turn per position, in units of 2^-64 (the product with
        // 2^64 in two exact halves: a double holds 53 bits of it).
        const double turns = inv_freq[i] / 6.283185307179586476925286766559;
        const double frac = turns - std::floor(turns);
        const double hi = std::floor(frac * 4294967296.0);
        const double lo = (frac * 4294967296.0 - hi) * 4294967296.0;
        c->turns.turn[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
    }
    c->dev = dev;
    c->inject = kda::parse_inject(std::getenv("KDA_FAULT_INJECT"));
    cudaError_t e = cudaMalloc(&c->err_word, 16);
    if (e != cudaSuccess) {
        delete c;
        return kda::cuda_failed("cudaMalloc(error word)", e);
    }
    if ((e = cudaMemset(c->err_word, 0, 16)) != cudaSuccess) {
        cudaFree(c->err_word);
        delete c;
        return kda::cuda_failed("cudaMemset(error word)", e);
    }
    *out = c;
    return KDA_OK;
}

void kda_attn_destroy(kda_attn_ctx* ctx) {
    if (!ctx) return;
    if (ctx->err_word) cudaFree(ctx->err_word);
    delete ctx;
}

kda_status kda_attn_bind_cache(kda_attn_ctx* ctx, int num_pages, void* k_cache, void* v_cache) {
    if (!ctx || num_pages < 1 || !k_cache || !v_cache) return KDA_ERR_INVALID_ARG;
    if ((long long)num_pages * ctx->layer.Hkv > 0x7fffffffLL) {
        kda::set_error_text("num_pages (%d) * num_kv_heads (%d) exceeds 2^31 - 1", num_pages, ctx->layer.Hkv);
        return KDA_ERR_INVALID_ARG;
    }
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return KDA_ERR_ALIGNMENT;
    kda::AttnLayer l = ctx->layer;
    l.num_pages = num_pages;
    l.k_cache = k_cache;
    l.v_cache = v_cache;
    kda::AttnMaps maps;
    if (!kda::attn_decode_maps(l, maps) || !kda::attn_prefill_maps(l, maps)) {
        kda::set_error_text("cuTensorMapEncodeTiled failed for the cache");
        return KDA_ERR_CUDA;
    }
    ctx->layer = l;
    ctx->maps = maps;
    return KDA_OK;
}

kda_status kda_attn_plan(kda_attn_ctx* ctx, int B, int N, const int32_t* cache_lens, const int32_t* new_lens,
                         const int32_t* free_pages, int free_capacity, const int32_t* free_count,
                         int32_t* block_table, int max_pages, int32_t* cu_new, int32_t* kv_lens, int32_t* positions,
                         int64_t* slots, int32_t* info, void* stream) {
    if (!ctx || B < 0 || N < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;
    if (!cache_lens || !new_lens || free_capacity < 0 || (free_capacity && !free_pages) || !free_count ||
        !block_table || max_pages < 1 || !cu_new || !kv_lens || (N && (!positions || !slots)) || !info)
        return KDA_ERR_INVALID_ARG;
    const void* words[] = {cache_lens, new_lens, free_pages, free_count, block_table, cu_new, kv_lens, positions, info};
    for (const void* p : words)
        if (!aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    if (!aligned(slots, 8)) return KDA_ERR_ALIGNMENT;
    if ((long long)max_pages * ctx->layer.page_size > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (B > KDA_ATTN_MAX_PLAN_REQUESTS) {
        kda::set_error_text("%d requests in one plan, at most %d", B, KDA_ATTN_MAX_PLAN_REQUESTS);
        return KDA_ERR_UNSUPPORTED;
    }
    const kda::AttnPlanIO io{B, N, cache_lens, new_lens, free_pages, free_capacity, free_count, block_table,
                             max_pages, cu_new, kv_lens, positions, reinterpret_cast<long long*>(slots), info};
    return kda::launched(ctx, kda::kInjectPlan, "attn_plan launch", [&] {
        return kda::launch_attn_plan(ctx->layer, io, ctx->dev, static_cast<cudaStream_t>(stream));
    });
}

kda_status kda_attn_append(kda_attn_ctx* ctx, int N, const uint16_t* q, long long q_stride, const uint16_t* k,
                           long long k_stride, const uint16_t* v, long long v_stride, const int32_t* positions,
                           const int64_t* slots, uint16_t* q_out, void* stream) {
    if (!ctx || N < 0) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !positions || !slots || !q_out) return KDA_ERR_INVALID_ARG;
    const long long qd = (long long)ctx->layer.Hq * kda::kHeadDim, kd = (long long)ctx->layer.Hkv * kda::kHeadDim;
    if (q_stride < qd || k_stride < kd || v_stride < kd) {
        kda::set_error_text("token strides %lld, %lld, %lld below the heads' %lld, %lld, %lld elements", q_stride,
                            k_stride, v_stride, qd, kd, kd);
        return KDA_ERR_INVALID_ARG;
    }
    if (q == q_out && q_stride != qd) {
        kda::set_error_text("q_out is dense: q may be it only with a token stride of %lld elements", qd);
        return KDA_ERR_INVALID_ARG;
    }
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(q_out, 16) || !aligned(positions, 4) || !aligned(slots, 8))
        return KDA_ERR_ALIGNMENT;
    if (const kda_status s = kda::need_cache(ctx); s != KDA_OK) return s;
    const kda::AttnAppendIO io{N, q, k, v, q_stride, k_stride, v_stride, positions,
                               reinterpret_cast<const long long*>(slots), q_out};
    return kda::launched(ctx, kda::kInjectAppend, "attn_append launch", [&] {
        return kda::launch_attn_append(ctx->layer, ctx->turns, io, ctx->dev, ctx->err_word,
                                       static_cast<cudaStream_t>(stream));
    });
}

size_t kda_attn_workspace_bytes(const kda_attn_ctx* ctx) {
    return ctx ? kda::workspace_bytes_of(ctx) : 0;
}

kda_status kda_attn_decode(kda_attn_ctx* ctx, int B, const uint16_t* q, const int32_t* block_table, int max_pages,
                           const int32_t* kv_lens, const float* gate_logit, void* o, int o_f32, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!ctx || B < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;
    const kda::AttnIO io{B, B, nullptr, q, block_table, max_pages, kv_lens, gate_logit, o, o_f32 != 0, lse, workspace,
                         (ctx->inject & kda::kInjectDrop) ? 1 : 0};
    if (const kda_status s = kda::check_attend(ctx, io, workspace_bytes); s != KDA_OK) return s;
    return kda::launched(ctx, kda::kInjectDecode, "attn_decode launch", [&] {
        return kda::launch_attn_few_rows(ctx->layer, ctx->maps, io, ctx->dev, ctx->err_word,
                                         static_cast<cudaStream_t>(stream), false);
    });
}

kda_status kda_attn_prefill(kda_attn_ctx* ctx, int B, int N, const int32_t* cu_new, const uint16_t* q,
                            const int32_t* block_table, int max_pages, const int32_t* kv_lens,
                            const float* gate_logit, void* o, int o_f32, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (!ctx || B < 0 || N < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return KDA_OK;
    if (!cu_new) return KDA_ERR_INVALID_ARG;
    const kda::AttnIO io{B, N, cu_new, q, block_table, max_pages, kv_lens, gate_logit, o, o_f32 != 0, lse, workspace,
                         (ctx->inject & kda::kInjectDrop) ? 1 : 0};
    if (const kda_status s = kda::check_attend(ctx, io, workspace_bytes); s != KDA_OK) return s;
    return kda::launched(ctx, kda::kInjectPrefill, "attn_prefill launch", [&] {
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        const bool many = !kda::attn_few_rows(N, ctx->layer.G);   // else no request can have more rows
        const bool all = many && kda::attn_all_many(B, N, ctx->layer.G);
        if (many) {
            kda::AttnIO m = io;
            m.workspace = static_cast<uint8_t*>(workspace) + kda::attn_decode_workspace_bytes(ctx->dev);
            const cudaError_t e = kda::launch_attn_many_rows(ctx->layer, ctx->maps, m, ctx->dev, ctx->err_word, st, all);
            if (e != cudaSuccess || all) return e;
        }
        return kda::launch_attn_few_rows(ctx->layer, ctx->maps, io, ctx->dev, ctx->err_word, st, many);
    });
}

kda_status kda_attn_sync_status(kda_attn_ctx* ctx, void* stream) {
    if (!ctx) return KDA_ERR_INVALID_ARG;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return kda::cuda_failed("cudaStreamSynchronize", e);
    int word = 0;
    if ((e = cudaMemcpy(&word, ctx->err_word, sizeof(int), cudaMemcpyDeviceToHost)) != cudaSuccess)
        return kda::cuda_failed("cudaMemcpy(error word)", e);
    if (word == 0) return KDA_OK;
    const bool index = (word & ~kda::kErrAttnIndex) == 0;
    kda::set_error_text(index ? "kernel error word 0x%x (a page id or slot outside the cache, or row offsets that are not ascending)"
                              : "kernel error word 0x%x (bounded wait gave up)", word);
    if ((e = cudaMemset(ctx->err_word, 0, sizeof(int))) != cudaSuccess)
        return kda::cuda_failed("cudaMemset(error word)", e);
    return index ? KDA_ERR_INVALID_ARG : KDA_ERR_TIMEOUT;
}

}  // extern "C"
