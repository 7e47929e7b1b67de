// ha_serve_api.cu -- the C entry points of the serving operators (include/hyper_attn.h, "serving"): argument checks
// and launches. Nothing is allocated, copied or waited for, so that every call can be captured into a graph.
#include <cmath>
#include <new>

#include "ha_handle.h"

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

int esize(hyper_attn_t h) { return h->opt.dtype == HA_DTYPE_BF16 ? 2 : 4; }
int out_type(hyper_attn_t h) { return h->opt.out_dtype < 0 ? h->opt.dtype : h->opt.out_dtype; }

// No C++ exception leaves a C entry point: the error text is the only thing here that allocates host memory.
template <typename F>
int guarded(hyper_attn_t h, F &&f) {
    if (!h) return HA_ERR_INVALID_ARG;
    try {
        h->err.clear();
        DeviceGuard g(h->device);
        return f();
    } catch (...) {
        return HA_ERR_OOM;
    }
}

int check_heads(hyper_attn_t h, int heads, int kv_heads, int d) {
    if (d != 64 && d != 128) return fail(h, HA_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d);
    if (heads <= 0 || kv_heads <= 0) return fail(h, HA_ERR_INVALID_ARG, "heads and kv_heads must be positive");
    if (heads % kv_heads) return fail(h, HA_ERR_INVALID_ARG, "heads (%d) must be a multiple of kv_heads (%d)", heads, kv_heads);
    if (heads / kv_heads > 128)
        return fail(h, HA_ERR_UNSUPPORTED, "at most 128 query heads share a key head (got %d)", heads / kv_heads);
    if (heads > 65536) return fail(h, HA_ERR_UNSUPPORTED, "at most 65536 heads (got %d)", heads);
    return HA_OK;
}

// Strides of a [tokens, heads, d] tensor. A dimension of one element has no stride: it gets one that fits.
int check_strides(hyper_attn_t h, const char *what, int64_t tokens, int heads, int d, int esz, int64_t *token, int64_t *head,
                  bool written) {
    if (heads == 1) *head = d;
    if (tokens == 1) *token = static_cast<int64_t>(heads) * (*head > d ? *head : d);
    const int64_t unit = 16 / esz, most = int64_t(1) << 36;
    if (*token < d || *head < d || *token % unit || *head % unit || *token > most || *head > most)
        return fail(h, HA_ERR_INVALID_ARG, "%s: strides must be at least d, of 16-byte multiples (got %lld, %lld)", what,
                    (long long)*token, (long long)*head);
    if (*token > (int64_t(1) << 62) / tokens || *head > (int64_t(1) << 62) / heads)
        return fail(h, HA_ERR_INVALID_ARG, "%s: strides too large", what);
    if (written && *token < (heads - 1) * *head + d && *head < (tokens - 1) * *token + d)
        return fail(h, HA_ERR_INVALID_ARG, "%s: rows overlap", what);
    return HA_OK;
}

int pick_family(hyper_attn_t h, bool *tc) {
    *tc = h->opt.kernel != HA_KERNEL_SIMT && h->opt.dtype == HA_DTYPE_BF16;
    if (h->opt.kernel == HA_KERNEL_TC && h->opt.dtype != HA_DTYPE_BF16)
        return fail(h, HA_ERR_UNSUPPORTED, "tensor-core kernels need bf16 inputs");
    return HA_OK;
}

int check_cache(hyper_attn_t h, const ha_cache *c, ha::ServeCache *out) {
    if (!c) return fail(h, HA_ERR_INVALID_ARG, "null cache");
    if (c->d != 64 && c->d != 128) return fail(h, HA_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", c->d);
    int shift = 4;
    while (shift < 8 && (1 << shift) != c->page) ++shift;
    if ((1 << shift) != c->page) return fail(h, HA_ERR_UNSUPPORTED, "pages have 16, 32, 64, 128 or 256 rows (got %d)", c->page);
    if (c->layers < 1 || c->layers > 16384 || c->pages < 1 || c->pages > 0x7fffffff || c->slots < 1 ||
        c->slots > 0x7fffffff || c->max_pages < 1 || c->max_pages > kMaxTokens / c->page || c->kv_heads < 1 ||
        c->kv_heads > 65536)
        return fail(h, HA_ERR_INVALID_ARG, "cache sizes out of range");
    if (!c->k || !c->v || !c->table || !c->lens || !c->held || !c->refs) return fail(h, HA_ERR_INVALID_ARG, "null cache pointer");
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->refs))
        return fail(h, HA_ERR_INVALID_ARG, "the cache's k, v and refs must be 16-byte aligned");
    *out = {c->k, c->v, c->table, c->lens, c->held, c->refs, c->layers, c->pages, c->slots, c->max_pages,
            c->kv_heads, c->page, shift, c->d};
    return HA_OK;
}

int check_count(hyper_attn_t h, int64_t n, int64_t most = 16384) {
    if (n < 0 || n > most) return fail(h, HA_ERR_INVALID_ARG, "n must lie in [0, %lld] (got %lld)", (long long)most, (long long)n);
    return HA_OK;
}

int launched(hyper_attn_t h, int k, const char *what) {
    if (k == -2) return fail(h, HA_ERR_UNSUPPORTED, "%s: sizes or strides that this kernel does not take", what);
    if (k < 0) return fail(h, HA_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(cudaGetLastError()));
    h->last_launches = k;
    return HA_OK;
}

}  // namespace

extern "C" {

int hyper_attn_capturing(hyper_attn_t h) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (!h || cudaStreamIsCapturing(static_cast<cudaStream_t>(h->opt.stream), &s) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return s != cudaStreamCaptureStatusNone;
}

size_t hyper_attn_prompt_workspace(hyper_attn_t h, int64_t tokens, int64_t seqs, int64_t max_len, int heads, int kv_heads) {
    if (!h || tokens < 0 || seqs < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads) return 0;
    const bool tc = h->opt.kernel != HA_KERNEL_SIMT && h->opt.dtype == HA_DTYPE_BF16;
    return ha::serve_prompt_workspace(tc, tokens, seqs, max_len, kv_heads, heads / kv_heads, h->sms);
}

int hyper_attn_prompt(hyper_attn_t h, const ha_prompt_args *p) {
    return guarded(h, [&]() -> int {
        if (!p) return fail(h, HA_ERR_INVALID_ARG, "null arguments");
        int rc = check_heads(h, p->heads, p->kv_heads, p->d);
        if (rc) return rc;
        if (p->tokens < 0 || p->tokens > kMaxTokens) return fail(h, HA_ERR_INVALID_ARG, "tokens must lie in [0, 2^30]");
        if (p->seqs < 0 || p->seqs > (1 << 20)) return fail(h, HA_ERR_INVALID_ARG, "seqs must lie in [0, 2^20]");
        if (p->max_len < 1) return fail(h, HA_ERR_INVALID_ARG, "max_len must be positive");
        if (!(p->scale > 0.f) || std::isinf(p->scale)) return fail(h, HA_ERR_INVALID_ARG, "scale must be positive and finite");
        bool tc;
        if ((rc = pick_family(h, &tc))) return rc;
        h->last_launches = 0;
        h->last_kernel = tc ? HA_KERNEL_TC : HA_KERNEL_SIMT;
        if (p->tokens == 0 || p->seqs == 0) return HA_OK;
        if (!p->q || !p->k || !p->v || !p->o || !p->offsets) return fail(h, HA_ERR_INVALID_ARG, "null tensor pointer");
        if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->o))
            return fail(h, HA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
        const int ei = esize(h), eo = out_type(h) == HA_DTYPE_BF16 ? 2 : 4;
        ha::ServeArgs a{};
        a.q = p->q; a.k = p->k; a.v = p->v; a.o = p->o; a.lse = p->lse;
        a.q_tok = p->q_token; a.q_head = p->q_head; a.k_tok = p->k_token; a.k_head = p->k_head;
        a.v_tok = p->v_token; a.v_head = p->v_head; a.o_tok = p->o_token; a.o_head = p->o_head;
        if ((rc = check_strides(h, "q", p->tokens, p->heads, p->d, ei, &a.q_tok, &a.q_head, false))) return rc;
        if ((rc = check_strides(h, "k", p->tokens, p->kv_heads, p->d, ei, &a.k_tok, &a.k_head, false))) return rc;
        if ((rc = check_strides(h, "v", p->tokens, p->kv_heads, p->d, ei, &a.v_tok, &a.v_head, false))) return rc;
        if ((rc = check_strides(h, "o", p->tokens, p->heads, p->d, eo, &a.o_tok, &a.o_head, true))) return rc;
        if (p->o == p->q || p->o == p->k || p->o == p->v) return fail(h, HA_ERR_INVALID_ARG, "O must not alias Q, K or V");
        const size_t need = ha::serve_prompt_workspace(tc, p->tokens, p->seqs, p->max_len, p->kv_heads, p->heads / p->kv_heads, h->sms);
        if (need && (!p->workspace || !aligned16(p->workspace) || p->workspace_bytes < need))
            return fail(h, HA_ERR_INVALID_ARG, "workspace of %zu bytes needed, 16-byte aligned", need);
        a.tokens = p->tokens;
        a.heads = p->heads; a.kv_heads = p->kv_heads; a.group = p->heads / p->kv_heads; a.d = p->d;
        a.cu = p->offsets;
        a.seqs = static_cast<int>(p->seqs);
        a.max_len = static_cast<int>(p->max_len < p->tokens ? p->max_len : p->tokens);
        a.scale = p->scale;
        a.out_dtype = out_type(h);
        a.status = h->serve_status;
        a.ws = p->workspace;
        a.sms = h->sms;
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_PROMPT, "ha:prompt", st);
        const int k = tc ? ha::launch_prompt_tc(a, st) : ha::launch_prompt_simt(a, h->opt.dtype, st);
        prof.end(k);
        return launched(h, k, "prompt attention");
    });
}

size_t hyper_attn_tree_workspace(hyper_attn_t h, int d) {
    if (!h || (d != 64 && d != 128)) return 0;
    return ha::serve_tree_workspace(h->sms, d);
}

int hyper_attn_tree(hyper_attn_t h, const ha_cache *cache, const ha_tree_args *p) {
    return guarded(h, [&]() -> int {
        if (!p) return fail(h, HA_ERR_INVALID_ARG, "null arguments");
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc) return rc;
        if ((rc = check_heads(h, p->heads, c.kv_heads, c.d))) return rc;
        if (p->tokens < 0 || p->tokens > kMaxTokens) return fail(h, HA_ERR_INVALID_ARG, "tokens must lie in [0, 2^30]");
        if (p->seqs < 0 || p->seqs > 65536) return fail(h, HA_ERR_INVALID_ARG, "seqs must lie in [0, 65536]");
        if (p->max_draft < 1 || p->max_draft > 64) return fail(h, HA_ERR_INVALID_ARG, "max_draft must lie in [1, 64]");
        if (p->layer < 0 || p->layer >= c.layers) return fail(h, HA_ERR_INVALID_ARG, "layer out of range");
        if (!(p->scale > 0.f) || std::isinf(p->scale)) return fail(h, HA_ERR_INVALID_ARG, "scale must be positive and finite");
        bool tc;
        if ((rc = pick_family(h, &tc))) return rc;
        h->last_launches = 0;
        h->last_kernel = tc ? HA_KERNEL_TC : HA_KERNEL_SIMT;
        if (p->tokens == 0 || p->seqs == 0) return HA_OK;
        if (!p->q || !p->o || !p->offsets) return fail(h, HA_ERR_INVALID_ARG, "null tensor pointer");
        if (!aligned16(p->q) || !aligned16(p->o))
            return fail(h, HA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
        const int ei = esize(h), eo = out_type(h) == HA_DTYPE_BF16 ? 2 : 4;
        ha::ServeArgs a{};
        a.q = p->q; a.o = p->o; a.lse = p->lse;
        a.q_tok = p->q_token; a.q_head = p->q_head; a.o_tok = p->o_token; a.o_head = p->o_head;
        if ((rc = check_strides(h, "q", p->tokens, p->heads, c.d, ei, &a.q_tok, &a.q_head, false))) return rc;
        if ((rc = check_strides(h, "o", p->tokens, p->heads, c.d, eo, &a.o_tok, &a.o_head, true))) return rc;
        if (p->o == p->q) return fail(h, HA_ERR_INVALID_ARG, "O must not alias Q");
        const size_t need = ha::serve_tree_workspace(h->sms, c.d);
        if (!p->workspace || !aligned16(p->workspace) || p->workspace_bytes < need)
            return fail(h, HA_ERR_INVALID_ARG, "workspace of %zu bytes needed, 16-byte aligned", need);
        a.tokens = p->tokens;
        a.heads = p->heads; a.kv_heads = c.kv_heads; a.group = p->heads / c.kv_heads; a.d = c.d;
        a.cu = p->offsets;
        a.seqs = static_cast<int>(p->seqs);
        a.max_len = p->max_draft;
        a.scale = p->scale;
        a.out_dtype = out_type(h);
        a.status = h->serve_status;
        const int64_t layer_bytes = c.pages * c.kv_heads * c.page * static_cast<int64_t>(c.d) * ei;
        a.kp = static_cast<const char *>(c.k) + p->layer * layer_bytes;
        a.vp = static_cast<const char *>(c.v) + p->layer * layer_bytes;
        a.slots = p->slots;
        a.mask = p->mask;
        a.table = c.table; a.lens = c.lens; a.held = c.held;
        a.pages = c.pages; a.max_slots = c.slots; a.max_pages = c.max_pages;
        a.page_shift = c.page_shift;
        a.ws = p->workspace;
        a.sms = h->sms;
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_TREE, "ha:tree", st);
        const int k = tc ? ha::launch_tree_tc(a, st) : ha::launch_tree_simt(a, h->opt.dtype, st);
        prof.end(k);
        return launched(h, k, "tree attention");
    });
}

int hyper_attn_cache_free(hyper_attn_t h, const ha_cache *cache, const int32_t *slots, int64_t n) {
    return guarded(h, [&]() -> int {
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc || (rc = check_count(h, n))) return rc;
        h->last_launches = 0;
        if (n == 0) return HA_OK;
        if (!slots) return fail(h, HA_ERR_INVALID_ARG, "null list");
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_CACHE, "ha:cache", st);
        const int k = ha::launch_cache_free(c, slots, static_cast<int>(n), h->serve_status, st);
        prof.end(k);
        return launched(h, k, "cache free");
    });
}

int hyper_attn_cache_fork(hyper_attn_t h, const ha_cache *cache, const int32_t *src, const int32_t *dst, int64_t n) {
    return guarded(h, [&]() -> int {
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc || (rc = check_count(h, n))) return rc;
        h->last_launches = 0;
        if (n == 0) return HA_OK;
        if (!src || !dst) return fail(h, HA_ERR_INVALID_ARG, "null list");
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_CACHE, "ha:cache", st);
        const int k = ha::launch_cache_fork(c, src, dst, static_cast<int>(n), h->serve_status, st);
        prof.end(k);
        return launched(h, k, "cache fork");
    });
}

size_t hyper_attn_cache_workspace(int64_t n, int64_t pages) {
    return n < 0 || pages < 0 ? 0 : ha::cache_workspace(n, pages);
}

int hyper_attn_cache_reserve(hyper_attn_t h, const ha_cache *cache, const int32_t *slots, const int32_t *add, int64_t n,
                             int32_t *granted, void *workspace, size_t workspace_bytes) {
    return guarded(h, [&]() -> int {
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc || (rc = check_count(h, n))) return rc;
        h->last_launches = 0;
        if (n == 0) return HA_OK;
        if (!slots || !add) return fail(h, HA_ERR_INVALID_ARG, "null list");
        const size_t need = ha::cache_workspace(n, c.pages);
        if (!workspace || !aligned16(workspace) || workspace_bytes < need)
            return fail(h, HA_ERR_INVALID_ARG, "workspace of %zu bytes needed, 16-byte aligned", need);
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_CACHE, "ha:cache", st);
        const int k = ha::launch_cache_reserve(c, esize(h), slots, add, static_cast<int>(n), granted, workspace,
                                               h->serve_status, st);
        prof.end(k);
        return launched(h, k, "cache reserve");
    });
}

int hyper_attn_cache_append(hyper_attn_t h, const ha_cache *cache, const int32_t *slots, const int32_t *offsets, int64_t n,
                            int64_t tokens, const void *k, const void *v, const int64_t k_strides[3],
                            const int64_t v_strides[3], int64_t layer, int64_t layers) {
    return guarded(h, [&]() -> int {
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc || (rc = check_count(h, n, 65536))) return rc;
        if (tokens < 0 || tokens > kMaxTokens) return fail(h, HA_ERR_INVALID_ARG, "tokens must lie in [0, 2^30]");
        if (layer < 0 || layers < 1 || layer > c.layers - layers) return fail(h, HA_ERR_INVALID_ARG, "layers out of range");
        h->last_launches = 0;
        if (n == 0 || tokens == 0) return HA_OK;
        if (!slots || !offsets || !k || !v || !k_strides || !v_strides) return fail(h, HA_ERR_INVALID_ARG, "null pointer");
        if (!aligned16(k) || !aligned16(v)) return fail(h, HA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
        const int esz = esize(h);
        int64_t ks[3], vs[3];
        for (int i = 0; i < 3; ++i) {
            ks[i] = k_strides[i];
            vs[i] = v_strides[i];
            if (layers == 1 && i == 0) ks[i] = vs[i] = 0;
            if (tokens == 1 && i == 1) ks[i] = vs[i] = 0;
            if (c.kv_heads == 1 && i == 2) ks[i] = vs[i] = 0;
            const int64_t unit = 16 / esz, most = int64_t(1) << 36;
            if (ks[i] < 0 || vs[i] < 0 || ks[i] % unit || vs[i] % unit || ks[i] > most || vs[i] > most)
                return fail(h, HA_ERR_INVALID_ARG, "strides must be of 16-byte multiples and not negative");
        }
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_CACHE, "ha:cache", st);
        const int r = ha::launch_cache_append(c, esz, slots, offsets, static_cast<int>(n), tokens, k, v, ks, vs, layer,
                                              layers, h->serve_status, st);
        prof.end(r);
        return launched(h, r, "cache append");
    });
}

int hyper_attn_cache_commit(hyper_attn_t h, const ha_cache *cache, const int32_t *slots, const int32_t *counts,
                            const int32_t *keep, int64_t max_keep, int64_t n) {
    return guarded(h, [&]() -> int {
        ha::ServeCache c;
        int rc = check_cache(h, cache, &c);
        if (rc || (rc = check_count(h, n))) return rc;
        if (keep && (max_keep < 1 || max_keep > kMaxTokens)) return fail(h, HA_ERR_INVALID_ARG, "max_keep out of range");
        h->last_launches = 0;
        if (n == 0) return HA_OK;
        if (!slots || !counts) return fail(h, HA_ERR_INVALID_ARG, "null list");
        cudaStream_t st = static_cast<cudaStream_t>(h->opt.stream);
        ProfScope prof(h, HA_KC_CACHE, "ha:cache", st);
        const int k = ha::launch_cache_commit(c, esize(h), slots, counts, keep, max_keep, static_cast<int>(n),
                                              h->serve_status, st);
        prof.end(k);
        return launched(h, k, "cache commit");
    });
}

}  // extern "C"
