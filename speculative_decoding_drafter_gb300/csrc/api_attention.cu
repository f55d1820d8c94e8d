// api_attention.cu -- C-ABI entry points of the attention-side operators (rotary positions, the
// paged cache, attention over it): argument checks and launches.  No allocation, no sync.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "dflash2.h"
#include "internal.h"

namespace df2 {
namespace {

df2_status check_rows(const df2_heads *r, int heads)
{
    if (!r || !r->data || !aligned(r->data, 16) || r->heads != heads || heads < 1)
        return DF2_ERR_INVALID_ARG;
    if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride % 8 != 0 || r->head_stride % 8 != 0)
        return DF2_ERR_INVALID_ARG;
    return DF2_OK;
}

// Rows that are written: distinct (token, head) rows must not share elements.
df2_status check_out_rows(const df2_heads *r, int heads, long long N, int dim)
{
    DF2_TRY(check_rows(r, heads));
    const bool head_inner = r->head_stride >= dim && (N <= 1 || r->token_stride >= (heads - 1) * r->head_stride + dim);
    const bool token_inner = r->token_stride >= dim && (heads <= 1 || r->head_stride >= (N - 1) * r->token_stride + dim);
    const bool one_head = heads == 1 && (N <= 1 || r->token_stride >= dim);
    return head_inner || token_inner || one_head ? DF2_OK : DF2_ERR_INVALID_ARG;
}

HeadRows rows_of(const df2_heads *r)
{
    HeadRows h;
    if (r) {
        h.data = static_cast<uint16_t *>(r->data);
        h.heads = r->heads;
        h.token_stride = r->token_stride;
        h.head_stride = r->head_stride;
    }
    return h;
}

df2_status check_rope(const df2_rope *r, int dim)
{
    if (!r || !r->table || !aligned(r->table, 4) || r->max_pos < 1 || r->rot < 2 || r->rot % 2 != 0 || r->rot > dim)
        return DF2_ERR_INVALID_ARG;
    return DF2_OK;
}

RopeTable rope_of(const df2_rope *r)
{
    RopeTable t;
    if (r) {
        t.table = r->table;
        t.max_pos = r->max_pos;
        t.rot = r->rot;
        t.interleaved = r->interleaved != 0;
    }
    return t;
}

df2_status check_cache_limits(const df2_cache *c)
{
    if (!c || c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->dim < 1 || c->type < DF2_CACHE_BF16 ||
        c->type > DF2_CACHE_INT8)
        return DF2_ERR_INVALID_ARG;
    if (c->page_size % 8 != 0 || c->page_size > 1024 || c->dim % 16 != 0 || c->dim > 128 || c->heads > 1024)
        return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

df2_status check_cache(const df2_cache *c)
{
    DF2_TRY(check_cache_limits(c));
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return DF2_ERR_INVALID_ARG;
    if (c->type != DF2_CACHE_BF16 &&
        (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
        return DF2_ERR_INVALID_ARG;
    return DF2_OK;
}

df2_status check_tokens_limits(const df2_tokens *t)
{
    if (!t || t->B < 1 || t->N < 0 || t->max_new < 0 || t->max_new > t->N || t->max_pages < 0 ||
        (t->N > 0 && t->max_new < 1))
        return DF2_ERR_INVALID_ARG;
    if (t->B > 2048)
        return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

df2_status check_tokens(const df2_tokens *t, int page_size)
{
    DF2_TRY(check_tokens_limits(t));
    if (!t->token_start || !t->kv_len || !aligned(t->token_start, 4) || !aligned(t->kv_len, 4) ||
        (t->max_pages > 0 && (!t->page_table || !aligned(t->page_table, 4))))
        return DF2_ERR_INVALID_ARG;
    if (static_cast<long long>(t->max_pages) * page_size > (1LL << 30))
        return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

PagedCache cache_of(const df2_cache &c)
{
    PagedCache p;
    p.pages = c.pages;
    p.page_size = c.page_size;
    p.heads = c.heads;
    p.dim = c.dim;
    p.type = c.type;
    p.k = c.k;
    p.v = c.v;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    return p;
}

TokenBatch tokens_of(const df2_tokens &t)
{
    TokenBatch b;
    b.B = t.B;
    b.N = t.N;
    b.max_new = t.max_new;
    b.max_pages = t.max_pages;
    b.token_start = t.token_start;
    b.kv_len = t.kv_len;
    b.page_table = t.page_table;
    return b;
}

df2_status check_q_heads(const df2_cache &c, const df2_tokens &t, int q_heads)
{
    if (q_heads < 1 || q_heads % c.heads != 0)
        return DF2_ERR_INVALID_ARG;
    if (q_heads / c.heads > 64 || static_cast<long long>(t.N) * q_heads >= (1LL << 31))
        return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

}  // namespace
}  // namespace df2

using namespace df2;

extern "C" {

df2_status dflash2_rope_table(const df2_rope_scaling *s, int32_t max_pos, int32_t rot, float *table, void *stream)
{
    const TraceRange range("dflash2_rope_table");
    if (!s || !table || !aligned(table, 4) || max_pos < 1 || rot < 2 || rot % 2 != 0 || s->kind < DF2_ROPE_PLAIN ||
        s->kind > DF2_ROPE_BAND)
        return DF2_ERR_INVALID_ARG;
    if (rot > 256)
        return DF2_ERR_UNSUPPORTED;
    if (!(s->theta > 1.0) || !std::isfinite(s->theta) || !(s->multiplier > 0.0) || !std::isfinite(s->multiplier))
        return DF2_ERR_INVALID_ARG;
    if (s->kind != DF2_ROPE_PLAIN && (!(s->factor > 0.0) || !std::isfinite(s->factor)))
        return DF2_ERR_INVALID_ARG;
    if (s->kind == DF2_ROPE_BASE && rot == 2)
        return DF2_ERR_INVALID_ARG;
    if ((s->kind == DF2_ROPE_RAMP || s->kind == DF2_ROPE_BAND) &&
        (!(s->original_len > 0.0) || !std::isfinite(s->original_len) || !(s->low > 0.0) || !(s->high > s->low) ||
         !std::isfinite(s->high)))
        return DF2_ERR_INVALID_ARG;
    cudaGetLastError();
    const RopeScaling sc{s->kind, s->theta, s->factor, s->original_len, s->low, s->high, s->multiplier};
    return from_cuda(launch_rope_table(sc, max_pos, rot, table, static_cast<cudaStream_t>(stream)));
}

df2_status dflash2_rope(const df2_rope *rope, int32_t N, int32_t dim, const df2_heads *x, const int32_t *positions,
                        int32_t inverse, const df2_heads *y, void *stream)
{
    const TraceRange range("dflash2_rope");
    if (N < 0 || dim < 1 || !x || !y)
        return DF2_ERR_INVALID_ARG;
    if (dim % 8 != 0 || dim > 256)
        return DF2_ERR_UNSUPPORTED;
    DF2_TRY(check_rope(rope, dim));
    if (N == 0)
        return DF2_OK;
    if (!positions || !aligned(positions, 4))
        return DF2_ERR_INVALID_ARG;
    DF2_TRY(check_rows(x, x->heads));
    DF2_TRY(check_out_rows(y, x->heads, N, dim));
    if (x->data == y->data && (x->token_stride != y->token_stride || x->head_stride != y->head_stride))
        return DF2_ERR_INVALID_ARG;
    if (static_cast<long long>(N) * x->heads >= (1LL << 31) - 1024)
        return DF2_ERR_UNSUPPORTED;
    cudaGetLastError();
    return from_cuda(launch_rope(rope_of(rope), N, dim, rows_of(x), positions, inverse ? -1.f : 1.f, rows_of(y),
                                 static_cast<cudaStream_t>(stream)));
}

df2_status dflash2_cache_append(const df2_cache *cache, const df2_tokens *tokens, const df2_rope *rope,
                                const df2_heads *q, const df2_heads *q_out, const df2_heads *k, const df2_heads *v,
                                void *stream)
{
    const TraceRange range("dflash2_cache_append");
    DF2_TRY(check_cache(cache));
    DF2_TRY(check_tokens(tokens, cache->page_size));
    if (rope)
        DF2_TRY(check_rope(rope, cache->dim));
    if ((q == nullptr) != (q_out == nullptr))
        return DF2_ERR_INVALID_ARG;
    if (tokens->N == 0)
        return DF2_OK;
    DF2_TRY(check_rows(k, cache->heads));
    DF2_TRY(check_rows(v, cache->heads));
    if (q) {
        DF2_TRY(check_rows(q, q->heads));
        DF2_TRY(check_out_rows(q_out, q->heads, tokens->N, cache->dim));
        if (q->data == q_out->data &&
            (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
            return DF2_ERR_INVALID_ARG;
    }
    if (static_cast<long long>(tokens->N) * ((q ? q->heads : 0) + 2LL * cache->heads) >= (1LL << 31) - 1024)
        return DF2_ERR_UNSUPPORTED;
    cudaGetLastError();
    return from_cuda(launch_cache_append(cache_of(*cache), tokens_of(*tokens), rope_of(rope), rows_of(q),
                                         rows_of(q_out), rows_of(k), rows_of(v), static_cast<cudaStream_t>(stream)));
}

df2_status dflash2_cache_read(const df2_cache *cache, const df2_tokens *tokens, const df2_heads *k_out,
                              const df2_heads *v_out, void *stream)
{
    const TraceRange range("dflash2_cache_read");
    DF2_TRY(check_cache(cache));
    DF2_TRY(check_tokens(tokens, cache->page_size));
    if (tokens->N == 0)
        return DF2_OK;
    if (!k_out && !v_out)
        return DF2_ERR_INVALID_ARG;
    if (k_out)
        DF2_TRY(check_out_rows(k_out, cache->heads, tokens->N, cache->dim));
    if (v_out)
        DF2_TRY(check_out_rows(v_out, cache->heads, tokens->N, cache->dim));
    if (static_cast<long long>(tokens->N) * 2 * cache->heads >= (1LL << 31) - 1024)
        return DF2_ERR_UNSUPPORTED;
    cudaGetLastError();
    return from_cuda(launch_cache_read(cache_of(*cache), tokens_of(*tokens), rows_of(k_out), rows_of(v_out),
                                       static_cast<cudaStream_t>(stream)));
}

size_t dflash2_paged_attention_workspace_bytes(const df2_cache *cache, const df2_tokens *tokens, int32_t q_heads)
{
    if (check_cache_limits(cache) != DF2_OK || check_tokens_limits(tokens) != DF2_OK ||
        check_q_heads(*cache, *tokens, q_heads) != DF2_OK)
        return 0;
    return kAlign + round_up(paged_attention_scratch(cache_of(*cache), tokens_of(*tokens), q_heads));
}

df2_status dflash2_paged_attention(const df2_cache *cache, const df2_tokens *tokens, const df2_attention *options,
                                   const df2_heads *q, const df2_heads *out, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream)
{
    const TraceRange range("dflash2_paged_attention");
    DF2_TRY(check_cache(cache));
    DF2_TRY(check_tokens(tokens, cache->page_size));
    if (!options || !std::isfinite(options->scale) || options->window < 0 || !q || !out)
        return DF2_ERR_INVALID_ARG;
    DF2_TRY(check_q_heads(*cache, *tokens, q->heads));
    if (tokens->N == 0)
        return DF2_OK;
    DF2_TRY(check_rows(q, q->heads));
    DF2_TRY(check_out_rows(out, q->heads, tokens->N, cache->dim));
    if (lse && !aligned(lse, 4))
        return DF2_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, kAlign) ||
        workspace_bytes < dflash2_paged_attention_workspace_bytes(cache, tokens, q->heads))
        return DF2_ERR_WORKSPACE;
    cudaGetLastError();
    AttentionOptions opt;
    opt.scale = options->scale;
    opt.causal = options->causal != 0;
    opt.window = options->window;
    return from_cuda(launch_paged_attention(cache_of(*cache), tokens_of(*tokens), opt, rows_of(q), rows_of(out), lse,
                                            static_cast<uint32_t *>(workspace),
                                            static_cast<uint8_t *>(workspace) + kAlign,
                                            static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
