// kv_api.hip -- the C ABI (include/moe.h) of the paged cache, its attention and pages,
// the few-token int4 products and beam search's selection: host-side validation and launches.  As in
// moe_api.hip nothing here touches device memory from the host or synchronises.
#include "moe.h"
#include "moe_launch.h"

#include <initializer_list>

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int check_shape(const moe_kv_shape *s)
{
    if (!s) return MOE_ERR_NULL;
    if (s->n_seq < 0 || s->rows < 0 || s->max_rows < 0 || s->max_rows > s->rows || s->max_len < 0) return MOE_ERR_SHAPE;
    if (s->q_heads <= 0 || s->kv_heads <= 0 || s->q_heads % s->kv_heads || s->head_dim <= 0) return MOE_ERR_SHAPE;
    if (s->kv_bits != 8 && s->kv_bits != 16) return MOE_ERR_SHAPE;
    if (s->page_tokens <= 0 || s->n_pages < 0 || s->max_pages < 0 || s->window < 0) return MOE_ERR_SHAPE;
    if (s->kv_bits == 8 && s->n_slots < 0) return MOE_ERR_SHAPE;
    if (!(s->scale - s->scale == 0.0f)) return MOE_ERR_SHAPE;  // infinite or NaN
    if ((int64_t)s->max_pages * s->page_tokens > 1 << 30 || s->max_len > 1 << 30) return MOE_ERR_SHAPE;
    if (s->q_heads > 1 << 22) return MOE_ERR_SHAPE;
    if ((int64_t)s->rows * s->q_heads > INT32_MAX / 32 || (int64_t)s->n_seq * s->kv_heads > INT32_MAX / 32)
        return MOE_ERR_SHAPE;
    // what the gfx950 kernels cover
    if (s->head_dim != 64 && s->head_dim != 128) return MOE_ERR_UNSUPPORTED;
    if (s->page_tokens != 16 && s->page_tokens != 32 && s->page_tokens != 64 && s->page_tokens != 128)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool empty(const moe_kv_shape *s) { return s->rows == 0 || s->max_rows == 0 || s->n_seq == 0; }

int check_tables(const moe_kv_shape *s, const moe_kv_batch *b, const moe_kv_cache *c)
{
    if (!b || !c || !b->row_start || !b->kv_len) return MOE_ERR_NULL;
    if (s->max_pages > 0 && !b->pages) return MOE_ERR_NULL;
    if (!aligned(b->row_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->pages, 4) || !aligned(b->slots, 4))
        return MOE_ERR_ALIGN;
    if (s->n_pages > 0 && (!c->k || !c->v)) return MOE_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return MOE_ERR_ALIGN;
    if (s->kv_bits == 8) {
        if (s->n_pages > 0 && (!c->k_scale || !c->v_scale)) return MOE_ERR_NULL;
        if (s->n_slots > 0 && (!c->k_tail || !c->v_tail)) return MOE_ERR_NULL;
        if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->k_tail, 16) || !aligned(c->v_tail, 16))
            return MOE_ERR_ALIGN;
    }
    return MOE_OK;
}

// rows of `heads` heads, `stride` elements apart
int check_rows(const void *p, int64_t stride, int heads, int dim)
{
    if (!p) return MOE_ERR_NULL;
    if (stride < (int64_t)heads * dim) return MOE_ERR_SHAPE;
    if (!aligned(p, 16) || stride % 8) return MOE_ERR_ALIGN;
    return MOE_OK;
}

moe::KvArgs args_of(const moe_kv_shape *s, const moe_kv_batch *b, const moe_kv_cache *c)
{
    moe::KvArgs a = {};
    a.n_seq = s->n_seq;
    a.rows = s->rows;
    a.max_rows = s->max_rows;
    a.max_len = s->max_len;
    a.q_heads = s->q_heads;
    a.kv_heads = s->kv_heads;
    a.head_dim = s->head_dim;
    a.kv_bits = s->kv_bits;
    a.page_log2 = __builtin_ctz((unsigned)s->page_tokens);
    a.n_pages = s->n_pages;
    a.max_pages = s->max_pages;
    a.n_slots = s->kv_bits == 8 ? s->n_slots : 0;
    a.window = s->window;
    a.causal = (s->flags & MOE_KV_NONCAUSAL) ? 0 : 1;
    a.scale = s->scale != 0.0f ? s->scale : s->head_dim == 64 ? 0.125f : 0.08838834764831845f;
    if (b) {
        a.row_start = b->row_start;
        a.kv_len = b->kv_len;
        a.pages = b->pages;
        a.slots = b->slots;
    }
    if (c) {
        a.k = c->k;
        a.v = c->v;
        a.k_scale = c->k_scale;
        a.v_scale = c->v_scale;
        a.k_tail = c->k_tail;
        a.v_tail = c->v_tail;
    }
    return a;
}

}  // namespace

extern "C" int moe_kv_append(const moe_kv_shape *shape, const moe_kv_batch *batch, const moe_kv_cache *cache,
                             const moe_kv_rotary *rot, const moe_bf16 *k, int64_t k_row_stride, const moe_bf16 *v,
                             int64_t v_row_stride, const moe_bf16 *q, int64_t q_row_stride, moe_bf16 *q_out,
                             void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (rot) {
        if (rot->rot_dim < 0 || rot->rot_dim > shape->head_dim || rot->rot_dim % 2 || rot->n_pos < 0)
            return MOE_ERR_SHAPE;
        if (rot->rot_dim % 16) return MOE_ERR_UNSUPPORTED;
    }
    if (empty(shape)) return MOE_OK;
    if (const int r = check_tables(shape, batch, cache)) return r;
    if (const int r = check_rows(k, k_row_stride, shape->kv_heads, shape->head_dim)) return r;
    if (const int r = check_rows(v, v_row_stride, shape->kv_heads, shape->head_dim)) return r;
    if (q) {
        if (const int r = check_rows(q, q_row_stride, shape->q_heads, shape->head_dim)) return r;
        if (!q_out) return MOE_ERR_NULL;
        if (!aligned(q_out, 16)) return MOE_ERR_ALIGN;
        // in place only where a row's result lies where the row was: else it would meet rows not read yet
        if (q_out == q && shape->rows > 1 && q_row_stride != (int64_t)shape->q_heads * shape->head_dim) return MOE_ERR_SHAPE;
    }
    moe::KvAppend n = {};
    if (rot) {
        if (rot->rot_dim && rot->n_pos > 0 && (!rot->cos || !rot->sin)) return MOE_ERR_NULL;
        if (!aligned(rot->cos, 16) || !aligned(rot->sin, 16) || !aligned(rot->pos, 4) || !aligned(rot->q_norm, 16) ||
            !aligned(rot->k_norm, 16))
            return MOE_ERR_ALIGN;
        n.cos = rot->cos;
        n.sin = rot->sin;
        n.pos = rot->pos;
        n.n_pos = rot->n_pos;
        n.rot_dim = rot->rot_dim;
        n.q_norm = rot->q_norm;
        n.k_norm = rot->k_norm;
        n.eps = rot->eps;
    }
    n.pairs = (shape->flags & MOE_KV_ROPE_PAIRS) ? 1 : 0;
    n.k = k;
    n.v = v;
    n.q = q;
    n.k_stride = k_row_stride;
    n.v_stride = v_row_stride;
    n.q_stride = q_row_stride;
    n.q_out = q_out;
    return hip_status(moe::launch_kv_append(args_of(shape, batch, cache), n, (hipStream_t)stream));
}

extern "C" size_t moe_kv_attention_sinks_workspace_bytes(const moe_kv_shape *shape, int32_t sink_tokens)
{
    if (check_shape(shape) != MOE_OK || sink_tokens < 0 || sink_tokens > 1 << 30) return 0;
    const size_t n = moe::kv_attention_workspace(args_of(shape, nullptr, nullptr), shape->window ? sink_tokens : 0);
    return n < 256 ? 256 : (n + 255) / 256 * 256;
}

extern "C" size_t moe_kv_workspace_bytes(const moe_kv_shape *shape) { return moe_kv_attention_sinks_workspace_bytes(shape, 0); }

extern "C" int moe_kv_attention_sinks(const moe_kv_shape *shape, int32_t sink_tokens, const moe_kv_batch *batch,
                                      const moe_kv_cache *cache, const moe_bf16 *q, int64_t q_row_stride, void *out,
                                      float *lse, void *ws, size_t ws_bytes, void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (sink_tokens < 0 || sink_tokens > 1 << 30) return MOE_ERR_SHAPE;
    if (empty(shape)) return MOE_OK;
    if (const int r = check_tables(shape, batch, cache)) return r;
    if (const int r = check_rows(q, q_row_stride, shape->q_heads, shape->head_dim)) return r;
    if (!out) return MOE_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4)) return MOE_ERR_ALIGN;
    if (ws_bytes < moe_kv_attention_sinks_workspace_bytes(shape, sink_tokens)) return MOE_ERR_WORKSPACE;
    if (!ws) return MOE_ERR_NULL;
    if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
    return hip_status(moe::launch_kv_attention(args_of(shape, batch, cache), sink_tokens, q, q_row_stride, out,
                                               (shape->flags & MOE_OUT_F32) ? 1 : 0, lse, ws, (hipStream_t)stream));
}

extern "C" int moe_kv_attention(const moe_kv_shape *shape, const moe_kv_batch *batch, const moe_kv_cache *cache,
                                const moe_bf16 *q, int64_t q_row_stride, void *out, float *lse, void *ws,
                                size_t ws_bytes, void *stream)
{
    return moe_kv_attention_sinks(shape, 0, batch, cache, q, q_row_stride, out, lse, ws, ws_bytes, stream);
}

extern "C" int moe_kv_read(const moe_kv_shape *shape, const moe_kv_batch *batch, const moe_kv_cache *cache,
                           moe_bf16 *k, moe_bf16 *v, void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (empty(shape)) return MOE_OK;
    if (const int r = check_tables(shape, batch, cache)) return r;
    if (!k || !v) return MOE_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_ALIGN;
    return hip_status(moe::launch_kv_read(args_of(shape, batch, cache), k, v, (hipStream_t)stream));
}

// ---- the cache's pages

static bool misaligned(std::initializer_list<const void *> tables)
{
    for (const void *p : tables)
        if (!aligned(p, 4)) return true;
    return false;
}

extern "C" size_t moe_kv_pool_workspace_bytes(const moe_kv_shape *shape)
{
    if (check_shape(shape) != MOE_OK) return 0;
    return (moe::kv_pool_workspace(shape->n_pages) + 255) / 256 * 256;
}

static int check_pool_ws(const moe_kv_shape *shape, const void *ws, size_t ws_bytes)
{
    if (ws_bytes < moe_kv_pool_workspace_bytes(shape)) return MOE_ERR_WORKSPACE;
    if (!ws) return MOE_ERR_NULL;
    return aligned(ws, 256) ? MOE_OK : MOE_ERR_ALIGN;
}

extern "C" int moe_kv_release(const moe_kv_shape *shape, int32_t sink_tokens, const int32_t *kv_len, int32_t *pages,
                              int32_t *refs, void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (sink_tokens < 0 || sink_tokens > 1 << 30) return MOE_ERR_SHAPE;
    if (shape->n_seq == 0 || shape->max_pages == 0) return MOE_OK;
    if (!kv_len || !pages || (shape->n_pages > 0 && !refs)) return MOE_ERR_NULL;
    if (misaligned({kv_len, pages, refs})) return MOE_ERR_ALIGN;
    moe::KvArgs a = args_of(shape, nullptr, nullptr);
    a.kv_len = kv_len;
    return hip_status(moe::launch_kv_release(a, sink_tokens, pages, refs, (hipStream_t)stream));
}

extern "C" int moe_kv_fork(const moe_kv_shape *shape, const moe_kv_batch *batch, const int32_t *parent, int32_t *kv_len,
                           int32_t *pages, int32_t *slots, int32_t *refs, int32_t *slot_src, int32_t *slot_dst,
                           void *stream)
{
    static_assert(MOE_KV_FORK_MAX == moe::KV_FORK_MAX, "");
    if (const int r = check_shape(shape)) return r;
    if (shape->n_seq > MOE_KV_FORK_MAX) return MOE_ERR_UNSUPPORTED;
    if (shape->n_seq == 0) return MOE_OK;
    if (!batch || !batch->kv_len || !parent || !kv_len) return MOE_ERR_NULL;
    if (shape->max_pages > 0 && (!batch->pages || !pages || (shape->n_pages > 0 && !refs))) return MOE_ERR_NULL;
    const bool with_slots = shape->kv_bits == 8;
    if (with_slots && (!slots || !slot_src || !slot_dst)) return MOE_ERR_NULL;
    if (misaligned({batch->kv_len, batch->pages, batch->slots, parent, kv_len, pages, slots, refs, slot_src, slot_dst}))
        return MOE_ERR_ALIGN;
    if (batch->kv_len == kv_len || (shape->max_pages > 0 && batch->pages == pages) || (with_slots && batch->slots == slots))
        return MOE_ERR_SHAPE;  // rows are read while others are written
    return hip_status(moe::launch_kv_fork(args_of(shape, batch, nullptr), parent, kv_len, pages, with_slots ? slots : nullptr,
                                          refs, slot_src, slot_dst, (hipStream_t)stream));
}

extern "C" int moe_kv_reserve(const moe_kv_shape *shape, const moe_kv_batch *batch, int32_t *pages, int32_t *refs,
                              int32_t *copy_src, int32_t *copy_dst, int32_t *missing, void *ws, size_t ws_bytes,
                              void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (shape->n_seq == 0) return MOE_OK;
    if (!batch || !batch->row_start || !batch->kv_len) return MOE_ERR_NULL;
    if (shape->max_pages > 0 && (!pages || (shape->n_pages > 0 && !refs))) return MOE_ERR_NULL;
    const bool copies = shape->kv_bits == 16;
    if (copies && (!copy_src || !copy_dst)) return MOE_ERR_NULL;
    if (misaligned({batch->row_start, batch->kv_len, pages, refs, copy_src, copy_dst, missing})) return MOE_ERR_ALIGN;
    if (const int r = check_pool_ws(shape, ws, ws_bytes)) return r;
    return hip_status(moe::launch_kv_reserve(args_of(shape, batch, nullptr), pages, refs, copies ? copy_src : nullptr,
                                             copies ? copy_dst : nullptr, missing, ws, (hipStream_t)stream));
}

extern "C" int moe_kv_compact(const moe_kv_shape *shape, int32_t *pages, int32_t *refs, int32_t max_moves,
                              int32_t *copy_src, int32_t *copy_dst, int32_t *n_live, void *ws, size_t ws_bytes,
                              void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (max_moves < 0 || max_moves > shape->n_pages / 2) return MOE_ERR_SHAPE;
    if (shape->n_pages > 0 && !refs) return MOE_ERR_NULL;
    if (max_moves > 0 && (!copy_src || !copy_dst)) return MOE_ERR_NULL;
    if (shape->n_seq > 0 && shape->max_pages > 0 && !pages) return MOE_ERR_NULL;
    if (misaligned({pages, refs, copy_src, copy_dst, n_live})) return MOE_ERR_ALIGN;
    if (const int r = check_pool_ws(shape, ws, ws_bytes)) return r;
    return hip_status(moe::launch_kv_compact(args_of(shape, nullptr, nullptr), pages, refs, max_moves, copy_src, copy_dst,
                                             n_live, ws, (hipStream_t)stream));
}

extern "C" int moe_kv_copy(const moe_kv_shape *shape, const moe_kv_cache *cache, int32_t n_pages_listed,
                           const int32_t *page_src, const int32_t *page_dst, int32_t n_slots_listed,
                           const int32_t *slot_src, const int32_t *slot_dst, void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (n_pages_listed < 0 || n_slots_listed < 0) return MOE_ERR_SHAPE;
    const int32_t n_slots = shape->kv_bits == 8 && shape->n_slots > 0 ? n_slots_listed : 0;
    const int32_t n_pages = shape->n_pages > 0 ? n_pages_listed : 0;
    if (n_pages == 0 && n_slots == 0) return MOE_OK;
    if (!cache || (n_pages && (!page_src || !page_dst)) || (n_slots && (!slot_src || !slot_dst))) return MOE_ERR_NULL;
    if (misaligned({page_src, page_dst, slot_src, slot_dst})) return MOE_ERR_ALIGN;
    if (n_pages && (!cache->k || !cache->v)) return MOE_ERR_NULL;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16)) return MOE_ERR_ALIGN;
    if (shape->kv_bits == 8) {
        if (n_pages && (!cache->k_scale || !cache->v_scale)) return MOE_ERR_NULL;
        if (n_slots && (!cache->k_tail || !cache->v_tail)) return MOE_ERR_NULL;
        if (misaligned({cache->k_scale, cache->v_scale}) || !aligned(cache->k_tail, 16) || !aligned(cache->v_tail, 16))
            return MOE_ERR_ALIGN;
    }
    return hip_status(moe::launch_kv_copy(args_of(shape, nullptr, cache), n_pages, page_src, page_dst, n_slots, slot_src,
                                          slot_dst, (hipStream_t)stream));
}

// ---- beam search

static int check_beam(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out)
{
    if (requests < 0 || beams < 1 || vocab < 1 || vocab > 1 << 30 || n_out < 1) return MOE_ERR_SHAPE;
    if (beams > 128 || n_out > 128) return MOE_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)requests * beams;
    if (rows >= 1 << 22 || rows * vocab > (int64_t)1 << 36) return MOE_ERR_SHAPE;  // a launch below 2^32 lanes
    return MOE_OK;
}

extern "C" size_t moe_beam_workspace_bytes(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out)
{
    if (check_beam(requests, beams, vocab, n_out) != MOE_OK) return 0;
    const size_t n = moe::beam_workspace((int64_t)requests * beams, vocab, n_out);
    return n < 256 ? 256 : (n + 255) / 256 * 256;
}

extern "C" int moe_beam_select(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out, const void *logits,
                               int32_t logits_format, int64_t row_stride, const float *scores, const uint8_t *done,
                               int32_t end_token, int32_t *parent, int32_t *token, float *score, uint8_t *done_out,
                               float *lse, void *ws, size_t ws_bytes, void *stream)
{
    if (const int r = check_beam(requests, beams, vocab, n_out)) return r;
    if (logits_format != MOE_SRC_F32 && logits_format != MOE_SRC_BF16) return MOE_ERR_SHAPE;
    if (row_stride < vocab || row_stride > (int64_t)1 << 40 || (done && end_token < 0)) return MOE_ERR_SHAPE;
    if (requests == 0) return MOE_OK;
    if (!logits || !scores || !parent || !token || !score) return MOE_ERR_NULL;
    if (!aligned(logits, logits_format == MOE_SRC_F32 ? 4 : 2) || misaligned({scores, parent, token, score, lse}))
        return MOE_ERR_ALIGN;
    if (ws_bytes < moe_beam_workspace_bytes(requests, beams, vocab, n_out)) return MOE_ERR_WORKSPACE;
    if (!ws) return MOE_ERR_NULL;
    if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
    moe::BeamSelect a = {};
    a.requests = requests;
    a.beams = beams;
    a.vocab = vocab;
    a.n_out = n_out;
    a.end_token = end_token;
    a.logits = logits;
    a.bf16 = logits_format == MOE_SRC_BF16;
    a.row_stride = row_stride;
    a.scores = scores;
    a.done = done;
    a.parent = parent;
    a.token = token;
    a.score = score;
    a.lse = lse;
    a.done_out = done_out;
    return hip_status(moe::launch_beam_select(a, ws, (hipStream_t)stream));
}

extern "C" size_t moe_linear_q4_workspace_bytes(int32_t T, int32_t N, int32_t K)
{
    return T < 0 || N < 0 || K <= 0 ? 0 : 256;  // reserved: no kernel uses it
}

extern "C" int moe_linear_q4(int32_t T, int32_t N, int32_t K, int32_t group, const moe_bf16 *x, int64_t x_row_stride,
                             const void *q, const void *scales, int32_t scale_format, const moe_bf16 *residual,
                             void *out, uint32_t flags, void *ws, size_t ws_bytes, void *stream)
{
    if (T < 0 || N < 0 || K <= 0 || group <= 0 || K % group || x_row_stride < K) return MOE_ERR_SHAPE;
    if (scale_format != MOE_SRC_F32 && scale_format != MOE_SRC_BF16) return MOE_ERR_SHAPE;
    if ((int64_t)T * N > ((int64_t)1 << 40)) return MOE_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
    if (x_row_stride > 1 << 25) return MOE_ERR_UNSUPPORTED;  // 32-bit offsets inside a workgroup (K is no larger)
    if (T == 0 || N == 0) return MOE_OK;
    if (!x || !q || !scales || !out) return MOE_ERR_NULL;
    if (!aligned(x, 16) || x_row_stride % 8 || !aligned(q, 16) || !aligned(scales, 16)) return MOE_ERR_ALIGN;
    if (!aligned(residual, 2) || !aligned(out, (flags & MOE_OUT_F32) ? 4 : 2)) return MOE_ERR_ALIGN;
    if (ws_bytes < moe_linear_q4_workspace_bytes(T, N, K)) return MOE_ERR_WORKSPACE;
    if (!ws) return MOE_ERR_NULL;
    if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
    moe::LinearQ4 a = {};
    a.T = T;
    a.N = N;
    a.K = K;
    a.group = group;
    a.x = x;
    a.x_stride = x_row_stride;
    a.q = (const uint8_t *)q;
    a.scales = scales;
    a.scales_bf16 = scale_format == MOE_SRC_BF16;
    a.residual = residual;
    a.out = out;
    a.out_f32 = (flags & MOE_OUT_F32) ? 1 : 0;
    return hip_status(moe::launch_linear_q4(a, (hipStream_t)stream));
}
