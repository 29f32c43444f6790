// kv_api.hip -- the C ABI (include/moe.h) of the paged cache, its attention and
// the few-token int4 products: host-side validation and launches.  As in
// moe_api.hip nothing here touches device memory from the host or synchronises.
#include "moe.h"
#include "moe_launch.h"

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

extern "C" size_t moe_kv_workspace_bytes(const moe_kv_shape *shape)
{
    if (check_shape(shape) != MOE_OK) return 0;
    const size_t n = moe::kv_attention_workspace(args_of(shape, nullptr, nullptr));
    return n < 256 ? 256 : (n + 255) / 256 * 256;
}

extern "C" int moe_kv_attention(const moe_kv_shape *shape, const moe_kv_batch *batch, const moe_kv_cache *cache,
                                const moe_bf16 *q, int64_t q_row_stride, void *out, float *lse, void *ws,
                                size_t ws_bytes, void *stream)
{
    if (const int r = check_shape(shape)) return r;
    if (empty(shape)) return MOE_OK;
    if (const int r = check_tables(shape, batch, cache)) return r;
    if (const int r = check_rows(q, q_row_stride, shape->q_heads, shape->head_dim)) return r;
    if (!out) return MOE_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4)) return MOE_ERR_ALIGN;
    if (ws_bytes < moe_kv_workspace_bytes(shape)) return MOE_ERR_WORKSPACE;
    if (!ws) return MOE_ERR_NULL;
    if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
    return hip_status(moe::launch_kv_attention(args_of(shape, batch, cache), q, q_row_stride, out,
                                               (shape->flags & MOE_OUT_F32) ? 1 : 0, lse, ws, (hipStream_t)stream));
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
