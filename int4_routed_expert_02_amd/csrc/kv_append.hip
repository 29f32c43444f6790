// kv_append.hip -- new keys and values into the paged cache, with the per-head
// norm and the position rotation on the way; and the stored values back.
//
// A head of one row is x (D values).  With a norm, y = x * rsqrt(mean x^2 + eps)
// * w; the first R values are rotated, (a, b) -> (a c - b s, a s + b c) with c, s
// of the row's position; the result is rounded to bf16 once.  In 8 bits a page
// of one head (P x D values) gets scale = max|v| / 127 and codes rint(v / scale)
// when its last row comes, from the bf16 values, so the codes are the same
// however the rows arrived.
//
// One workgroup per (sequence, touched page, head, k or v): a page's codes need
// all its rows anyway, and this is also the unit that a transposed store (v is
// [D][P]) wants in LDS.  Eight values of a row per lane (16-byte loads); D / 8
// lanes hold a row, so the norm's sum is a butterfly over them.  Queries take
// the same arithmetic in workgroups of the same launch.
//
// What bounds it: memory for prompts (each value read once, written once, the
// older rows of the one partial page read again): 7677 rows of 64 + 2 x 8 heads
// of 128, six chunks into a bf16 cache, move 0.31 GB in 70 us, 4.5 TB/s, and reading
// their pages back takes 16 us.  A decode step is bound by its launch: 32 rows of 16 + 2 x 4
// heads of 64 take 6.4 us on the device, three dependent reads (tables, rows, the page).
// Table rows shared by four query heads of a lane measured slower (75 us: fewer,
// longer waves), codes without divisions the same.
#include "kv_device.h"

namespace moe {

constexpr int KVA_THREADS = 256;

// A launch's workgroups: for pages, for each sequence's queries, all of them; and the pages of a sequence.
struct KvaGroups {
    int pages, queries, all, touched;
};

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 r = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, r);
}

// Eight values at element e of a head (16-byte aligned) after norm and
// rotation, in bf16.  All D / 8 lanes of the row call it together.
template <int D>
__device__ __forceinline__ u32x4 normed_rotated(const uint16_t *head, int e, const float *norm, const KvAppend &n,
                                                int pos)
{
    const u32x4 raw = *(const u32x4 *)(head + e);
    const bool rotated = e < n.rot_dim;
    if (!norm && !rotated) return raw;
    const int half = n.rot_dim >> 1;
    const int pe = n.pairs || !rotated ? e : e < half ? e + half : e - half;  // the partners' place
    const u32x4 praw = *(const u32x4 *)(head + pe);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(raw[i]);
        x[2 * i + 1] = bf16_hi(raw[i]);
        y[2 * i] = bf16_lo(praw[i]);
        y[2 * i + 1] = bf16_hi(praw[i]);
    }
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor(ss, o, WAVE);
        const float r = rsqrtf(ss * (1.0f / D) + n.eps);
        const f32x4 *w = (const f32x4 *)(norm + e), *pw = (const f32x4 *)(norm + pe);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * r * w[i / 4][i % 4];
            y[i] = y[i] * r * pw[i / 4][i % 4];
        }
    }
    if (rotated) {
        const bool in_table = (unsigned)pos < (unsigned)n.n_pos;
        const int64_t row = (int64_t)(in_table ? pos : 0) * half;
        if (n.pairs) {
            f32x4 c, s;
            if (in_table) {
                c = *(const f32x4 *)(n.cos + row + e / 2);
                s = *(const f32x4 *)(n.sin + row + e / 2);
            } else {
                c = s = f32x4{NAN, NAN, NAN, NAN};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * c[i] - b * s[i];
                x[2 * i + 1] = a * s[i] + b * c[i];
            }
        } else {
            const bool first = e < half;
            const int j = first ? e : e - half;
            f32x4 c[2], s[2];
            if (in_table) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    c[i] = *(const f32x4 *)(n.cos + row + j + 4 * i);
                    s[i] = *(const f32x4 *)(n.sin + row + j + 4 * i);
                }
            } else {
                c[0] = c[1] = s[0] = s[1] = f32x4{NAN, NAN, NAN, NAN};
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = y[i] * s[i / 4][i % 4];
                x[i] = x[i] * c[i / 4][i % 4] + (first ? -t : t);
            }
        }
    }
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = to_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
}

// The largest |value| of eight bf16 as its bits: NaN above infinity above the
// finite values, so a page's maximum keeps them.
__device__ __forceinline__ uint32_t abs_bits_max(uint32_t m, u32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    return m;
}

// A page of one head in LDS, [P][D + 2] bf16: rows are written along D; the
// extra dword a row puts the 16-row groups that a transposed read takes
// together on different banks.
template <int D>
struct PageTile {
    static constexpr int ROW = D + 2;
    uint16_t *t;
    __device__ void put(int row, int e, u32x4 v) const
    {
        uint32_t *p = (uint32_t *)(t + row * ROW + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = v[i];
    }
    __device__ u32x4 get(int row, int e) const
    {
        const uint32_t *p = (const uint32_t *)(t + row * ROW + e);
        return u32x4{p[0], p[1], p[2], p[3]};
    }
};

// Columns [lo, hi) of a page's transposed values: dst [D][P] at rows d, from
// the tile.  Whole groups of eight tokens are stored as vectors.
template <int D>
__device__ __forceinline__ void store_transposed(uint16_t *dst, int log2p, PageTile<D> tile, int lo, int hi)
{
    const int c0 = lo >> 3, nc = ((hi + 7) >> 3) - c0;
    for (int i = threadIdx.x; i < nc * D; i += KVA_THREADS) {
        const int d = i / nc, c = c0 + i - d * nc;
        uint16_t *out = dst + ((int64_t)d << log2p) + c * 8;
        if (c * 8 >= lo && c * 8 + 8 <= hi) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = (uint32_t)tile.t[(c * 8 + 2 * j) * tile.ROW + d] |
                       ((uint32_t)tile.t[(c * 8 + 2 * j + 1) * tile.ROW + d] << 16);
            }
            *(u32x4 *)out = v;
        } else {
            for (int j = 0; j < 8; ++j)
                if (c * 8 + j >= lo && c * 8 + j < hi) out[j] = tile.t[(c * 8 + j) * tile.ROW + d];
        }
    }
}

template <int D, int BITS, bool EVEN, bool IS_V>
__device__ __forceinline__ void append_page(const KvArgs &a, const KvAppend &n, int s, int t, int h, uint16_t *lds,
                                            uint32_t *red)
{
    constexpr int LPR = D / 8, RPP = KVA_THREADS / LPR;  // lanes a row, rows a pass
    const KvSeq sq = kv_seq(a, s);
    const int start = sq.len - sq.n_pos, log2p = a.page_log2, P = 1 << log2p;
    // In 8 bits the page that max_len cuts is stored whole: its codes need all its rows, and who reads below
    // max_len finds them there once the sequence is past the page.
    const int L = BITS == 16 ? kv_limit(a, sq)
                             : min(min(sq.len, (a.max_len + P - 1) & -P), a.max_pages << log2p);
    // this call's rows that have a place: positions [lo_all, hi_all)
    const int lo_all = max(start, 0), hi_all = min(L, start + sq.n);
    if ((!EVEN && t < 0) || hi_all <= lo_all) return;
    const int first = lo_all >> log2p, last = (hi_all - 1) >> log2p, page = first + t;
    if (EVEN ? page > last : t > last - first) return;
    const int id = kv_page(a, s, page), slot = BITS == 8 ? kv_slot(a, s) : -1;
    const PageTile<D> tile{lds};
    const int lane_row = threadIdx.x / LPR, e = (threadIdx.x % LPR) * 8;
    const uint16_t *src = IS_V ? n.v : n.k;
    const int64_t stride = IS_V ? n.v_stride : n.k_stride;

    auto row8 = [&](int p) -> u32x4 {  // position p's new row
        const int row = sq.row0 + p - start;
        const uint16_t *head = src + row * stride + h * D;
        if (IS_V) return *(const u32x4 *)(head + e);
        return normed_rotated<D>(head, e, n.k_norm, n, n.pos ? n.pos[row] : p);
    };

    if constexpr (BITS == 16) {
        if (id < 0) return;
        const int lo = max(lo_all, page << log2p), hi = min(hi_all, (page + 1) << log2p);
        const int64_t at = kv_block_at(a, id, h);
        for (int p = lo + lane_row; p < hi; p += RPP) {
            const u32x4 v = row8(p);
            if (IS_V) tile.put(p & (P - 1), e, v);
            else *(u32x4 *)((uint16_t *)a.k + at + (p & (P - 1)) * D + e) = v;
        }
        if (IS_V) {
            __syncthreads();
            store_transposed<D>((uint16_t *)a.v + at, log2p, tile, lo & (P - 1), ((hi - 1) & (P - 1)) + 1);
        }
        return;
    } else {
        if (slot < 0) return;
        uint16_t *tails = IS_V ? a.v_tail : a.k_tail;
        // Older rows are read from the first page's half when it fills up.  A
        // newer page of this call that keeps its rows in the same half must not
        // overwrite them first, so the first page's workgroup stores those rows
        // too, after it has read.
        const bool first_reads = ((first + 1) << log2p) <= hi_all && lo_all > (first << log2p);
        const int newer = last - ((last - first) & 1);
        auto store_rows = [&](int pg) {  // the new rows of page pg: into the tile, and its open page
            const int lo = max(lo_all, pg << log2p), hi = min(hi_all, (pg + 1) << log2p);
            const int64_t at = kv_block_at(a, (int64_t)slot * 2 + (pg & 1), h);
            uint32_t m = 0;
            for (int p = lo + lane_row; p < hi; p += RPP) {
                const u32x4 v = row8(p);
                m = abs_bits_max(m, v);
                tile.put(p & (P - 1), e, v);
            }
            return m;
        };
        auto keep_rows = [&](int pg) {  // from the tile into the open page
            const int lo = max(lo_all, pg << log2p), hi = min(hi_all, (pg + 1) << log2p);
            uint16_t *tail = tails + kv_block_at(a, (int64_t)slot * 2 + (pg & 1), h);
            if (IS_V) {
                store_transposed<D>(tail, log2p, tile, lo & (P - 1), ((hi - 1) & (P - 1)) + 1);
            } else {
                for (int p = lo + lane_row; p < hi; p += RPP)
                    *(u32x4 *)(tail + (p & (P - 1)) * D + e) = tile.get(p & (P - 1), e);
            }
        };
        const bool full = ((page + 1) << log2p) <= hi_all;
        const bool reads = t == 0 && first_reads;
        const bool keeps = page >= last - 1 && !(t > 0 && first_reads && page == newer);
        if (!full && !keeps) return;
        uint32_t m = store_rows(page);
        if (reads) {  // the page's older rows
            const uint16_t *tail = tails + kv_block_at(a, (int64_t)slot * 2 + (page & 1), h);
            const int older = lo_all & (P - 1);
            if (IS_V) {
                const int nc = (older + 7) >> 3;
                for (int i = threadIdx.x; i < nc * D; i += KVA_THREADS) {
                    const int d = i / nc, c = i - d * nc;
                    const u32x4 v = *(const u32x4 *)(tail + ((int64_t)d << log2p) + c * 8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t b = (j & 1) ? v[j / 2] >> 16 : v[j / 2] & 0xFFFFu;
                        if (c * 8 + j < older) {
                            tile.t[(c * 8 + j) * tile.ROW + d] = (uint16_t)b;
                            m = max(m, b & 0x7FFFu);
                        }
                    }
                }
            } else {
                for (int r = lane_row; r < older; r += RPP) {
                    const u32x4 v = *(const u32x4 *)(tail + r * D + e);
                    m = abs_bits_max(m, v);
                    tile.put(r, e, v);
                }
            }
        }
        if (full) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, WAVE));
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        }
        __syncthreads();
        if (keeps) keep_rows(page);
        if (full && id >= 0) {
            m = max(max(red[0], red[1]), max(red[2], red[3]));
            const float amax = bf16_to_f32((uint16_t)m);
            // a page with an infinity or NaN has no codes: its scale is NaN
            const float scale = m < 0x7F80u ? __fdiv_rn(amax, 127.0f) : NAN, inv = __frcp_rn(scale);
            if (threadIdx.x == 0) (IS_V ? a.v_scale : a.k_scale)[(int64_t)id * a.kv_heads + h] = scale;
            uint8_t *codes = (uint8_t *)(IS_V ? a.v : a.k) + kv_block_at(a, id, h);
            // sixteen codes a store: a sixteenth of a row's D (k) or of a page's tokens (v)
            for (int i = threadIdx.x; i < (P * D) / 16; i += KVA_THREADS) {
                u32x4 out;
                const int row = IS_V ? (i & ((P >> 4) - 1)) * 16 : i / (D / 16);
                const int col = IS_V ? i >> (log2p - 4) : (i % (D / 16)) * 16;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t word = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int o = w * 4 + j;
                        const float x = bf16_to_f32(IS_V ? tile.t[(row + o) * tile.ROW + col]
                                                         : tile.t[row * tile.ROW + col + o]);
                        word |= (amax == 0.0f ? 0u : qz_code(x, scale, inv, 127.0f) & 0xFFu) << (8 * j);
                    }
                    out[w] = word;
                }
                *(u32x4 *)(codes + (int64_t)i * 16) = out;
            }
        }
        if (reads && newer > first) {  // the rows that share the half just read
            __syncthreads();
            store_rows(newer);
            __syncthreads();
            keep_rows(newer);
        }
    }
}

// The sequence and touched page of the b-th unit: `touched` pages of every sequence, or as many as the rows of
// each can touch.
template <bool EVEN>
__device__ __forceinline__ int page_unit(const KvArgs &a, int b, int touched, int &t)
{
    if (!EVEN) return kv_unit(a, b, 1, a.page_log2, 2, t);
    t = b % touched;
    return b / touched;
}

template <int D, int BITS, bool EVEN>
__global__ __launch_bounds__(KVA_THREADS) void k_kv_append(KvArgs a, KvAppend n, KvaGroups g)
{
    extern __shared__ __align__(16) uint16_t kva_tile[];
    __shared__ uint32_t red[KVA_THREADS / WAVE];
    int b = EVEN ? (int)blockIdx.x : kv_block();
    if (b < g.pages) {
        const int is_v = b & 1;
        b >>= 1;
        const int h = b % a.kv_heads;
        int t;
        const int s = page_unit<EVEN>(a, b / a.kv_heads, g.touched, t);
        if (is_v) append_page<D, BITS, EVEN, true>(a, n, s, t, h, kva_tile, red);
        else append_page<D, BITS, EVEN, false>(a, n, s, t, h, kva_tile, red);
        return;
    }
    if (!EVEN && b >= g.all) return;
    // queries: g.queries workgroups a sequence, or all rows of the batch one after another
    b -= g.pages;
    int s = 0;
    if (EVEN) {
        s = b / g.queries;
        b %= g.queries;
    }
    const int64_t i = (int64_t)b * KVA_THREADS + threadIdx.x;
    const int64_t head_row = i / (D / 8);
    const int e = (int)(i % (D / 8)) * 8;
    int r = (int)(head_row / a.q_heads);
    const int h = (int)(head_row % a.q_heads);
    if (!EVEN) s = kv_unit(a, r, 1, 0, 0, r);
    const KvSeq sq = kv_seq(a, s);
    if (r < 0 || r >= sq.n) return;  // the lanes of a row leave together
    const int row = sq.row0 + r, p = sq.len - sq.n_pos + r;
    const u32x4 v = normed_rotated<D>(n.q + row * n.q_stride + h * D, e, n.q_norm, n, n.pos ? n.pos[row] : p);
    *(u32x4 *)(n.q_out + ((int64_t)row * a.q_heads + h) * D + e) = v;
}

// ---------------------------------------------------------------- read

template <int D, int BITS, bool EVEN, bool IS_V>
__device__ __forceinline__ void read_page(const KvArgs &a, uint16_t *out, int s, int t, int h, uint16_t *lds)
{
    const KvSeq sq = kv_seq(a, s);
    const int L = kv_limit(a, sq), start = sq.len - sq.n_pos, log2p = a.page_log2, P = 1 << log2p;
    // the first touched page is the one of the first row with a position (rows before it read as 0)
    if (!EVEN && (unsigned)t > (unsigned)(((sq.n - 1) >> log2p) + 1)) return;
    const int first = max(start, 0) >> log2p, page = first + t;
    const int lo = max(t == 0 ? start : (page << log2p), start), hi = min((page + 1) << log2p, start + sq.n);
    if (hi <= lo) return;
    const uint16_t *half = nullptr;
    int64_t id = kv_page(a, s, page);
    float scale = 1.0f;
    if (BITS == 8) {
        if (id >= 0 && (page << log2p) >= kv_full(a, sq)) {  // still open
            const int slot = kv_slot(a, s);
            if (slot >= 0) half = (IS_V ? a.v_tail : a.k_tail) + kv_block_at(a, (int64_t)slot * 2 + (page & 1), h);
            id = -1;
        }
        if (id >= 0) scale = (IS_V ? a.v_scale : a.k_scale)[id * a.kv_heads + h];
    } else if (id >= 0) {
        half = (const uint16_t *)(IS_V ? a.v : a.k) + kv_block_at(a, id, h);
    }
    const uint8_t *codes = BITS == 8 && id >= 0 ? (const uint8_t *)(IS_V ? a.v : a.k) + kv_block_at(a, id, h) : nullptr;
    const PageTile<D> tile{lds};
    auto decoded = [&](u32x2 w) {
        u32x4 r;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const int32_t c = (int32_t)w[d];
            r[2 * d] = to_bf16x2((float)((c << 24) >> 24) * scale, (float)((c << 16) >> 24) * scale);
            r[2 * d + 1] = to_bf16x2((float)((c << 8) >> 24) * scale, (float)(c >> 24) * scale);
        }
        return r;
    };
    if (IS_V) {
        // eight tokens of one d at a time into the tile
        const int nc = P >> 3;
        for (int i = threadIdx.x; i < nc * D; i += KVA_THREADS) {
            const int d = i / nc, c = i - d * nc;
            u32x4 v = {0, 0, 0, 0};
            if (codes) v = decoded(*(const u32x2 *)(codes + ((int64_t)d << log2p) + c * 8));
            else if (half) v = *(const u32x4 *)(half + ((int64_t)d << log2p) + c * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tile.t[(c * 8 + j) * tile.ROW + d] = (uint16_t)((j & 1) ? v[j / 2] >> 16 : v[j / 2]);
        }
        __syncthreads();
    }
    constexpr int LPR = D / 8, RPP = KVA_THREADS / LPR;
    const int e = (threadIdx.x % LPR) * 8;
    for (int p = lo + threadIdx.x / LPR; p < hi; p += RPP) {
        u32x4 v = {0, 0, 0, 0};
        if (p >= 0 && p < L) {
            const int r = p & (P - 1);
            if (IS_V) v = tile.get(r, e);
            else if (codes) v = decoded(*(const u32x2 *)(codes + r * D + e));
            else if (half) v = *(const u32x4 *)(half + r * D + e);
        }
        *(u32x4 *)(out + ((int64_t)(sq.row0 + p - start) * a.kv_heads + h) * D + e) = v;
    }
}

template <int D, int BITS, bool EVEN>
__global__ __launch_bounds__(KVA_THREADS) void k_kv_read(KvArgs a, uint16_t *k, uint16_t *v, KvaGroups g)
{
    extern __shared__ __align__(16) uint16_t kva_tile[];
    int b = EVEN ? (int)blockIdx.x : kv_block();
    if (!EVEN && b >= g.all) return;
    const int is_v = b & 1;
    b >>= 1;
    const int h = b % a.kv_heads;
    int t;
    const int s = page_unit<EVEN>(a, b / a.kv_heads, g.touched, t);
    if (is_v) read_page<D, BITS, EVEN, true>(a, v, s, t, h, kva_tile);
    else read_page<D, BITS, EVEN, false>(a, k, s, t, h, kva_tile);
}

// Workgroups are laid out evenly, as many for each sequence as the longest may need (pages that max_rows rows can touch
// wherever they start, and query rows), or by the sequences' own rows, which costs a search in row_start.  Evenly
// unless that makes more than twice as many and a thousand more (6 sequences of 876 to 1501 rows, bf16: 69 us
// evenly, 100 by rows; 32 of one row: 6.8, 7.5; one of 512 rows and 31 of one: 9.0, 8.1; one of 8192 rows and 63 of
// one: 1260, 153), so their number goes by the rows whatever max_rows is.
static bool groups_of(const KvArgs &a, bool queries, KvaGroups &g)
{
    const int64_t heads = (int64_t)a.kv_heads * 2, row = queries ? (int64_t)a.q_heads * (a.head_dim / 8) : 0;
    g.touched = ((a.max_rows - 2) >> a.page_log2) + 2;
    const int64_t each = (a.max_rows * row + KVA_THREADS - 1) / KVA_THREADS, pages = a.n_seq * heads * g.touched;
    const int64_t own_pages = ((a.rows >> a.page_log2) + 2 * (int64_t)a.n_seq) * heads;
    const int64_t own = own_pages + (a.rows * row + KVA_THREADS - 1) / KVA_THREADS;
    const bool even = pages + each * a.n_seq <= 2 * own + 1024 && pages + each * a.n_seq <= KV_GRID_X;
    g.pages = (int)(even ? pages : own_pages);
    g.queries = (int)(even ? each : 0);
    g.all = (int)(even ? pages + each * a.n_seq : own);
    return even;
}

template <int D>
static size_t tile_bytes(const KvArgs &a) { return ((size_t)PageTile<D>::ROW << a.page_log2) * 2; }

template <int D, int BITS>
static hipError_t append(const KvArgs &a, const KvAppend &n, hipStream_t st)
{
    KvaGroups g;
    if (groups_of(a, n.q, g))
        hipLaunchKernelGGL((k_kv_append<D, BITS, true>), kv_grid(g.all), dim3(KVA_THREADS), tile_bytes<D>(a), st, a, n, g);
    else
        hipLaunchKernelGGL((k_kv_append<D, BITS, false>), kv_grid(g.all), dim3(KVA_THREADS), tile_bytes<D>(a), st, a, n, g);
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvArgs &a, const KvAppend &n, hipStream_t st)
{
    if (a.head_dim == 64) return a.kv_bits == 8 ? append<64, 8>(a, n, st) : append<64, 16>(a, n, st);
    return a.kv_bits == 8 ? append<128, 8>(a, n, st) : append<128, 16>(a, n, st);
}

template <int D, int BITS>
static hipError_t read(const KvArgs &a, uint16_t *k, uint16_t *v, hipStream_t st)
{
    KvaGroups g;
    if (groups_of(a, false, g))
        hipLaunchKernelGGL((k_kv_read<D, BITS, true>), kv_grid(g.all), dim3(KVA_THREADS), tile_bytes<D>(a), st, a, k, v, g);
    else
        hipLaunchKernelGGL((k_kv_read<D, BITS, false>), kv_grid(g.all), dim3(KVA_THREADS), tile_bytes<D>(a), st, a, k, v, g);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs &a, uint16_t *k, uint16_t *v, hipStream_t st)
{
    if (a.head_dim == 64) return a.kv_bits == 8 ? read<64, 8>(a, k, v, st) : read<64, 16>(a, k, v, st);
    return a.kv_bits == 8 ? read<128, 8>(a, k, v, st) : read<128, 16>(a, k, v, st);
}

}  // namespace moe
