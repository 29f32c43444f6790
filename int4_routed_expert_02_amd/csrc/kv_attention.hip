// kv_attention.hip -- attention over the paged cache.
//
// For a row q at position p and the positions j it sees: z_j = scale q.k_j,
// out = sum exp(z_j - m) v_j / sum exp(z_j - m) with m = max z_j, taken in one
// pass over the cache with a running m, sum and accumulator (each rescaled
// when m grows), all in f32.
//
// Both kernels, the one for few rows and the one for many, compute S^T = K Q^T and
// O^T = V^T P^T on the matrix cores, so a lane holds scores of one query row: the
// weights of a row go from the first product's accumulator into the second
// product's operand without leaving the lane.  The rows of the K operand are taken
// in an order that makes each lane's scores belong to consecutive positions, so a
// lane reads V^T (stored [D][P]) in 16-byte pieces of 16 consecutive positions,
// which lie in one page whatever its size, with one pair of scales.
//
// An int8 code is exact in bf16, so codes, keys and queries enter the products as
// they are; a page's key scale (times log2(e) * scale) is applied to its scores in
// f32 and its value scale to its weights.  A weight enters the second product as
// the sum of two bf16 values, 2^-16 relative at any distance from the maximum.
// One bf16 value (2^-8) makes an output's error half as large again as its own
// rounding, and f16 loses weights far below the maximum.
//
// What bounds them.  Few rows (k_attn_dec): the cache's bytes.  One row each of 8
// sequences of 75639..131072 positions, 8 x 128 in 8 bits: 1.69 GB in 303 us, 5.6 TB/s; three to
// five drafted rows of 16 sequences, a window of 8192 positions of 8 x 128 in bf16: 0.54 GB in
// 109 us, 5.0 TB/s; 32 sequences of 2324..4096 positions, 4 x 64 in 8 bits: 50 MB in 20 us, a few
// tiles a wave between two launches.  Many rows (k_attn_tile): vector
// and matrix instructions together.  Two waves on one SIMD overlap them only in part
// (118 us of products and 144 us of vector work alone take 233 us side by side), so a
// tile costs about its vector work and 0.7 of its products: 720 TFLOP/s (the weights'
// second halves not counted) for 3707 rows over 16384 and 8465 positions with heads of
// 128, 400 for a causal prompt of 4096 rows with heads of 64, whose softmax is twice as
// large a share.
//
// Sinks (positions that stay visible in front of a window) are a range of tiles of their own before the window's,
// so a row's work goes by window and sinks: one row of 8 sequences of 75639..131072 positions, window 98304, 500 sinks,
// 8 x 128 in 8 bits: 1.53 GB in 277 us, 5.5 TB/s; 32 sequences, window 1024, four sinks, 4 x 64: 12.6 us;
// 3707 rows behind a window of 4096, 16 sinks, 8 x 128: 387 us, 645 TFLOP/s, in bf16 385.
#include "kv_device.h"

namespace moe {

constexpr float LOG2E = 1.44269504088896341f;
constexpr float M_NONE = -0x1.fffffep127f;  // running maximum before any score: no finite score lies below it
// The running maximum m is set this far (in powers of two) above the largest score, and
// raised only when a score passes it: no weight is above 1, so sums pass f32's range no
// sooner than sums of the values themselves, and most tiles skip the reduction over
// lanes and the rescaling of the accumulator.
constexpr float M_SLACK = 8.0f;
// Where every position is seen, a weight's exponent is z c - m in one fused step: z c unrounded,
// m a rounded one, so it may pass 0 by half of m's spacing.  Up to this size that is half a unit; in a
// tile with a larger maximum z c is rounded first, like the m that it is compared with.
constexpr float M_FUSED = 0x1p24f;

struct KvAttend {
    const uint16_t *q;
    int64_t q_stride;
    void *out;
    float *lse;
    float *part;  // partial results: [ns][rows][q_heads] of (D accumulators), then the same of (m, sum)
    int out_f32, ns, group;
    int sinks;    // behind a window: positions below this stay visible (0: none)
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    const bf16x2 r = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, r);
}

// Two weights as hi + lo in bf16: hi the upper halves as they are (truncated),
// lo the rest rounded; together 2^-16 relative.
__device__ __forceinline__ void split_bf16x2(float e0, float e1, uint32_t &hi, uint32_t &lo)
{
    hi = __builtin_amdgcn_perm(__float_as_uint(e1), __float_as_uint(e0), 0x07060302u);
    lo = cvt_bf16x2(e0 - __uint_as_float(__float_as_uint(e0) & 0xFFFF0000u),
                    e1 - __uint_as_float(__float_as_uint(e1) & 0xFFFF0000u));
}

// Eight int8 codes to bf16: small integers are their f32's upper halves.
__device__ __forceinline__ u32x4 codes_bf16(u32x2 w)
{
    u32x4 r;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const int32_t v = (int32_t)w[d];
        const float f0 = (float)((v << 24) >> 24), f1 = (float)((v << 16) >> 24), f2 = (float)((v << 8) >> 24), f3 = (float)(v >> 24);
        r[2 * d] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
        r[2 * d + 1] = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
    }
    return r;
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// What a row of the batch sees: positions [lo, hi), and with sinks those below both sinks and hi.
__device__ __forceinline__ void kv_sees(const KvArgs &a, const KvSeq &sq, int L, int i, int &lo, int &hi)
{
    const int p = sq.len - sq.n_pos + i;
    hi = a.causal ? min(max(p + 1, 0), L) : L;
    lo = a.window ? max(0, max(p + 1, 0) - a.window) : 0;  // the difference of two numbers from 0 on stays in 32 bits
}

// Tiles of 64 positions with sinks: the first n_sink hold the sinks, the others the window from w0
// on; tile t of these begins at w0 + 64 (t - n_sink).  What lies between is never read, so a row's work
// goes by its window however long the sequence is.  Where the sinks' tiles reach the window's,
// both are one run from position 0.  Otherwise the sinks' tiles lie below the last page that is full:
// an open page spans two tiles at most, and the window's first tile holds its end or begins before it.
__device__ __forceinline__ int sink_tiles(int sinks, int hi, int &w0)
{
    if (sinks == 0) return 0;
    const int n = (min(sinks, max(hi, 0)) + 63) >> 6;
    if (w0 > 64 * n) return n;
    w0 = 0;
    return 0;
}

// ---------------------------------------------------------------- few rows

// How the tiles of 64 positions of a sequence are cut into parts: first the
// tiles of full pages, then those of the open page (8 bits), from position F on.
// Tile t of full pages begins at t0 + 64 t, or at 64 t for the first n_sink.
struct DecTiles {
    int t0, F, n_codes, total, parts, per, n_sink;
};

// Waves of a workgroup: they take a part's tiles in turn, and join their results in LDS.
constexpr int DEC_WAVES = 8;

__device__ __forceinline__ DecTiles dec_tiles(const KvArgs &a, const KvSeq &sq, int L, int ns, int bits, int sinks)
{
    int lo, hi, lo1, hi1;
    kv_sees(a, sq, L, 0, lo, hi);
    kv_sees(a, sq, L, max(sq.n - 1, 0), lo1, hi1);
    DecTiles t;
    t.F = bits == 8 ? min(kv_full(a, sq), hi1) : hi1;
    int w0 = lo & ~63;
    t.n_sink = sink_tiles(sinks, hi1, w0);
    t.t0 = w0 - 64 * t.n_sink;
    t.n_codes = t.n_sink + (t.F > w0 ? (t.F - w0 + 63) >> 6 : 0);
    int n_open = 0;
    if (bits == 8) {
        t.F = max(kv_full(a, sq), w0);
        n_open = hi1 > t.F ? (hi1 - t.F + 63) >> 6 : 0;
    }
    t.total = t.n_codes + n_open;
    // a part gives each wave a tile at least
    t.parts = max(1, min(ns, (t.total + DEC_WAVES - 1) / DEC_WAVES));
    t.per = (t.total + t.parts - 1) / t.parts;
    return t;
}

// One wave's running softmax of 16 * NT query rows; a lane has rows (lane % 16)
// + 16 n and, of a tile, the positions 16 g .. 16 g + 15 with g = lane / 16.
template <int D, int NT>
struct DecState {
    f32x4 o[NT][D / 16];  // o[n][dt][i]: value d = 16 dt + 4 g + i of the lane's row n
    float m[NT], l[NT];   // maximum (the same in a row's four lanes), this lane's share of the sum

    __device__ void clear()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t] = zero4();
            m[n] = M_NONE;
            l[n] = 0.f;
        }
    }

    // xm: this lane's new largest scores
    __device__ __forceinline__ void raise(const float (&xm)[NT])
    {
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) up |= xm[n] > m[n];
        if (!__builtin_amdgcn_ballot_w64(up)) return;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x = xm[n];
            x = fmaxf(x, __shfl_xor(x, 16, WAVE));
            x = fmaxf(x, __shfl_xor(x, 32, WAVE));
            const float mn = x > m[n] ? x + M_SLACK : m[n], f = __builtin_amdgcn_exp2f(m[n] - mn);
            m[n] = mn;
            l[n] *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t] *= f;
        }
    }
};

template <int D, int BITS, int NT, bool SINK>
__global__ __launch_bounds__(DEC_WAVES *WAVE, D == 64 && NT == 1 ? 4 : 2) void k_attn_dec(KvArgs a, KvAttend t)
{
    constexpr int DT = D / 16, KS = D / 32;  // d tiles, contraction steps of a score
    extern __shared__ __align__(16) float dec_lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r16 = lane & 15;
    int b = blockIdx.x;
    const int split = b % t.ns;
    b /= t.ns;
    const int kh = b % a.kv_heads, s = b / a.kv_heads;
    const KvSeq sq = kv_seq(a, s);
    if (sq.n == 0) return;
    const int L = kv_limit(a, sq), log2p = a.page_log2, P = 1 << log2p;
    const int sinks = SINK ? t.sinks : 0;
    const DecTiles tl = dec_tiles(a, sq, L, t.ns, BITS, sinks);
    auto tile_at = [&](int tile) { return (SINK && tile < tl.n_sink ? 0 : tl.t0) + 64 * tile; };
    if (split >= tl.parts) return;
    const int begin = split * tl.per, end = min(tl.total, begin + tl.per);
    const int rows = sq.n * t.group;

    // the lane's query rows: what they see, and their operand
    int lo[NT], hi[NT];
    u32x4 q[NT][KS];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = min(r16 + 16 * n, rows - 1), i = r / t.group, h = kh * t.group + r % t.group;
        kv_sees(a, sq, L, i, lo[n], hi[n]);
        const uint16_t *src = t.q + (sq.row0 + i) * t.q_stride + h * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) q[n][k] = *(const u32x4 *)(src + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
    }
    if (a.scale < 0.f) {  // the sign goes to q, so that a maximum of products is one of scores
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < KS; ++k) q[n][k] ^= 0x80008000u;
    }
    const float zscale = fabsf(a.scale) * LOG2E;
    // positions that every row sees need no masks
    int lo_all, hi_all, x0, x1;
    kv_sees(a, sq, L, sq.n - 1, lo_all, x1);
    kv_sees(a, sq, L, 0, x0, hi_all);

    DecState<D, NT> st;
    st.clear();

    // Scores of a tile -> weights in the second product's operand order, as the
    // sum of two bf16 values (2^-16 relative): the matrix cores have time for the
    // second product here, where the cache's bytes are what is waited for.
    auto softmax = [&](f32x4 (&z)[NT][4], float c, float vs, int b0, bool full, bool valid, uint32_t (&p)[NT][2][8]) {
        const int j0 = b0 + 16 * g;
        float xm[NT];
        if (full) {
            bool large = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float m = z[n][0][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) m = fmaxf(m, z[n][i / 4][i % 4]);
                xm[n] = m * c;
                large |= fabsf(xm[n]) > M_FUSED;
            }
            if (__builtin_amdgcn_ballot_w64(large)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int u = 0; u < 4; ++u) z[n][u] *= c;
                c = 1.0f;
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                xm[n] = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool see = valid && (j0 + i >= lo[n] || (SINK && j0 + i < sinks)) && j0 + i < hi[n];
                    z[n][i / 4][i % 4] = see ? z[n][i / 4][i % 4] * c : -INFINITY;
                    xm[n] = fmaxf(xm[n], z[n][i / 4][i % 4]);
                }
            }
        }
        st.raise(xm);
        const float cc = full ? c : 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float e[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float zz = z[n][i / 4][i % 4 + j];
                    e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(zz, cc, -st.m[n]));
                    st.l[n] += e[j];
                    if (BITS == 8) e[j] *= vs;
                    if (!full) e[j] = zz == -INFINITY ? 0.f : e[j];  // 0 * NaN scale
                }
                split_bf16x2(e[0], e[1], p[n][0][i / 2], p[n][1][i / 2]);
            }
        }
    };
    // o += V^T P^T for one d tile: vb the 64 positions' values in two steps
    auto values = [&](int d, const u32x4 (&vb)[2], const uint32_t (&p)[NT][2][8]) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    st.o[n][d] = mfma_bf16(vb[k], u32x4{p[n][w][4 * k], p[n][w][4 * k + 1], p[n][w][4 * k + 2],
                                                        p[n][w][4 * k + 3]}, st.o[n][d]);
    };
    // operand row r16 of step u is position 16 kchunk + 4 u + krow of the tile
    const int krow = r16 & 3, kchunk = r16 >> 2;

    // ---- tiles of int8 codes
    if constexpr (BITS == 8) {
        const int last = min(end, tl.n_codes);
        int tile = begin + wave;
        if (tile < last) {
            const int8_t *kc = (const int8_t *)a.k, *vc = (const int8_t *)a.v;
            const int64_t head_at = (int64_t)kh * D << log2p;
            const int64_t page_elems = ((int64_t)a.kv_heads * D) << log2p;
            auto page_at = [&](int tl_, int chunk) {
                const int j = tile_at(tl_) + 16 * chunk;
                return j < tl.F ? kv_page(a, s, j >> log2p) : -1;
            };
            u32x4 kq[4][D / 64], vq[DT];
            float ks, vs;
            auto load_k = [&](int tl_, int id) {
                const int j = tile_at(tl_) + 16 * kchunk;
                const int8_t *src = kc + max(id, 0) * page_elems + head_at + ((j & (P - 1)) + krow) * D + 16 * g;
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) kq[u][k] = *(const u32x4 *)(src + 4 * u * D + 64 * k);
            };
            auto load_v = [&](int tl_, int id) {
                const int j = tile_at(tl_) + 16 * g;
                const int8_t *src = vc + max(id, 0) * page_elems + head_at + (r16 << log2p) + (j & (P - 1));
#pragma unroll
                for (int d = 0; d < DT; ++d) vq[d] = *(const u32x4 *)(src + ((16 * d) << log2p));
                ks = a.k_scale[(int64_t)max(id, 0) * a.kv_heads + kh];
                vs = a.v_scale[(int64_t)max(id, 0) * a.kv_heads + kh];
            };
            int idk = page_at(tile, kchunk), idg = page_at(tile, g);
            load_k(tile, idk);
            load_v(tile, idg);
            int next = tile + DEC_WAVES;
            int idk1 = page_at(min(next, last - 1), kchunk), idg1 = page_at(min(next, last - 1), g);
            while (true) {
                const bool more = next < last;
                f32x4 z[NT][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) z[n][u] = zero4();
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const u32x4 w = kq[u][k >> 1];
                        const u32x4 kb = codes_bf16((k & 1) ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]});
#pragma unroll
                        for (int n = 0; n < NT; ++n) z[n][u] = mfma_bf16(kb, q[n][k], z[n][u]);
                    }
                }
                if (more) load_k(next, idk1);
                const int b0 = tile_at(tile);
                const bool valid = idg >= 0;
                const bool full = ((b0 >= lo_all) | (SINK && b0 + 64 <= sinks)) && b0 + 64 <= min(hi_all, tl.F) && !__builtin_amdgcn_ballot_w64(!valid);
                uint32_t p[NT][2][8];
                softmax(z, valid ? ks * zscale : 0.f, valid ? vs : 0.f, b0, full, valid, p);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const u32x4 vb[2] = {codes_bf16(u32x2{vq[d][0], vq[d][1]}), codes_bf16(u32x2{vq[d][2], vq[d][3]})};
                    values(d, vb, p);
                }
                if (!more) break;
                idg = idg1;
                load_v(next, idg);
                tile = next;
                next += DEC_WAVES;
                idk1 = page_at(min(next, last - 1), kchunk);
                idg1 = page_at(min(next, last - 1), g);
            }
        }
    }

    // ---- tiles of bf16 values: every page of a bf16 cache, the open page of an 8-bit one
    const int slot = BITS == 8 ? kv_slot(a, s) : -1;
    int first16 = BITS == 8 ? tl.n_codes : 0;
    int tile16 = begin + wave;
    if (tile16 < first16) tile16 += (first16 - tile16 + DEC_WAVES - 1) / DEC_WAVES * DEC_WAVES;
    // The next tile's loads fly while one is used where the registers hold both (heads of 128, 16 rows);
    // elsewhere the other waves of the SIMD fill the wait.
    constexpr bool AHEAD = BITS == 16 && D == 128 && NT == 1;
    if (tile16 < end && (BITS == 16 || a.n_slots > 0)) {
        const uint16_t *const ka = BITS == 8 ? a.k_tail : (const uint16_t *)a.k;
        const uint16_t *const va = BITS == 8 ? a.v_tail : (const uint16_t *)a.v;
        auto first_of = [&](int tile) { return BITS == 8 ? tl.F + 64 * (tile - first16) : tile_at(tile); };
        // the block of a chunk: a page of the cache, or the sequence's open page (only where its id is there)
        auto block_of = [&](int b0, int chunk) -> int {
            const int j = b0 + 16 * chunk;
            const int id = j < L ? kv_page(a, s, j >> log2p) : -1;
            if (BITS == 8) return id >= 0 && slot >= 0 ? slot * 2 + ((j >> log2p) & 1) : -1;
            return id;
        };
        u32x4 kb[4][KS], vb[DT][2];
        auto load_k = [&](int b0, int block) {
            const uint16_t *src = ka + kv_block_at(a, max(block, 0), kh) + (((b0 + 16 * kchunk) & (P - 1)) + krow) * D + 16 * g;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < KS; ++k) kb[u][k] = *(const u32x4 *)(src + 4 * u * D + 64 * (k >> 1) + 8 * (k & 1));
        };
        auto load_v = [&](int b0, int block) {
            const uint16_t *src = va + kv_block_at(a, max(block, 0), kh) + (r16 << log2p) + ((b0 + 16 * g) & (P - 1));
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int k = 0; k < 2; ++k) vb[d][k] = *(const u32x4 *)(src + ((16 * d) << log2p) + 8 * k);
        };
        int b0 = first_of(tile16), bg = block_of(b0, g);
        if (AHEAD) {
            load_k(b0, block_of(b0, kchunk));
            load_v(b0, bg);
        }
        while (true) {
            if (!AHEAD) {
                bg = block_of(b0, g);
                load_k(b0, block_of(b0, kchunk));
                load_v(b0, bg);
            }
            const int next = tile16 + DEC_WAVES;
            const bool more = next < end;
            const int b1 = first_of(next);
            int bk1 = -1, bg1 = -1;
            if (AHEAD && more) {
                bk1 = block_of(b1, kchunk);
                bg1 = block_of(b1, g);
            }
            f32x4 z[NT][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    z[n][u] = zero4();
#pragma unroll
                    for (int k = 0; k < KS; ++k) z[n][u] = mfma_bf16(kb[u][k], q[n][k], z[n][u]);
                }
            }
            if (AHEAD && more) load_k(b1, bk1);
            const bool valid = bg >= 0;
            const bool full = ((b0 >= lo_all) | (SINK && b0 + 64 <= sinks)) && b0 + 64 <= min(hi_all, L) && !__builtin_amdgcn_ballot_w64(!valid);
            uint32_t p[NT][2][8];
            softmax(z, zscale, 1.0f, b0, full, valid, p);
            if (!full) {
                // places that no row sees may hold anything: 0 in their stead, since 0 * NaN is not 0
                int lo_min, hi_max, y;
                kv_sees(a, sq, L, 0, lo_min, y);
                kv_sees(a, sq, L, sq.n - 1, y, hi_max);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int j = b0 + 16 * g + 8 * k + 2 * w;
                        auto some = [&](int p) { return (p >= lo_min || (SINK && p < sinks)) && p < hi_max; };
                        const uint32_t keep = !valid ? 0u : (some(j) ? 0xFFFFu : 0u) | (some(j + 1) ? 0xFFFF0000u : 0u);
#pragma unroll
                        for (int d = 0; d < DT; ++d) vb[d][k][w] &= keep;
                    }
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) values(d, vb[d], p);
            if (!more) break;
            if (AHEAD) load_v(b1, bg1);
            tile16 = next;
            b0 = b1;
            bg = bg1;
        }
    }

    // ---- the waves' results together: maxima and sums first, then the accumulators pairwise
    float *sm = dec_lds, *sl = sm + DEC_WAVES * 16 * NT;
    float *so = sl + DEC_WAVES * 16 * NT;  // [DEC_WAVES / 2][DT][64 lanes][4]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        st.l[n] += __shfl_xor(st.l[n], 16, WAVE);
        st.l[n] += __shfl_xor(st.l[n], 32, WAVE);
        if (lane < 16) {
            sm[wave * 16 * NT + 16 * n + r16] = st.m[n];
            sl[wave * 16 * NT + 16 * n + r16] = st.l[n];
        }
    }
    __syncthreads();
    float m_all[NT], l_all[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m_all[n] = M_NONE;
        for (int w = 0; w < DEC_WAVES; ++w) m_all[n] = fmaxf(m_all[n], sm[w * 16 * NT + 16 * n + r16]);
        l_all[n] = 0.f;
        for (int w = 0; w < DEC_WAVES; ++w)
            l_all[n] += sl[w * 16 * NT + 16 * n + r16] *
                        __builtin_amdgcn_exp2f(sm[w * 16 * NT + 16 * n + r16] - m_all[n]);
        const float f = __builtin_amdgcn_exp2f(st.m[n] - m_all[n]);
#pragma unroll
        for (int d = 0; d < DT; ++d) st.o[n][d] *= f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        for (int half = DEC_WAVES / 2; half > 0; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int d = 0; d < DT; ++d) *(f32x4 *)(so + (((wave - half) * DT + d) * 64 + lane) * 4) = st.o[n][d];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int d = 0; d < DT; ++d) st.o[n][d] += *(const f32x4 *)(so + ((wave * DT + d) * 64 + lane) * 4);
            }
            __syncthreads();
        }
    }
    if (wave) return;
    int group = t.group;
    asm("" : "+s"(group));  // divided by anew: the constant of the first division would take a register through the loops
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r16 + 16 * n;
        if (r >= rows) continue;
        const int64_t at = (int64_t)(sq.row0 + r / group) * a.q_heads + kh * group + r % group;
        if (tl.parts > 1) {
            const int64_t pt = (int64_t)split * a.rows * a.q_heads + at;
#pragma unroll
            for (int d = 0; d < DT; ++d) *(f32x4 *)(t.part + pt * D + 16 * d + 4 * g) = st.o[n][d];
            if (g == 0) {
                float *ml = t.part + (int64_t)t.ns * a.rows * a.q_heads * D + pt * 2;
                ml[0] = m_all[n];
                ml[1] = l_all[n];
            }
            continue;
        }
        // a row that sees nothing has sum 0; a NaN sum stays one
        const float inv = l_all[n] == 0.f ? 0.f : 1.0f / l_all[n];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const f32x4 v = st.o[n][d] * inv;
            if (t.out_f32) *(f32x4 *)((float *)t.out + at * D + 16 * d + 4 * g) = v;
            else *(u32x2 *)((uint16_t *)t.out + at * D + 16 * d + 4 * g) = u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
        }
        if (t.lse && g == 0) t.lse[at] = l_all[n] == 0.f ? -INFINITY : (m_all[n] + __log2f(l_all[n])) * (1.0f / LOG2E);
    }
}

// ---------------------------------------------------------------- many rows

constexpr int TILE_MIN = 8;  // tiles of 64 positions in a part, at least

// The sequence that is r-th by length, longest first (ties in their order): its
// workgroups are started first, so that no long one is left for the end.  Up to 64
// sequences; more go in their order.
__device__ __forceinline__ int kv_ranked(const KvArgs &a, int r, int lane)
{
    if (a.n_seq > WAVE || a.n_seq == 1) return r;
    const int len = lane < a.n_seq ? a.kv_len[lane] : INT32_MIN;
    int rank = 0;
    for (int j = 0; j < a.n_seq; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane) ? 1 : 0;
    }
    return __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < a.n_seq && rank == r));
}

// Waves of a workgroup, 32 query rows each.
// With heads of 128 eight share a tile's staging (2048 and 1659 rows over 16384 and 8465 positions: 1024 us,
// four 1109); with heads of 64 four leave two workgroups a compute unit (a prompt of 4096 rows: 88 us, eight 122).
constexpr int tile_waves(int dim) { return dim == 64 ? 4 : 8; }

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32_bf16(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// The tiles that the rt-th `rows` query rows of a sequence and head look at, and
// how they are cut into parts.
struct RowTile {
    int lo, hi;         // positions some row sees lie in [lo, hi), or below both sinks and hi
    int t0, total;      // tile t begins at t0 + 64 t; tiles
    int parts, per;
    int n_sink;         // the first tiles, of sinks: tile t of these begins at 64 t
};

__device__ __forceinline__ RowTile row_tile(const KvArgs &a, const KvSeq &sq, int L, const KvAttend &at, int rt, int rows)
{
    const int group = at.group;
    const int i0 = rt * rows / group, i1 = min((rt * rows + rows - 1) / group, sq.n - 1);
    RowTile t;
    int x;
    kv_sees(a, sq, L, i0, t.lo, x);
    kv_sees(a, sq, L, i1, x, t.hi);
    int w0 = t.lo & ~63;
    t.n_sink = sink_tiles(at.sinks, t.hi, w0);
    t.t0 = w0 - 64 * t.n_sink;
    t.total = t.n_sink + (t.hi > w0 ? (t.hi - w0 + 63) >> 6 : 0);
    t.parts = max(1, min(at.ns, (t.total + TILE_MIN - 1) / TILE_MIN));
    t.per = (t.total + t.parts - 1) / t.parts;
    return t;
}

// Tiles of 64 positions in LDS, two of them (one is filled while the other is used):
//   K  [64 rows][D] bf16, position t of the tile in row t with bits 2 and 3 of t exchanged, so
//      that a lane's 16 scores of a 32 x 32 product belong to runs of 8 consecutive positions,
//      which is what the second product takes from a lane; 16-byte units of a row XORed with
//      the row, so that the 32 rows of an operand read lie on different banks;
//   V  [D rows][64 positions] bf16, 16-byte units XORed with the row;
//   of each of the tile's four chunks of 16 positions: score scales, log2 of the value scales, their
//   inverses, the value scales (negative where the chunk is absent); whether no scale needs care.
template <int D>
struct TileLds {
    static constexpr int KB = 64 * D * 2, BYTES = 2 * KB + 80;
    char *base;
    __device__ u32x4 *k(int buf, int row, int unit) const
    {
        return (u32x4 *)(base + buf * BYTES + row * D * 2 + ((unit ^ (row & (D / 8 - 1))) << 4));
    }
    __device__ u32x4 *v(int buf, int d, int unit) const
    {
        return (u32x4 *)(base + buf * BYTES + KB + d * 128 + ((unit ^ (d & 7)) << 4));
    }
    __device__ f32x4 *chunks(int buf) const { return (f32x4 *)(base + buf * BYTES + 2 * KB); }
};

template <int D, int BITS, bool SINK>
__global__ __launch_bounds__(tile_waves(D) * WAVE, 2) void k_attn_tile(KvArgs a, KvAttend t, int row_tiles, int units)
{
    constexpr int QS = D / 16, DT = D / 32;     // contraction steps of a score, d tiles
    constexpr int TW = tile_waves(D), TILE_ROWS = 32 * TW, THREADS = TW * WAVE;
    // What a thread stages of a tile: KC values of one position's K, and 8 * VU positions of VN rows of V.
    constexpr int KC = D / TW, VN = KC > 16 ? KC / 16 : 1, VU = KC / 8 / VN, VP = 8 / VU;  // VP threads a row of V
    static_assert(KC % 8 == 0 && VU <= 2, "");
    extern __shared__ __align__(16) char tile_lds[];
    const TileLds<D> lds{tile_lds};
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h32 = lane >> 5, c32 = lane & 31;
    // kv head fastest (a head's workgroups share an L2), then the longest rows first: where most positions
    // are cached ones, a long sequence's rows before a shorter one's (2048 and 1659 rows over 16384 and
    // 8465 positions: 1024 us, 1264 with the sequences in turn), else the last rows of every sequence (3 x 1000
    // rows: 31 us, 36 by sequences)
    int b = blockIdx.x;
    const int kh = b % a.kv_heads;
    b /= a.kv_heads;
    const int split = b % t.ns;
    b /= t.ns;
    int s, rt;
    if (units) {  // the sequences' row tiles one after another (ns is 1)
        s = kv_unit(a, b, t.group, __builtin_ctz(TILE_ROWS), 1, rt);
        if ((unsigned)rt >= (unsigned)row_tiles) return;
    } else {
        const bool by_length = a.max_len / 2 >= a.max_rows;
        s = kv_ranked(a, by_length ? b / row_tiles : b % a.n_seq, lane);
        rt = row_tiles - 1 - (by_length ? b % row_tiles : b / a.n_seq);
    }
    const KvSeq sq = kv_seq(a, s);
    const int rows = sq.n * t.group;
    if (rt * TILE_ROWS >= rows) return;
    const int L = kv_limit(a, sq), log2p = a.page_log2, P = 1 << log2p;
    if (!SINK) t.sinks = 0;
    const int sinks = SINK ? t.sinks : 0;
    const RowTile tl = row_tile(a, sq, L, t, rt, TILE_ROWS);
    auto tile_at = [&](int tile) { return (SINK && tile < tl.n_sink ? 0 : tl.t0) + 64 * tile; };
    if (split >= tl.parts) return;
    const int begin = split * tl.per, end = min(tl.total, begin + tl.per);
    const int F = BITS == 8 ? kv_full(a, sq) : 0;  // from here on: the open page
    const int slot = BITS == 8 ? kv_slot(a, s) : -1;

    // the wave's rows, the lane's row
    const int r0 = rt * TILE_ROWS + wave * 32, r = min(r0 + c32, rows - 1);
    const int i = r / t.group, head = kh * t.group + r % t.group;
    int lo, hi, lo_all, hi_all, x;
    kv_sees(a, sq, L, i, lo, hi);
    kv_sees(a, sq, L, min(r0, rows - 1) / t.group, x, hi_all);
    int lo_min = x, hi_max;
    kv_sees(a, sq, L, min(r0 + 31, rows - 1) / t.group, lo_all, hi_max);
    u32x4 q[QS];
    {
        const uint16_t *src = t.q + (sq.row0 + i) * t.q_stride + head * D + 8 * h32;
#pragma unroll
        for (int k = 0; k < QS; ++k) q[k] = *(const u32x4 *)(src + 16 * k);
        if (a.scale < 0.f) {
#pragma unroll
            for (int k = 0; k < QS; ++k) q[k] ^= 0x80008000u;
        }
    }
    const float zscale = fabsf(a.scale) * LOG2E;

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] = 0.f;
    float m = M_NONE, l = 0.f;

    // ---- staging
    const int kt = tid / TW, kq = tid % TW;                             // position, part of its values
    const int vd = tid / VP, vt = (tid % VP) * (8 * VU), vc = vt >> 4;  // row (+ THREADS / VP each), first position, its chunk
    typedef uint32_t raw_t __attribute__((ext_vector_type(2 * (BITS / 8))));  // eight values
    raw_t kr[KC / 8], vr[VN * VU];
    float ks = 0.f, vs = 0.f;            // wave 0: chunk lane % 4
    int idk = -1, idv = -1, idc = -1;    // pages of the position, of the V chunk, of chunk lane % 4 of the tile to load next
    auto page_of = [&](int tile, int chunk) {
        const int j = tile_at(tile) + 16 * chunk;
        return j < L ? kv_page(a, s, j >> log2p) : -1;
    };
    auto ids_of = [&](int tile) {
        idk = page_of(tile, kt >> 4);
        idv = page_of(tile, vc);
        if (wave == 0) idc = page_of(tile, lane & 3);
    };
    const int64_t page_elems = ((int64_t)a.kv_heads * D) << log2p, head_at = (int64_t)kh * D << log2p;
    constexpr int EB = BITS / 8;
    auto load = [&](int tile) {
        const int b0 = tile_at(tile), jk = b0 + kt, jv = b0 + vt;
        const char *sk = (const char *)a.k + (max(idk, 0) * page_elems + head_at + (jk & (P - 1)) * D + kq * KC) * EB;
#pragma unroll
        for (int n = 0; n < KC / 8; ++n) kr[n] = *(const raw_t *)(sk + 8 * n * EB);
        const char *sv = (const char *)a.v + (max(idv, 0) * page_elems + head_at + (vd << log2p) + (jv & (P - 1))) * EB;
#pragma unroll
        for (int n = 0; n < VN; ++n)
#pragma unroll
            for (int u = 0; u < VU; ++u)
                vr[n * VU + u] = *(const raw_t *)(sv + (((int64_t)(THREADS / VP * n) << log2p) + 8 * u) * EB);
        if (BITS == 8 && wave == 0) {
            ks = a.k_scale[(int64_t)max(idc, 0) * a.kv_heads + kh];
            vs = a.v_scale[(int64_t)max(idc, 0) * a.kv_heads + kh];
        }
    };
    auto bf16s = [&](raw_t v) -> u32x4 {
        if constexpr (BITS == 8) return codes_bf16(v);
        else return v;
    };
    const int krow = (kt & 0x33) | ((kt & 4) << 1) | ((kt & 8) >> 1);
    // wave 0, lanes 0..3: what a chunk's scores and weights are multiplied by
    auto put_chunk = [&](int buf, bool valid, float c, float v) {
        if (wave) return;
        const bool nice = valid && v >= 0x1p-60f && v <= 0x1p60f;
        const int care = __builtin_amdgcn_ballot_w64(lane < 4 && !nice) ? 1 : 0;
        if (lane < 4) {
            float *f = (float *)lds.chunks(buf) + lane;
            f[0] = c;
            f[4] = __log2f(v);
            f[8] = __builtin_amdgcn_rcpf(v);
            f[12] = valid ? v : -1.0f;
            if (lane == 0) f[16] = __int_as_float(care);
        }
    };
    // Eight bf16 values from position j on, 0 in the place of those no row here
    // sees: these may hold anything, and 0 * NaN is not 0.
    auto seen = [&](u32x4 v, int j) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int jj = j + 2 * w;
            auto some = [&](int p) { return (p >= tl.lo || (SINK && p < sinks)) && p < tl.hi; };
            v[w] &= (some(jj) ? 0xFFFFu : 0u) | (some(jj + 1) ? 0xFFFF0000u : 0u);
        }
        return v;
    };
    auto put = [&](int buf, int tile) {
#pragma unroll
        for (int n = 0; n < KC / 8; ++n) *lds.k(buf, krow, kq * (KC / 8) + n) = bf16s(kr[n]);
        const int j = tile_at(tile) + vt;
        const bool whole = BITS == 8 || (idv >= 0 && (j >= tl.lo || (SINK && j + 8 * VU <= sinks)) && j + 8 * VU <= tl.hi);
#pragma unroll
        for (int n = 0; n < VN; ++n)
#pragma unroll
            for (int u = 0; u < VU; ++u) {
                u32x4 v = bf16s(vr[n * VU + u]);
                if (BITS == 16 && !whole) v = idv < 0 ? u32x4{0, 0, 0, 0} : seen(v, j + 8 * u);
                *lds.v(buf, vd + THREADS / VP * n, (vt >> 3) + u) = v;
            }
        if (BITS == 8) put_chunk(buf, idc >= 0, ks * zscale, vs);
        else put_chunk(buf, idc >= 0, zscale, 1.0f);
    };
    // a tile with chunks of the open page, loaded where it is needed
    auto put_open = [&](int buf, int tile) {
        const int b0 = tile_at(tile), jk = b0 + kt, jv = b0 + vt;
        const bool openk = jk >= F, openv = jv >= F;
#pragma unroll
        for (int n = 0; n < KC / 8; ++n) {
            const int at = (jk & (P - 1)) * D + kq * KC + 8 * n;
            u32x4 v = {0, 0, 0, 0};
            if (idk >= 0 && openk && slot >= 0)
                v = *(const u32x4 *)(a.k_tail + kv_block_at(a, (int64_t)slot * 2 + ((jk >> log2p) & 1), kh) + at);
            else if (idk >= 0 && !openk)
                v = codes_bf16(*(const u32x2 *)((const char *)a.k + idk * page_elems + head_at + at));
            *lds.k(buf, krow, kq * (KC / 8) + n) = v;
        }
#pragma unroll
        for (int n = 0; n < VN; ++n)
#pragma unroll
            for (int u = 0; u < VU; ++u) {
                const int at = ((vd + THREADS / VP * n) << log2p) + (jv & (P - 1)) + 8 * u;
                u32x4 v = {0, 0, 0, 0};
                if (idv >= 0 && openv && slot >= 0)
                    v = seen(*(const u32x4 *)(a.v_tail + kv_block_at(a, (int64_t)slot * 2 + ((jv >> log2p) & 1), kh) + at),
                             jv + 8 * u);
                else if (idv >= 0 && !openv)
                    v = codes_bf16(*(const u32x2 *)((const char *)a.v + idv * page_elems + head_at + at));
                *lds.v(buf, vd + THREADS / VP * n, (vt >> 3) + u) = v;
            }
        const bool openc = b0 + 16 * (lane & 3) >= F, valid = idc >= 0 && (!openc || slot >= 0);
        float cks = 1.f, cvs = 1.f;
        if (valid && !openc) {
            cks = a.k_scale[(int64_t)idc * a.kv_heads + kh];
            cvs = a.v_scale[(int64_t)idc * a.kv_heads + kh];
        }
        put_chunk(buf, valid, cks * zscale, cvs);
    };

    // ---- one tile: scores, weights, values
    auto step = [&](int buf, int tile) {
        const int b0 = tile_at(tile);
        if (b0 >= hi_max || (b0 + 64 <= lo_min && !(SINK && b0 < sinks))) return;  // nothing for this wave
        f32x16 z[2];
#pragma unroll
        for (int T = 0; T < 2; ++T)
#pragma unroll
            for (int j = 0; j < 16; ++j) z[T][j] = 0.f;
#pragma unroll
        for (int k = 0; k < QS; ++k)
#pragma unroll
            for (int T = 0; T < 2; ++T) z[T] = mfma32_bf16(*lds.k(buf, 32 * T + c32, 2 * k + h32), q[k], z[T]);
        // z[n / 2][8 (n % 2) + j]: chunk n, position b0 + 16 n + 8 h32 + j
        f32x4 c = lds.chunks(buf)[0];
        const int care = __builtin_amdgcn_readfirstlane(*(const int *)(lds.chunks(buf) + 4));
        float xm = -INFINITY;
        auto raise = [&]() {
            if (!__builtin_amdgcn_ballot_w64(xm > m)) return;
            xm = fmaxf(xm, __shfl_xor(xm, 32, WAVE));
            const float mn = xm > m ? xm + M_SLACK : m, f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
        };
        auto values = [&](int n, const float (&e)[8]) {
            u32x4 p[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi_, lo_;
                split_bf16x2(e[2 * j], e[2 * j + 1], hi_, lo_);
                p[0][j] = hi_;
                p[1][j] = lo_;
            }
            u32x4 vb[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) vb[d] = *lds.v(buf, 32 * d + c32, 2 * n + h32);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] = mfma32_bf16(vb[d], p[w], o[d]);
        };
        // (tiles of sinks take the way with masks: asked for here, the compiler's other order of the two ways
        // costs 70 registers to memory, and 2048 and 1659 rows behind a window of 4096 positions 728 us)
        if (!care && b0 >= lo_all && b0 + 64 <= hi_all) {
            // every row sees every position: the value scale goes into the exponent, and a chunk's
            // sum is divided by it once
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float mx = z[n >> 1][(n & 1) * 8];
#pragma unroll
                for (int j = 1; j < 8; ++j) mx = fmaxf(mx, z[n >> 1][(n & 1) * 8 + j]);
                xm = fmaxf(xm, mx * c[n]);
            }
            if (__builtin_amdgcn_ballot_w64(fabsf(xm) > M_FUSED)) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[n >> 1][(n & 1) * 8 + j] *= c[n];
                    c[n] = 1.0f;
                }
            }
            raise();
            const f32x4 lv = lds.chunks(buf)[1], iv = lds.chunks(buf)[2];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float sub = BITS == 8 ? lv[n] - m : -m;
                float e[8], sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[n >> 1][(n & 1) * 8 + j], c[n], sub));
                    sum += e[j];
                }
                l = BITS == 8 ? __builtin_fmaf(sum, iv[n], l) : l + sum;
                values(n, e);
            }
            return;
        }
        const f32x4 scale = lds.chunks(buf)[3];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool valid = !(scale[n] < 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = b0 + 16 * n + 8 * h32 + j;
                const bool see = SINK ? valid & ((pos >= lo) | (pos < sinks)) & (pos < hi) : valid && pos >= lo && pos < hi;
                const float v = see ? z[n >> 1][(n & 1) * 8 + j] * c[n] : -INFINITY;
                z[n >> 1][(n & 1) * 8 + j] = v;
                xm = fmaxf(xm, v);
            }
        }
        raise();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = z[n >> 1][(n & 1) * 8 + j];
                e[j] = __builtin_amdgcn_exp2f(v - m);
                l += e[j];
                e[j] = v == -INFINITY ? 0.f : e[j] * scale[n];  // 0 * NaN scale
            }
            values(n, e);
        }
    };

    // tiles without an open page: the next one's loads fly while one is used
    const int closed = BITS == 8 ? min(end, max(begin, (F - tl.t0) >> 6)) : end;
    if (begin < closed) {
        ids_of(begin);
        load(begin);
        put(begin & 1, begin);
        if (begin + 1 < closed) ids_of(begin + 1);
        __syncthreads();
        for (int tile = begin; tile < closed; ++tile) {
            const bool more = tile + 1 < closed;
            if (more) load(tile + 1);
            step(tile & 1, tile);
            if (more) {
                put((tile + 1) & 1, tile + 1);
                if (tile + 2 < closed) ids_of(tile + 2);
            }
            __syncthreads();
        }
    }
    if (BITS == 8) {
        for (int tile = closed; tile < end; ++tile) {
            ids_of(tile);
            put_open(0, tile);
            __syncthreads();
            step(0, tile);
            __syncthreads();
        }
    }

    l += __shfl_xor(l, 32, WAVE);
    if (r0 + c32 >= rows) return;
    const int64_t at = (int64_t)(sq.row0 + i) * a.q_heads + head;
    const bool whole = tl.parts == 1;
    const int64_t pt = (int64_t)split * a.rows * a.q_heads + at;
    const float f = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = 32 * d + 8 * j + 4 * h32;
            const f32x4 v = f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]} * f;
            if (!whole) *(f32x4 *)(t.part + pt * D + e) = v;
            else if (t.out_f32) *(f32x4 *)((float *)t.out + at * D + e) = v;
            else *(u32x2 *)((uint16_t *)t.out + at * D + e) = u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
        }
    if (h32) return;
    if (!whole) {
        float *ml = t.part + (int64_t)t.ns * a.rows * a.q_heads * D + pt * 2;
        ml[0] = m;
        ml[1] = l;
    } else if (t.lse) {
        t.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * (1.0f / LOG2E);
    }
}

// The parts of a sequence's rows together, in order.  D / 4 lanes a row and head.
template <int D>
__global__ __launch_bounds__(256) void k_attn_parts(KvArgs a, KvAttend t, int groups, int few)
{
    const int s = blockIdx.x / groups;
    const KvSeq sq = kv_seq(a, s);
    const int L = kv_limit(a, sq);
    const int64_t idx = (int64_t)(blockIdx.x % groups) * 256 + threadIdx.x;
    const int64_t rh = idx / (D / 4);
    const int i = (int)(rh / a.q_heads), h = (int)(rh % a.q_heads), d = (int)(idx % (D / 4)) * 4;
    if (i >= sq.n) return;
    const int parts = few ? dec_tiles(a, sq, L, t.ns, a.kv_bits, t.sinks).parts
                          : row_tile(a, sq, L, t, (i * t.group + h % t.group) / (32 * tile_waves(D)), 32 * tile_waves(D)).parts;
    if (parts == 1) return;
    const int64_t at = (int64_t)(sq.row0 + i) * a.q_heads + h, step = (int64_t)a.rows * a.q_heads;
    const float *ml = t.part + t.ns * step * D;
    // eight parts' loads at a time are in flight together; a part past the last adds nothing
    float m = M_NONE, l = 0.f;
    f32x4 o = zero4();
    for (int p0 = 0; p0 < parts; p0 += 8) {
        float pm[8], pl[8], mn = m;
        f32x4 po[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t pt = min(p0 + u, parts - 1) * step + at;
            pm[u] = p0 + u < parts ? ml[pt * 2] : M_NONE;
            pl[u] = p0 + u < parts ? ml[pt * 2 + 1] : 0.f;
            po[u] = *(const f32x4 *)(t.part + pt * D + d);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mn = fmaxf(mn, pm[u]);
        const float f0 = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f0;
        o *= f0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (p0 + u >= parts) break;
            const float f = __builtin_amdgcn_exp2f(pm[u] - m);
            l += pl[u] * f;
            o += po[u] * f;
        }
    }
    o *= l == 0.f ? 0.f : 1.0f / l;
    if (t.out_f32) *(f32x4 *)((float *)t.out + at * D + d) = o;
    else *(u32x2 *)((uint16_t *)t.out + at * D + d) = u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
    if (t.lse && d == 0) t.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * (1.0f / LOG2E);
}


// The same for few rows and many parts: a workgroup a row and head, its lanes
// share out the parts.
template <int D>
__global__ __launch_bounds__(256) void k_attn_parts_few(KvArgs a, KvAttend t)
{
    constexpr int LANES = D / 4, PL = 256 / LANES;  // lanes of a row, parts at a time
    __shared__ f32x4 so[256];
    __shared__ float sm[PL], sl[PL];
    const int h = blockIdx.x % a.q_heads, i = (blockIdx.x / a.q_heads) % a.max_rows, s = blockIdx.x / a.q_heads / a.max_rows;
    const KvSeq sq = kv_seq(a, s);
    const int L = kv_limit(a, sq), d = threadIdx.x % LANES * 4, pl = threadIdx.x / LANES;
    if (i >= sq.n) return;
    const int parts = dec_tiles(a, sq, L, t.ns, a.kv_bits, t.sinks).parts;
    if (parts == 1) return;
    const int64_t at = (int64_t)(sq.row0 + i) * a.q_heads + h, step = (int64_t)a.rows * a.q_heads;
    const float *ml = t.part + t.ns * step * D;
    float m = M_NONE, l = 0.f;
    f32x4 o = zero4();
    for (int p = pl; p < parts; p += PL) {
        const int64_t pt = p * step + at;
        const float pm = ml[pt * 2], pv = ml[pt * 2 + 1];
        const f32x4 po = *(const f32x4 *)(t.part + pt * D + d);
        const float mn = fmaxf(m, pm), f0 = __builtin_amdgcn_exp2f(m - mn), f = __builtin_amdgcn_exp2f(pm - mn);
        m = mn;
        l = l * f0 + pv * f;
        o = o * f0 + po * f;
    }
    so[threadIdx.x] = o;
    if (d == 0) {
        sm[pl] = m;
        sl[pl] = l;
    }
    __syncthreads();
    if (pl) return;
    for (int u = 1; u < PL; ++u) m = fmaxf(m, sm[u]);
    l = 0.f;
    o = zero4();
#pragma unroll
    for (int u = 0; u < PL; ++u) {
        const float f = __builtin_amdgcn_exp2f(sm[u] - m);
        l += sl[u] * f;
        o += so[u * LANES + threadIdx.x] * f;
    }
    o *= l == 0.f ? 0.f : 1.0f / l;
    if (t.out_f32) *(f32x4 *)((float *)t.out + at * D + d) = o;
    else *(u32x2 *)((uint16_t *)t.out + at * D + d) = u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
    if (t.lse && d == 0) t.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * (1.0f / LOG2E);
}

// ---------------------------------------------------------------- launches

constexpr int DEC_TARGET = 512;  // workgroups that fill the chip: 2 per compute unit
constexpr int DEC_UNITS = 256;   // compute units

// Rounds of a part's waves over its tiles, of `tiles` cut into `parts`.
static int64_t dec_rounds(int64_t tiles, int64_t parts) { return ((tiles + parts - 1) / parts + DEC_WAVES - 1) / DEC_WAVES; }

// Parts behind a window with sinks.  Windows make the sequences alike, so parts only fill the chip: as many as run at once,
// one workgroup a compute unit.  A second one there costs more than its parts save (us for one row with heads of 64 in 8 bits
// behind 4096: 192 key/value heads whole 28.7, in two parts 29.6; 8 rows 37.4 and 46.9; heads of 128 42.4 and 51.7).
// And the parts have to save rounds worth their join, which costs 1.5 to 3 us: a round is 1.2 to 2.5 us with heads of 64 in
// 8 bits, 3 and more with other heads and bits (128 key/value heads, whole and in two parts, behind 1024: 11.4 / 11.8 saving one
// round with heads of 64 in 8 bits, 15.3 / 14.3 in 16, 17.8 / 17.0 with heads of 128 in 8 bits, 23.3 / 20.8 in 16; behind 2048,
// saving two: 17.0 / 15.5, 22.3 / 19.5, 25.8 / 22.4, 37.1 / 28.6).  Over 720 calls of 8 to 384 key/value heads,
// windows of 300 to 8192 and 1 and 8 rows, the parts taken here cost 1% more than the best ones; most where a few more
// parts than compute units would run (160 heads of 64 behind 8192: 47.8 us whole, 36.3 in three parts).
static int window_parts(const KvArgs &a, int sinks, int64_t len)
{
    int64_t span = len;  // positions between the first and the last that some row sees, behind the sinks
    if (a.causal && span > (int64_t)a.window + a.max_rows - 1) span = (int64_t)a.window + a.max_rows - 1;
    int64_t tiles = (span + 62) / 64 + 1 + ((int64_t)(sinks < len ? sinks : len) + 63) / 64;
    if (tiles > (len + 63) / 64) tiles = (len + 63) / 64;
    const int64_t base = (int64_t)a.n_seq * a.kv_heads, most = (tiles + DEC_WAVES - 1) / DEC_WAVES;
    int64_t ns = base > 0 ? DEC_UNITS / base : 1;
    if (ns > most) ns = most;
    const int saved = a.head_dim == 64 && a.kv_bits == 8 ? 2 : 1;
    return ns > 1 && dec_rounds(tiles, 1) - dec_rounds(tiles, ns) >= saved ? (int)ns : 1;
}

// Parts that a sequence's tiles may be cut into, so that few sequences still fill the chip.
static int dec_parts(const KvArgs &a, int sinks)
{
    int64_t len = a.max_len < ((int64_t)a.max_pages << a.page_log2) ? a.max_len : (int64_t)a.max_pages << a.page_log2;
    if (sinks) return window_parts(a, sinks, len);
    if (a.window && a.causal && len > (int64_t)a.window + a.max_rows) len = (int64_t)a.window + a.max_rows;
    const int64_t tiles = len / 64 + 3, most = (tiles + DEC_WAVES - 1) / DEC_WAVES;
    const int64_t base = (int64_t)a.n_seq * a.kv_heads;
    int64_t ns = base > 0 ? (DEC_TARGET + base - 1) / base : 1;
    if (ns > most) ns = most;
    return (int)(ns < 1 ? 1 : ns);
}

static int64_t row_tiles_of(const KvArgs &a)
{
    const int rows = 32 * tile_waves(a.head_dim);
    return ((int64_t)a.max_rows * (a.q_heads / a.kv_heads) + rows - 1) / rows;
}

// Parts that the positions of a many-row call are cut into, as long as its
// workgroups are fewer than this.  A part's accumulators go through memory: with heads of 128
// that costs more than an even load gains once the chip is full (4000 causal rows, 504
// workgroups: 195 us whole, 267 in three parts), with heads of 64 less (4096 causal rows, 512
// workgroups: 111 us whole, 87 in three parts).
static int tile_parts(const KvArgs &a)
{
    const int64_t target = a.head_dim == 64 ? 1536 : 512;
    const int64_t len = a.max_len < ((int64_t)a.max_pages << a.page_log2) ? a.max_len : (int64_t)a.max_pages << a.page_log2;
    const int64_t most = (len / 64 + TILE_MIN) / TILE_MIN, base = (int64_t)a.n_seq * a.kv_heads * row_tiles_of(a);
    int64_t ns = base > 0 ? target / base : 1;
    if (ns > most) ns = most;
    return (int)(ns < 1 ? 1 : ns);
}

constexpr int FEW_ROWS = 32;  // rows of a key/value head that the few-row kernel holds

static bool few_rows(const KvArgs &a) { return (int64_t)a.max_rows * (a.q_heads / a.kv_heads) <= FEW_ROWS; }

static int parts_of(const KvArgs &a, int sinks) { return few_rows(a) ? dec_parts(a, sinks) : tile_parts(a); }

size_t kv_attention_workspace(const KvArgs &a, int sinks)
{
    const int ns = parts_of(a, sinks);
    return ns > 1 ? (size_t)ns * a.rows * a.q_heads * (a.head_dim + 2) * 4 : 256;
}

template <int D, int BITS, int NT, bool SINK>
static hipError_t attend_few(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    const size_t lds = (2 * DEC_WAVES * 16 * NT + (DEC_WAVES / 2) * (D / 16) * 64 * 4) * sizeof(float);
    const int64_t grid = (int64_t)a.n_seq * a.kv_heads * t.ns;
    hipLaunchKernelGGL((k_attn_dec<D, BITS, NT, SINK>), dim3((unsigned)grid), dim3(DEC_WAVES * WAVE), lds, st, a, t);
    return hipGetLastError();
}

template <int D, int BITS, bool SINK>
static hipError_t attend_many(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    // Row tiles are laid out evenly, for each sequence as many as the longest may have, as long as that fits one
    // dimension of a launch; else by the sequences' own rows, with a search for a tile's sequence.
    const int64_t tiles = row_tiles_of(a);
    int64_t grid = tiles * a.n_seq * a.kv_heads * t.ns, units = 0;
    if (grid > KV_GRID_X) {  // below 2^19 for the rows and 2^22 for the sequences
        units = ((int64_t)a.rows * t.group) / (32 * tile_waves(D)) + a.n_seq;
        grid = units * a.kv_heads;
    }
    constexpr size_t lds = 2 * TileLds<D>::BYTES;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = lds > 64 << 10 ? allow_lds((const void *)k_attn_tile<D, BITS, SINK>, (int)lds, done) : hipSuccess;
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attn_tile<D, BITS, SINK>), dim3((unsigned)grid), dim3(tile_waves(D) * WAVE), lds, st, a, t,
                       (int)tiles, (int)units);
    return hipGetLastError();
}

template <int D, int BITS, bool SINK>
static hipError_t attend(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    const int64_t rows = (int64_t)a.max_rows * t.group;
    hipError_t e;
    if (few_rows(a)) {
        e = rows <= 16 ? attend_few<D, BITS, 1, SINK>(a, t, st) : attend_few<D, BITS, 2, SINK>(a, t, st);
    } else {
        e = attend_many<D, BITS, SINK>(a, t, st);
    }
    if (e != hipSuccess || t.ns == 1) return e;
    // More than one round of loads for a lane that takes all parts, so the parts go over lanes (one
    // sequence of 30000 positions: 12.8 us, 19.9 in one lane).
    const int64_t each = (int64_t)a.n_seq * a.max_rows * a.q_heads;
    if (few_rows(a) && t.ns > 8 && each <= 65536) {
        hipLaunchKernelGGL((k_attn_parts_few<D>), dim3((unsigned)each), dim3(256), 0, st, a, t);
        return hipGetLastError();
    }
    const int64_t groups = ((int64_t)a.max_rows * a.q_heads * (D / 4) + 255) / 256;
    hipLaunchKernelGGL((k_attn_parts<D>), dim3((unsigned)(groups * a.n_seq)), dim3(256), 0, st, a, t, (int)groups,
                       few_rows(a) ? 1 : 0);
    return hipGetLastError();
}

template <bool SINK>
static hipError_t attend_any(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    if (a.head_dim == 64) return a.kv_bits == 8 ? attend<64, 8, SINK>(a, t, st) : attend<64, 16, SINK>(a, t, st);
    return a.kv_bits == 8 ? attend<128, 8, SINK>(a, t, st) : attend<128, 16, SINK>(a, t, st);
}

hipError_t launch_kv_attention(const KvArgs &args, int sinks, const uint16_t *q, int64_t q_stride, void *out, int out_f32,
                               float *lse, void *ws, hipStream_t st)
{
    KvArgs a = args;
    if (a.n_pages == 0) a.max_len = 0;  // no page can be present: every row sees nothing
    KvAttend t = {};
    t.q = q;
    t.q_stride = q_stride;
    t.out = out;
    t.out_f32 = out_f32;
    t.lse = lse;
    t.part = (float *)ws;
    t.sinks = a.window ? sinks : 0;  // without a window every position is seen anyway
    t.ns = parts_of(args, t.sinks);
    t.group = a.q_heads / a.kv_heads;
    // at most as many sequences together as one dimension of a launch holds (more than that are never cut into parts)
    const int together = (int)(KV_GRID_X / a.kv_heads);
    for (int s0 = 0; s0 < args.n_seq; s0 += together) {
        a.n_seq = args.n_seq - s0 < together ? args.n_seq - s0 : together;
        a.row_start = args.row_start + s0;
        a.kv_len = args.kv_len + s0;
        a.pages = args.pages + (int64_t)s0 * a.max_pages;
        if (args.slots) {
            a.slots = args.slots + s0;
        } else if (s0 && a.n_slots) {  // sequence s has slot s
            const int64_t first = s0 < args.n_slots ? s0 : args.n_slots;
            a.n_slots = args.n_slots - (int)first;
            a.k_tail = args.k_tail + (first * 2 * a.kv_heads * a.head_dim << a.page_log2);
            a.v_tail = args.v_tail + (first * 2 * a.kv_heads * a.head_dim << a.page_log2);
        }
        const hipError_t e = t.sinks ? attend_any<true>(a, t, st) : attend_any<false>(a, t, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
