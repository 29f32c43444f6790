// kv_attention.hip -- attention over the paged cache.
//
// For a row q at position p and the positions j it sees: z_j = scale q.k_j,
// out = sum exp(z_j - m) v_j / sum exp(z_j - m) with m = max z_j, taken in one
// pass over the cache with a running m, sum and accumulator (each rescaled
// when m grows), all in f32.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T on the matrix cores, so a
// lane holds scores of one query row: the weights of a row go from the first
// product's accumulator into the second product's operand without leaving the
// lane.  The rows of the K operand are taken in an order that makes each lane's
// scores belong to consecutive positions, so a lane reads V^T (stored [D][P])
// in 16-byte pieces of 16 consecutive positions, which lie in one page whatever
// its size, with one pair of scales.
//
// An int8 code is exact in bf16 and in f16.  Scores: q and the codes in bf16,
// the page's scale times log2(e) * scale after the product.  Values: codes in
// f16, and the weight times the page's scale relative to the largest seen (a
// power of two), rounded to f16 (2^-11 relative; f16 keeps what is within 2^-24
// of the largest, the rest cannot be seen in a 32-bit sum either).  bf16 pages
// and open pages: weights rounded to bf16 (2^-8), so that values keep their range.
#include "kv_device.h"

namespace moe {

constexpr float LOG2E = 1.44269504088896341f;
constexpr float M_NONE = -1e30f;  // running maximum before any score
// The running maximum is raised only when a score passes it by more than this
// (in powers of two): weights stay below 2^8, far inside f16, and most tiles skip
// the reduction over lanes and the rescaling of the accumulator.
constexpr float M_SLACK = 8.0f;

struct KvAttend {
    const uint16_t *q;
    int64_t q_stride;
    void *out;
    float *lse;
    float *part;  // partial results: [ns][rows][q_heads] of (D accumulators), then the same of (m, l)
    int out_f32, ns, group;
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    const bf16x2 r = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, r);
}

// Two weights to f16, rounded toward zero (one instruction; below 2^-10
// relative, while a rounding to nearest takes three).
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
}

// Eight int8 codes to exact f16: code + 1152 by byte permutes, then the packed subtraction.
__device__ __forceinline__ u32x4 codes_f16(u32x2 w)
{
    const f16x8 v = __builtin_bit_cast(f16x8, unpack_int8x8_f16(w)) - (_Float16)INT8_F16_BIAS;
    return __builtin_bit_cast(u32x4, v);
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// What a row of the batch sees: positions [lo, hi).
__device__ __forceinline__ void kv_sees(const KvArgs &a, const KvSeq &sq, int L, int i, int &lo, int &hi)
{
    const int p = sq.len - sq.n_pos + i;
    hi = a.causal ? min(max(p + 1, 0), L) : L;
    lo = a.window ? max(0, p - a.window + 1) : 0;
}

// The smallest power of two that is not below v (2^-100 at least).
__device__ __forceinline__ float pow2_above(float v)
{
    uint32_t u = __float_as_uint(v);
    u = min((u & 0x7F800000u) + ((u & 0x7FFFFFu) ? 0x800000u : 0u), 253u << 23);
    return __uint_as_float(max(u, 27u << 23));
}

// ---------------------------------------------------------------- few rows

// How the tiles of 64 positions of a sequence are cut into parts: first the
// tiles of full pages, then those of the open page (8 bits), from position F on.
struct DecTiles {
    int t0, F, n_codes, total, parts, per;
};

constexpr int DEC_WAVES = 8;

__device__ __forceinline__ DecTiles dec_tiles(const KvArgs &a, const KvSeq &sq, int L, int ns)
{
    int lo, hi, lo1, hi1;
    kv_sees(a, sq, L, 0, lo, hi);
    kv_sees(a, sq, L, max(sq.n - 1, 0), lo1, hi1);
    DecTiles t;
    t.F = a.kv_bits == 8 ? min((L >> a.page_log2) << a.page_log2, hi1) : hi1;
    t.t0 = lo & ~63;
    t.n_codes = t.F > t.t0 ? (t.F - t.t0 + 63) >> 6 : 0;
    int n_open = 0;
    if (a.kv_bits == 8) {
        t.F = max((L >> a.page_log2) << a.page_log2, t.t0);
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
    f32x4 o[NT][D / 16];  // o[n][dt][i]: value d = 16 dt + 4 g + i of the lane's row n, over vref
    float m[NT], l[NT];   // maximum (the same in a row's four lanes), this lane's share of the sum
    float vref, ivref;    // power of two the accumulator's values are relative to, and its inverse

    __device__ void clear(float v)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t] = zero4();
            m[n] = M_NONE;
            l[n] = 0.f;
        }
        vref = v;
        ivref = 1.0f / v;
    }

    // New largest scores xm (this lane's) and, in 8 bits, its page's value scale.
    __device__ __forceinline__ void raise(const float (&xm)[NT], float vs)
    {
        bool up = vs > vref;
#pragma unroll
        for (int n = 0; n < NT; ++n) up |= xm[n] > m[n] + M_SLACK;
        if (!__builtin_amdgcn_ballot_w64(up)) return;
        float v = vs == vs ? vs : 0.f;
        v = fmaxf(v, __shfl_xor(v, 16, WAVE));
        v = fmaxf(v, __shfl_xor(v, 32, WAVE));
        float fv = 1.0f;
        if (v > vref) {
            const float r = pow2_above(v);
            fv = vref / r;
            vref = r;
            ivref = __uint_as_float((254u << 23) - __float_as_uint(r));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x = xm[n];
            x = fmaxf(x, __shfl_xor(x, 16, WAVE));
            x = fmaxf(x, __shfl_xor(x, 32, WAVE));
            const float mn = fmaxf(m[n], x), f = __builtin_amdgcn_exp2f(m[n] - mn);
            m[n] = mn;
            l[n] *= f;
            const float fo = f * fv;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t] *= fo;
        }
    }
};

template <int D, int BITS, int NT>
__global__ __launch_bounds__(DEC_WAVES *WAVE, 2) void k_attn_dec(KvArgs a, KvAttend t)
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
    const DecTiles tl = dec_tiles(a, sq, L, t.ns);
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
    st.clear(BITS == 8 ? 0x1p-100f : 1.0f);

    // scores of a tile -> weights in the second product's operand order
    auto softmax = [&](f32x4 (&z)[NT][4], float c, float vs, int b0, bool full, bool valid, uint32_t (&p)[NT][8],
                       bool f16) {
        const int j0 = b0 + 16 * g;
        float xm[NT];
        if (full) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float m = z[n][0][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) m = fmaxf(m, z[n][i / 4][i % 4]);
                xm[n] = m * c;
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                xm[n] = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool see = valid && j0 + i >= lo[n] && j0 + i < hi[n];
                    z[n][i / 4][i % 4] = see ? z[n][i / 4][i % 4] * c : -INFINITY;
                    xm[n] = fmaxf(xm[n], z[n][i / 4][i % 4]);
                }
            }
        }
        st.raise(xm, vs);
        const float w = vs * st.ivref, cc = full ? c : 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[n][i / 4][i % 4], cc, -st.m[n]));
                st.l[n] += e[i];
                e[i] *= w;
                if (!full) e[i] = z[n][i / 4][i % 4] == -INFINITY ? 0.f : e[i];  // 0 * NaN scale
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) p[n][i] = f16 ? cvt_f16x2(e[2 * i], e[2 * i + 1]) : cvt_bf16x2(e[2 * i], e[2 * i + 1]);
        }
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
                const int j = tl.t0 + 64 * tl_ + 16 * chunk;
                return j < tl.F ? kv_page(a, s, j >> log2p) : -1;
            };
            u32x4 kq[4][D / 64], vq[DT];
            float ks, vs;
            auto load_k = [&](int tl_, int id) {
                const int j = tl.t0 + 64 * tl_ + 16 * kchunk;
                const int8_t *src = kc + max(id, 0) * page_elems + head_at + ((j & (P - 1)) + krow) * D + 16 * g;
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) kq[u][k] = *(const u32x4 *)(src + 4 * u * D + 64 * k);
            };
            auto load_v = [&](int tl_, int id) {
                const int j = tl.t0 + 64 * tl_ + 16 * g;
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
                        const u32x4 kb = unpack_int8x8((k & 1) ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]});
#pragma unroll
                        for (int n = 0; n < NT; ++n) z[n][u] = mfma_bf16(kb, q[n][k], z[n][u]);
                    }
                }
                if (more) load_k(next, idk1);
                const int b0 = tl.t0 + 64 * tile;
                const bool valid = idg >= 0;
                const bool full = b0 >= lo_all && b0 + 64 <= min(hi_all, tl.F) && !__builtin_amdgcn_ballot_w64(!valid);
                uint32_t p[NT][8];
                softmax(z, valid ? ks * zscale : 0.f, valid ? vs : 0.f, b0, full, valid, p, true);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const u32x4 vb = codes_f16(k ? u32x2{vq[d][2], vq[d][3]} : u32x2{vq[d][0], vq[d][1]});
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            st.o[n][d] = mfma_f16(vb, u32x4{p[n][4 * k], p[n][4 * k + 1], p[n][4 * k + 2], p[n][4 * k + 3]},
                                                  st.o[n][d]);
                    }
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
    for (; tile16 < end; tile16 += DEC_WAVES) {
        const int b0 = BITS == 8 ? tl.F + 64 * (tile16 - first16) : tl.t0 + 64 * tile16;
        // the block of a chunk: a page of the cache, or the sequence's open page (only where its id is there)
        auto block_of = [&](int chunk) -> int64_t {
            const int j = b0 + 16 * chunk;
            const int id = j < L ? kv_page(a, s, j >> log2p) : -1;
            if (BITS == 8) return id >= 0 && slot >= 0 ? (int64_t)slot * 2 + ((j >> log2p) & 1) : -1;
            return id;
        };
        const int64_t bk = block_of(kchunk), bg = block_of(g);
        const bool valid = bg >= 0;
        const uint16_t *kt = (BITS == 8 ? a.k_tail : (const uint16_t *)a.k) + kv_block_at(a, max(bk, (int64_t)0), kh);
        const uint16_t *vt = (BITS == 8 ? a.v_tail : (const uint16_t *)a.v) + kv_block_at(a, max(bg, (int64_t)0), kh);
        const bool have = BITS == 16 || a.n_slots > 0;
        u32x4 kb[4][KS], vb[DT][2];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                kb[u][k] = have ? *(const u32x4 *)(kt + (((b0 + 16 * kchunk) & (P - 1)) + krow + 4 * u) * D + 64 * (k >> 1) +
                                                   16 * g + 8 * (k & 1))
                                : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                vb[d][k] = have ? *(const u32x4 *)(vt + ((16 * d + r16) << log2p) + ((b0 + 16 * g) & (P - 1)) + 8 * k)
                                : u32x4{0, 0, 0, 0};
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
        const bool full = b0 >= lo_all && b0 + 64 <= min(hi_all, L) && !__builtin_amdgcn_ballot_w64(!valid);
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
                    const uint32_t keep = !valid ? 0u
                                                 : (j >= lo_min && j < hi_max ? 0xFFFFu : 0u) |
                                                       (j + 1 >= lo_min && j + 1 < hi_max ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int d = 0; d < DT; ++d) vb[d][k][w] &= keep;
                }
        }
        uint32_t p[NT][8];
        softmax(z, zscale, valid ? 1.0f : 0.f, b0, full, valid, p, false);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    st.o[n][d] = mfma_bf16(vb[d][k], u32x4{p[n][4 * k], p[n][4 * k + 1], p[n][4 * k + 2], p[n][4 * k + 3]},
                                           st.o[n][d]);
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
        const float f = __builtin_amdgcn_exp2f(st.m[n] - m_all[n]) * st.vref;
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
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r16 + 16 * n;
        if (r >= rows) continue;
        const int64_t at = (int64_t)(sq.row0 + r / t.group) * a.q_heads + kh * t.group + r % t.group;
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

// The parts of a sequence's rows together, in order.  D / 4 lanes a row and head.
template <int D>
__global__ __launch_bounds__(256) void k_attn_parts(KvArgs a, KvAttend t, int groups)
{
    const int s = blockIdx.x / groups;
    const KvSeq sq = kv_seq(a, s);
    const int L = kv_limit(a, sq);
    if (sq.n == 0) return;
    const int parts = dec_tiles(a, sq, L, t.ns).parts;
    if (parts == 1) return;
    const int64_t idx = (int64_t)(blockIdx.x % groups) * 256 + threadIdx.x;
    const int64_t rh = idx / (D / 4);
    const int i = (int)(rh / a.q_heads), h = (int)(rh % a.q_heads), d = (int)(idx % (D / 4)) * 4;
    if (i >= sq.n) return;
    const int64_t at = (int64_t)(sq.row0 + i) * a.q_heads + h, step = (int64_t)a.rows * a.q_heads;
    const float *ml = t.part + t.ns * step * D;
    float m = M_NONE;
    for (int p = 0; p < parts; ++p) m = fmaxf(m, ml[(p * step + at) * 2]);
    float l = 0.f;
    f32x4 o = zero4();
    for (int p = 0; p < parts; ++p) {
        const float f = __builtin_amdgcn_exp2f(ml[(p * step + at) * 2] - m);
        l += ml[(p * step + at) * 2 + 1] * f;
        o += *(const f32x4 *)(t.part + (p * step + at) * D + d) * f;
    }
    o *= l == 0.f ? 0.f : 1.0f / l;
    if (t.out_f32) *(f32x4 *)((float *)t.out + at * D + d) = o;
    else *(u32x2 *)((uint16_t *)t.out + at * D + d) = u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
    if (t.lse && d == 0) t.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * (1.0f / LOG2E);
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void k_attn_row(KvArgs a, const uint16_t *q, int64_t q_stride, void *out,
                                                  int out_f32, float *lse)
{
    __shared__ float qs[D], w[256], red[4], acc4[256];
    const int tid = threadIdx.x, h = blockIdx.y, i = blockIdx.x % a.max_rows, s = blockIdx.x / a.max_rows;
    const KvSeq sq = kv_seq(a, s);
    if (i >= sq.n) return;
    const int row = sq.row0 + i, p = sq.len - sq.n_pos + i, L = kv_limit(a, sq), P = 1 << a.page_log2;
    const int kh = h / (a.q_heads / a.kv_heads);
    const int hi = a.causal ? min(L, p + 1) : L, lo = a.window ? max(0, p - a.window + 1) : 0;
    const int slot = BITS == 8 ? kv_slot(a, s) : -1;
    if (tid < D) qs[tid] = bf16_to_f32(q[row * q_stride + h * D + tid]) * a.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;  // acc: value tid % D over a share of the positions
    constexpr int SH = 256 / D;
    auto block_of = [&](int j, const uint16_t *&half, const uint16_t *&vhalf, int64_t &id) {
        const int pg = j >> a.page_log2;
        id = kv_page(a, s, pg);
        half = vhalf = nullptr;
        if (id < 0) return false;
        if (BITS == 16) {
            half = (const uint16_t *)a.k + kv_block_at(a, id, kh);
            vhalf = (const uint16_t *)a.v + kv_block_at(a, id, kh);
        } else if (((pg + 1) << a.page_log2) > L) {
            if (slot < 0) return false;
            const int64_t at = kv_block_at(a, (int64_t)slot * 2 + (pg & 1), kh);
            half = a.k_tail + at;
            vhalf = a.v_tail + at;
        }
        return true;
    };
    for (int c = lo; c < hi; c += 256) {
        const int j = c + tid;
        float z = -INFINITY;
        const uint16_t *half, *vhalf;
        int64_t id;
        if (j < hi && block_of(j, half, vhalf, id)) {
            z = 0.f;
            const int r = j & (P - 1);
            if (half) {
                for (int d = 0; d < D; ++d) z += qs[d] * bf16_to_f32(half[r * D + d]);
            } else {
                const int8_t *kc = (const int8_t *)a.k + kv_block_at(a, id, kh) + r * D;
                for (int d = 0; d < D; ++d) z += qs[d] * (float)kc[d];
                z *= a.k_scale[id * a.kv_heads + kh];
            }
        }
        float mx = z;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, WAVE));
        if ((tid & 63) == 0) red[tid >> 6] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float base = mn > -INFINITY ? mn : 0.f;
        const float e = z > -INFINITY || z != z ? __expf(z - base) : 0.f, f = m > -INFINITY ? __expf(m - base) : 0.f;
        w[tid] = e;
        __syncthreads();
        float sum = e;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, WAVE);
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        acc *= f;
        const int d = tid % D;
        for (int t = tid / D; t < 256 && c + t < hi; t += SH) {
            if (w[t] == 0.f || !block_of(c + t, half, vhalf, id)) continue;
            const int r = (c + t) & (P - 1);
            if (half) acc += w[t] * bf16_to_f32(vhalf[d * P + r]);
            else
                acc += w[t] * (float)((const int8_t *)a.v)[kv_block_at(a, id, kh) + d * P + r] *
                       a.v_scale[id * a.kv_heads + kh];
        }
        __syncthreads();
        l = l * f + red[0] + red[1] + red[2] + red[3];
        m = mn;
        __syncthreads();
    }
    acc4[tid] = acc;
    __syncthreads();
    if (tid < D) {
        float o = 0.f;
        for (int t = 0; t < SH; ++t) o += acc4[tid + t * D];
        o = l > 0.f || l != l ? o / l : 0.f;
        const int64_t at = ((int64_t)row * a.q_heads + h) * D + tid;
        if (out_f32) ((float *)out)[at] = o;
        else ((__bf16 *)out)[at] = (__bf16)o;
        if (lse && tid == 0) lse[(int64_t)row * a.q_heads + h] = l > 0.f || l != l ? m + __logf(l) : -INFINITY;
    }
}


// ---------------------------------------------------------------- launches

constexpr int DEC_TARGET = 512;  // workgroups that fill the chip: 2 per compute unit

// Parts that a sequence's tiles may be cut into, so that few sequences still fill the chip.
static int dec_parts(const KvArgs &a)
{
    int64_t len = a.max_len < ((int64_t)a.max_pages << a.page_log2) ? a.max_len : (int64_t)a.max_pages << a.page_log2;
    if (a.window && a.causal && len > (int64_t)a.window + a.max_rows) len = (int64_t)a.window + a.max_rows;
    const int64_t tiles = len / 64 + 3, most = (tiles + DEC_WAVES - 1) / DEC_WAVES;
    const int64_t base = (int64_t)a.n_seq * a.kv_heads;
    int64_t ns = base > 0 ? (DEC_TARGET + base - 1) / base : 1;
    if (ns > most) ns = most;
    return (int)(ns < 1 ? 1 : ns);
}

size_t kv_attention_workspace(const KvArgs &a)
{
    if ((int64_t)a.max_rows * (a.q_heads / a.kv_heads) > 32) return 256;
    const int ns = dec_parts(a);
    return ns > 1 ? (size_t)ns * a.rows * a.q_heads * (a.head_dim + 2) * 4 : 256;
}

template <int D, int BITS, int NT>
static hipError_t attend_few(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    const size_t lds = (2 * DEC_WAVES * 16 * NT + (DEC_WAVES / 2) * (D / 16) * 64 * 4) * sizeof(float);
    const int64_t grid = (int64_t)a.n_seq * a.kv_heads * t.ns;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_attn_dec<D, BITS, NT>), dim3((unsigned)grid), dim3(DEC_WAVES * WAVE), lds, st, a, t);
    return hipGetLastError();
}

template <int D, int BITS>
static hipError_t attend(const KvArgs &a, const KvAttend &t, hipStream_t st)
{
    const int64_t rows = (int64_t)a.max_rows * t.group;
    if (rows > 32) {
        const int64_t gx = (int64_t)a.n_seq * a.max_rows;
        if (gx > INT32_MAX / 256 || a.q_heads > 65535) return hipErrorInvalidValue;
        hipLaunchKernelGGL((k_attn_row<D, BITS>), dim3((unsigned)gx, a.q_heads), dim3(256), 0, st, a, t.q, t.q_stride,
                           t.out, t.out_f32, t.lse);
        return hipGetLastError();
    }
    const hipError_t e = rows <= 16 ? attend_few<D, BITS, 1>(a, t, st) : attend_few<D, BITS, 2>(a, t, st);
    if (e != hipSuccess || t.ns == 1) return e;
    const int64_t groups = ((int64_t)a.max_rows * a.q_heads * (D / 4) + 255) / 256;
    hipLaunchKernelGGL((k_attn_parts<D>), dim3((unsigned)(groups * a.n_seq)), dim3(256), 0, st, a, t, (int)groups);
    return hipGetLastError();
}

hipError_t launch_kv_attention(const KvArgs &args, const uint16_t *q, int64_t q_stride, void *out, int out_f32,
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
    t.ns = dec_parts(args);
    t.group = a.q_heads / a.kv_heads;
    if (a.head_dim == 64) return a.kv_bits == 8 ? attend<64, 8>(a, t, st) : attend<64, 16>(a, t, st);
    return a.kv_bits == 8 ? attend<128, 8>(a, t, st) : attend<128, 16>(a, t, st);
}

}  // namespace moe
