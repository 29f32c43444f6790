// linear_q4.hip -- few-token products with packed int4 weights and group scales:
//   y[t][n] = sum_g s[n][g] * sum_{k in g} x[t][k] * c[n][k]  (+ residual[t][n]).
//
// Weights are read once, so their bytes are its floor: N * K / 2 and the scales.  A
// wave takes 16 * RT output columns, all tokens and a slice of K: the codes go
// from memory into the operand of the 16 x 16 x 32 matrix product (tokens x k
// times k x columns), so any number of tokens up to 16 costs what one does.  A
// workgroup's waves have the same columns and share out K; their sums meet in
// LDS, in order, so one launch does it and few columns still fill the chip.
//
// A lane's 16 bytes are 32 codes of one column.  The four lanes of a column hold
// 128 consecutive ones; exchanged between the lanes (a 4 x 4 transpose of dwords,
// four lane swaps) they become four operands of 32 consecutive k each, so a
// product never mixes two groups.  Unpacking: nibble c + 8 in the mantissa of 1
// gives the bf16 of (c + 24) / 16, one shift and one bit operation for two codes;
// the offset comes out with -1.5 * sum x of the group, taken by one product
// against a constant whose result is where the group's accumulators start.  The
// scale (times 16) joins a group's sum in f32.  Where that leaves f32's range the
// output is infinite or NaN and is taken from the definition instead (lq_defined).
//
// What it reaches: 5 x 50257 x 2048, 58 MB in 14.9 us, 3.9 TB/s (reading alone in this
// pattern takes 10.4 us).  32 x 6144 x 8192, 26 MB in 14.7 us: every workgroup reads all
// activations (100 MB from the L2s); without products and activations the weights take
// 9.5 us.  1 x 1536 x 1024 takes 3 us on the device and is bound by the call.
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

constexpr int LQ_BLOCK = 128;  // k of one step: a 16-byte piece for each of a column's four lanes

// Eight nibbles -> eight bf16 of (code + 24) / 16, in the order of unpack_int4x8.
__device__ __forceinline__ u32x4 lq_unpack(uint32_t w)
{
    u32x4 r;
    r[0] = (((w << 3) ^ 0x00400040u) & 0x00780078u) | 0x3F803F80u;
    r[1] = (((w >> 1) ^ 0x00400040u) & 0x00780078u) | 0x3F803F80u;
    r[2] = (((w >> 5) ^ 0x00400040u) & 0x00780078u) | 0x3F803F80u;
    r[3] = (((w >> 9) ^ 0x00400040u) & 0x00780078u) | 0x3F803F80u;
    return r;
}

// Lane group g's dword j becomes lane group j's dword g.
__device__ __forceinline__ u32x4 lq_transpose(u32x4 v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// A load that touches 16 rows costs the memory pipeline as much for 4 bytes a row
// as for 64, about 64 cycles, so only the codes come straight into their lanes.  A
// wave's activations (TR rows of a block of 128 k) and scales come in runs
// along k and go through a piece of LDS of its own: no barriers, so the
// waves drift apart and one loads while another computes.
//
// More than 16 tokens, where 16 bytes of a column's scales last for four blocks: a wave has a run of
// consecutive blocks and takes their scales in such pieces (32 x 6144 x 8192, bf16 scales of 128: 14.4 us,
// 15.6 with the waves' blocks in turn and their scales one by one).  Elsewhere the waves take the blocks in
// turn (5 x 50257 x 2048: 15.3 us against 16.4; 24 x 6144 x 4096, f32 scales of 32: 8.5 against 8.8).
template <int GROUP, bool SB, int RT, int TR, int WAVES>
struct LqLds {
    static constexpr int GB = LQ_BLOCK / GROUP, TT = (TR + 15) / 16;
    static constexpr bool RUNS = TR > 16 && (SB ? 8 : 4) / GB >= 4;
    static constexpr int NS = RUNS ? (SB ? 8 : 4) : GB, SCB = NS / GB;           // scales of a load, blocks they are for
    static constexpr int SROW = RUNS ? NS + 1 : GB;                              // a column's scales in LDS
    static constexpr int XROW = LQ_BLOCK * 2 + 16;                               // bytes of a token's row
    static constexpr int X_BYTES = TR * XROW, WAVE_BYTES = X_BYTES + 16 * RT * SROW * 4;
    static constexpr int R_BYTES = WAVES * RT * TT * 1024;                       // the waves' sums
    // From 5 tokens on, as many workgroups as are resident together take tile after tile of columns, the next
    // tile's first loads under way while one is summed up (32 x 50257 x 2048: 31 us, 36.5 with a workgroup a
    // tile; 5 x 50257 x 2048: 14.7, 15.3).  With fewer tokens a workgroup a tile is no slower (1 x 50257 x 2048:
    // 13.6 us, 14.0 in a loop).
    static constexpr bool LOOP = RT == 2 && TR >= 16;
    // in a loop the sums have two places of their own, else they come where the activations were
    static constexpr int R_AT = LOOP ? WAVES * WAVE_BYTES : 0;
    static constexpr int BYTES = LOOP ? R_AT + 2 * R_BYTES : WAVES * WAVE_BYTES > R_BYTES ? WAVES * WAVE_BYTES : R_BYTES;
};

// N scales from an address of their own alignment
template <bool SB, int N>
__device__ __forceinline__ void lq_scales(const char *p, float (&s)[N])
{
    if constexpr (SB) {
        typedef uint16_t v_t __attribute__((ext_vector_type(N), aligned(2)));
        const v_t v = *(const v_t *)p;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = bf16_to_f32(v[i]);
    } else {
        typedef float v_t __attribute__((ext_vector_type(N), aligned(4)));
        const v_t v = *(const v_t *)p;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = v[i];
    }
}

// Whether a token has a NaN.  16 lanes have the same token; those that are here share its row.
__device__ __forceinline__ bool lq_has_nan(const u32x4 *x, int n, int lane)
{
    const uint32_t here = __builtin_amdgcn_ballot_w64(true) >> (lane & 48) & 0xFFFFu;
    const int step = __builtin_popcount(here);
    uint32_t m = 0;  // the largest |value| as its bits
    for (int j = __builtin_popcount(here & ((1u << (lane & 15)) - 1)); j < n; j += step) {
        const u32x4 v = x[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    }
    return __builtin_amdgcn_ballot_w64(m > 0x7F80u) >> (lane & 48) & 0xFFFFu;
}

// One output from the definition, in 64 bits.  With an infinite activation the offset makes infinity less
// infinity; finite ones above 1.7e38, or scales above 2.1e37, pass f32's range on the way with no need.  Every
// such output comes out infinite or NaN, and only these are taken anew, where the token has no NaN (32 x 6144 x
// 8192: 15 us, 37 with a NaN in every token, 393 with an infinity in one).
template <int GROUP, bool SB>
__device__ __forceinline__ float lq_defined(const LinearQ4 &a, int token, int n)
{
    int K = a.K, lane = threadIdx.x & 63;
    asm volatile("" : "+v"(token), "+v"(n), "+v"(lane), "+s"(K));  // nothing of this is made ready outside the rare branch
    const uint32_t *q = (const uint32_t *)(a.q + (int64_t)n * (K / 2));
    const u32x4 *x = (const u32x4 *)(a.x + (int64_t)token * a.x_stride);
    if (lq_has_nan(x, K / 8, lane)) return NAN;
    const char *s = (const char *)a.scales + (int64_t)n * (K / GROUP) * (SB ? 2 : 4);
    double y = 0.0;
    for (int g = 0; g < K / GROUP; ++g) {
        double sum = 0.0;
#pragma unroll 1
        for (int j = 0; j < GROUP / 8; ++j) {
            const uint32_t w = q[g * (GROUP / 8) + j];
            const u32x4 v = x[g * (GROUP / 8) + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum += (double)bf16_lo(v[i]) * (double)((int32_t)(w << (28 - 8 * i)) >> 28);
                sum += (double)bf16_hi(v[i]) * (double)((int32_t)(w << (24 - 8 * i)) >> 28);
            }
        }
        float sg[1];
        lq_scales<SB, 1>(s + g * (SB ? 2 : 4), sg);
        y += sum * (double)sg[0];
    }
    return (float)y;
}

// 16 * RT columns at a time, up to TR tokens; the workgroup's waves share out the blocks of K.
template <int GROUP, bool SB, int RT, int TR, int WAVES>
__global__ __launch_bounds__(WAVES *WAVE, TR <= 16 ? 4 : 2) void k_linear_q4(LinearQ4 a, int t0, int tile0)
{
    using Lds = LqLds<GROUP, SB, RT, TR, WAVES>;
    constexpr int TT = Lds::TT, GB = Lds::GB, THREADS = WAVES * WAVE, XU = TR / 4, SS = SB ? 2 : 4;
    constexpr int NS = Lds::NS, SCB = Lds::SCB, SROW = Lds::SROW;
    extern __shared__ __align__(16) char lq_lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, c16 = lane & 15;
    const int tok0 = t0 + blockIdx.y * TR, tokens = min(a.T - tok0, TR);
    const int groups = a.K / GROUP, tiles = (a.N - 1) / (16 * RT) + 1;
    const int blocks = (a.K + LQ_BLOCK - 1) / LQ_BLOCK;

    // Offsets of the lane's loads from a tile's first row: rows past an edge are some row that is there,
    // and their results are dropped.
    uint32_t wo[RT], xo[XU], so;
    const char *wbase, *sbase;
    auto columns = [&](int tile) {
        const int n0 = tile * 16 * RT, cols = min(16 * RT, a.N - n0);
#pragma unroll
        for (int r = 0; r < RT; ++r) wo[r] = (uint32_t)min(16 * r + c16, cols - 1) * (uint32_t)(a.K / 2) + 16 * g;
        so = (uint32_t)min(lane & (16 * RT - 1), cols - 1) * (uint32_t)(groups * SS);
        wbase = (const char *)a.q + (int64_t)n0 * (a.K / 2);
        sbase = (const char *)a.scales + (int64_t)n0 * groups * SS;
    };
#pragma unroll
    for (int i = 0; i < XU; ++i) xo[i] = (uint32_t)min(g + 4 * i, tokens - 1) * (uint32_t)(a.x_stride * 2) + 16 * c16;
    const char *xbase = (const char *)(a.x + (int64_t)tok0 * a.x_stride);

    u32x4 w[RT], x[XU];
    float s[NS];
    // the scales of the SCB blocks from b on, 0 past the last group
    auto all_scales = [&](int b) { lq_scales<SB, NS>(sbase + so + b * (GB * SS), s); };
    auto last_scales = [&](int b) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float v[1];
            lq_scales<SB, 1>(sbase + so + min(b * GB + i, groups - 1) * SS, v);
            s[i] = b * GB + i < groups ? v[0] : 0.f;
        }
    };
    auto load = [&](int b, bool scales) {
        const char *wt = wbase + b * (LQ_BLOCK / 2), *xt = xbase + b * (LQ_BLOCK * 2);
        if ((b + 1) * LQ_BLOCK <= a.K) {
#pragma unroll
            for (int r = 0; r < RT; ++r) w[r] = *(const u32x4 *)(wt + wo[r]);
#pragma unroll
            for (int i = 0; i < XU; ++i)
                if (4 * i < tokens) x[i] = *(const u32x4 *)(xt + xo[i]);
            if (scales) {
                if (SCB == 1 || (b + SCB) * GB <= groups) all_scales(b);
                else last_scales(b);
            }
        } else {
            // the last block ends early: activations (and scales) are 0 from K on, the codes there are the
            // block's first ones (its first 32 are always there)
            const int left = a.K - b * LQ_BLOCK;
#pragma unroll
            for (int r = 0; r < RT; ++r) w[r] = *(const u32x4 *)(wt + (32 * g < left ? wo[r] : wo[r] - 16 * g));
#pragma unroll
            for (int i = 0; i < XU; ++i) {
                x[i] = *(const u32x4 *)(xt + (8 * c16 < left ? xo[i] : xo[i] - 16 * c16));
                if (8 * c16 >= left) x[i] = u32x4{0, 0, 0, 0};
            }
            if (scales) last_scales(b);
        }
    };
    char *const mine = lq_lds + wave * Lds::WAVE_BYTES;
    char *const xput = mine + g * Lds::XROW + 16 * c16;
    float *const sc = (float *)(mine + Lds::X_BYTES);
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < XU; ++i)
            if (4 * i < tokens) *(u32x4 *)(xput + 4 * i * Lds::XROW) = interleave_bf16x8(x[i]);
    };
    auto put_scales = [&]() {
        if (lane < 16 * RT) {
#pragma unroll
            for (int i = 0; i < NS; ++i) sc[lane * SROW + i] = s[i] * 16.0f;
        }
    };

    const u32x4 offset = {0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u};  // -1.5
    const char *xget[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xget[t] = mine + min(16 * t + c16, tokens - 1) * Lds::XROW + 16 * g;

    const int per = (blocks + WAVES - 1) / WAVES;
    const int b0 = Lds::RUNS ? wave * per : wave, b1 = Lds::RUNS ? min(blocks, b0 + per) : blocks;
    constexpr int STEP = Lds::RUNS ? 1 : WAVES;
    const int stride = gridDim.x;
    int tile = tile0 + blockIdx.x;
    columns(tile);
    if (b0 < b1) load(b0, true);
    char *red_at = lq_lds + Lds::R_AT;
    do {
        f32x4 y[RT][TT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) y[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int b = b0; b < b1; b += STEP) {
            const int sj = SCB > 1 ? (b - b0) % SCB : 0;  // the block's place in its piece of scales
            if (sj == 0) put_scales();
            put();
            // the wave's own writes, read by its other lanes: LDS keeps their order, the compiler is told to
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            u32x4 wb[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) wb[r] = lq_transpose(w[r]);
            const bool same = b + STEP < b1;  // else the next tile's first block
            if (same || (Lds::LOOP && tile + stride < tiles)) {
                if (!same) columns(tile + stride);
                const int nb = same ? b + STEP : b0;
                load(nb, !same || sj == SCB - 1);
            }
#pragma unroll
            for (int i = 0; i < GB; ++i) {
                f32x4 acc[RT][TT], off[TT];
                u32x4 xb[TT][GROUP / 32];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    off[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < GROUP / 32; ++j) {
                        xb[t][j] = *(const u32x4 *)(xget[t] + (i * (GROUP / 32) + j) * 64);
                        off[t] = mfma_bf16(xb[t][j], offset, off[t]);
                    }
                }
#pragma unroll
                for (int j = 0; j < GROUP / 32; ++j)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const u32x4 v = lq_unpack(wb[r][i * (GROUP / 32) + j]);
#pragma unroll
                        for (int t = 0; t < TT; ++t) acc[r][t] = mfma_bf16(xb[t][j], v, j ? acc[r][t] : off[t]);
                    }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float sv = sc[(16 * r + c16) * SROW + sj * GB + i];
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[r][t][e] = __builtin_fmaf(sv, acc[r][t][e], y[r][t][e]);
                }
            }
        }

        // The waves' sums together.  In a loop the next tile's loads are under way, and its sums go to the
        // other place: a wave is there only after all have passed this barrier once more.
        if (!Lds::LOOP) __syncthreads();
        float *red = (float *)red_at;  // [waves][RT][TT][64 lanes][4]
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) *(f32x4 *)(red + (((wave * RT + r) * TT + t) * 64 + lane) * 4) = y[r][t];
        __syncthreads();
        // one value a thread and turn: column n, token t
        for (int i = tid; i < RT * TT * 256; i += THREADS) {
            const int c = i & 15, t16 = (i >> 4) & 15, t = (i >> 8) % TT, r = (i >> 8) / TT;
            const int n = tile * 16 * RT + 16 * r + c, tok = 16 * t + t16;
            if (n >= a.N || tok >= tokens) continue;
            const float *src = red + ((r * TT + t) * 64 + (t16 >> 2) * 16 + c) * 4 + (t16 & 3);
            float v = 0.f;
#pragma unroll
            for (int u = 0; u < WAVES; ++u) v += src[u * RT * TT * 256];
            if (__builtin_expect(!(fabsf(v) < INFINITY), 0)) v = lq_defined<GROUP, SB>(a, tok0 + tok, n);
            const int64_t at = (int64_t)(tok0 + tok) * a.N + n;
            if (a.residual) v += bf16_to_f32(a.residual[at]);
            if (a.out_f32) ((float *)a.out)[at] = v;
            else ((__bf16 *)a.out)[at] = (__bf16)v;
        }
        red_at = lq_lds + 2 * Lds::R_AT + Lds::R_BYTES - (red_at - lq_lds);
        tile += stride;
    } while (Lds::LOOP && tile < tiles);
}

template <int GROUP, bool SB, int RT, int TR, int WAVES>
static hipError_t linear(const LinearQ4 &a, hipStream_t st)
{
    using Lds = LqLds<GROUP, SB, RT, TR, WAVES>;
    constexpr int lds = Lds::BYTES;
    if (lds > 64 << 10) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_lds((const void *)k_linear_q4<GROUP, SB, RT, TR, WAVES>, lds, done);
        if (e != hipSuccess) return e;
    }
    const int tiles = (a.N - 1) / (16 * RT) + 1;
    const int fit = TR == 16 ? 512 : 256;  // workgroups that are resident together, by their registers
    constexpr int most = 1 << 21;  // workgroups in one dimension: it holds fewer than 2^32 lanes
    for (int64_t t0 = 0; t0 < a.T; t0 += 32768 * TR) {
        const int64_t left = (a.T - t0 + TR - 1) / TR;
        for (int tile0 = 0; tile0 < tiles; tile0 += Lds::LOOP ? tiles : most) {
            const int gx = tiles - tile0 < (Lds::LOOP ? fit : most) ? tiles - tile0 : Lds::LOOP ? fit : most;
            hipLaunchKernelGGL((k_linear_q4<GROUP, SB, RT, TR, WAVES>),
                               dim3((unsigned)gx, (unsigned)(left < 32768 ? left : 32768)), dim3(WAVES * WAVE), lds, st, a,
                               (int)t0, tile0);
        }
    }
    return hipGetLastError();
}

template <int GROUP, bool SB>
static hipError_t linear_tiles(const LinearQ4 &a, hipStream_t st)
{
    // Two tiles of columns a workgroup where they still fill the chip, else one: 32 x 6144 x 8192 takes 16.1 us
    // against 22.7 (graph replays, as the next figures), a fifth more with three tiles; at 1 x 1536 x 1024 (96
    // tiles) one is faster.  Sixteen waves for a few tokens of a long K and few columns (1 x 6144 x 8192: 10.2 us,
    // eight waves 11.1), four for many columns (1 x 50257 x 2048: 14.8 us, two 15.7).  From 5 tokens on eight:
    // sixteen leave a wave 128 registers, too few for 32 tokens (2.5 times the time), and are slower at 5 x 50257
    // x 2048 too; twelve are no faster.  Above 32 tokens one tile for 64 of them together; two do not fit the
    // registers.  Two blocks of 32 tokens with two tiles measured faster than that (33 x 6144 x 8192: 24 us, 28
    // as it is; 64 x 6144 x 8192: 27, 35; 450 x 1536 x 1024: 11.5, 13.4) and have still to take its place.
    const int64_t tiles = ((int64_t)a.N + 15) / 16;
    if (a.T > 32) return linear<GROUP, SB, 1, 64, 8>(a, st);
    if (a.T > 16) return tiles >= 256 ? linear<GROUP, SB, 2, 32, 8>(a, st) : linear<GROUP, SB, 1, 32, 8>(a, st);
    if (a.T > 4) return tiles >= 256 ? linear<GROUP, SB, 2, 16, 8>(a, st) : linear<GROUP, SB, 1, 16, 8>(a, st);
    if (tiles < 256) return linear<GROUP, SB, 1, 4, 8>(a, st);
    return tiles < 1024 ? linear<GROUP, SB, 2, 4, 16>(a, st) : linear<GROUP, SB, 2, 4, 4>(a, st);
}

hipError_t launch_linear_q4(const LinearQ4 &a, hipStream_t st)
{
    if (a.scales_bf16) {
        if (a.group == 32) return linear_tiles<32, true>(a, st);
        return a.group == 64 ? linear_tiles<64, true>(a, st) : linear_tiles<128, true>(a, st);
    }
    if (a.group == 32) return linear_tiles<32, false>(a, st);
    return a.group == 64 ? linear_tiles<64, false>(a, st) : linear_tiles<128, false>(a, st);
}

}  // namespace moe
