// linear_q4.hip -- few-token products with packed int4 weights and group scales:
//   y[t][n] = sum_g s[n][g] * sum_{k in g} x[t][k] * c[n][k]  (+ residual[t][n]).
//
// Weights are read once, so their bytes bound it: N * K / 2 and the scales.  A
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
// scale (times 16) joins a group's sum in f32.
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

constexpr int LQ_BLOCK = 128;  // k of one step: a 16-byte piece for each of a column's four lanes
// Waves of a workgroup: sixteen where 128 registers do, else eight.
constexpr int lq_max_waves(int rt, int tt) { return rt * tt <= 2 ? 16 : 8; }

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

// RT tiles of 16 columns, TT of 16 tokens a wave; the workgroup's waves share K.
template <int GROUP, bool SB, int RT, int TT>
__global__ __launch_bounds__(lq_max_waves(RT, TT) * WAVE) void k_linear_q4(LinearQ4 a, int t0)
{
    constexpr int GB = LQ_BLOCK / GROUP;  // groups of a block
    extern __shared__ __align__(16) float lq_red[];  // [waves][RT][TT][64 lanes][4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int g = lane >> 4, c16 = lane & 15;
    const int tokens = min(a.T - t0 - (int)blockIdx.y * 16 * TT, 16 * TT), tok0 = t0 + blockIdx.y * 16 * TT;
    const int n0 = blockIdx.x * 16 * RT, blocks = (a.K + LQ_BLOCK - 1) / LQ_BLOCK;
    const int per = (blocks + waves - 1) / waves, b0 = wave * per, b1 = min(blocks, b0 + per);
    const int groups = a.K / GROUP;

    const uint8_t *wp[RT];
    int64_t sp[RT];
    const uint16_t *xp[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t n = min(n0 + 16 * r + c16, a.N - 1);
        wp[r] = a.q + n * (a.K / 2);
        sp[r] = n * groups;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) xp[t] = a.x + (int64_t)(tok0 + min(16 * t + c16, tokens - 1)) * a.x_stride + 8 * g;

    u32x4 w[RT], x[TT][4];
    float s[RT][GB];
    auto load = [&](int b) {
        const int k0 = b * LQ_BLOCK;
        // the last block of a K that is no multiple of 128 ends early: its missing pieces are read
        // from its first one and not used
        const int piece = k0 + 32 * g < a.K ? 16 * g : 0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            w[r] = *(const u32x4 *)(wp[r] + k0 / 2 + piece);
#pragma unroll
            for (int i = 0; i < GB; ++i) {
                const int64_t at = sp[r] + min(b * GB + i, groups - 1);
                s[r][i] = SB ? bf16_to_f32(((const uint16_t *)a.scales)[at]) : ((const float *)a.scales)[at];
            }
        }
    };
    auto load_x = [&](int b) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[t][j] = *(const u32x4 *)(xp[t] + min(b * LQ_BLOCK + 32 * j, a.K - 32));
    };
    // the next block's activations are loaded ahead too where the registers are there
    constexpr bool AHEAD = TT <= 2;

    f32x4 y[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) y[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 offset = {0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u};  // -1.5
    if (b0 < b1) {
        load(b0);
        if (AHEAD) load_x(b0);
    }
    for (int b = b0; b < b1; ++b) {
        if (!AHEAD) load_x(b);
        u32x4 wb[RT], xb[TT][4];
        float sb[RT][GB];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            wb[r] = lq_transpose(w[r]);
#pragma unroll
            for (int i = 0; i < GB; ++i) sb[r][i] = s[r][i] * 16.0f;
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) xb[t][j] = interleave_bf16x8(x[t][j]);
        const int steps = min(4, (a.K - b * LQ_BLOCK) / 32);
        if (b + 1 < b1) {
            load(b + 1);
            if (AHEAD) load_x(b + 1);
        }
#pragma unroll
        for (int i = 0; i < GB; ++i) {
            f32x4 acc[RT][TT];
            if (i * (GROUP / 32) >= steps) break;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = i * (GROUP / 32); j < (i + 1) * (GROUP / 32); ++j) c = mfma_bf16(xb[t][j], offset, c);
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r][t] = c;
            }
#pragma unroll
            for (int j = i * (GROUP / 32); j < (i + 1) * (GROUP / 32); ++j)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const u32x4 v = lq_unpack(wb[r][j]);
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[r][t] = mfma_bf16(xb[t][j], v, acc[r][t]);
                }
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[r][t][e] = __builtin_fmaf(sb[r][i], acc[r][t][e], y[r][t][e]);
        }
    }

#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) *(f32x4 *)(lq_red + (((wave * RT + r) * TT + t) * 64 + lane) * 4) = y[r][t];
    __syncthreads();
    // one value a thread and turn: column n, token t
    for (int i = threadIdx.x; i < RT * TT * 256; i += blockDim.x) {
        const int c = i & 15, t16 = (i >> 4) & 15, t = (i >> 8) % TT, r = (i >> 8) / TT;
        const int n = n0 + 16 * r + c, tok = 16 * t + t16;
        if (n >= a.N || tok >= tokens) continue;
        const float *src = lq_red + ((r * TT + t) * 64 + (t16 >> 2) * 16 + c) * 4 + (t16 & 3);
        float v = 0.f;
        for (int u = 0; u < waves; ++u) v += src[u * RT * TT * 256];
        const int64_t at = (int64_t)(tok0 + tok) * a.N + n;
        if (a.residual) v += bf16_to_f32(a.residual[at]);
        if (a.out_f32) ((float *)a.out)[at] = v;
        else ((__bf16 *)a.out)[at] = (__bf16)v;
    }
}

size_t linear_q4_workspace(int, int, int) { return 256; }

template <int GROUP, bool SB, int RT, int TT>
static hipError_t linear(const LinearQ4 &a, int waves, hipStream_t st)
{
    const unsigned gx = (a.N + 16 * RT - 1) / (16 * RT);
    for (int t0 = 0; t0 < a.T; t0 += 32768 * 16 * TT) {
        const int64_t left = ((int64_t)a.T - t0 + 16 * TT - 1) / (16 * TT);
        hipLaunchKernelGGL((k_linear_q4<GROUP, SB, RT, TT>), dim3(gx, (unsigned)(left < 32768 ? left : 32768)),
                           dim3(waves * WAVE), waves * RT * TT * 1024, st, a, t0);
    }
    return hipGetLastError();
}

template <int GROUP, bool SB>
static hipError_t linear_tiles(const LinearQ4 &a, hipStream_t st)
{
    const int tiles = (a.N + 15) / 16, blocks = (a.K + LQ_BLOCK - 1) / LQ_BLOCK;
    const int tt = a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4;
    const int rt = tiles >= 512 || (tt >= 2 && tiles >= 256) ? 2 : 1;
    int waves = lq_max_waves(rt, tt);
    while (waves > 4 && (waves > blocks || tiles / rt * waves > 256 * 32)) waves /= 2;
    if (rt == 1) {
        if (tt == 1) return linear<GROUP, SB, 1, 1>(a, waves, st);
        if (tt == 2) return linear<GROUP, SB, 1, 2>(a, waves, st);
        return linear<GROUP, SB, 1, 4>(a, waves, st);
    }
    if (tt == 1) return linear<GROUP, SB, 2, 1>(a, waves, st);
    if (tt == 2) return linear<GROUP, SB, 2, 2>(a, waves, st);
    return linear<GROUP, SB, 2, 4>(a, waves, st);
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
