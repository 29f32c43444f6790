// beam.hip -- beam search's selection over a request's beams and the vocabulary.
//
// c(r, v) = (score_r - lse_r) + x_rv, the n largest of a request.  Within a row the order of the sums is that
// of the logits, so one pass over the logits finds both: the row's sum of exponentials and its n largest
// logits.  First launch: a workgroup a piece of a row, the piece in registers.  Second launch: a workgroup a
// request joins the pieces' sums and merges their lists.
//
// The n largest of a piece without sorting it: each wave finds the k-th largest of its 64 lanes' maxima, k = n / waves
// rounded up (a search over the leading bits of the value with ballots).  So at least n values reach the least
// of the waves' bounds, and few more.  These go to LDS, where each counts how many are ahead of it: its place.
// Where the waves are not alike (a row's last piece) their lanes are counted together, a barrier for each bit.
//
// The exponentials and their sums are 64 bits wide: a token's place among those of other rows hangs on the
// difference of two log-sums, and 2^-24 of it changes places (one in some thousand steps with 32 beams).
//
// What bounds it.  Few rows: latency, two launches of 5 to 8 us (4 beams over 50257 tokens: 7.6 + 6.1 us).  Many: the vector
// units.  A value takes 17 instructions of 64 bits for its exponential (a subtraction, the reduction, nine steps
// of a polynomial, the exponent, the sum) and some 19 others, most of them for the values that reach the bound: 512
// rows of 131071 f32 logits, 268 MB, 86 us (3.1 TB/s; the instructions alone 61), 256 rows of 50257 in bf16 21 us, where a
// copy's rate would take 52 and 5.
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

constexpr int BEAM_T1 = 256, BEAM_T2 = 512;  // threads of a piece, of a request
constexpr int BEAM_CAP = 1024, BEAM_CAP2 = 1024;  // values that reach the bound and are ranked by counting

// Order-preserving bits of a value (both zeros the same); numbers from the lowest finite one on reach ORDER_FINITE.
constexpr uint32_t ORDER_FINITE = 0x00800000u;

__device__ __forceinline__ uint32_t order32(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value32(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

__device__ __forceinline__ uint64_t order64(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x == 0. ? 0. : x);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ double value64(uint64_t o) { return __builtin_bit_cast(double, o ^ ((o >> 63) ? 1ull << 63 : ~0ull)); }

// e^(x - top) for x <= top, top finite: (x - top) log2 e = k + f with a whole k and |f| <= 1/2, 1 + f q(f) with the
// polynomial q of degree 8 through (2^f - 1) / f at the Chebyshev points (2^-44.6 relative at most), times 2^k.  1 at x = top,
// exactly: a row that allows one token has that logit as its log-sum.  (Its sum (score - x) + x is the score to a step of 64
// bits, and the score itself where score - x loses nothing: where both lie between 2^-24 and 2^5, say.)  k comes from the low bits of a sum with 3 * 2^51 and goes into the result's exponent.  From e^-690 down (so -infinity
// too) it is e^-690, nothing beside the 1 that the largest adds.  Positive NaN or infinity as x is the caller's.
// A row's log-sum takes it three times (value to wave, wave to piece, piece to row), 3 * 2^-44.62 = 0.98 * 2^-43 of the sum; the
// additions are a thread's 31, 6 and 4 over a wave and a piece and, of the row's pieces of 8192, one after another every 64th:
// under 2^-47 up to 2^19 tokens, 0.5 * 2^-43 at 2^28, 2.05 * 2^-43 at 2^30; the rest (f's constant, the logarithm) under 2^-46.  So
// 2^-42 up to 2^28 tokens, 2^-41 above, beside 2^-52 of the log-sum itself.
// The constants are made once and stay in scalar registers: as literals the compiler moves them there again for every value, a
// third of the loop's instructions, and in vector registers they leave fewer waves (119 us against 105 at 16 x 32 x 131071).
struct ExpBelow {
    double c[10], log2e, round, low;
    __device__ __forceinline__ ExpBelow()
    {
        constexpr double C[10] = {1.0, 0x1.62e42fefa39efp-1, 0x1.ebfbdff823cedp-3, 0x1.c6b08d7047e52p-5,
                                  0x1.3b2ab7181b755p-7, 0x1.5d87fe86fe88ep-10, 0x1.4308ac85aa947p-13, 0x1.ffcb9515a8016p-17,
                                  0x1.63d136366db24p-20, 0x1.b63880a30e9ffp-24};
#pragma unroll
        for (int i = 0; i < 10; ++i) c[i] = held(C[i]);
        log2e = held(0x1.71547652b82fep+0);
        round = held(0x1.8p52);
        low = held(-690.0);
    }
    static __device__ __forceinline__ double held(double x)
    {
        asm("" : "+s"(x));
        return x;
    }
    __device__ __forceinline__ double operator()(double x, double top) const
    {
        const double d = fmax(x - top, low);
        const double t = __builtin_fma(d, log2e, round), f = __builtin_fma(d, log2e, round - t);
        double p = c[9];
#pragma unroll
        for (int i = 8; i >= 1; --i) p = __builtin_fma(p, f, c[i]);
        p = __builtin_fma(p, f, 1.0);
        u32x2 bits = __builtin_bit_cast(u32x2, p);
        bits[1] += __builtin_bit_cast(u32x2, t)[0] << 20;
        return __builtin_bit_cast(double, bits);
    }
};

__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, WAVE);
    return x;
}

__device__ __forceinline__ int wave_reach(uint32_t v, uint32_t trial)
{
    return __builtin_popcountll(__builtin_amdgcn_ballot_w64(v >= trial));
}

// The k-th largest of the wave's 64 values, rounded down to their BITS leading bits; k <= 64.
template <int BITS>
__device__ __forceinline__ uint32_t wave_kth(uint32_t v, int k)
{
    uint32_t t = 0;
#pragma unroll 1
    for (int b = 31; b > 31 - BITS; --b) {
        const uint32_t trial = t | 1u << b;
        if (wave_reach(v, trial) >= k) t = trial;
    }
    return t;
}

// A bound that n of the workgroup's values reach, W waves: the n-th largest, to its BITS leading bits, by a count over the
// workgroup for each.  wave_count(trial): how many of the wave's values reach it.  0 where there are fewer.
template <int BITS, int W, typename F>
__device__ __forceinline__ uint32_t group_kth(int n, int (*counts)[W], F wave_count)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t t = 0;
#pragma unroll 1
    for (int b = 31; b > 31 - BITS; --b) {
        const uint32_t trial = t | 1u << b;
        const int c = wave_count(trial);
        if (lane == 0) counts[b & 1][wave] = c;
        __syncthreads();  // (the other half is written next, this one again behind the next barrier)
        int all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) all += counts[b & 1][w];
        if (all >= n) t = trial;
    }
    return t;
}

// f(i, part, parts) for i < n, part < parts: as many lanes next to each other (`parts`, a power of two up to a wave) share
// each i as T threads allow; the sum of their results goes to done(i, sum), of which one lane writes.
template <int T, typename F, typename G>
__device__ __forceinline__ void shared_count(int n, F f, G done)
{
    int log = 0;
    while (log < 6 && n << (log + 1) <= T) ++log;
    const int part = threadIdx.x & ((1 << log) - 1);
    for (int i = threadIdx.x >> log; i < n; i += T >> log) {
        int c = f(i, part, 1 << log);
#pragma unroll 1
        for (int d = 1; d < 1 << log; d <<= 1) c += __shfl_xor(c, d, WAVE);
        if (part == 0) done(i, c);
    }
}

// What a piece leaves for the second launch.
struct BeamPiece {
    double sum;  // of exp(x - top)
    float top;   // largest logit, -infinity where there is none
    int pad;
};

struct BeamWs {
    BeamPiece *pieces;  // [rows][pieces of a row]
    uint64_t *keys;     // [rows][pieces][n_out]: order32(logit) << 32 | ~token, descending, 0 behind the last
    int n;              // pieces of a row
};

// A piece of 256 * V values of one row.  A thread's values lie 16 bytes together; which thread has which
// depends on their place in the row alone, so equal rows have equal sums.
template <typename T, int V>
__global__ __launch_bounds__(BEAM_T1) void k_beam_piece(BeamSelect a, BeamWs w)
{
    constexpr int E = 16 / sizeof(T), LOADS = V / E, W = BEAM_T1 / WAVE;
    __shared__ uint64_t cand[BEAM_CAP];
    __shared__ double sums[W];
    __shared__ float tops[W];
    __shared__ uint32_t bounds[W];
    __shared__ int found, counts[2][W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / w.n;
    const int piece = blockIdx.x % w.n;
    constexpr int N = BEAM_T1 * V;
    const T *src = (const T *)a.logits + row * a.row_stride + (int64_t)piece * N;
    const int left = a.vocab - piece * N;  // values from here on, N of them at most are this piece's
    if (tid == 0) found = 0;

    float x[V], top = -INFINITY;
    {
        u32x4 raw[LOADS];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int i = tid * E + u * (BEAM_T1 * E);
            if (i + E <= left) {
                __builtin_memcpy(&raw[u], src + i, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (E == 4) {
                        raw[u][j] = i + j < left ? __float_as_uint(src[i + j]) : 0xFF800000u;
                    } else {
                        const uint32_t lo = i + 2 * j < left ? src[i + 2 * j] : 0xFF80u, hi = i + 2 * j + 1 < left ? src[i + 2 * j + 1] : 0xFF80u;
                        raw[u][j] = hi << 16 | lo;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float y = E == 4 ? __uint_as_float(raw[u][j]) : (j & 1) ? bf16_hi(raw[u][j / 2]) : bf16_lo(raw[u][j / 2]);
                x[u * E + j] = y;
                top = __builtin_elementwise_maximum(top, y);  // (NaN stays)
            }
    }
    // a wave's sum is taken from its own largest
    float wtop = top;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) wtop = __builtin_elementwise_maximum(wtop, __shfl_xor(wtop, d, WAVE));
    const ExpBelow exp_below;
    double sum = 0.;
    if (wtop > -INFINITY) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum += exp_below(x[i], wtop);
    }
    sum = wave_sum(sum);
    if (!(wtop < INFINITY)) sum = __builtin_nan("");  // a NaN or +infinity among them
    // the last piece of a row: its lanes' largest counted together, or where these are few for n_out, all its values (32
    // bf16 rows of 9000 tokens, 100 of them: 21 us, 34 by the lanes; always all values: 128 of 2 x 128 x 131071 108 us, 100)
    uint32_t bound;
    if (N <= left) {
        bound = wave_kth<16>(order32(top), (a.n_out + W - 1) / W);
    } else if (2 * a.n_out <= min(left / E, BEAM_T1)) {
        const uint32_t v = order32(top);
        bound = group_kth<16, W>(a.n_out, counts, [&](uint32_t trial) { return wave_reach(v, trial); });
    } else {
        bound = group_kth<16, W>(a.n_out, counts, [&](uint32_t trial) {
            const float y = value32(trial);  // (not a number below all numbers: the bound stays 0)
            int c = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x[i] >= y));
            return c;
        });
    }
    if (lane == 0) {
        sums[wave] = sum;
        tops[wave] = wtop;
        bounds[wave] = bound;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) bound = min(bound, bounds[i]);
    const float t = value32(max(bound, ORDER_FINITE));
    auto key = [&](int i) {
        return (uint64_t)order32(x[i]) << 32 | (uint32_t)~(uint32_t)(piece * N + tid * E + i / E * (BEAM_T1 * E) + i % E);
    };
    // one place for the wave's values, which lie there value by value
    int mine = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mine += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x[i] >= t));
    if (mine) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&found, mine);
        at = __builtin_amdgcn_readfirstlane(at);
        if (at + mine <= BEAM_CAP) {
            // compared again: 32 masks of 64 lanes that are kept cost more than that
            float again = t;
            asm("" : "+s"(again));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool reach = x[i] >= again;
                const uint64_t m = __builtin_amdgcn_ballot_w64(reach);
                if (!m) continue;
                if (reach) cand[__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, at))] = key(i);
                at += __builtin_popcountll(m);
            }
        }
    }
    __syncthreads();
    int n = found;
    if (n > BEAM_CAP) {
        // many equal values: the n_out-th largest key itself, bit by bit
        uint64_t bit_t = 0;
        for (int b = 63; b >= 0; --b) {
            const uint64_t trial = bit_t | 1ull << b;
            int c = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) c += x[i] >= t && key(i) >= trial;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) c += __shfl_xor(c, d, WAVE);
            __syncthreads();
            if (lane == 0) counts[0][wave] = c;
            __syncthreads();
            c = 0;
            for (int i = 0; i < W; ++i) c += counts[0][i];
            if (c >= a.n_out) bit_t = trial;
        }
        if (tid == 0) found = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (x[i] >= t && key(i) >= bit_t) cand[atomicAdd(&found, 1)] = key(i);  // n_out of them
        __syncthreads();
        n = found;
    }
    uint64_t *out = w.keys + (row * w.n + piece) * a.n_out;
    shared_count<BEAM_T1>(
        n,
        [&](int i, int part, int parts) {
            const uint64_t mine = cand[i];
            int ahead = 0;
#pragma unroll 4
            for (int j = part; j < n; j += parts) ahead += cand[j] > mine;
            return ahead;
        },
        [&](int i, int ahead) {
            if (ahead < a.n_out) out[ahead] = cand[i];
        });
    for (int i = n + tid; i < a.n_out; i += BEAM_T1) out[i] = 0;
    if (tid == 0) {
        float m = -INFINITY;
        for (int i = 0; i < W; ++i) m = fmaxf(m, tops[i]);
        double s = 0.;
        for (int i = 0; i < W; ++i) {
            if (sums[i] != sums[i]) s = sums[i];
            else if (tops[i] > -INFINITY) s += sums[i] * exp_below(tops[i], m);
        }
        w.pieces[row * w.n + piece] = {s, m, 0};
    }
}

// A candidate's place: the larger sum, then the lower row, then the larger key (logit, then lower token).
struct BeamCand {
    uint64_t c, key;
    int row;
    __device__ bool ahead_of(const BeamCand &o) const
    {
        return c != o.c ? c > o.c : row != o.row ? row < o.row : key > o.key;
    }
};

__global__ __launch_bounds__(BEAM_T2) void k_beam_request(BeamSelect a, BeamWs w)
{
    constexpr int W = BEAM_T2 / WAVE;
    __shared__ uint64_t cs[BEAM_CAP2], ks[BEAM_CAP2];
    __shared__ uint8_t rs[BEAM_CAP2], state[128];  // state of a row: 0 nothing to offer, 1 its lists, 2 done
    __shared__ double base[128];
    __shared__ uint32_t bounds[W];
    __shared__ int counts[2][W];
    __shared__ BeamCand heads[W];
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    if (tid == 0) found = 0;

    // a list is a piece of a row, the pieces of a row one after another; the first eight keys of a list are a thread's
    // each, and the first of these keys are on their way early.  Neighbours are mostly one row's, so the best row's wave
    // alone gives a close bound.  Where lists are so few that more keys of each fit the threads, more are taken: a
    // bound from eight keys of few lists lets most of all keys through (4 x 8 beams of 2000 tokens, 128 of them: 27 us, 198)
    const int lists = a.beams * w.n, n_out = a.n_out;
    constexpr int A = 4;
    int log_depth = 3;
    while (log_depth < 6 && 1 << log_depth < n_out && lists << (log_depth + 1) <= BEAM_T2) ++log_depth;
    const int depth = 1 << log_depth, at_once = BEAM_T2 >> log_depth;
    const int my_list = tid >> log_depth, my_depth = tid & (depth - 1);
    auto keys_of = [&](int list) { return w.keys + (row0 * w.n + list) * n_out; };
    const double per_piece = 1.0 / w.n;
    auto row_of = [&](int list) { return (int)(((double)list + 0.5) * per_piece); };  // half a piece away from the next row
    uint64_t keys[A];
    auto load_keys = [&](int l0, int d0) {
#pragma unroll
        for (int j = 0; j < A; ++j) {
            const int list = l0 + j * at_once + my_list, d = d0 + my_depth;
            keys[j] = list < lists && d < n_out ? keys_of(list)[d] : 0;
        }
    };
    load_keys(0, 0);

    // the rows' sums: as many lanes next to each other as a row has pieces, a wave at most
    const ExpBelow exp_below;
    int per = 1;
    while (per < min(w.n, WAVE)) per *= 2;
    for (int r0 = 0; r0 < a.beams; r0 += BEAM_T2 / per) {
        const int r = r0 + tid / per, i0 = tid % per;
        const bool live = r < a.beams;
        const BeamPiece *p = w.pieces + (row0 + (live ? r : 0)) * w.n;
        const double score = a.scores[row0 + (live ? r : 0)];
        const bool ended = a.done && a.done[row0 + (live ? r : 0)];
        float m = -INFINITY;
        for (int i = i0; i < w.n; i += per) m = fmaxf(m, p[i].top);
#pragma unroll 1
        for (int d = per / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, WAVE));
        double s = 0.;
        for (int i = i0; i < w.n; i += per) {
            const BeamPiece x = p[i];
            if (x.sum != x.sum) s = x.sum;
            else if (x.top > -INFINITY) s += x.sum * exp_below(x.top, m);
        }
#pragma unroll 1
        for (int d = per / 2; d > 0; d >>= 1) s += __shfl_xor(s, d, WAVE);
        if (live && i0 == 0) {
            const double lse = s == 0. ? -INFINITY : (double)m + log(s), b = score - lse;
            base[r] = ended ? score : b;
            state[r] = fabs(base[r]) < INFINITY ? ended ? 2 : 1 : 0;
            if (a.lse) a.lse[row0 + r] = (float)lse;
        }
    }
    __syncthreads();

    // what a key of a list is worth; without one the key is 0
    auto worth = [&](int list, uint64_t key, bool first) {
        BeamCand x = {0, 0, row_of(list)};
        const int st = state[x.row];
        if (st == 1 && key) {
            x.key = key;
            x.c = order64(base[x.row] + (double)value32((uint32_t)(key >> 32)));
        } else if (st == 2 && first && list == x.row * w.n) {
            x.c = order64(base[x.row]);
            x.key = 1ull << 32 | (uint32_t)~a.end_token;
        }
        return x;
    };
    auto candidate = [&](int list, int d) { return worth(list, keys_of(list)[d], d == 0); };
    // a bound that at least n_out candidates reach, from the keys that are here; of more lists, from each one's first,
    // one list after another in another wave
    uint32_t most = 0;
    if (lists <= A * at_once) {
#pragma unroll
        for (int j = 0; j < A; ++j)
            if (j * at_once + my_list < lists) most = max(most, (uint32_t)(worth(j * at_once + my_list, keys[j], my_depth == 0).c >> 32));
    } else {
        for (int l = lane * W + wave; l < lists; l += BEAM_T2) most = max(most, (uint32_t)(worth(l, keys_of(l)[0], true).c >> 32));
    }
    uint32_t t = 0;
    if (n_out > 16) {
        t = group_kth<22, W>(n_out, counts, [&](uint32_t trial) { return wave_reach(most, trial); });
    } else {
        // few: the best wave's n_out-th lane says about as much, without barriers.  Both ways, counted together / the best
        // wave: 16 of 4 x 50257 16.8 / 14.8 us, of 32 x 8 x 50257 29.4 / 27.8, of 8 x 16 x 50257 23.3 / 21.9; 20 of them 17.1 / 14.9,
        // 29.4 / 28.9, 23.6 / 25.6; 64 of them 19.7 / 24.6, 36.8 / 188, 27.2 / 156
        const uint32_t b = wave_kth<22>(most, n_out);
        if (lane == 0) bounds[wave] = b;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) t = max(t, bounds[i]);
    }
    int n;
    for (bool again = false;; again = true) {
        // the candidates that reach it; a list all of whose keys here do has more to look at
        bool deeper = false;
        for (int d0 = 0; d0 < n_out; d0 += depth) {
            for (int l0 = 0; l0 < lists; l0 += A * at_once) {
                if (l0 || d0 || again) load_keys(l0, d0);
#pragma unroll
                for (int j = 0; j < A; ++j) {
                    const int list = l0 + j * at_once + my_list;
                    BeamCand x = {0, 0, 0};
                    if (list < lists) x = worth(list, keys[j], d0 + my_depth == 0);
                    const bool reach = x.key && (uint32_t)(x.c >> 32) >= t;
                    const uint64_t m = __builtin_amdgcn_ballot_w64(reach);
                    if (!m) continue;
                    deeper |= reach && my_depth == depth - 1;
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&found, (int)__builtin_popcountll(m));
                    at = __builtin_amdgcn_readfirstlane(at) + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
                    if (reach && at < BEAM_CAP2) {
                        cs[at] = x.c;
                        ks[at] = x.key;
                        rs[at] = (uint8_t)x.row;
                    }
                }
            }
            if (!__syncthreads_or(deeper)) break;
            deeper = false;
        }
        __syncthreads();
        n = found;
        if (n <= BEAM_CAP2) break;
        // too many (few rows are alive): the candidates that are here give a higher bound
        const uint32_t v0 = (uint32_t)(cs[tid] >> 32), v1 = (uint32_t)(cs[tid + BEAM_T2] >> 32);
        const uint32_t higher = group_kth<32, W>(n_out, counts, [&](uint32_t trial) { return wave_reach(v0, trial) + wave_reach(v1, trial); });
        if (higher <= t) break;
        t = higher;
        if (tid == 0) found = 0;
        __syncthreads();
    }
    const int64_t out0 = (int64_t)blockIdx.x * n_out;
    auto put = [&](int i, const BeamCand &x) {
        const bool none = x.key == 0;
        const int token = none ? -1 : (int)~(uint32_t)x.key;
        a.parent[out0 + i] = none ? -1 : (int)(row0 + x.row);
        a.token[out0 + i] = token;
        a.score[out0 + i] = none ? -INFINITY : (float)value64(x.c);
        if (a.done_out) a.done_out[out0 + i] = none || state[x.row] == 2 || (a.end_token >= 0 && token == a.end_token);
    };
    if (n <= BEAM_CAP2) {
        shared_count<BEAM_T2>(
            n,
            [&](int i, int part, int parts) {
                const uint64_t mine = cs[i];
                int ahead = 0, equal = 0;
#pragma unroll 4
                for (int j = part; j < n; j += parts) {
                    const uint64_t c = cs[j];
                    ahead += c > mine;
                    equal += c == mine;
                }
                if (equal > (i % parts == part)) {
                    const uint64_t key = ks[i];
                    const int row = rs[i];
#pragma unroll 4
                    for (int j = part; j < n; j += parts)
                        ahead += (cs[j] == mine) & ((rs[j] < row) | ((rs[j] == row) & (ks[j] > key)));
                }
                return ahead;
            },
            [&](int i, int ahead) {
                if (ahead < n_out) put(ahead, BeamCand{cs[i], ks[i], rs[i]});
            });
        for (int i = n + tid; i < n_out; i += BEAM_T2) put(i, BeamCand{0, 0, 0});
        return;
    }
    // very many equal sums: the lists merged one candidate at a time, each round from the lists' beginnings.  Inputs that
    // get here have more than 1024 sums alike in 32 bits: 16 x 32 rows of 131071 that allow three tokens, the others at the
    // type's lowest value, 64 asked for 427 us (94 where the logits differ), 128 rows with 128 asked for 1.2 ms (75); all
    // logits equal 1.2 and 2.9 ms
    BeamCand last = {~0ull, ~0ull, -1};
    for (int i = 0; i < n_out; ++i) {
        BeamCand best = {0, 0, 0};
        for (int l = tid; l < lists; l += BEAM_T2)
            for (int d = 0; d < n_out; ++d) {
                const BeamCand x = candidate(l, d);
                if (x.key == 0) break;
                if (!last.ahead_of(x)) continue;
                if (best.key == 0 || x.ahead_of(best)) best = x;
                break;
            }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const BeamCand o = {__shfl_xor(best.c, d, WAVE), __shfl_xor(best.key, d, WAVE), __shfl_xor(best.row, d, WAVE)};
            if (o.key && (best.key == 0 || o.ahead_of(best))) best = o;
        }
        __syncthreads();
        if (lane == 0) heads[wave] = best;
        __syncthreads();
        best = heads[0];
        for (int j = 1; j < W; ++j)
            if (heads[j].key && (best.key == 0 || heads[j].ahead_of(best))) best = heads[j];
        if (tid == 0) put(i, best);
        last = best;
    }
}

// ---------------------------------------------------------------- launches

// Values of a thread: pieces of 8192, where these are too few for the chip of 4096 (bf16, us for 16 / 32 values: one row of
// 131071 13.3 / 14.3, 4 x 4 of 50257 16.8 / 19.0, 32 x 8 26.5 / 26.5, 2 x 32 of 131071 35.6 / 29.7), and half or a quarter of
// that where it saves a fifth of the places in a row's last piece (128 x 8 of 2000, 8 / 16 / 32 values: 14.9 / 16.7 / 20.2, of
// 4000 18.7 / 16.3 / 19.8, of 12000 34.4 / 27.6 / 28.4).
static int beam_values(int64_t rows, int64_t vocab)
{
    auto padded = [&](int v) { return (vocab + BEAM_T1 * v - 1) / (BEAM_T1 * v) * (BEAM_T1 * v); };
    int v = rows * ((vocab + 8191) / 8192) < 256 ? 16 : 32;
    while (v > 8 && padded(v / 2) * 5 <= padded(v) * 4) v /= 2;
    return v;
}

static int beam_pieces(int64_t rows, int vocab)
{
    const int64_t piece = (int64_t)BEAM_T1 * beam_values(rows, vocab);
    return (int)((vocab + piece - 1) / piece);
}

size_t beam_workspace(int64_t rows, int vocab, int n_out)
{
    return (size_t)rows * beam_pieces(rows, vocab) * (sizeof(BeamPiece) + (size_t)n_out * 8);
}

template <typename T>
static hipError_t pieces(const BeamSelect &a, const BeamWs &w, int64_t rows, hipStream_t st)
{
    const dim3 grid((unsigned)(rows * w.n)), block(BEAM_T1);
    const int v = beam_values(rows, a.vocab);
    if (v == 8) hipLaunchKernelGGL((k_beam_piece<T, 8>), grid, block, 0, st, a, w);
    else if (v == 16) hipLaunchKernelGGL((k_beam_piece<T, 16>), grid, block, 0, st, a, w);
    else hipLaunchKernelGGL((k_beam_piece<T, 32>), grid, block, 0, st, a, w);
    return hipGetLastError();
}

hipError_t launch_beam_select(const BeamSelect &a, void *ws, hipStream_t st)
{
    const int64_t rows = (int64_t)a.requests * a.beams;
    BeamWs w;
    w.n = beam_pieces(rows, a.vocab);
    w.pieces = (BeamPiece *)ws;
    w.keys = (uint64_t *)(w.pieces + rows * w.n);
    const hipError_t e = a.bf16 ? pieces<uint16_t>(a, w, rows, st) : pieces<float>(a, w, rows, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_beam_request, dim3((unsigned)a.requests), dim3(BEAM_T2), 0, st, a, w);
    return hipGetLastError();
}

}  // namespace moe
