// beam.hip -- beam search's selection over a request's beams and the vocabulary.
//
// c(r, v) = (score_r - lse_r) + x_rv, the n largest of a request.  Within a row the order of the sums is that
// of the logits, so one pass over the logits finds both: the row's sum of exponentials and its n largest
// logits.  First launch: a workgroup a piece of a row, the piece in registers.  Second launch: a workgroup a
// request joins the pieces' sums and merges their lists.
//
// The n largest of a piece without sorting it: each wave finds the k-th largest of its 64 lanes' maxima
// (a search over the leading bits of the value with ballots).  With k = n / g, rounded up, k lanes of each of
// the g waves with the largest such bounds reach the g-th of them, so at least n values do, and few more.
// These go to LDS, where each counts how many are ahead of it: its place.
//
// The exponentials and their sums are 64 bits wide: a token's place among those of other rows hangs on the
// difference of two log-sums, and 2^-24 of it changes places (one in some thousand steps with 32 beams).
#include "moe_device.h"
#include "moe_launch.h"
#include <cstdlib>

namespace moe {

constexpr int BEAM_T1 = 256, BEAM_T2 = 512;  // threads of a piece, of a request
constexpr int BEAM_CAP = 1024, BEAM_CAP2 = 1024;  // values that reach the bound and are ranked by counting

// Order-preserving bits of a value (both zeros the same); numbers from the lowest finite one on reach ORDER_FINITE.
constexpr uint32_t ORDER_FINITE = 0x00800000u, ORDER_INF = 0xFF800000u;

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

// e^(x - top) for x <= top, top finite: (x - top) log2 e = k + f with a whole k and |f| <= 1/2, the polynomial of
// degree 9 through 2^f at the Chebyshev points (2^-45.6 relative at most), times 2^k.  k comes from the low bits of a
// sum with 3 * 2^51 and goes into the result's exponent.  From e^-690 down (so -infinity too) it is e^-690, nothing
// beside the 1 that the largest adds.  Positive NaN or infinity as x is the caller's.
// The constants are kept in vector registers: the compiler otherwise moves them there for every value, a third
// of the loop's instructions.
struct ExpBelow {
    double c[10], log2e, round, low;
    __device__ __forceinline__ ExpBelow()
    {
        constexpr double C[10] = {0x1.000000000003dp+0, 0x1.62e42fefa39f7p-1, 0x1.ebfbdff8149f2p-3, 0x1.c6b08d7044119p-5,
                                  0x1.3b2ab72b175eep-7, 0x1.5d87fe908f88ap-10, 0x1.43088e257f341p-13, 0x1.ffcb76789860fp-17,
                                  0x1.63ef969a64d3cp-20, 0x1.b6571de2f2351p-24};
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
        for (int i = 8; i >= 0; --i) p = __builtin_fma(p, f, c[i]);
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

// The k-th largest of the wave's 64 values, rounded down to their BITS leading bits; k <= 64.
template <int BITS>
__device__ __forceinline__ uint32_t wave_kth(uint32_t v, int k)
{
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b > 31 - BITS; --b) {
        const uint32_t trial = t | 1u << b;
        if (__builtin_popcountll(__builtin_amdgcn_ballot_w64(v >= trial)) >= k) t = trial;
    }
    return t;
}

// The waves' bounds for g = 2^i of W waves, in bounds[i][W]: at least n of the values whose largest of each lane is
// v reach what waves_bound() makes of them.  All waves together say most where their values are alike, one wave
// (for n above its lanes, two) where others have few.
template <int BITS, int W>
__device__ __forceinline__ void wave_bounds(uint32_t v, int n, bool alike, uint32_t (*bounds)[W])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i <= (W == 8 ? 3 : 2); ++i) {
        const int k = (n + (1 << i) - 1) >> i;
        uint32_t b = 0;
        if (1 << i == W || (!alike && i == (n > WAVE))) b = wave_kth<BITS>(v, k);
        if (lane == 0) bounds[i][wave] = b;
    }
}

template <int W>
__device__ __forceinline__ uint32_t waves_bound(const uint32_t (*bounds)[W])
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i <= (W == 8 ? 3 : 2); ++i) {
        const int lane = threadIdx.x & 63;
        const uint32_t mine = lane < W ? bounds[i][lane] : 0u;
        int reach = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) reach += bounds[i][w] >= mine ? 1 : 0;
        uint32_t b = reach >= 1 << i ? mine : 0u;
#pragma unroll
        for (int d = 1; d < WAVE; d <<= 1) b = max(b, (uint32_t)__shfl_xor((int)b, d, WAVE));
        t = max(t, b);
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
    __shared__ uint32_t bounds[3][W];
    __shared__ int found, counts[W];
    static_assert(W == 4, "");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / w.n;
    const int piece = blockIdx.x % w.n;
    const T *src = (const T *)a.logits + row * a.row_stride;
    const int64_t first = (int64_t)piece * (BEAM_T1 * V) + tid * E;
    if (tid == 0) found = 0;

    float x[V];
    uint32_t o[V], most = 0, least = ~0u;
    {
        u32x4 raw[LOADS];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int64_t i = first + u * (BEAM_T1 * E);
            if (i + E <= a.vocab) {
                __builtin_memcpy(&raw[u], src + i, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (E == 4) {
                        raw[u][j] = i + j < a.vocab ? __float_as_uint(src[i + j]) : 0xFF800000u;
                    } else {
                        const uint32_t lo = i + 2 * j < a.vocab ? src[i + 2 * j] : 0xFF80u, hi = i + 2 * j + 1 < a.vocab ? src[i + 2 * j + 1] : 0xFF80u;
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
                o[u * E + j] = order32(y);
                most = max(most, o[u * E + j]);
                least = min(least, o[u * E + j]);
            }
    }
    // a wave's sum is taken from its own largest
    uint32_t wmost = most;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) wmost = max(wmost, (uint32_t)__shfl_xor((int)wmost, d, WAVE));
    const float top = value32(wmost);
    const ExpBelow exp_below;
    double sum = 0.;
    if (wmost >= ORDER_FINITE) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum += exp_below(x[i], top);
    }
    sum = wave_sum(sum);
    // NaN of either sign or +infinity: above the numbers, or below -infinity
    if (__builtin_amdgcn_ballot_w64(most >= ORDER_INF || least < ORDER_FINITE - 1)) sum = __builtin_nan("");
    wave_bounds<16, W>(most, a.n_out, (piece + 1) * (int64_t)(BEAM_T1 * V) <= a.vocab, bounds);
    if (lane == 0) {
        sums[wave] = sum;
        tops[wave] = wmost >= ORDER_FINITE ? top : -INFINITY;
    }
    __syncthreads();
    const uint32_t t = max(waves_bound<W>(bounds), ORDER_FINITE);
    auto key = [&](int i) { return (uint64_t)o[i] << 32 | (uint32_t)~(uint32_t)(first + i / E * (BEAM_T1 * E) + i % E); };
    // one place for the wave's values, which lie there value by value
    int mine = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mine += __builtin_popcountll(__builtin_amdgcn_ballot_w64(o[i] >= t));
    if (mine) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&found, mine);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t m = __builtin_amdgcn_ballot_w64(o[i] >= t);
            if (!m) continue;
            const int to = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
            if (o[i] >= t && to < BEAM_CAP) cand[to] = key(i);
            at += __builtin_popcountll(m);
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
            for (int i = 0; i < V; ++i) c += o[i] >= ORDER_FINITE && key(i) >= trial;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) c += __shfl_xor(c, d, WAVE);
            __syncthreads();
            if (lane == 0) counts[wave] = c;
            __syncthreads();
            c = 0;
            for (int i = 0; i < W; ++i) c += counts[i];
            if (c >= a.n_out) bit_t = trial;
        }
        if (tid == 0) found = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (o[i] >= ORDER_FINITE && key(i) >= bit_t) cand[atomicAdd(&found, 1)] = key(i);  // n_out of them
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
        float m = tops[0];
        for (int i = 1; i < W; ++i) m = fmaxf(m, tops[i]);
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
    __shared__ uint32_t bounds[4][W];
    __shared__ BeamCand heads[W];
    static_assert(W == 8, "");
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    if (tid == 0) found = 0;

    // a list is piece list / beams of row list % beams; the first keys of the thread's first one are on their way early
    const int lists = a.beams * w.n, n_out = a.n_out;
    auto keys_of = [&](int list) { return w.keys + ((row0 + list % a.beams) * w.n + list / a.beams) * n_out; };
    uint64_t ahead8[8];
    auto load8 = [&](int list, int d0) {
        const uint64_t *src = keys_of(list) + d0;
#pragma unroll
        for (int j = 0; j < 8; ++j) ahead8[j] = d0 + j < n_out ? src[j] : 0;
    };
    if (tid < lists) load8(tid, 0);

    // the rows' sums
    const ExpBelow exp_below;
    for (int r = wave; r < a.beams; r += W) {
        const BeamPiece *p = w.pieces + (row0 + r) * w.n;
        float m = -INFINITY;
        for (int i = lane; i < w.n; i += WAVE) m = fmaxf(m, p[i].top);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, WAVE));
        double s = 0.;
        for (int i = lane; i < w.n; i += WAVE) {
            const BeamPiece x = p[i];
            if (x.sum != x.sum) s = x.sum;
            else if (x.top > -INFINITY) s += x.sum * exp_below(x.top, m);
        }
        s = wave_sum(s);
        if (lane == 0) {
            const double lse = s == 0. ? -INFINITY : (double)m + log(s), score = a.scores[row0 + r], b = score - lse;
            const bool ended = a.done && a.done[row0 + r];
            base[r] = ended ? score : b;
            state[r] = fabs(base[r]) < INFINITY ? ended ? 2 : 1 : 0;
            if (a.lse) a.lse[row0 + r] = (float)lse;
        }
    }
    __syncthreads();

    // what a key of a list is worth; without one the key is 0
    auto worth = [&](int list, uint64_t key, bool first) {
        BeamCand x = {0, 0, list % a.beams};
        const int st = state[x.row];
        if (st == 1 && key) {
            x.key = key;
            x.c = order64(base[x.row] + (double)value32((uint32_t)(key >> 32)));
        } else if (st == 2 && first && list < a.beams) {
            x.c = order64(base[x.row]);
            x.key = 1ull << 32 | (uint32_t)~a.end_token;
        }
        return x;
    };
    auto candidate = [&](int list, int d) { return worth(list, keys_of(list)[d], d == 0); };
    // a bound that at least n_out candidates reach, from the first ones of the lists
    const int depth = (n_out + lists - 1) / lists;
    uint32_t most = tid < lists ? (uint32_t)(worth(tid, ahead8[0], true).c >> 32) : 0u;
    for (int e = tid + BEAM_T2; e < lists * depth; e += BEAM_T2) most = max(most, (uint32_t)(candidate(e % lists, e / lists).c >> 32));
    if (lists < BEAM_T2 && tid >= lists && tid < lists * depth) most = (uint32_t)(candidate(tid % lists, tid / lists).c >> 32);
    wave_bounds<22, W>(most, n_out, false, bounds);
    __syncthreads();
    const uint32_t t = waves_bound<W>(bounds);
    for (int l = tid; l < lists; l += BEAM_T2)
        for (int d0 = 0; d0 < n_out; d0 += 8) {
            if (l != tid || d0) load8(l, d0);
            bool more = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const BeamCand x = worth(l, ahead8[j], d0 + j == 0);
                more = x.key && (uint32_t)(x.c >> 32) >= t;
                if (!more) continue;
                const int at = atomicAdd(&found, 1);
                if (at >= BEAM_CAP2) continue;
                cs[at] = x.c;
                ks[at] = x.key;
                rs[at] = (uint8_t)x.row;
            }
            if (!more) break;
        }
    __syncthreads();
    const int n = found;
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
                    const BeamCand x = {mine, ks[i], rs[i]};
                    for (int j = part; j < n; j += parts)
                        if (cs[j] == mine) ahead += BeamCand{mine, ks[j], rs[j]}.ahead_of(x);
                }
                return ahead;
            },
            [&](int i, int ahead) {
                if (ahead < n_out) put(ahead, BeamCand{cs[i], ks[i], rs[i]});
            });
        for (int i = n + tid; i < n_out; i += BEAM_T2) put(i, BeamCand{0, 0, 0});
        return;
    }
    // very many equal sums: the lists merged one candidate at a time
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

// Values of a thread: pieces of 8192, or of 2048 where the larger ones would be too few for the chip.
static int beam_values(int64_t rows, int64_t vocab) { if (const char *e = getenv("BV")) return atoi(e); return rows * ((vocab + 8191) / 8192) < 512 ? 8 : 32; }

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
