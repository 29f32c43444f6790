// beam.hip -- beam search's selection over a request's beams and the vocabulary.
//
// c(r, v) = (score_r - lse_r) + x_rv, the n largest of a request.  Within a row the order of the sums is that
// of the logits, so one pass over the logits finds both: the row's sum of exponentials and its n largest
// logits.  First launch: a workgroup a piece of a row, the piece in registers.  Second launch: a workgroup a
// request joins the pieces' sums and merges their lists.
//
// The n largest of a piece without sorting it: each wave finds the k-th largest of its 64 lanes' maxima
// (k = n / waves, a search over the bits of the value with ballots).  k lanes of every wave have a value that
// large, so at least n values reach the least of the waves' bounds, and few more do.  These go to LDS,
// where each counts how many are ahead of it: its place.
//
// The exponentials and their sums are 64 bits wide: a token's place among those of other rows hangs on the
// difference of two log-sums, and 2^-24 of it changes places (one in some thousand steps with 32 beams).
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

constexpr int BEAM_T1 = 256, BEAM_T2 = 512;  // threads of a piece, of a request
constexpr int BEAM_CAP = 512, BEAM_CAP2 = 1024;  // values that reach the bound and are ranked by counting

// Order-preserving bits of a value, above 0 for every number.
__device__ __forceinline__ uint32_t order32(float x)
{
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float value32(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

__device__ __forceinline__ uint64_t order64(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x == 0. ? 0. : x);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ double value64(uint64_t o) { return __builtin_bit_cast(double, o ^ ((o >> 63) ? 1ull << 63 : ~0ull)); }

// e^d for d <= 0: d = k ln 2 + r with |r| <= ln 2 / 2, the series of e^r up to r^11 / 11! (rest below 7e-15), 2^k.
// ln 2 in two parts, the first its 40 leading bits, so k times it is exact.  NaN stays NaN; below -745 it is 0.
__device__ __forceinline__ double exp_neg(double d)
{
    const double k = __builtin_rint(fmax(d, -800.0) * 1.4426950408889634074);
    const double r = __builtin_fma(k, -0x1.9ef35793c7673p-41, __builtin_fma(k, -0x1.62e42fefa2000p-1, d));
    double p = 1.0 / 39916800.0;
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return d < -745.0 ? 0.0 : __builtin_ldexp(p, (int)k);
}

__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, WAVE);
    return x;
}

// The k-th largest of the wave's 64 values (the largest v that k of them reach), k <= 64.
__device__ __forceinline__ uint32_t wave_kth(uint32_t v, int k)
{
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 0; --b) {
        const uint32_t trial = t | 1u << b;
        if (__builtin_popcountll(__builtin_amdgcn_ballot_w64(v >= trial)) >= k) t = trial;
    }
    return t;
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
    __shared__ int found, counts[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / w.n;
    const int piece = blockIdx.x % w.n;
    const T *src = (const T *)a.logits + row * a.row_stride;
    const int64_t first = (int64_t)piece * (BEAM_T1 * V) + tid * E;
    if (tid == 0) found = 0;

    uint32_t o[V];
    float top = -INFINITY;
    uint32_t most = 0;
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
                const float x = E == 4 ? __uint_as_float(raw[u][j]) : (j & 1) ? bf16_hi(raw[u][j / 2]) : bf16_lo(raw[u][j / 2]);
                top = fmaxf(top, x);
                o[u * E + j] = __float_as_uint(x);
            }
    }
    // a wave's sum is taken from its own largest
    float wtop = top;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) wtop = fmaxf(wtop, __shfl_xor(wtop, d, WAVE));
    double sum = 0.;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float x = __uint_as_float(o[i]);
        nan |= x != x || x == INFINITY;
        if (wtop > -INFINITY) sum += exp_neg((double)x - (double)wtop);
        o[i] = x > -INFINITY ? order32(x) : 0u;
        most = most > o[i] ? most : o[i];
    }
    if (__builtin_amdgcn_ballot_w64(nan)) sum = __builtin_nan("");
    sum = wave_sum(sum);
    const uint32_t bound = wave_kth(most, (a.n_out + W - 1) / W);
    if (lane == 0) {
        sums[wave] = sum;
        tops[wave] = wtop;
        bounds[wave] = bound;
    }
    __syncthreads();
    uint32_t t = bounds[0];
#pragma unroll
    for (int i = 1; i < W; ++i) t = t < bounds[i] ? t : bounds[i];
    t = t ? t : 1u;
    auto key = [&](int i) { return (uint64_t)o[i] << 32 | (uint32_t)~(uint32_t)(first + i / E * (BEAM_T1 * E) + i % E); };
    if (most >= t) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (o[i] >= t) {
                const int at = atomicAdd(&found, 1);
                if (at < BEAM_CAP) cand[at] = key(i);
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
            for (int i = 0; i < V; ++i) c += o[i] && key(i) >= trial;
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
            if (o[i] && key(i) >= bit_t) cand[atomicAdd(&found, 1)] = key(i);  // n_out of them
        __syncthreads();
        n = found;
    }
    uint64_t *out = w.keys + (row * w.n + piece) * a.n_out;
    for (int i = tid; i < n; i += BEAM_T1) {
        const uint64_t mine = cand[i];
        int ahead = 0;
        for (int j = 0; j < n; ++j) ahead += cand[j] > mine;
        if (ahead < a.n_out) out[ahead] = mine;
    }
    for (int i = n + tid; i < a.n_out; i += BEAM_T1) out[i] = 0;
    if (tid == 0) {
        float m = tops[0];
        for (int i = 1; i < W; ++i) m = fmaxf(m, tops[i]);
        double s = 0.;
        for (int i = 0; i < W; ++i)
            if (tops[i] > -INFINITY || sums[i] != sums[i]) s += sums[i] * exp_neg((double)tops[i] - (double)m);
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
    __shared__ BeamCand heads[W];
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    if (tid == 0) found = 0;

    // the rows' sums
    for (int r = wave; r < a.beams; r += W) {
        const BeamPiece *p = w.pieces + (row0 + r) * w.n;
        float m = -INFINITY;
        for (int i = lane; i < w.n; i += WAVE) m = fmaxf(m, p[i].top);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, WAVE));
        double s = 0.;
        for (int i = lane; i < w.n; i += WAVE) {
            const BeamPiece x = p[i];
            if (x.top > -INFINITY || x.sum != x.sum) s += x.sum * exp_neg((double)x.top - (double)m);
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

    const int lists = a.beams * w.n, n_out = a.n_out;
    // the d-th candidate of a list (the lists of a row: its pieces); without one the key is 0
    auto candidate = [&](int list, int d) {
        BeamCand x = {0, 0, list / w.n};
        const int st = state[x.row];
        if (st == 1) {
            x.key = w.keys[((row0 + x.row) * w.n + list % w.n) * n_out + d];
            if (x.key) x.c = order64(base[x.row] + (double)value32((uint32_t)(x.key >> 32)));
        } else if (st == 2 && list % w.n == 0 && d == 0) {
            x.c = order64(base[x.row]);
            x.key = 1ull << 32 | (uint32_t)~a.end_token;
        }
        return x;
    };
    // a bound that at least n_out of the lists' first candidates reach
    const int depth = min(n_out, (BEAM_T2 + lists - 1) / lists);
    uint32_t most = 0;
    for (int e = tid; e < lists * depth; e += BEAM_T2) {
        const uint32_t c = (uint32_t)(candidate(e % lists, e / lists).c >> 32);
        most = most > c ? most : c;
    }
    const uint32_t bound = wave_kth(most, (n_out + W - 1) / W);
    if (lane == 0) bounds[wave] = bound;
    __syncthreads();
    uint32_t t = bounds[0];
#pragma unroll
    for (int i = 1; i < W; ++i) t = t < bounds[i] ? t : bounds[i];
    for (int l = tid; l < lists; l += BEAM_T2)
        for (int d = 0; d < n_out; ++d) {
            const BeamCand x = candidate(l, d);
            if (x.key == 0 || (uint32_t)(x.c >> 32) < t) break;
            const int at = atomicAdd(&found, 1);
            if (at >= BEAM_CAP2) break;
            cs[at] = x.c;
            ks[at] = x.key;
            rs[at] = (uint8_t)x.row;
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
        for (int i = tid; i < n; i += BEAM_T2) {
            const BeamCand x = {cs[i], ks[i], rs[i]};
            int ahead = 0;
            for (int j = 0; j < n; ++j) ahead += BeamCand{cs[j], ks[j], rs[j]}.ahead_of(x);
            if (ahead < n_out) put(ahead, x);
        }
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
static int beam_values(int64_t rows, int64_t vocab) { return rows * ((vocab + 8191) / 8192) < 512 ? 8 : 32; }

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
    if (beam_values(rows, a.vocab) == 8) hipLaunchKernelGGL((k_beam_piece<T, 8>), grid, block, 0, st, a, w);
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
