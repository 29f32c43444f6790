// kv_pool.hip -- the pages of a cache: given back, shared by forked sequences, handed out, moved
// together, copied.
//
// A pool's state is the page tables and one count a page, refs: how many entries name it.  There is no
// list of free pages: a page is free when its count is 0, and the lowest free pages are found by
// reading the counts (4 bytes a page: 131072 pages are half a megabyte).  So there is nothing that could
// disagree with the counts, and who gets which page does not depend on the order of atomics: those
// only add to counts, whose sums do not depend on it, or take the least of numbers.
//
// What bounds them: latency.  A table's or count's line is written by one kernel and read by the next from memory
// behind the chip's eight L2 caches, so a kernel takes its launch (2 us) and 0.5 to 1 us for each load that waits for
// another: release 3.0 us (32 x 64 entries), fork 3.5 (32 sequences), reserve 6.8 (32 sequences, one token each) and 9.7
// (16 groups of eight that share their last page), compact 5.1 (1710 pages) or 15.4 in three launches (38731 pages).  So
// loads that do not depend on one another are sent together, and what can be looked up lies in LDS.  The copies
// run at the rate of the memory: 9211 pages of 64 KB, 1.21 GB read and written, 241 us, 5.0 TB/s; a large copy 5.2.
//
// Every page id and parent that comes from a device table is brought inside the sizes of the shape
// where it is read, so no access depends on what a table holds.
#include "kv_device.h"

namespace moe {

constexpr int CHUNK = 16 * WAVE;         // pages that a wave looks at together: 16 of a lane
constexpr int BLOCK_WAVES = 4;
constexpr int BLOCK = BLOCK_WAVES * CHUNK;  // pages of a workgroup's step
constexpr int MAX_BLOCKS = 8192;         // workgroups over the counts, each with as many steps as it needs

struct PoolBlocks {
    int n, steps;  // workgroups, steps of each
};

static PoolBlocks pool_blocks(int n_pages)
{
    const int64_t all = ((int64_t)n_pages + BLOCK - 1) / BLOCK;
    const int64_t steps = (all + MAX_BLOCKS - 1) / MAX_BLOCKS;
    return {(int)(steps ? (all + steps - 1) / steps : 0), (int)steps};
}

// Workspace: [MAX_BLOCKS] counts, [n_pages] a list of free pages or the move of each page, [n_pages] PageUse.
struct PageUse {
    unsigned long long leader;  // the first block of the call that names the page: sequence << 32 | block
    int blocks, refs;           // blocks of the call that name it, its count before the call
};

static size_t list_at() { return MAX_BLOCKS * sizeof(int32_t); }
static size_t use_at(int n_pages) { return list_at() + ((size_t)n_pages * 4 + 255) / 256 * 256; }

size_t kv_pool_workspace(int n_pages) { return use_at(n_pages) + (size_t)n_pages * sizeof(PageUse); }

// The number of blocks that hold positions below len.
__device__ __forceinline__ int blocks_of(const KvArgs &a, int len)
{
    len = min(max(len, 0), 1 << 30);
    return min((len + (1 << a.page_log2) - 1) >> a.page_log2, a.max_pages);
}

__device__ __forceinline__ bool in_cache(const KvArgs &a, int page) { return (unsigned)page < (unsigned)a.n_pages; }

// Which of the CHUNK pages from p0 on are in use: bit l of word(u) is page p0 + 64 u + l, 0 from n_pages on.  Lane u
// holds word u, so that loops over the words stay loops.
struct ChunkBits {
    uint32_t lo, hi;
    int n;
    __device__ __forceinline__ uint64_t word(int u) const
    {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, u) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)lo, u);
    }
};

__device__ __forceinline__ ChunkBits chunk_live(const int32_t *refs, int64_t p0, int64_t n_pages, int lane)
{
    ChunkBits c = {0, 0, 0};
    if (p0 >= n_pages) return c;
    // every lane loads, past the end the last page: loads under a condition wait for one another (4.3 us for 16)
    int r[16];
    const int32_t *at = refs + p0;
    const int last = (int)min(n_pages - p0, (int64_t)CHUNK) - 1;
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = at[min(64 * i + lane, last)];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint64_t m = __builtin_amdgcn_ballot_w64(r[i] > 0 && 64 * i + lane <= last);
        c.n += __builtin_popcountll(m);
        c.lo = lane == i ? (uint32_t)m : c.lo;
        c.hi = lane == i ? (uint32_t)(m >> 32) : c.hi;
    }
    return c;
}

// Bits of m below the lane's own.
__device__ __forceinline__ int below(uint64_t m)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Sum over the lanes up to each one's own (of a wave, or of each row of 16 lanes).
template <bool ROW>
__device__ __forceinline__ int lanes_scan(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4 and 8 lanes below in the row
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    if (ROW) return x;
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // the last lane of rows 0 and 2 to rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
    return x;
}

// Sum of the workgroup's values before mine (`total`: of all), T threads, T / 64 at most 16 waves.  `waves` has 16 places.
template <int T>
__device__ __forceinline__ int group_scan(int v, int *waves, int &total)
{
    constexpr int W = T / WAVE;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, x = lanes_scan<false>(v);
    __syncthreads();
    if (lane == 63) waves[wave] = x;
    __syncthreads();
    const int sums = lanes_scan<true>((lane & 15) < W ? waves[lane & 15] : 0);
    total = __builtin_amdgcn_readlane(sums, W - 1);
    const int before = __builtin_amdgcn_readlane(sums, max(wave - 1, 0));
    return (wave ? before : 0) + x - v;
}

// ---------------------------------------------------------------- given back

// One entry a thread.
__global__ __launch_bounds__(256) void k_kv_release(KvArgs a, int sinks, int32_t *__restrict__ pages, int32_t *__restrict__ refs)
{
    const int64_t total = (int64_t)a.n_seq * a.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int s = (int)(i / a.max_pages), b = (int)(i % a.max_pages);
        const int len = min(max(a.kv_len[s], 0), 1 << 30);
        const int64_t first = (int64_t)b << a.page_log2, next = first + (1 << a.page_log2);
        const bool behind = a.window && next <= (int64_t)len - a.window + 1 && first >= sinks;
        if (first < len && !behind) continue;
        const int page = pages[i];
        if (page == -1) continue;
        pages[i] = -1;
        if (in_cache(a, page)) atomicSub(refs + page, 1);
    }
}

// ---------------------------------------------------------------- forked

constexpr int FORK_ENTRIES = 2048;   // entries of a row that a workgroup takes at a time
constexpr int FORK_PARTS = 256;      // workgroups of a row, at most

// The first workgroup: lengths, slots and the slots' copies.  The others: a part of one
// row's table each, as a continuation (its entries from the parent) and as a parent (its pages'
// counts change by the continuations less one).
__global__ __launch_bounds__(256) void k_kv_fork(KvArgs a, const int32_t *__restrict__ parent, int32_t *__restrict__ len_out,
                                                 int32_t *__restrict__ pages_out, int32_t *__restrict__ slots_out,
                                                 int32_t *__restrict__ refs, int32_t *__restrict__ slot_src,
                                                 int32_t *__restrict__ slot_dst, int parts)
{
    __shared__ int first[KV_FORK_MAX];
    __shared__ uint16_t left[KV_FORK_MAX];
    __shared__ int waves[16];
    const int tid = threadIdx.x, n = a.n_seq;
    auto parent_of = [&](int s) {
        const int p = parent[s];
        return (unsigned)p < (unsigned)n ? p : -1;
    };
    auto len_of = [&](int s) { return min(max(a.kv_len[s], 0), 1 << 30); };
    if (blockIdx.x == 0) {
        for (int s = tid; s < n; s += 256) {
            const int p = parent_of(s);
            len_out[s] = p >= 0 ? len_of(p) : 0;
            first[s] = INT32_MAX;
        }
        if (!slots_out) return;
        __syncthreads();
        for (int s = tid; s < n; s += 256)
            if (const int p = parent_of(s); p >= 0) atomicMin(&first[p], s);
        __syncthreads();
        int total = 0;
        for (int s0 = 0, at = 0; s0 < n; s0 += 256, at += total) {   // sequences that none goes on from
            const int s = s0 + tid, none = s < n && first[s] == INT32_MAX;
            const int rank = group_scan<256>(none, waves, total);
            if (none) left[at + rank] = (uint16_t)s;
        }
        __syncthreads();
        auto slot_of = [&](int s) { return a.slots ? a.slots[s] : s; };
        for (int s0 = 0, at = 0; s0 < n; s0 += 256, at += total) {   // as many as there are sequences without a slot
            const int s = s0 + tid, p = s < n ? parent_of(s) : -1;
            const int extra = s < n && (p < 0 || first[p] != s);
            const int rank = group_scan<256>(extra, waves, total);
            if (s >= n) continue;
            const int slot = slot_of(extra ? left[at + rank] : p);
            const bool copied = extra && p >= 0 && len_of(p) > 0;
            slots_out[s] = slot;
            slot_src[s] = copied ? slot_of(p) : -1;
            slot_dst[s] = copied ? slot : -1;
        }
        return;
    }
    const int s = (blockIdx.x - 1) / parts, part = (blockIdx.x - 1) % parts, p = parent_of(s);
    const int taken = p >= 0 ? blocks_of(a, a.kv_len[p]) : 0, held = blocks_of(a, a.kv_len[s]);
    int c = 0;
    for (int t = tid; t < n; t += 256) c += parent[t] == s ? 1 : 0;
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) c += __shfl_xor(c, d, WAVE);
    if ((tid & 63) == 0) waves[tid >> 6] = c;
    __syncthreads();
    const int go_on = waves[0] + waves[1] + waves[2] + waves[3];
    const int32_t *mine = a.pages + (int64_t)s * a.max_pages, *theirs = a.pages + (int64_t)max(p, 0) * a.max_pages;
    int32_t *out = pages_out + (int64_t)s * a.max_pages;
    for (int e = part * FORK_ENTRIES; e < a.max_pages; e += parts * FORK_ENTRIES)
        for (int b = e + tid; b < min(e + FORK_ENTRIES, a.max_pages); b += 256) {
            const int page = b < taken ? theirs[b] : -1;
            out[b] = in_cache(a, page) ? page : -1;
            const int change = b < held ? go_on - 1 : -1;
            if (change == 0) continue;
            const int named = mine[b];
            if (in_cache(a, named)) atomicAdd(refs + named, change);
        }
}

// ---------------------------------------------------------------- handed out

// The blocks of a sequence that its coming rows are in: first, how many, and whether the first has rows before them.
struct Wanted {
    int first, n;
    bool partial;
};

__device__ __forceinline__ Wanted wanted_blocks(const KvArgs &a, int s)
{
    const KvSeq q = kv_seq(a, s);
    const int start = max(q.len - q.n_pos, 0), end = kv_limit(a, q);
    Wanted w = {start >> a.page_log2, 0, (start & ((1 << a.page_log2) - 1)) != 0};
    if (q.n_pos > 0 && end > start) w.n = ((end - 1) >> a.page_log2) - w.first + 1;
    return w;
}

// First launch: the number of free pages of every block of pages; for every page that a wanted block
// names its count now and room for who else wants it; the lists' empty state.
__global__ __launch_bounds__(256) void k_kv_reserve_count(KvArgs a, const int32_t *__restrict__ pages, const int32_t *__restrict__ refs,
                                                          int32_t *__restrict__ copy_src, int32_t *__restrict__ copy_dst,
                                                          int32_t *__restrict__ missing, int32_t *__restrict__ counts,
                                                          PageUse *__restrict__ use, int blocks, int steps)
{
    __shared__ int waves[BLOCK_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if ((int)blockIdx.x < blocks) {
        int n = 0;
        for (int i = 0; i < steps; ++i) {
            const int64_t p0 = ((int64_t)blockIdx.x * steps + i) * BLOCK + wave * CHUNK;
            const int64_t there = min(max((int64_t)a.n_pages - p0, (int64_t)0), (int64_t)CHUNK);
            n += (int)there - chunk_live(refs, p0, a.n_pages, lane).n;
        }
        if (lane == 0) waves[wave] = n;
        __syncthreads();
        if (tid == 0) counts[blockIdx.x] = waves[0] + waves[1] + waves[2] + waves[3];
        return;
    }
    // a wave for each sequence
    for (int64_t s = (int64_t)(blockIdx.x - blocks) * 4 + wave; s < a.n_seq; s += (int64_t)(gridDim.x - blocks) * 4) {
        if (lane == 0) {
            if (copy_src) copy_src[s] = copy_dst[s] = -1;
            if (missing) missing[s] = 0;
        }
        const Wanted w = wanted_blocks(a, (int)s);
        for (int i = lane; i < w.n; i += WAVE) {
            const int page = pages[s * a.max_pages + w.first + i];
            if (in_cache(a, page)) use[page] = {~0ull, 0, refs[page]};
        }
    }
}

// Second launch, one workgroup: the wanted blocks in order, 1024 at a time.  Who shares which page
// first; then how many pages are needed; their list; then the hand-out.  Sequences of one token that have their page / that
// all need one, both launches, in a pool nine tenths full: 32 over 70000 pages 13 / 19 us, over a million 13 / 23 (10 / 10 over
// 60000 in the one launch below), 512 over a million 14 / 26, 20000 149 / 166; a prompt of 8192 blocks 78.
constexpr int RT = 1024;

__global__ __launch_bounds__(RT) void k_kv_reserve(KvArgs a, int32_t *pages, int32_t *refs, int32_t *copy_src, int32_t *copy_dst,
                                                   int32_t *missing, const int32_t *counts, int32_t *list, PageUse *use,
                                                   int blocks, int steps)
{
    __shared__ int begin[RT], from[RT], waves[RT / WAVE], base[MAX_BLOCKS];
    __shared__ uint8_t inside[RT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int total;

    // The wanted blocks one after another: f(sequence, block, whether it is its sequence's first and has older rows).
    // Every thread calls f, those past the end with sequence -1.  Rows that ascend lie in at most rows / P + 2 blocks of
    // each sequence; whatever else the tables hold, no more than that are looked at.
    auto each = [&](auto f) {
        int left = (a.rows >> a.page_log2) + 2 * a.n_seq;
        for (int s0 = 0; s0 < a.n_seq; s0 += RT) {
            const int s = s0 + tid;
            Wanted w = {0, 0, false};
            if (s < a.n_seq) w = wanted_blocks(a, s);
            const int at = group_scan<RT>(w.n, waves, total);
            const int all = min(total, left);
            left -= max(all, 0);
            begin[tid] = at;
            from[tid] = w.first;
            inside[tid] = w.partial;
            __syncthreads();
            for (int i0 = 0; i0 < all; i0 += RT) {
                const int i = i0 + tid;
                int lo = 0, hi = RT;   // the last sequence that begins at or below i
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (begin[mid] <= i) lo = mid;
                    else hi = mid;
                }
                const int b = i - begin[lo], block = from[lo] + b;
                const bool is = i < all && s0 + lo < a.n_seq && (unsigned)block < (unsigned)a.max_pages;
                f(is ? s0 + lo : -1, block, is && b == 0 && inside[lo]);  // one call for all lanes: f has barriers
            }
            __syncthreads();
        }
    };
    auto entry = [&](int s, int b) { return pages[(int64_t)s * a.max_pages + b]; };
    auto key = [](int s, int b) { return (unsigned long long)s << 32 | (unsigned)b; };

    each([&](int s, int b, bool) {
        if (s < 0) return;
        const int page = entry(s, b);
        if (!in_cache(a, page) || use[page].refs <= 1) return;
        atomicAdd(&use[page].blocks, 1);
        atomicMin(&use[page].leader, key(s, b));
    });
    __threadfence();
    __syncthreads();

    // Of a wanted block: 0 it has its page, 1 it needs one, 2 it needs one in another's place, 3 its older rows are gone.
    // first: of all that name the page of another here, which then is left with `rest` entries.
    bool first = false;
    int rest = 0;
    auto state = [&](int s, int b, bool partial, int &page) {
        first = false;
        page = entry(s, b);
        if (!in_cache(a, page)) {
            page = -1;
            return partial ? 3 : 1;
        }
        const int held = use[page].refs;
        if (held <= 1) return 0;
        const int wanted = __hip_atomic_load(&use[page].blocks, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        first = __hip_atomic_load(&use[page].leader, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == key(s, b);
        rest = wanted == held ? 1 : held - wanted;
        return wanted == held && first ? 0 : 2;
    };
    int need = 0;
    each([&](int s, int b, bool partial) {
        int page;
        const int st = s >= 0 ? state(s, b, partial, page) : 0;
        need += st == 1 || st == 2;
    });
    group_scan<RT>(need, waves, need);

    // the lowest `need` free pages
    int have = 0;
    if (need) {
        for (int b0 = 0; b0 < blocks; b0 += RT) {
            const int i = b0 + tid;
            const int before = group_scan<RT>(i < blocks ? counts[i] : 0, waves, total);
            if (i < blocks) base[i] = have + before;
            have += total;
        }
        __syncthreads();
        have = min(have, need);
        for (int i = wave; i < blocks; i += RT / WAVE) {
            int at = base[i];
            if (at >= have) break;
            if (counts[i] == 0) continue;
            for (int c = 0; c < steps * BLOCK_WAVES && at < have; ++c) {
                const int64_t p0 = (int64_t)i * steps * BLOCK + c * CHUNK;
                const ChunkBits live = chunk_live(refs, p0, a.n_pages, lane);
#pragma unroll 1
                for (int u = 0; u < 16; ++u) {
                    const int64_t p = p0 + 64 * u;
                    uint64_t free = ~live.word(u);
                    if (p + 64 > a.n_pages) free &= p >= a.n_pages ? 0ull : ~0ull >> (64 - (int)(a.n_pages - p));
                    const int mine = at + below(free);
                    if ((free >> lane & 1) && mine < have) list[mine] = (int32_t)(p + lane);
                    at += __builtin_popcountll(free);
                }
            }
        }
        __threadfence();
        __syncthreads();
    }

    int given = 0;
    each([&](int s, int b, bool partial) {
        int page = -1;
        const int st = s >= 0 ? state(s, b, partial, page) : 0;
        const bool needs = st == 1 || st == 2;
        const int rank = given + group_scan<RT>(needs, waves, total);
        given += total;
        if (s >= 0 && first) refs[page] = rest;
        if (st == 0) return;
        const int got = needs && rank < have ? list[rank] : -1;
        if (got < 0 && missing) atomicAdd(missing + s, 1);
        if (st == 3) return;
        pages[(int64_t)s * a.max_pages + b] = got;
        if (got < 0) return;
        refs[got] = 1;
        if (st == 2 && partial && copy_src) {
            copy_src[s] = page;
            copy_dst[s] = got;
        }
    });
}

// The same in one launch where the wanted blocks are at most 1024 and the pages few: who shares a page is
// found by comparing the blocks in LDS, and a block finds its free page in the pages' bits there.
constexpr int RESERVE_PAGES = 64 * RT;  // pages, at most: a word of bits for each thread

__global__ __launch_bounds__(RT) void k_kv_reserve_small(KvArgs a, int32_t *__restrict__ pages, int32_t *__restrict__ refs,
                                                         int32_t *__restrict__ copy_src, int32_t *__restrict__ copy_dst,
                                                         int32_t *__restrict__ missing)
{
    __shared__ int begin[RT], from[RT], free_before[RT], waves[RT / WAVE];
    __shared__ __align__(16) int shared[RT];
    __shared__ uint64_t free_pages[RT];
    __shared__ uint8_t inside[RT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll 1
    for (int chunk = wave; chunk < RT / 16; chunk += RT / WAVE) {
        const int p0 = chunk * CHUNK, rest = a.n_pages - p0 - 64 * lane;  // lane u: word u
        if (p0 >= a.n_pages) {
            if (lane < 16) free_pages[chunk * 16 + lane] = 0;
            continue;
        }
        const ChunkBits live = chunk_live(refs, p0, a.n_pages, lane);
        const uint64_t there = rest >= 64 ? ~0ull : rest <= 0 ? 0ull : ~0ull >> (64 - rest);
        if (lane < 16) free_pages[chunk * 16 + lane] = ~((uint64_t)live.hi << 32 | live.lo) & there;
    }
    Wanted w = {0, 0, false};
    if (tid < a.n_seq) {
        w = wanted_blocks(a, tid);
        if (copy_src) copy_src[tid] = copy_dst[tid] = -1;
        if (missing) missing[tid] = 0;
    }
    int all, have, total;
    const int at = group_scan<RT>(w.n, waves, all);
    all = min(all, RT);
    begin[tid] = at;
    from[tid] = w.first;
    inside[tid] = w.partial;
    free_before[tid] = group_scan<RT>((int)__builtin_popcountll(free_pages[tid]), waves, have);
    __syncthreads();
    // the thread's block
    int s = 0, hi = RT, page = -1, held = 0;
#pragma unroll 1
    while (hi - s > 1) {
        const int mid = (s + hi) / 2;
        if (begin[mid] <= tid) s = mid;
        else hi = mid;
    }
    const int block = from[s] + tid - begin[s];
    const bool mine = tid < all && s < a.n_seq && (unsigned)block < (unsigned)a.max_pages;
    const bool partial = mine && tid == begin[s] && inside[s];
    if (mine) page = pages[(int64_t)s * a.max_pages + block];
    if (in_cache(a, page)) held = refs[page];
    else page = -1;
    bool needs = mine && page < 0 && !partial;
    shared[tid] = held > 1 ? page : -1;
    if (__syncthreads_or(held > 1) && held > 1) {
        int wanted = 0, before = 0;
#pragma unroll 4
        for (int i = 0; i < all; i += 4) {
            const u32x4 four = *(const u32x4 *)(shared + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool same = (int)four[j] == page;
                wanted += same;
                before += same && i + j < tid;
            }
        }
        needs = wanted != held || before;
        // all that name it here get another page, but for the first where no one else holds it
        if (!before) refs[page] = wanted == held ? 1 : held - wanted;
    }
    const int rank = group_scan<RT>(needs, waves, total);
    if (!mine) return;
    int got = -1;
    if (needs && rank < have) {
        // the rank-th free page: its word, then its bit
        int lo = 0, up = RT;
#pragma unroll 1
        while (up - lo > 1) {
            const int mid = (lo + up) / 2;
            if (free_before[mid] <= rank) lo = mid;
            else up = mid;
        }
        uint64_t bits = free_pages[lo];
        int left = rank - free_before[lo], bit = 0;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const int below_d = __builtin_popcountll(bits & ((1ull << d) - 1));
            if (left >= below_d) {
                left -= below_d;
                bits >>= d;
                bit += d;
            }
        }
        got = 64 * lo + bit;
    }
    if (!needs) {
        if (page < 0 && missing) atomicAdd(missing + s, 1);  // its older rows are gone
        return;
    }
    pages[(int64_t)s * a.max_pages + block] = got;
    if (got < 0) {
        if (missing) atomicAdd(missing + s, 1);
        return;
    }
    refs[got] = 1;
    if (page >= 0 && partial && copy_src) {
        copy_src[s] = page;
        copy_dst[s] = got;
    }
}

// ---------------------------------------------------------------- moved together

// All in one launch where pages and entries are few: the moves in LDS.
constexpr int COMPACT_PAGES = RT / WAVE * CHUNK, COMPACT_ENTRIES = 1 << 14;

__global__ __launch_bounds__(RT) void k_kv_compact_small(KvArgs a, int32_t *__restrict__ pages, int32_t *__restrict__ refs, int max_moves,
                                                         int32_t *__restrict__ src, int32_t *__restrict__ dst, int32_t *__restrict__ n_live)
{
    constexpr int STEPS = COMPACT_PAGES / RT;
    __shared__ uint16_t move[COMPACT_PAGES], hole[COMPACT_PAGES / 2];
    __shared__ int before[COMPACT_PAGES / 64], waves[RT / WAVE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // step i: pages RT i + tid
    int held[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) held[i] = a.n_pages > 0 ? refs[min(RT * i + tid, a.n_pages - 1)] : 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (RT * i + tid >= a.n_pages) held[i] = 0;
        const uint64_t m = __builtin_amdgcn_ballot_w64(held[i] > 0);
        if (lane == 0) before[16 * i + wave] = __builtin_popcountll(m);
    }
    __syncthreads();
    int all, moved, movers = 0;
    const int at = group_scan<RT>(tid < COMPACT_PAGES / 64 ? before[tid] : 0, waves, all);
    if (tid < COMPACT_PAGES / 64) before[tid] = at;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (RT * i >= a.n_pages) break;
        const int p = RT * i + tid;
        const bool used = held[i] > 0;
        const int rank = before[16 * i + wave] + below(__builtin_amdgcn_ballot_w64(used));  // pages in use below p
        int k = -1;
        if (used && p >= all) {
            ++movers;
            k = all - 1 - rank;
            if (k < max_moves) src[k] = p;
            else k = -1;
        } else if (!used && p < all && p - rank < max_moves) {
            hole[p - rank] = (uint16_t)p;
            dst[p - rank] = p;
        }
        move[p] = (uint16_t)k;
    }
    group_scan<RT>(movers, waves, moved);
    moved = min(moved, max_moves);
    for (int i = moved + tid; i < max_moves; i += RT) src[i] = dst[i] = -1;
    if (n_live && tid == 0) n_live[0] = all;
    for (int i = tid; i < a.n_seq * a.max_pages; i += RT) {
        const int page = pages[i];
        if (!in_cache(a, page)) continue;
        const int k = move[page];
        if (k != 0xFFFF) pages[i] = hole[k];
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int p = RT * i + tid, k = p < a.n_pages ? move[p] : 0xFFFF;
        if (k == 0xFFFF) continue;
        refs[hole[k]] = held[i];
        refs[p] = 0;
    }
}

// First launch: pages in use of every block; the lists' empty state.
__global__ __launch_bounds__(256) void k_kv_compact_count(const int32_t *__restrict__ refs, int n_pages, int steps, int max_moves,
                                                          int32_t *__restrict__ src, int32_t *__restrict__ dst, int32_t *__restrict__ counts)
{
    __shared__ int waves[BLOCK_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = blockIdx.x * 256 + tid; i < max_moves; i += gridDim.x * 256) src[i] = dst[i] = -1;
    int n = 0;
    for (int i = 0; i < steps; ++i)
        n += chunk_live(refs, ((int64_t)blockIdx.x * steps + i) * BLOCK + wave * CHUNK, n_pages, lane).n;
    if (lane == 0) waves[wave] = n;
    __syncthreads();
    if (tid == 0) counts[blockIdx.x] = waves[0] + waves[1] + waves[2] + waves[3];
}

// Second launch: of every page its move, or -1.  With n pages in use and r of them below page p, a free
// p < n is the (p - r)-th hole from below, and a p >= n in use the (n - 1 - r)-th page from above: holes and
// pages of one number go together.
__global__ __launch_bounds__(256) void k_kv_compact_plan(const int32_t *__restrict__ refs, int n_pages, int steps, int max_moves,
                                                         int32_t *__restrict__ src, int32_t *__restrict__ dst, int32_t *__restrict__ n_live,
                                                         const int32_t *__restrict__ counts, int32_t *__restrict__ move)
{
    __shared__ int waves[BLOCK_WAVES], sums[2][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int all = 0, before = 0;
    for (int i = tid; i < (int)gridDim.x; i += 256) {
        const int c = counts[i];
        all += c;
        before += i < (int)blockIdx.x ? c : 0;
    }
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
        all += __shfl_xor(all, d, WAVE);
        before += __shfl_xor(before, d, WAVE);
    }
    if (lane == 0) {
        sums[0][wave] = all;
        sums[1][wave] = before;
    }
    __syncthreads();
    all = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    before = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
    if (n_live && blockIdx.x == 0 && tid == 0) n_live[0] = all;
    for (int i = 0; i < steps; ++i) {
        const int64_t p0 = ((int64_t)blockIdx.x * steps + i) * BLOCK + wave * CHUNK;
        const ChunkBits live = chunk_live(refs, p0, n_pages, lane);
        __syncthreads();
        if (lane == 0) waves[wave] = live.n;
        __syncthreads();
        int r = before;
        for (int w = 0; w < BLOCK_WAVES; ++w) {
            r += w < wave ? waves[w] : 0;
            before += waves[w];
        }
#pragma unroll 1
        for (int u = 0; u < 16; ++u) {
            const uint64_t m = live.word(u);
            const int64_t p = p0 + 64 * u + lane;
            const bool used = m >> lane & 1;
            const int rank = r + below(m);
            r += __builtin_popcountll(m);
            if (p >= n_pages) continue;
            int to = -1;
            if (used && p >= all) {
                const int k = all - 1 - rank;
                if (k < max_moves) {
                    src[k] = (int)p;
                    to = k;
                }
            } else if (!used && p < all) {
                const int k = (int)p - rank;
                if (k < max_moves) dst[k] = (int)p;
            }
            move[p] = to;
        }
    }
}

// Third launch: the tables' entries and the counts.
__global__ __launch_bounds__(256) void k_kv_compact_apply(KvArgs a, int32_t *__restrict__ pages, int32_t *__restrict__ refs, int max_moves,
                                                          const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                                                          const int32_t *__restrict__ move)
{
    const int64_t entries = (int64_t)a.n_seq * a.max_pages, total = entries + max_moves;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        if (i < entries) {
            const int page = pages[i];
            if (!in_cache(a, page)) continue;
            const int k = move[page];
            if (k >= 0) pages[i] = dst[k];
        } else {
            const int from = src[i - entries], to = dst[i - entries];
            if (from < 0) continue;
            refs[to] = refs[from];
            refs[from] = 0;
        }
    }
}

// ---------------------------------------------------------------- copied

struct KvCopyList {
    const int32_t *src, *dst;
    int n, limit;          // pairs; ids are below this
    char *k, *v;           // what is copied of an id: `bytes` of k and of v from id * bytes on
    float *ks, *vs;        // and `heads` scales of each (null: none)
    int64_t bytes;
    int heads, parts;      // parts of a pair
};

constexpr int COPY_UNITS = 4;                          // 16-byte pieces of a thread, on their way together
constexpr int COPY_PART = 256 * COPY_UNITS;            // of a part

// One pair's part: k and v as one run of 16-byte pieces.
__device__ __forceinline__ void copy_part(const KvCopyList &l, int src, int dst, int part)
{
    const int tid = threadIdx.x;
    const int64_t per = l.bytes / 16, i0 = (int64_t)part * COPY_PART + tid;
    u32x4 x[COPY_UNITS];
#pragma unroll
    for (int u = 0; u < COPY_UNITS; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i < 2 * per) x[u] = *(const u32x4 *)((i < per ? l.k + 16 * i : l.v + 16 * (i - per)) + src * l.bytes);
    }
#pragma unroll
    for (int u = 0; u < COPY_UNITS; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i < 2 * per) *(u32x4 *)((i < per ? l.k + 16 * i : l.v + 16 * (i - per)) + dst * l.bytes) = x[u];
    }
    if (l.ks && part == 0)
        for (int h = tid; h < l.heads; h += 256) {
            l.ks[(int64_t)dst * l.heads + h] = l.ks[(int64_t)src * l.heads + h];
            l.vs[(int64_t)dst * l.heads + h] = l.vs[(int64_t)src * l.heads + h];
        }
}

// Workgroups take every gridDim.x-th part of the lists' pairs.  A wave looks 64 of its workgroup's parts up at a
// time, so pairs that are not there cost a 64th of a look.
__global__ __launch_bounds__(256) void k_kv_copy(KvCopyList pages, KvCopyList slots)
{
    const int lane = threadIdx.x & 63;
    auto list = [&](const KvCopyList &l) {
        const int64_t total = (int64_t)l.n * l.parts;
        for (int64_t i0 = blockIdx.x; i0 < total; i0 += (int64_t)WAVE * gridDim.x) {
            const int64_t i = i0 + (int64_t)lane * gridDim.x;
            int src = -1, dst = -1;
            if (i < total) {
                src = l.src[i / l.parts];
                dst = l.dst[i / l.parts];
            }
            const bool there = (unsigned)src < (unsigned)l.limit && (unsigned)dst < (unsigned)l.limit && src != dst;
            uint64_t todo = __builtin_amdgcn_ballot_w64(there);
            while (todo) {
                const int u = __builtin_ctzll(todo);
                todo &= todo - 1;
                copy_part(l, __builtin_amdgcn_readlane(src, u), __builtin_amdgcn_readlane(dst, u),
                          (int)((i0 + (int64_t)u * gridDim.x) % l.parts));
            }
        }
    };
    if (pages.n) list(pages);
    if (slots.n) list(slots);
}

// ---------------------------------------------------------------- launches

static unsigned groups_of(int64_t items, int64_t per, int64_t most = 1 << 16)
{
    const int64_t n = (items + per - 1) / per;
    return (unsigned)(n < 1 ? 1 : n > most ? most : n);
}

hipError_t launch_kv_release(const KvArgs &a, int sinks, int32_t *pages, int32_t *refs, hipStream_t st)
{
    hipLaunchKernelGGL(k_kv_release, dim3(groups_of((int64_t)a.n_seq * a.max_pages, 256)), dim3(256), 0, st, a, sinks, pages, refs);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const KvArgs &a, const int32_t *parent, int32_t *len_out, int32_t *pages_out, int32_t *slots_out,
                          int32_t *refs, int32_t *slot_src, int32_t *slot_dst, hipStream_t st)
{
    const int parts = (int)groups_of(a.max_pages, FORK_ENTRIES, FORK_PARTS);
    hipLaunchKernelGGL(k_kv_fork, dim3((unsigned)(1 + parts * a.n_seq)), dim3(256), 0, st, a, parent, len_out, pages_out, slots_out, refs,
                       slot_src, slot_dst, parts);
    return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvArgs &a, int32_t *pages, int32_t *refs, int32_t *copy_src, int32_t *copy_dst, int32_t *missing,
                             void *ws, hipStream_t st)
{
    // rows lie in at most rows / P + 2 blocks of a sequence
    if ((int64_t)(a.rows >> a.page_log2) + 2 * (int64_t)a.n_seq <= RT && a.n_pages <= RESERVE_PAGES) {
        hipLaunchKernelGGL(k_kv_reserve_small, dim3(1), dim3(RT), 0, st, a, pages, refs, copy_src, copy_dst, missing);
        return hipGetLastError();
    }
    const PoolBlocks b = pool_blocks(a.n_pages);
    int32_t *counts = (int32_t *)ws, *list = (int32_t *)((char *)ws + list_at());
    PageUse *use = (PageUse *)((char *)ws + use_at(a.n_pages));
    hipLaunchKernelGGL(k_kv_reserve_count, dim3(b.n + groups_of(a.n_seq, 4)), dim3(256), 0, st, a, pages, refs, copy_src, copy_dst,
                       missing, counts, use, b.n, b.steps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.rows == 0 || a.max_pages == 0) return e;
    hipLaunchKernelGGL(k_kv_reserve, dim3(1), dim3(RT), 0, st, a, pages, refs, copy_src, copy_dst, missing, counts, list, use, b.n,
                       b.steps);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvArgs &a, int32_t *pages, int32_t *refs, int max_moves, int32_t *src, int32_t *dst, int32_t *n_live,
                             void *ws, hipStream_t st)
{
    if (a.n_pages <= COMPACT_PAGES && (int64_t)a.n_seq * a.max_pages <= COMPACT_ENTRIES) {
        hipLaunchKernelGGL(k_kv_compact_small, dim3(1), dim3(RT), 0, st, a, pages, refs, max_moves, src, dst, n_live);
        return hipGetLastError();
    }
    const PoolBlocks b = pool_blocks(a.n_pages);
    int32_t *counts = (int32_t *)ws, *move = (int32_t *)((char *)ws + list_at());
    const unsigned n = b.n ? b.n : 1;  // without a page: n_live 0
    hipLaunchKernelGGL(k_kv_compact_count, dim3(n), dim3(256), 0, st, refs, a.n_pages, b.steps, max_moves, src, dst, counts);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL(k_kv_compact_plan, dim3(n), dim3(256), 0, st, refs, a.n_pages, b.steps, max_moves, src, dst, n_live, counts, move);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (max_moves == 0) return hipSuccess;
    hipLaunchKernelGGL(k_kv_compact_apply, dim3(groups_of((int64_t)a.n_seq * a.max_pages + max_moves, 256)), dim3(256), 0, st, a, pages,
                       refs, max_moves, src, dst, move);
    return hipGetLastError();
}

constexpr int COPY_GROUPS = 4096;  // workgroups that keep the memory busy, with parts left to even out

hipError_t launch_kv_copy(const KvArgs &a, int n_pages, const int32_t *page_src, const int32_t *page_dst, int n_slots,
                          const int32_t *slot_src, const int32_t *slot_dst, hipStream_t st)
{
    const int64_t values = (int64_t)a.kv_heads * a.head_dim << a.page_log2;
    auto list = [&](const int32_t *src, const int32_t *dst, int n, int limit, void *k, void *v, float *ks, float *vs, int64_t bytes) {
        const int64_t parts = (2 * bytes / 16 + COPY_PART - 1) / COPY_PART;
        return KvCopyList{src, dst, n, limit, (char *)k, (char *)v, ks, vs, bytes, a.kv_heads, (int)parts};
    };
    const bool codes = a.kv_bits == 8;
    const KvCopyList p = list(page_src, page_dst, n_pages, a.n_pages, a.k, a.v, codes ? a.k_scale : nullptr, codes ? a.v_scale : nullptr,
                              values * (a.kv_bits / 8));
    const KvCopyList s = list(slot_src, slot_dst, codes ? n_slots : 0, a.n_slots, a.k_tail, a.v_tail, nullptr, nullptr, 2 * values * 2);
    const int64_t parts = (int64_t)p.n * p.parts > (int64_t)s.n * s.parts ? (int64_t)p.n * p.parts : (int64_t)s.n * s.parts;
    hipLaunchKernelGGL(k_kv_copy, dim3(groups_of(parts, 1, COPY_GROUPS)), dim3(256), 0, st, p, s);
    return hipGetLastError();
}

}  // namespace moe
