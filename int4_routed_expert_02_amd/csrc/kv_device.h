// kv_device.h -- what the cache kernels share: the arguments as the kernels take
// them, and the reading of the batch's tables.  Every value that comes from a
// device table is brought inside the sizes of the shape here, so no access
// depends on what a table holds.
#pragma once

#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

// One sequence of the batch: its rows, its length after them.
struct KvSeq {
    int row0;   // first row in the batch's tensors
    int n;      // rows, inside the batch's tensors and at most max_rows
    int n_pos;  // rows as the table has them: row i has position len - n_pos + i
    int len;    // kv_len as the table has it, from 0 to 2^30
};

__device__ __forceinline__ KvSeq kv_seq(const KvArgs &a, int s)
{
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1];
    KvSeq q;
    q.row0 = min(max(r0, 0), a.rows);
    const int n = max(min(r1, a.rows) - q.row0, 0);
    q.n = min(n, a.max_rows);
    q.n_pos = n;
    q.len = min(max(a.kv_len[s], 0), 1 << 30);
    return q;
}

// Positions a kernel may look at: inside the page table and the host's bound.
__device__ __forceinline__ int kv_limit(const KvArgs &a, const KvSeq &q)
{
    return min(min(q.len, a.max_len), a.max_pages << a.page_log2);
}

// The workgroup's number in a launch of kv_grid().
__device__ __forceinline__ int kv_block() { return (int)blockIdx.x + (int)blockIdx.y * (int)KV_GRID_X; }

// Units of 2^log2 rows of `heads` heads, counted through the batch: sequence s has them
// from (row_start[s] * heads >> log2) + extra * s on, so `extra` more than its rows fill
// for each sequence.  Of unit u: the last sequence that begins at or below it, and the
// unit's number in that sequence (below 0 before the first; the callers bound it above).
__device__ __forceinline__ int kv_unit(const KvArgs &a, int u, int heads, int log2, int extra, int &t)
{
    auto begin = [&](int s) { return (min(max(a.row_start[s], 0), a.rows) * heads >> log2) + extra * s; };
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (begin(mid) <= u) lo = mid;
        else hi = mid;
    }
    t = u - begin(lo);
    return lo;
}

// Positions below this lie in full pages (8 bits: these have their codes, the
// rows of the page from here on are in the sequence's open page).  That goes by
// the sequence's length: a smaller max_len opens no page.
__device__ __forceinline__ int kv_full(const KvArgs &a, const KvSeq &q) { return (q.len >> a.page_log2) << a.page_log2; }

// The page of a sequence's position block, -1 where it is absent.
__device__ __forceinline__ int kv_page(const KvArgs &a, int s, int block)
{
    if ((unsigned)block >= (unsigned)a.max_pages) return -1;
    const int p = a.pages[(int64_t)s * a.max_pages + block];
    return (unsigned)p < (unsigned)a.n_pages ? p : -1;
}

__device__ __forceinline__ int kv_slot(const KvArgs &a, int s)
{
    const int t = a.slots ? a.slots[s] : s;
    return (unsigned)t < (unsigned)a.n_slots ? t : -1;
}

// Element offset of a page's (or an open page's) values of one head: both
// orders, [P][D] and [D][P], take P * D elements.
__device__ __forceinline__ int64_t kv_block_at(const KvArgs &a, int64_t block, int head)
{
    return (block * a.kv_heads + head) * ((int64_t)a.head_dim << a.page_log2);
}

}  // namespace moe
