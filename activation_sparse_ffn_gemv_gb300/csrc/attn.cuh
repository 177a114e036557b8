// attn.cuh -- device code shared by the attention kernels: the split of a
// draft-tree call's work over the CTAs, the partial results and their layout.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace sffn {

// ---------------------------------------------------------------------------
// How sffn_attn_tree's work is split
//
// A sequence's new tokens are cut into row tiles of `tile_tokens` tokens (times
// the G query heads of a key head: one row each).  An item is a (sequence, key head,
// row tile); it reads ceil(positions / 64) units of 64 cached positions.  On one line, item
// after item, each takes its units and kTreeItemCost more in front of them for what an
// item costs by itself; CTA w of W takes [w total / W, (w + 1) total / W) of the line, whatever
// the lengths.  (48 sequences of one token, some a few positions long: 132 us without the extra
// cost, because one CTA got all the short items of a sequence group, 92 with 2 units, 66 with 4, 65.5
// with 5, 67 with 7; 32 with large draft trees, kernel and join on the device, 144, 130, 124.6 and 124.4, which a call
// from Python among others takes 132 for.  It also cuts a short call into more pieces: one token over 300
// positions, 32 heads, 12.2 us with 4, 13 with 5.)  Row tiles of
// one key head are neighbours, so that they read its keys at about the same time.  An
// item whose units lie in one CTA's range is finished there; the pieces of a cut item are
// written as partial results (unnormalised output, running maximum and sum) and joined by
// k_tree_join in the order of the CTAs.  The cut depends on the lengths alone.
// ---------------------------------------------------------------------------

constexpr int kTreeUnit = 64;
constexpr int kTreeItemCost = 5;
constexpr int kTreeMaxTokens = 64;
constexpr int kTreeMaxCtx = 0x7fff0000;  // positions stay below 2^31 with room for a tile

struct TreeSeq {
    int t0, n, ctx;   // first new token, new tokens, committed positions
    int tiles, units; // row tiles, units of each item
    SFFN_DEV int span() const { return units + kTreeItemCost; }  // an item's length on the line
};

// A sequence's numbers, checked; one that breaks the contract has no rows.
SFFN_DEV TreeSeq tree_seq(const TreeArgs &a, int s, bool record) {
    TreeSeq q;
    q.t0 = a.cu_tokens[s];
    const int t1 = a.cu_tokens[s + 1];
    q.ctx = a.ctx_lens[s];
    const long long n = (long long)t1 - q.t0;
    const bool ok = q.t0 >= 0 && t1 <= a.T && n >= 0 && n <= kTreeMaxTokens && q.ctx >= 0 &&
                    q.ctx + n <= ((long long)a.table_width << a.page_shift) && q.ctx <= kTreeMaxCtx;
    if (!ok) {
        if (record) record_error(a.err, SFFN_ERR_DEVICE);
        q.t0 = q.n = q.ctx = q.tiles = q.units = 0;
        return q;
    }
    q.n = (int)n;
    q.tiles = (q.n + a.tile_tokens - 1) / a.tile_tokens;
    q.units = (int)((q.ctx + n + kTreeUnit - 1) / kTreeUnit);
    return q;
}

// pre[s] = length of the line before sequence s, pre[n_seq] = all of it (shared memory, every thread of
// the CTA takes part; scratch: >= 33 long longs).
SFFN_DEV void tree_prefix(const TreeArgs &a, long long *pre, long long *scratch, bool record) {
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = nt >> 5;
    long long base = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += nt) {
        const int s = s0 + threadIdx.x;
        long long v = 0;
        if (s < a.n_seq) {
            const TreeSeq q = tree_seq(a, s, record);
            v = (long long)q.tiles * a.n_kv_heads * q.span();
        }
        long long incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) scratch[warp] = incl;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) before += scratch[w];
            all += scratch[w];
        }
        if (s < a.n_seq) pre[s] = base + before + incl - v;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[a.n_seq] = base;
    __syncthreads();
}

// Last sequence s with pre[s] <= u (u < pre[n_seq]): the one that place u of the line belongs to.
SFFN_DEV int tree_find(const long long *pre, int n_seq, long long u) {
    int lo = 0, hi = n_seq;  // pre[lo] <= u < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// CTAs that take part: none has an empty range.
SFFN_HOST_DEV int tree_ctas(long long total, int grid) { return total < grid ? (int)total : grid; }

// First place of CTA w, and the CTA that place u falls to.
SFFN_HOST_DEV long long tree_cut(long long total, int w, int W) { return total * w / W; }
SFFN_HOST_DEV int tree_owner(long long total, long long u, int W) { return (int)(((u + 1) * W - 1) / total); }

// The piece of an item at place u of the line, in a range that ends at u1.
struct TreePiece {
    int s, h, tile;  // sequence, key head, row tile
    int un0, un1;    // units; none if the range ends before the first
    long long next;  // where the range goes on
};
SFFN_DEV TreePiece tree_piece(const TreeArgs &a, const long long *pre, long long u, long long u1, TreeSeq &q) {
    TreePiece p;
    p.s = tree_find(pre, a.n_seq, u);
    q = tree_seq(a, p.s, false);
    const long long local = u - pre[p.s];
    const int item = (int)(local / q.span()), at = (int)(local - (long long)item * q.span());
    p.h = item / q.tiles;
    p.tile = item - p.h * q.tiles;
    const int end = (int)min((long long)q.span(), at + (u1 - u));
    p.un0 = max(0, at - kTreeItemCost);
    p.un1 = max(0, end - kTreeItemCost);
    p.next = u + (end - at);
    return p;
}

// Partial result slots: a CTA's range cuts at most one item at its front (slot 2 w)
// and one at its end (slot 2 w + 1).  A slot holds rows_max rows of D floats, then
// rows_max (maximum, sum) pairs, and is a multiple of 16 bytes long whatever the rows.
SFFN_HOST_DEV size_t tree_slot_floats(int rows_max, int D) {
    return (size_t)rows_max * D + (size_t)((2 * rows_max + 3) & ~3);
}

}  // namespace sffn
