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

struct SeqTokens {
    int t0, n, ctx;   // first new token, new tokens, committed positions
};

// A sequence's numbers, checked; one that breaks the contract has no tokens.
SFFN_DEV SeqTokens seq_tokens(const SeqArgs &a, int s, bool record) {
    SeqTokens q;
    q.t0 = a.cu_tokens[s];
    const int t1 = a.cu_tokens[s + 1];
    q.ctx = a.ctx_lens[s];
    const long long n = (long long)t1 - q.t0;
    const bool ok = q.t0 >= 0 && t1 <= a.T && n >= 0 && n <= kTreeMaxTokens && q.ctx >= 0 &&
                    q.ctx + n <= ((long long)a.table_width << a.page_shift) && q.ctx <= kTreeMaxCtx;
    if (!ok) {
        if (record) record_error(a.err, SFFN_ERR_DEVICE);
        q.t0 = q.n = q.ctx = 0;
        return q;
    }
    q.n = (int)n;
    return q;
}

struct TreeSeq : SeqTokens {
    int tiles, units; // row tiles, units of each item
    SFFN_DEV int span() const { return units + kTreeItemCost; }  // an item's length on the line
};
SFFN_DEV TreeSeq tree_seq(const TreeArgs &a, int s, bool record) {
    TreeSeq q;
    static_cast<SeqTokens &>(q) = seq_tokens(a, s, record);
    q.tiles = (q.n + a.tile_tokens - 1) / a.tile_tokens;
    q.units = (int)(((long long)q.ctx + q.n + kTreeUnit - 1) / kTreeUnit);
    return q;
}

// pre[i] = sum of length(0) .. length(i - 1), pre[n] = all of it (shared memory, every thread of
// the CTA takes part; scratch: >= 33 long longs).
template <typename F>
SFFN_DEV void line_prefix(int n, long long *pre, long long *scratch, F length) {
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = nt >> 5;
    long long base = 0;
    for (int i0 = 0; i0 < n; i0 += nt) {
        const int i = i0 + threadIdx.x;
        const long long v = i < n ? length(i) : 0;
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
        if (i < n) pre[i] = base + before + incl - v;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[n] = base;
    __syncthreads();
}

// Length of the line before each sequence, and all of it.
SFFN_DEV void tree_prefix(const TreeArgs &a, long long *pre, long long *scratch, bool record) {
    line_prefix(a.n_seq, pre, scratch, [&](int s) {
        const TreeSeq q = tree_seq(a, s, record);
        return (long long)q.tiles * a.n_kv_heads * q.span();
    });
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

// A row of a cut item, put together by one warp from partial results: M = max of the pieces' maxima,
// out = sum(exp(m_i - M) o_i) / sum(exp(m_i - M) l_i), the pieces in the order in which they are added.
// A lane holds C = D / 32 consecutive columns.
template <int C>
struct JoinedRow {
    float o[C], l, M;
    SFFN_DEV JoinedRow() : l(0.f), M(-INFINITY) {
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = 0.f;
    }
    // Pieces i0 .. i1: sums_of(i) points to a piece's (maximum, sum), row_of(i) to its unnormalised row.
    template <typename Sums, typename Row>
    SFFN_DEV void add(int i0, int i1, int lane, Sums sums_of, Row row_of) {
        for (int b = i0; b <= i1; b += 32) {  // 32 pieces at a time
            const int n = min(32, i1 - b + 1);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) ml = __ldcg(reinterpret_cast<const float2 *>(sums_of(b + lane)));
            const float Mn = fmaxf(M, warp_max(ml.x)), ref = Mn == -INFINITY ? 0.f : Mn;
            // a piece without a key that this row sees has no weight
            const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : expf(ml.x - ref), keep = expf(M - ref);
            l = l * keep + warp_sum(f * ml.y);
#pragma unroll
            for (int i = 0; i < C; ++i) o[i] *= keep;
            M = Mn;
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const float *p = row_of(b + k) + lane * C;
                if constexpr (C == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(p));
                    o[0] += fk * x.x, o[1] += fk * x.y, o[2] += fk * x.z, o[3] += fk * x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(p));
                    o[0] += fk * x.x, o[1] += fk * x.y;
                }
            }
        }
    }
    template <typename T>
    SFFN_DEV void write(T *row, int lane) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T *dst = row + lane * C;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (sizeof(T) == 4) dst[i] = o[i] * inv;
            else dst[i] = __float2bfloat16_rn(o[i] * inv);
        }
    }
};

}  // namespace sffn
