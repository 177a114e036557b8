// attn_pages.cu -- attention of each token over its chosen pages of the paged cache (sm_103a).
//
// An item is a (token, key head, row tile): up to 32 of the G rows (of 128 elements 16; in fp32 8) against the
// n_sel chosen pages, taken one after the other as if they were consecutive positions.  The work of all items is
// one line as in attn.cuh (units of 64 or 16 positions and kItemCost more per item), token by token and head by
// head, cut evenly over the warps; items that lie in one range are finished there, the pieces of a cut item are
// joined by k_pages_join.
#include "attn_few.cuh"
#include "attn_tc.cuh"

namespace sffn {

namespace {

// Units that an item costs by itself (48 tokens of up to 2048 positions, 8 key heads: 55.5 us with 1,
// 57.1 with 2, 57.5 with 4).
constexpr int kItemCost = 1;

// Pages of token t, 0 if it reads none; -1: its row is left as it is (padding, or it breaks the contract).
SFFN_DEV int pages_of(const PagesArgs &a, int t, bool record) {
    const int pos = a.at.positions[t], seq = a.at.seqs[t], n = a.n_sel[t];
    if (pos < 0) return -1;
    if (seq < 0 || seq >= a.at.n_seq || (pos >> a.at.page_shift) >= a.at.table_width || n < 0 || n > a.n_keep) {
        if (record) record_error(a.err, SFFN_ERR_DEVICE);
        return -1;
    }
    return n;
}

SFFN_DEV int pages_units(const PagesArgs &a, int n) {
    return (int)((((long long)n << a.at.page_shift) + (1 << a.unit_shift) - 1) >> a.unit_shift);
}
SFFN_DEV int pages_span(const PagesArgs &a, int n) { return n > 0 ? pages_units(a, n) + kItemCost : 0; }

// A piece of an item.
struct PagesPiece {
    int t, h, n;   // token, key head, its pages
    int tile;      // row tile
    int un0, un1;  // units
    bool whole;
};

// A warp's walk along the line.
struct PagesWalk {
    const PagesArgs &a;
    long long u, u1;  // next place, end of the range
    long long at;     // where the item of place u (or the one before it, all done) begins
    int t, n, span;   // token, its pages, length of its items
    int h, tile;      // the item
    int range;        // which range this is

    SFFN_DEV explicit PagesWalk(const PagesArgs &args) : a(args) {}

    // Every thread of the CTA: its warp's range, and the token at the range's beginning; rows of tokens without pages are zeroed (dealt to the CTAs by token); tells the join which item the beginning cuts.
    template <typename T, int D>
    SFFN_DEV void start() {
        constexpr int RANGES = few::kWarps;
        __shared__ long long s_scan[33], s_at[RANGES];
        __shared__ int s_t[RANGES];
        const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
        const int per = (a.T + nt - 1) / nt, t0 = min(a.T, tid * per), t1 = min(a.T, t0 + per);
        long long sum = 0;
        for (int i = t0; i < t1; ++i) {
            const int k = pages_of(a, i, blockIdx.x == 0);
            sum += pages_span(a, k);
            if (k == 0 && i % gridDim.x == blockIdx.x) {
                uint4 *row = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + (size_t)i * a.n_heads * D);
                for (int e = 0; e < a.n_heads * D * (int)sizeof(T) / 16; ++e) row[e] = make_uint4(0, 0, 0, 0);
            }
        }
        sum *= a.n_kv_heads * a.tiles;
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        long long before = incl - sum, total = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        const int W = tree_ctas(total, gridDim.x * RANGES);
        for (int r = 0; r < RANGES; ++r) {
            const int b = blockIdx.x * RANGES + r;
            if (b >= W) break;
            const long long place = tree_cut(total, b, W);
            if (before <= place && place < before + sum) {  // the token is one of this thread's
                long long begin = before;
                int i = t0;
                for (;; ++i) {
                    const long long len = (long long)pages_span(a, pages_of(a, i, false)) * a.n_kv_heads * a.tiles;
                    if (place < begin + len) break;
                    begin += len;
                }
                s_t[r] = i;
                s_at[r] = begin;
            }
        }
        __syncthreads();
        const int b = blockIdx.x * RANGES + warp;
        range = b;
        u = u1 = 0;
        h = tile = 0;
        int4 cut = make_int4(-1, 0, 0, 0);  // token, its item, first and last range of the cut item
        if (b < W) {
            u = tree_cut(total, b, W);
            u1 = tree_cut(total, b + 1, W);
            t = s_t[warp];
            n = pages_of(a, t, false);
            span = pages_span(a, n);
            const int item = (int)((u - s_at[warp]) / span);
            at = s_at[warp] + (long long)item * span;
            h = item / a.tiles;
            tile = item - h * a.tiles;
            const int w0 = tree_owner(total, at + kItemCost, W), w1 = tree_owner(total, at + span - 1, W);
            if (w0 < b && b <= w1) cut = make_int4(t, item, w0, w1);
        }
        if (lane == 0) a.cuts[b] = cut;
    }

    // The next piece with units (false: none is left).
    SFFN_DEV bool next(PagesPiece &p) {
        for (;;) {
            if (u >= u1) return false;
            if (u >= at + span) {  // on to the next item
                at += span;
                if (++tile == a.tiles) tile = 0, ++h;
                if (h == a.n_kv_heads) {
                    h = 0;
                    do n = pages_of(a, ++t, false); while (n <= 0);  // (place u is some token's)
                    span = pages_span(a, n);
                }
            }
            const int off = (int)(u - at), end = (int)min((long long)span, off + (u1 - u));
            u += end - off;
            p.t = t, p.h = h, p.tile = tile, p.n = n;
            p.un0 = max(0, off - kItemCost), p.un1 = max(0, end - kItemCost);
            p.whole = p.un0 == 0 && end == span;
            if (p.un0 < p.un1) return true;
        }
    }
};

SFFN_DEV const int32_t *list_of(const PagesArgs &a, int t, int h) { return a.sel + ((size_t)t * a.n_kv_heads + h) * a.n_keep; }

// Positions that a token sees in its n pages: of its own page those up to its own.
SFFN_DEV int seen(const PagesArgs &a, int t, int h, int n) {
    const int pos = a.at.positions[t], ps = 1 << a.at.page_shift;
    return (n - 1) * ps + (list_of(a, t, h)[n - 1] == pos >> a.at.page_shift ? (pos & (ps - 1)) + 1 : ps);
}

// Page of the cache behind place `j` of a token's pages; -1 (recorded) if there is none.
SFFN_DEV int cache_page(const PagesArgs &a, int t, int h, int j) {
    const int page = list_of(a, t, h)[j >> a.at.page_shift];
    if (page >= 0 && page <= a.at.positions[t] >> a.at.page_shift) {
        const int pg = a.at.page_table[(size_t)a.at.seqs[t] * a.at.table_width + page];
        if (pg >= 0 && pg < a.at.n_pages) return pg;
    }
    record_error(a.err, SFFN_ERR_DEVICE);
    return -1;
}

// Partial result slots as sffn_attn_tree's, two a range, of a row tile's rows.

// ---------------------------------------------------------------------------
// attn_few.cuh over the paged cache
// ---------------------------------------------------------------------------

template <typename T, int D>
struct PagesPolicy {
    const PagesArgs &a;
    PagesWalk walk;

    SFFN_DEV explicit PagesPolicy(const PagesArgs &args) : a(args), walk(args) {}

    SFFN_DEV bool next(few::Work &w) {
        PagesPiece p;
        if (!walk.next(p)) return false;
        w.q_row = p.t;
        w.h = p.h;
        w.r0 = p.tile * a.row_tile;
        w.rows = min(a.row_tile, a.group - w.r0);
        w.k0 = p.un0 << a.unit_shift;
        w.k1 = w.all = max(w.k0, min(seen(a, p.t, p.h, p.n), p.un1 << a.unit_shift));  // (none behind the last that it sees)
        w.whole = p.whole;
        w.slot = 2 * walk.range + (p.un0 > 0 ? 0 : 1);
        return true;
    }
    SFFN_DEV int page_of(const few::Work &w, int j) const {
        const int pg = cache_page(a, w.q_row, w.h, j);
        return pg < 0 ? a.at.n_pages : pg;
    }
    SFFN_DEV const T *query(const few::Work &w, int row) const {
        return static_cast<const T *>(a.q) + (size_t)w.q_row * a.q_stride + (size_t)(w.h * a.group + row) * D;
    }
    SFFN_DEV bool sees(const few::Work &, int, int) const { return false; }
    SFFN_DEV T *out_row(const few::Work &w, int row) const {
        return static_cast<T *>(a.out) + ((size_t)w.q_row * a.n_heads + (size_t)w.h * a.group + row) * D;
    }
    SFFN_DEV bool partial(const few::Work &w) const { return !w.whole; }
    SFFN_DEV float *part_row(const few::Work &w, int, int r) const {
        return a.part + tree_slot_floats(a.row_tile, D) * (size_t)w.slot + (size_t)r * D;
    }
    SFFN_DEV float2 *part_sums(const few::Work &w, int, int r) const {
        return reinterpret_cast<float2 *>(part_row(w, 0, a.row_tile) + 2 * r);
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(few::kThreads, 2)
    k_pages_few(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const PagesArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    griddep_wait();
    griddep_launch_dependents();
    PagesPolicy<__nv_bfloat16, D> policy(a);
    policy.walk.template start<__nv_bfloat16, D>();
    few::attention<D, NT>(policy, map_k, map_v, a.at.page_shift, a.n_kv_heads, a.scale, a.err, smem_raw);
}

template <int D, int R>
__global__ void __launch_bounds__(few::kThreads, 2) k_pages_few32(const PagesArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    griddep_wait();
    griddep_launch_dependents();
    PagesPolicy<float, D> policy(a);
    policy.walk.template start<float, D>();
    few::attention_f32<D, R>(policy, a.ck, a.cv, a.at.page_shift, a.at.n_pages, a.n_kv_heads, a.scale, a.err, smem_raw);
}

// ---------------------------------------------------------------------------
// bf16, many tokens of a sequence: attn_tc.cuh over the union of their pages
//
// Two row tiles have 2 TB = 2 (128 / G) consecutive tokens; a run of them that are of one sequence is an item (for each key
// head).  Neighbouring tokens choose mostly the same pages, so the item reads the union of their pages once, and a row's mask
// leaves out the pages that its token has not chosen: with 36 tokens of 48 of 480 pages each, about 120 pages are read
// where the tokens one by one read 1728.  k_pages_runs finds the runs and writes each token's pages, and each run's, as a bit
// set; the loading warp goes through a run's set and leaves each key tile's pages and the tokens that have them
// in a small ring.  That and the loads (64 KB a key tile) take the loading warp about 3000 cycles, and two row tiles' products
// as long (one row tile an item: 160 us for pieces of 1045 tokens).  Those, of 28/4 heads of 128, 48 pages of 32 each, take 151 us: 23 GFLOP
// for the pairs that tokens see, 28 % of an SM's tensor cycles over the whole unions, 29 MB of DRAM (one by one: 232 us).
// ---------------------------------------------------------------------------

constexpr int kUnionWidth = 4096;               // pages of a table row that a bit set holds
constexpr int kUnionWords = kUnionWidth / 32;

constexpr int kRunThreads = 256;  // tokens of two row tiles at the most

__global__ void __launch_bounds__(kRunThreads) k_pages_runs(const PagesArgs a, int tokens, int row_bytes) {
    constexpr int kWarps = kRunThreads / 32;
    __shared__ uint32_t s_set[kUnionWords], s_row[kWarps][kUnionWords];
    __shared__ int s_seq[kRunThreads], s_n[kRunThreads], s_run[kRunThreads], s_sum[kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0), h = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    if (tid < nt) {
        s_n[tid] = pages_of(a, t0 + tid, h == 0);
        s_seq[tid] = a.at.seqs[t0 + tid];
    }
    __syncthreads();
    if (tid < nt) {
        int len = 0;  // tokens of the run that begins here (0: none does)
        if (s_n[tid] > 0 && (tid == 0 || s_n[tid - 1] <= 0 || s_seq[tid - 1] != s_seq[tid]))
            for (len = 1; tid + len < nt && s_n[tid + len] > 0 && s_seq[tid + len] == s_seq[tid];) ++len;
        s_run[tid] = len;
        if (h == 0) a.runs[t0 + tid] = len;
        if (s_n[tid] == 0) {  // a token without pages has zeros
            uint4 *row = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(a.out) +
                                                   ((size_t)(t0 + tid) * a.n_heads + (size_t)h * a.group) * row_bytes);
            for (int e = 0; e < a.group * row_bytes / 16; ++e) row[e] = make_uint4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    const int words = (a.at.table_width + 31) / 32;
    for (int i = 0; i < nt; ++i) {
        const int len = s_run[i];
        if (len == 0) continue;
        for (int x = tid; x < words; x += kRunThreads) s_set[x] = 0;
        __syncthreads();
        for (int j = i + warp; j < i + len; j += kWarps) {  // a warp a token
            uint32_t *row = s_row[warp];
            for (int x = lane; x < words; x += 32) row[x] = 0;
            __syncwarp();
            const int32_t *list = list_of(a, t0 + j, h);
            const int mine = a.at.positions[t0 + j] >> a.at.page_shift;
            for (int k = lane; k < s_n[j]; k += 32) {
                const int page = list[k];
                if (page < 0 || page > mine) record_error(a.err, SFFN_ERR_DEVICE);
                else atomicOr(&row[page >> 5], 1u << (page & 31));
            }
            __syncwarp();
            uint32_t *dst = a.bits + ((size_t)(t0 + j) * a.n_kv_heads + h) * kUnionWords;
            for (int x = lane; x < words; x += 32) {
                dst[x] = row[x];
                if (row[x]) atomicOr(&s_set[x], row[x]);
            }
            __syncwarp();
        }
        __syncthreads();
        const size_t at = (size_t)(t0 + i) * a.n_kv_heads + h;
        int n = 0;
        for (int x = tid; x < words; x += kRunThreads) {
            a.union_bits[at * kUnionWords + x] = s_set[x];
            n += __popc(s_set[x]);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) s_sum[warp] = n;
        __syncthreads();
        if (tid == 0) {
            int all = 0;
            for (int x = 0; x < kWarps; ++x) all += s_sum[x];
            a.unions[at] = all;
        }
        __syncthreads();
    }
}

template <int D>
using TileCfg = atc::Cfg<D, D == 128 ? 4 : 8, true, false, false>;

// A key tile's pages (16 at most) and, for each token of the run, which of them it has.
struct TilePages {
    int page[16];            // -1: none
    uint16_t has[kRunThreads];
    int own;                 // whether a page may be some token's own, which it sees in part
};
constexpr int kTileRing = 16;  // key tiles that the loading warp may be ahead of the last softmax warp, and more
struct UnionSmem {
    TilePages ring[kTileRing];
    uint16_t pages[1024];  // of a run, in order: 32 words of its bit set at a time
};

// Q: tokens of two row tiles / 32, rounded up.
template <int D, int Q>
struct UnionPolicy {
    static constexpr bool kReread = true;
    static constexpr bool kWordMasks = true;
    const PagesArgs &a;
    TilePages *ring;
    uint16_t *pages;
    int G, TB, box, ps;   // box: cache rows of one copy (a page's, 64 at most)
    int piece, pieces;    // this CTA's next (pair of row tiles, key head), all of them
    int t, t1, h, base;   // next token of the row tiles, their end, key head; key tiles so far
    // the loading warp's place in a run's bit set (words, the stretch of 32 that is listed, how many are listed, the next of
    // them), and of tokens lane + 32 q the bit set's words `word` and the one after it
    int words, stretch, listed, upto, word;
    const uint32_t *set, *bits[Q];
    uint32_t now[Q], after[Q], got[Q];  // (got: which of the tile's pages the tokens have)
    bool has[2];  // whether this lane's box of the tile before the last one placed, and of that one, has a page
    int loaded, boxes, group;  // the tile whose boxes are known, how many, where this lane's lies

    struct RowInfo {
        int tok, page, off;  // token of the run; its own page and place in it
    };

    SFFN_DEV UnionPolicy(const PagesArgs &args, UnionSmem &sm)
        : a(args), ring(sm.ring), pages(sm.pages), G(args.group), TB(128 / args.group), box(min(64, 1 << args.at.page_shift)), ps(1 << args.at.page_shift) {}

    SFFN_DEV void start() {
        piece = blockIdx.x;
        pieces = (a.T + 2 * TB - 1) / (2 * TB) * a.n_kv_heads;
        t = t1 = base = 0;
        loaded = -1;
    }
    // The last tokens, whose contexts are the longest, first; forwards and backwards in turn.
    SFFN_DEV bool next_tile() {
        const int W = gridDim.x, round = piece / W, p = round & 1 ? 2 * round * W + W - 1 - piece : piece;
        if (p >= pieces) return false;  // (true of the last round alone)
        piece += W;
        h = p % a.n_kv_heads;
        t = (pieces / a.n_kv_heads - 1 - p / a.n_kv_heads) * 2 * TB;
        t1 = min(a.T, t + 2 * TB);
        return true;
    }
    // Lists the next pages of the run's set.
    SFFN_DEV void list_more(int lane) {
        do {
            uint32_t v = ++stretch * 32 + lane < words ? __ldg(set + stretch * 32 + lane) : 0u;
            const int n = __popc(v), end = warp_incl_scan(n, lane);
            listed = __shfl_sync(0xffffffffu, end, 31);
            __syncwarp();
            for (int i = end - n; v; v &= v - 1) pages[i++] = (uint16_t)((stretch * 32 + lane) * 32 + __ffs(v) - 1);
            __syncwarp();
        } while (listed == 0 && (stretch + 1) * 32 < words);
        upto = 0;
    }
    SFFN_DEV uint32_t bits_of(int q, int x) const { return bits[q] && x < words ? __ldg(bits[q] + x) : 0u; }
    SFFN_DEV bool next(atc::Work &w) {
        const int lane = threadIdx.x & 31;
        for (;;) {
            if (t >= t1 && !next_tile()) return false;
            const uint32_t heads = __ballot_sync(0xffffffffu, t + lane < t1 && a.runs[t + lane] > 0);
            if (!heads) {
                t += 32;
                continue;
            }
            t += __ffs(heads) - 1;
            break;
        }
        const int n = a.runs[t];
        const size_t head = (size_t)t * a.n_kv_heads + h;
        const int all = a.unions[head];
        set = a.union_bits + head * kUnionWords;
        words = (a.at.table_width + 31) / 32;
        stretch = word = -1;
        listed = upto = 0;
        int last = 0, first = 0x7fffffff, most = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int i = lane + 32 * q;
            bits[q] = nullptr;
            if (i < n) {
                bits[q] = a.bits + (head + (size_t)i * a.n_kv_heads) * kUnionWords;
                last = max(last, a.at.positions[t + i]);
                first = min(first, a.at.positions[t + i]);
                most = max(most, a.n_sel[t + i]);
            }
            now[q] = 0;
            after[q] = bits_of(q, 0);
        }
        w.h = h;
        w.q_row = t;
        w.nt = n;
        w.k0 = 0;
        w.k1 = __reduce_max_sync(0xffffffffu, most) * ps;  // (places of a token's own list: value_row)
        w.ctx = __reduce_max_sync(0xffffffffu, last);
        w.i0 = __reduce_min_sync(0xffffffffu, first) >> a.at.page_shift;
        w.seq = a.at.seqs[t];
        // (entries that are none of a table's pages are not counted: a run may have no page at all)
        w.tiles = (int)max(1ll, ((long long)all * ps + atc::kKeys - 1) / atc::kKeys);
        w.n[0] = w.tiles;
        w.n[1] = n > TB ? w.tiles : 0;
        w.mask_from[0] = w.mask_from[1] = 0;
        w.whole = true;
        w.base = base;
        base += w.tiles;
        t += n;
        return true;
    }
    // The pages of key tile j, and who has them; the table's entry of this lane's box.  (The loading warp has about as long
    // for a tile as its products take, 1600 cycles: four pages at a time, so that their chains of loads and
    // votes overlap.)
    SFFN_DEV int place(const atc::Work &w, int j, int lane) {
        TilePages &info = ring[(w.base + j) % kTileRing];
        const int n = ps < atc::kKeys ? atc::kKeys >> a.at.page_shift : 1;
        int mine = -1;  // this lane's box's page
        if (ps > atc::kKeys && (j * atc::kKeys & (ps - 1)) != 0) {  // the page goes on
            mine = ring[(w.base + j - 1) % kTileRing].page[0];
            if (lane == 0) info.page[0] = mine;
        } else {
            const int my_x = (lane * box) >> a.at.page_shift;
#pragma unroll
            for (int q = 0; q < Q; ++q) got[q] = 0;
            for (int x0 = 0; x0 < n; x0 += 4) {
                if (upto + 4 > listed) {  // near the end of what is listed: one at a time
                    for (int x = x0; x < min(n, x0 + 4); ++x) {
                        if (upto >= listed && (stretch + 1) * 32 < words) list_more(lane);
                        const int page = upto < listed ? pages[upto] : -1;
                        ++upto;
                        note(x, page);
                        if (lane == 0) info.page[x] = page;
                        if (x == my_x) mine = page;
                    }
                    continue;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (x0 + x >= n) break;
                    const int page = pages[upto + x];
                    note(x0 + x, page);
                    if (lane == 0) info.page[x0 + x] = page;
                    if (x0 + x == my_x) mine = page;
                }
                upto += min(4, n - x0);
            }
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) info.has[lane + 32 * q] = (uint16_t)got[q];
        // (pages ascend: a box that lies at or behind the first token's own page)
        const int own = __any_sync(0xffffffffu, lane * box < atc::kKeys && mine >= w.i0);
        if (lane == 0) info.own = own;
        __syncwarp();
        has[0] = has[1];
        has[1] = lane * box < atc::kKeys && mine >= 0;
        // the table's entry as it is: looked at when the tile is loaded, not before it has come
        return has[1] ? a.at.page_table[(size_t)w.seq * a.at.table_width + mine] : 0;
    }
    SFFN_DEV void to_word(int x) {
        const bool near = x == word + 1;
        word = x;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            now[q] = near ? after[q] : bits_of(q, x);
            after[q] = bits_of(q, x + 1);
        }
    }
    SFFN_DEV void note(int x, int page) {  // page (-1: none) is the tile's x-th
        if (page < 0) return;
        if (page >> 5 != word) to_word(page >> 5);
#pragma unroll
        for (int q = 0; q < Q; ++q) got[q] |= ((now[q] >> (page & 31)) & 1) << x;
    }
    SFFN_DEV void load_kv(const atc::Work &w, int j, int pg, const CUtensorMap *map, unsigned char *dst, uint64_t *bar,
                          int lane, uint64_t pol) {
        constexpr int H = TileCfg<D>::kHalves;
        if (loaded != w.base + j) {  // K; V of the tile follows
            loaded = w.base + j;
            // (the boxes of a tile that has them are its first; the next tile, if there is one, has been placed already)
            const bool mine = j + 1 < w.tiles ? has[0] : has[1], there = pg >= 0 && pg < a.at.n_pages;
            boxes = __popc(__ballot_sync(0xffffffffu, mine));
            if (!there && mine) record_error(a.err, SFFN_ERR_DEVICE);
            // 8-row group of the cache, past its end if there is no such page
            group = (((there ? pg : a.at.n_pages) * a.n_kv_heads + (there ? w.h : 0)) << (a.at.page_shift - 3)) +
                    (((j * atc::kKeys + lane * box) & (ps - 1)) >> 3);
        }
        const uint32_t to = smem_u32(dst), at = smem_u32(bar);
        tc::mbar_expect_tx_warp(at, (uint32_t)(boxes * box * 128 * H));
        for (int b = 0; b < boxes; ++b)
            tc::tma_load_rows_warp(to + b * box * 128 * H, map, __shfl_sync(0xffffffffu, group, b), at, pol);
    }
    SFFN_DEV bool exists(const atc::Work &w, int j, int row) const {
        const TilePages &info = ring[(w.base + j) % kTileRing];
        const int page = info.page[row >> a.at.page_shift];
        return page >= 0 && (long long)page * ps + ((j * atc::kKeys + row) & (ps - 1)) <= w.ctx;
    }
    SFFN_DEV RowInfo row_info(const atc::Work &w, int tok) const {
        const int pos = a.at.positions[w.q_row + tok];
        return RowInfo{tok, pos >> a.at.page_shift, pos & (ps - 1)};
    }
    SFFN_DEV void visible(const atc::Work &w, const RowInfo &r, int j, uint32_t (&vis)[4]) const {
        const TilePages &info = ring[(w.base + j) % kTileRing];
        const uint32_t has = info.has[r.tok];  // which of the tile's pages
        if (!info.own) {  // all of a page or nothing
            if (ps >= 32) {
#pragma unroll
                for (int q = 0; q < 4; ++q) vis[q] = 0u - ((has >> (32 * q >> a.at.page_shift)) & 1);
            } else {
                const uint32_t one = atc::low_bits(ps);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    vis[q] = 0;
                    for (int x = 0; x < 32 >> a.at.page_shift; ++x)
                        vis[q] |= (0u - ((has >> ((32 * q >> a.at.page_shift) + x)) & 1) & one) << (x << a.at.page_shift);
                }
            }
            return;
        }
        // keys of the tile's page x, from place `from` of the page on, that the row sees (32 or more: all)
        auto seen = [&](int x, int from) {
            return !((has >> x) & 1) ? 0 : (info.page[x] == r.page ? max(0, r.off + 1 - from) : 32);
        };
        if (ps >= 32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) vis[q] = atc::low_bits(seen(32 * q >> a.at.page_shift, (j * atc::kKeys + 32 * q) & (ps - 1)));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                vis[q] = 0;
                for (int x = 0; x < 32 >> a.at.page_shift; ++x)
                    vis[q] |= (atc::low_bits(seen((32 * q >> a.at.page_shift) + x, 0)) & atc::low_bits(ps)) << (x << a.at.page_shift);
            }
        }
    }
    SFFN_DEV const void *value_row(const atc::Work &w, const RowInfo &r, int key) const {
        const int tk = w.q_row + r.tok, k = key >> a.at.page_shift;
        if (k >= a.n_sel[tk]) return nullptr;
        const int page = list_of(a, tk, w.h)[k];
        if (page < 0 || page > r.page || (page == r.page && (key & (ps - 1)) > r.off)) return nullptr;
        const int pg = a.at.page_table[(size_t)w.seq * a.at.table_width + page];
        if (pg < 0 || pg >= a.at.n_pages) return nullptr;
        return static_cast<const uint16_t *>(a.cv) +
               ((((size_t)pg * a.n_kv_heads + w.h) << a.at.page_shift) + (key & (ps - 1))) * D;
    }
    SFFN_DEV bool partial(const atc::Work &) const { return false; }
    SFFN_DEV unsigned char *begin_row(const atc::Work &w, int tok, int head, bool valid, float, float l, float &inv) const {
        inv = l == 0.f ? 0.f : 1.f / l;
        if (!valid) return nullptr;
        return reinterpret_cast<unsigned char *>(static_cast<uint16_t *>(a.out) +
                                                 ((size_t)(w.q_row + tok) * a.n_heads + (size_t)w.h * G + head) * D);
    }
};

template <int D, int Q>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_pages_union(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const PagesArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ UnionSmem sm;
    UnionPolicy<D, Q> policy(a, sm);
    atc::attention_cta<TileCfg<D>, D>(policy, map_q, map_k, map_v, map_q, a.scale, a.group, a.err, smem_raw);
}

// ---------------------------------------------------------------------------
// Join: `parts` blocks for each place between two ranges; those of all the places that cut an
// item share its rows, a warp a row.
// ---------------------------------------------------------------------------

constexpr int kJoinWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_pages_join(const PagesArgs a, int parts) {
    const int lane = threadIdx.x & 31, w = 1 + blockIdx.x / parts, part = blockIdx.x % parts;
    griddep_wait();
    griddep_launch_dependents();
    const int4 cut = __ldcg(a.cuts + w);
    if (cut.x < 0) return;
    const int w0 = cut.z, w1 = cut.w, blocks = (w1 - w0) * parts, b = (w - w0 - 1) * parts + part;
    const size_t sf = tree_slot_floats(a.row_tile, D);
    const int h = cut.y / a.tiles, r0 = cut.y % a.tiles * a.row_tile, rows = min(a.row_tile, a.group - r0);
    auto slot = [&](int w) { return a.part + sf * (size_t)(2 * w + (w == w0 ? 1 : 0)); };
    for (int r = b * kJoinWarps + (threadIdx.x >> 5); r < rows; r += blocks * kJoinWarps) {
        JoinedRow<D / 32> j;
        j.add(w0, w1, lane, [&](int w) { return slot(w) + (size_t)a.row_tile * D + 2 * r; },
              [&](int w) { return slot(w) + (size_t)r * D; });
        j.write(static_cast<T *>(a.out) + ((size_t)cut.x * a.n_heads + (size_t)h * a.group + r0 + r) * D, lane);
    }
}

template <typename T, int D>
cudaError_t launch_join(const PagesArgs &a, int ranges, cudaStream_t s) {
    if (ranges < 2) return cudaSuccess;  // one: nothing is cut
    const int parts = (a.row_tile + 2 * kJoinWarps - 1) / (2 * kJoinWarps);
    return launch_k(k_pages_join<T, D>, dim3((unsigned)((ranges - 1) * parts)), dim3(32 * kJoinWarps), 0, s, a, parts);
}

template <int D, int R>
cudaError_t launch_few32(PagesArgs a, int grid, cudaStream_t s) {
    a.row_tile = a.group < R ? a.group : R;
    a.tiles = (a.group + a.row_tile - 1) / a.row_tile;
    // Units of 16 positions balance the warps better where there are more of 64 than warps (27 tokens of 512 positions, 64/8
    // heads: 26.6 us, with 64 36.5), and give a short list to more warps (4 tokens of 320: 13.6 and 16.6); between the two they
    // only make more pieces to join (5 tokens of 576: 21.7 and 17.5).
    const long long list = (long long)a.n_keep << a.at.page_shift;
    const long long units = (list + 63) / 64 * a.T * a.n_kv_heads * a.tiles;
    a.unit_shift = list <= 320 || units >= 2LL * grid * few::kWarps ? 4 : 6;
    constexpr int smem = few::Cfg32<D>::kSmem;
    cudaError_t e = set_max_smem((const void *)k_pages_few32<D, R>, smem);
    if (e == cudaSuccess) e = launch_k(k_pages_few32<D, R>, dim3(2 * grid), dim3(few::kThreads), smem, s, a);
    return e == cudaSuccess ? launch_join<float, D>(a, 2 * grid * few::kWarps, s) : e;
}

template <int D>
cudaError_t launch_f32(const PagesArgs &a, int grid, cudaStream_t s) {
    if (a.group == 1) return launch_few32<D, 1>(a, grid, s);
    if (a.group == 2) return launch_few32<D, 2>(a, grid, s);
    return a.group <= 4 ? launch_few32<D, 4>(a, grid, s) : launch_few32<D, 8>(a, grid, s);
}

template <int D, int NT>
cudaError_t launch_few(PagesArgs a, int grid, cudaStream_t s) {
    a.unit_shift = 6;
    const int ps = 1 << a.at.page_shift;
    a.row_tile = a.group < 8 * NT ? a.group : 8 * NT;
    a.tiles = (a.group + a.row_tile - 1) / a.row_tile;
    CUtensorMap mk, mv;
    // the cache as [8-row group][column block][row][64]: a box is 16 rows of a page, or the page, and all columns
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.at.n_pages * a.n_kv_heads * ps / 8}, sk[3] = {D * 2, 128, D * 16};
    const uint32_t bk[4] = {64, 8, D / 64, (uint32_t)(ps < few::kKeys ? ps : few::kKeys) / 8};
    if (!make_map_bf16(&mk, a.ck, 4, dk, sk, bk) || !make_map_bf16(&mv, a.cv, 4, dk, sk, bk)) return cudaErrorNotSupported;
    constexpr int smem = few::Cfg<D>::kSmem;
    cudaError_t e = set_max_smem((const void *)k_pages_few<D, NT>, smem);
    if (e == cudaSuccess) e = launch_k(k_pages_few<D, NT>, dim3(2 * grid), dim3(few::kThreads), smem, s, mk, mv, a);
    return e == cudaSuccess ? launch_join<__nv_bfloat16, D>(a, 2 * grid * few::kWarps, s) : e;
}

template <int D, int Q>
cudaError_t launch_union(const PagesArgs &a, int grid, cudaStream_t s) {
    const int G = a.group, TB = 128 / G, ps = 1 << a.at.page_shift;
    const unsigned tiles = (unsigned)((a.T + 2 * TB - 1) / (2 * TB));
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, sq[2] = {D * 2, (uint64_t)a.q_stride * 2};
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.at.n_pages * a.n_kv_heads * ps / 8}, sk[3] = {D * 2, 128, D * 16};
    const uint32_t bq[3] = {64, (uint32_t)G, (uint32_t)TB}, bk[4] = {64, 8, D / 64, (uint32_t)(ps < 64 ? ps : 64) / 8};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !make_map_bf16(&mk, a.ck, 4, dk, sk, bk) ||
        !make_map_bf16(&mv, a.cv, 4, dk, sk, bk))
        return cudaErrorNotSupported;
    cudaError_t e = launch_k(k_pages_runs, dim3(tiles, (unsigned)a.n_kv_heads), dim3(kRunThreads), 0, s, a, 2 * TB, D * 2);
    if (e == cudaSuccess) e = set_max_smem((const void *)k_pages_union<D, Q>, TileCfg<D>::kSmem);
    return e == cudaSuccess ? launch_k(k_pages_union<D, Q>, dim3(grid), dim3(atc::kThreads), TileCfg<D>::kSmem, s, mq, mk, mv, a) : e;
}

template <int D>
cudaError_t launch_bf16(const PagesArgs &a, int grid, cudaStream_t s) {
    // The union where the mean sequence has half a row tile of rows or more and the lists may hold 3 million positions: by
    // themselves the tokens take about 35 us a million, items 75 to 130 us for the first 152 of them.  Chunks of 28/4 heads, 1536
    // positions a token: 256 tokens 68 us by themselves and 102 by unions, 512 119 and 110, 2048 427 and 234; 32/8 heads,
    // 2048 positions: 256 tokens 146 and 125, 2048 1067 and 285; 33 sequences of 13 tokens, 1760 positions: 40 and 191.
    if ((long long)a.T * a.group >= 64LL * a.at.n_seq && a.at.table_width <= kUnionWidth &&
        (((long long)a.T * a.n_kv_heads * a.n_keep) << a.at.page_shift) >= 3000000)
        return a.group >= 4 ? launch_union<D, 2>(a, grid, s) : launch_union<D, 8>(a, grid, s);
    // (row tiles of as few rows as the group needs: the products of 8 more cost as much as the first)
    if (a.group <= 8) return launch_few<D, 1>(a, grid, s);
    return a.group <= 16 ? launch_few<D, 2>(a, grid, s) : launch_few<D, few::max_rows(D) / 8>(a, grid, s);
}

}  // namespace

PagesPlan make_pages_plan(int T, int n_heads, int n_kv_heads, int head_dim) {
    PagesPlan p = {};
    p.grid = device_sm_count();
    size_t o = align_up(kControlBytes);
    p.off_cuts = o;
    const size_t ranges = 2 * few::kWarps * (size_t)p.grid;
    o = align_up(o + sizeof(int4) * ranges);
    p.off_part = o;
    const int G = n_heads / n_kv_heads, most = few::max_rows(head_dim);
    o = align_up(o + sizeof(float) * 2 * ranges * tree_slot_floats(G < most ? G : most, head_dim));
    p.off_runs = o;
    o = align_up(o + sizeof(int32_t) * (size_t)T);
    p.off_unions = o;
    o = align_up(o + sizeof(int32_t) * (size_t)T * n_kv_heads);
    p.off_bits = o;
    p.union_words = (size_t)T * n_kv_heads * kUnionWords;
    o = align_up(o + sizeof(uint32_t) * 2 * p.union_words);
    p.total = o;
    return p;
}

sffn_status run_attn_pages(const PagesArgs &a, const PagesPlan &p, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16) e = head_dim == 128 ? launch_bf16<128>(a, p.grid, s) : launch_bf16<64>(a, p.grid, s);
    else e = head_dim == 128 ? launch_f32<128>(a, p.grid, s) : launch_f32<64>(a, p.grid, s);
    return e == cudaSuccess ? SFFN_OK : (e == cudaErrorNotSupported ? SFFN_ERR_UNSUPPORTED : SFFN_ERR_CUDA);
}

}  // namespace sffn
