// attn_shared.cu -- attention of new tokens over the paged cache for sequences that share
// prefixes (sm_103a).
//
// softmax over a prefix P and a sequence's own positions O splits into two partial results, each with its
// maximum m, sum l and unnormalised row o; they join as M = max(m_P, m_O),
//   out = (e^(m_P - M) o_P + e^(m_O - M) o_O) / (e^(m_P - M) l_P + e^(m_O - M) l_O).
// For the prefix the rows of one product are all the tokens of the group, times the query heads of a key
// head, so its keys are read once for all of them and the tensor cores have full tiles.
//
// The work is one line of items as in attn.cuh: first those of the groups' prefixes, then those of the sequences'
// own positions.  Two kernels can work on it: attn_tc.cuh (tcgen05, row tiles of 128, two an item) and attn_few.cuh
// (few rows, bound by the bytes).  By the rows of the mean group and of the mean sequence
//   few rows a group      attn_few.cuh takes the line;
//   few rows a sequence   attn_tc.cuh takes the prefixes and attn_few.cuh the own positions, at the same time: the
//                         first on as many SMs as its share of the work asks for (its other CTAs leave
//                         at once), the second on the rest, two CTAs an SM;
//   else                  attn_tc.cuh takes the line (large draft trees).
// In fp32 attn_rows.cuh has the place of attn_tc.cuh.
// Each cuts its part of the line evenly over its CTAs (attn_few.cuh: its warps).  An item leaves its result in `home` rows (one set for
// prefixes, one for own positions), the pieces of a cut item in the range's slots; k_shared_join adds both parts of
// each row.  Rows of a sequence without a shared page that no cut touches are written at once.
#include "attn_few.cuh"
#include "attn_rows.cuh"
#include "attn_tc.cuh"

namespace sffn {

namespace {

// Units (of 64 positions) that an item costs by itself.
constexpr int kCostTc = 5, kCostFew = 1, kCostRows = 5;
// Time of a prefix's place in attn_tc.cuh on an SM, in that of a place in attn_few.cuh: kPlaceTc / kPlaceFew.  With 9, 11, 12 and
// 16 / 4: 96 sequences on 24576 shared positions, 64/8 heads, 132, 127, 129, 124 us; 48 on 8192 63, 65, 65, 63; two groups of 32 on
// 16384, 32/8 heads, 64, 64, 66, 74; 64 of two tokens on 32768, 40/8 heads, 163, 172, 178, 206.
constexpr int kPlaceTc = 11, kPlaceFew = 4;
// The same in fp32 (64 sequences on 8192: 464 us with 8 / 4, 407 with 16 / 4, 374 with 32 / 4).
constexpr int kPlaceRows = 32, kPlaceFew32 = 4;
// fp32: rows of the mean sequence that attn_few.cuh takes, and of the mean group beside them.  The other way took: 1 row a
// sequence, 16 a group 337 us (few 118); 4 and 64 174 (73); 8 and 64 80 (40); 14 and 48 34 (45); 19 and 48 27 (28).  Groups of 64
// and 128 rows with prefixes by the row tiles of 64 67 and 204 us (few 73 and 259), of 16 153 (118).
constexpr int kFew32Own = 8, kFew32Pre = 64;
// Places of a range of attn_few.cuh at the least: shorter ones have more pieces to join (4 sequences on 1024 shared positions:
// 18.8 us with 1, 17.9 with 2, 19.3 with 3).
constexpr int kLeastFew = 2;
constexpr int kFewRanges = 2 * few::kWarps;  // warps of attn_few.cuh an SM has

// What a kernel works on.
enum { kLineAll = 0, kLinePrefixes = 1, kLineOwn = 2 };

// An entry of the line: a group's prefix or a sequence's own positions.
struct Part {
    int t0, n;         // first token, tokens
    int k0, ctx, end;  // first position, end of those that every token sees, end of all
    int row;           // row of the page table
    int rows;          // rows (token * G + query head) of a row tile
    int tiles, units;  // items of a key head, units of each item
    int cost, group;
    bool prefix, joint;  // joint: its rows have another part too
    SFFN_DEV int span() const { return units + cost; }
};

// The line, in shared memory.
struct Line {
    long long *scratch;                 // [33]
    long long *pre;                     // [entries + 1]: length before each entry, and of all
    int *seqs, *whole, *tok0, *tok1;    // a group's first sequence (and the last one's end), positions in whole pages
                                        // (-1: it breaks the contract), tokens
    int entries, n_groups;

    static SFFN_HOST_DEV size_t bytes(int n_groups, int n_seq) {
        return align16((size_t)(33 + n_groups + n_seq + 1) * sizeof(long long) + (size_t)(4 * n_groups + 1) * sizeof(int));
    }
    SFFN_DEV Line(const SharedArgs &a, unsigned char *mem) : entries(a.n_groups + a.n_seq), n_groups(a.n_groups) {
        scratch = reinterpret_cast<long long *>(mem);
        pre = scratch + 33;
        seqs = reinterpret_cast<int *>(pre + entries + 1);
        whole = seqs + n_groups + 1;
        tok0 = whole + n_groups;
        tok1 = tok0 + n_groups;
    }
    SFFN_DEV int group_of(int s) const {  // the last group that begins at sequence s or before
        int lo = 0, hi = n_groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seqs[mid] <= s) lo = mid; else hi = mid;
        }
        return lo;
    }
    SFFN_DEV Part prefix_part(const SharedArgs &a, int g) const {
        Part p = {};
        p.prefix = p.joint = true;
        p.group = g;
        p.rows = a.tile_rows[0];
        p.cost = a.cost[0];
        p.ctx = p.end = whole[g];
        p.row = seqs[g];
        p.t0 = tok0[g];
        if (p.end <= 0 || tok1[g] <= p.t0) return p;
        p.n = tok1[g] - p.t0;
        p.tiles = (p.n * a.group + p.rows - 1) / p.rows;
        p.units = (p.end + kTreeUnit - 1) / kTreeUnit;
        return p;
    }
    SFFN_DEV Part own_part(const SharedArgs &a, int s, bool record) const {
        Part p = {};
        p.row = s;
        p.rows = a.tile_rows[1];
        p.cost = a.cost[1];
        const SeqTokens q = seq_tokens(a, s, record);
        const int g = group_of(s), w = whole[g];
        p.group = g;
        if (s < seqs[g] || s >= seqs[g + 1] || w < 0 || a.ctx_lens[s] < w ||
            (q.n > 0 && (q.t0 < tok0[g] || q.t0 + q.n > tok1[g]))) {
            if (record) record_error(a.err, SFFN_ERR_DEVICE);
            return p;
        }
        p.joint = w > 0;
        p.t0 = q.t0;
        p.n = q.n;
        p.k0 = w;
        p.ctx = q.ctx;
        p.end = q.ctx + q.n;
        p.tiles = (q.n * a.group + p.rows - 1) / p.rows;
        p.units = (p.end - w + kTreeUnit - 1) / kTreeUnit;
        return p;
    }
    SFFN_DEV Part part(const SharedArgs &a, int i, bool record) const {
        return i < n_groups ? prefix_part(a, i) : own_part(a, i - n_groups, record);
    }
    SFFN_DEV void build(const SharedArgs &a, bool record) const {
        bool falls = false;
        for (int g = threadIdx.x; g <= n_groups; g += blockDim.x) {
            const int s0 = a.group_seqs[g];
            seqs[g] = s0;
            if (g == n_groups) break;
            const int s1 = a.group_seqs[g + 1], p = a.prefix_lens[g];
            const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.n_seq && p >= 0 && (p >> a.page_shift) <= a.table_width &&
                            p <= kTreeMaxCtx;
            falls |= s1 < s0;
            whole[g] = ok ? (p >> a.page_shift) << a.page_shift : -1;
            tok0[g] = ok ? min(max(a.cu_tokens[s0], 0), a.T) : 0;
            tok1[g] = ok ? min(max(a.cu_tokens[s1], 0), a.T) : 0;
        }
        // Where group_seqs falls, other groups may have the same sequences, and both would write their tokens' rows: none counts.
        if (__syncthreads_or(falls)) {
            for (int g = threadIdx.x; g < n_groups; g += blockDim.x) whole[g] = -1;
            __syncthreads();
        }
        line_prefix(entries, pre, scratch, [&](int i) {
            const Part p = part(a, i, record);
            return (long long)p.tiles * a.n_kv_heads * p.span();
        });
    }
};

// A kernel's stretch of the line and the ranges that it is cut into, a CTA's or a warp's (none is empty).
struct Stretch {
    long long first, length;
    int ranges;
    SFFN_DEV long long cut(int w) const { return first + tree_cut(length, w, ranges); }
};
// which: kLine...; per: ranges an SM has of the kernel that takes it.
SFFN_DEV Stretch stretch_of(const SharedArgs &a, const Line &line, int which, int per) {
    const int sms = a.sms;
    const long long all = line.pre[line.entries], pre = line.pre[line.n_groups], own = all - pre;
    if (which == kLineAll) return Stretch{0, all, tree_ctas((all + a.least - 1) / a.least, sms * per)};
    // SMs of the prefixes by their share of the time; the own positions always have one
    const long long tp = pre * a.place[0], to = own * a.place[1];
    int n = pre == 0 ? 0 : (int)(sms * tp / (tp + to));
    if (pre > 0 && n < 1) n = 1;
    if (own > 0 && n > sms - 1) n = sms - 1;
    if (which == kLinePrefixes) return Stretch{0, pre, tree_ctas(pre, n * per)};
    return Stretch{pre, own, tree_ctas((own + a.least - 1) / a.least, (sms - n) * per)};
}

// A piece of an item.
struct Piece {
    Part p;
    int h, tile;   // key head, row tile
    int un0, un1;  // units
    SFFN_DEV bool whole() const { return un0 == 0 && un1 == p.units; }
};

// A CTA's (or a warp's) walk over its range.
struct Walk {
    long long u, u1;  // next place, end of the range
    long long at;     // where the item of place u (or the one before it, all done) begins
    int entry;        // its entry of the line
    int range;        // which range this is
    Piece c;
    SFFN_DEV void start(const SharedArgs &a, const Line &line, const Stretch &s, int b) {
        range = b;
        u = b < s.ranges ? s.cut(b) : 0;
        u1 = b < s.ranges ? s.cut(b + 1) : 0;
        if (u >= u1) return;
        entry = tree_find(line.pre, line.entries, u);
        c.p = line.part(a, entry, false);
        const int item = (int)((u - line.pre[entry]) / c.p.span());
        at = line.pre[entry] + (long long)item * c.p.span();
        c.h = item / c.p.tiles;
        c.tile = item - c.h * c.p.tiles;
    }
    SFFN_DEV bool next(const SharedArgs &a, const Line &line) {  // c: the next piece with units
        for (;;) {
            if (u >= u1) return false;
            if (u >= at + c.p.span()) {  // on to the next item
                at += c.p.span();
                if (++c.tile == c.p.tiles) c.tile = 0, ++c.h;
                if (c.h == a.n_kv_heads) {
                    c.h = 0;
                    do c.p = line.part(a, ++entry, false); while (c.p.tiles == 0);  // (place u is some entry's)
                }
            }
            const int off = (int)(u - at), end = (int)min((long long)c.p.span(), off + (u1 - u));
            u += end - off;
            c.un0 = max(0, off - c.p.cost);
            c.un1 = max(0, end - c.p.cost);
            if (c.un0 < c.un1) return true;
        }
    }
};

// What the join has to know of a sequence, written by the first kernel that works on the line: of its group's prefix and
// of its own positions, which range of the line has a place, and where that range left its piece.
struct Half {
    const float *part;         // the slots of the pieces
    long long at, length;      // line of the stretch before the entry, all of it
    int ranges, rows_max;
    int t0, rows, tiles, units, cost, pad;
};
struct alignas(16) Entry {
    Half half[2];              // prefix, own positions
    int t0, n, joint, pad;
};
SFFN_DEV Half half_of(const SharedArgs &a, const Line &line, int entry, const Part &p) {
    const int kind = p.prefix ? 0 : 1;
    const Stretch st = stretch_of(a, line, a.split ? kind + 1 : kLineAll, a.per[kind]);
    return Half{a.parts[kind], line.pre[entry] - st.first, st.length, st.ranges, a.rows_max[kind], p.t0, p.rows, p.tiles, p.units, p.cost, 0};
}
SFFN_DEV void write_entries(const SharedArgs &a, const Line &line) {
    for (int s = blockIdx.x + threadIdx.x * gridDim.x; s < a.n_seq; s += gridDim.x * blockDim.x) {
        const Part own = line.own_part(a, s, false);
        Entry e = {};
        e.t0 = own.t0, e.n = own.n, e.joint = own.joint;
        if (own.n > 0) e.half[1] = half_of(a, line, line.n_groups + s, own);
        if (own.n > 0 && own.joint) e.half[0] = half_of(a, line, own.group, line.prefix_part(a, own.group));
        static_cast<Entry *>(a.entries)[s] = e;
        for (int i = 0; i < own.n; ++i) a.seq_of[own.t0 + i] = s;
    }
}

// Rows of whole items: D floats each, then (maximum, sum); prefixes first, own positions after them.
SFFN_HOST_DEV size_t home_floats(int T, int n_heads, int D) {
    const size_t rows = (size_t)T * n_heads;
    return rows * D + ((2 * rows + 3) & ~(size_t)3);
}
SFFN_DEV float *home_row(const SharedArgs &a, bool prefix, size_t row, int D) {
    return a.home + (prefix ? 0 : home_floats(a.T, a.n_heads, D)) + row * D;
}
SFFN_DEV float *home_sums(const SharedArgs &a, bool prefix, size_t row, int D) {
    return a.home + (prefix ? 0 : home_floats(a.T, a.n_heads, D)) + (size_t)a.T * a.n_heads * D + 2 * row;
}
// A CTA's slot for a cut item's piece.
SFFN_DEV float *slot_of(const SharedArgs &a, const Piece &c, int D) {
    const int kind = c.p.prefix ? 0 : 1;
    return a.parts[kind] + tree_slot_floats(a.rows_max[kind], D) * (size_t)(2 * blockIdx.x + (c.un0 > 0 ? 0 : 1));
}

// Which keys of its own sequence a token sees behind the committed ones.
SFFN_DEV uint64_t token_mask(const SharedArgs &a, int token, int i) {
    return a.tree_mask ? a.tree_mask[token] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
}

// ---------------------------------------------------------------------------
// fp32, many rows: attn_rows.cuh
// ---------------------------------------------------------------------------

// (Heads of 64: 224 registers at the most, so that a block of the join, 128 threads of 64, finds room beside a CTA and is there when
// this kernel ends.  5 sequences of 1 to 5 tokens, 16/2 heads: 29.2 us; with 228 registers 30.1.)
template <int D>
__global__ void __maxnreg__(D == 64 ? 224 : 255) k_shared_rows(const SharedArgs a, int which) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rows::Smem<D> &sm = *reinterpret_cast<rows::Smem<D> *>(smem_raw);
    const Line line(a, smem_raw + sizeof(rows::Smem<D>));
    __shared__ uint64_t mask[kTreeMaxTokens];
    griddep_wait();
    griddep_launch_dependents();
    line.build(a, blockIdx.x == 0);
    write_entries(a, line);
    Walk walk;
    walk.start(a, line, stretch_of(a, line, which, a.per[0]), blockIdx.x);
    const int tid = threadIdx.x, G = a.group, ps = 1 << a.page_shift;
    while (walk.next(a, line)) {
        const Piece &c = walk.c;
        const Part &p = c.p;
        const int tokens = p.rows / G, tk0 = c.tile * tokens, nt = min(tokens, p.n - tk0);
        const int32_t *table = a.page_table + (size_t)p.row * a.table_width;
        const int k0 = p.k0 + c.un0 * kTreeUnit, k1 = min(p.end, p.k0 + c.un1 * kTreeUnit);
        __syncthreads();
        if (tid < nt && !p.prefix) mask[tid] = token_mask(a, p.t0 + tk0 + tid, tk0 + tid);
        rows::Acc<D> acc;
        rows::attend<D>(
            sm, acc, nt * G, k0, k1, min(p.ctx, k1), a.scale,
            [&](int r) {
                return static_cast<const float *>(a.q) + (size_t)(p.t0 + tk0 + r / G) * a.q_stride +
                       (size_t)(c.h * G + r % G) * D;
            },
            [&](int j, int which) -> const float * {
                const int pg = table[j >> a.page_shift];
                if (pg < 0 || pg >= a.n_pages) {
                    record_error(a.err, SFFN_ERR_DEVICE);
                    return nullptr;
                }
                return static_cast<const float *>(which ? a.cv : a.ck) +
                       ((((size_t)pg * a.n_kv_heads + c.h) << a.page_shift) + (size_t)(j & (ps - 1))) * D;
            },
            [&](int r, int j) { return (mask[r / G] >> (j - p.ctx)) & 1; });
        const bool whole = c.whole();
        float *slot = slot_of(a, c, D);
        const int col = (tid % rows::Acc<D>::CT) * 4, g = (tid / rows::Acc<D>::CT) * rows::Acc<D>::RPT;
#pragma unroll
        for (int i = 0; i < rows::Acc<D>::RPT; ++i) {
            const int r = g + i;
            if (r >= nt * G) continue;
            const float4 o = acc.o[i];
            const size_t row = (size_t)(p.t0 + tk0 + r / G) * a.n_heads + (size_t)(c.h * G + r % G);
            if (whole && !p.joint) {
                const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * D + col) =
                    make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            } else {
                *reinterpret_cast<float4 *>((whole ? home_row(a, p.prefix, row, D) : slot + (size_t)r * D) + col) = o;
                if (col == 0) {
                    float *ml = whole ? home_sums(a, p.prefix, row, D) : slot + (size_t)a.rows_max[0] * D + 2 * r;
                    ml[0] = sm.m[r];
                    ml[1] = sm.l[r];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// bf16: attn_tc.cuh over the paged cache
// ---------------------------------------------------------------------------

// ONE row tile an item where the rows of a group fill no more; else two, which read each key tile together.
template <int D, bool ONE>
using Cfg = atc::Cfg<D, (D == 128 ? 1 : 2) * (ONE ? 5 : 4), true, ONE, false>;

template <int D, bool ONE>
struct SharedPolicy {
    static constexpr bool kReread = true;
    static constexpr bool kWordMasks = false;
    const SharedArgs &a;
    const Line &line;
    Walk walk;
    int which, G, box;  // box: cache rows of one copy (a page's, 64 at most)

    struct RowInfo {
        uint64_t mask;
    };

    SFFN_DEV SharedPolicy(const SharedArgs &args, const Line &l, int stretch)
        : a(args), line(l), which(stretch), G(args.group), box(min(64, 1 << args.page_shift)) {}

    SFFN_DEV void start() {
        line.build(a, blockIdx.x == 0);
        write_entries(a, line);
        walk.start(a, line, stretch_of(a, line, which, 1), blockIdx.x);
    }
    SFFN_DEV bool next(atc::Work &w) {
        if (!walk.next(a, line)) return false;
        const Piece &c = walk.c;
        const Part &p = c.p;
        const int tokens = p.rows / G, tk0 = c.tile * tokens;
        const int k0 = p.k0 + c.un0 * kTreeUnit, k1 = min(p.end, p.k0 + c.un1 * kTreeUnit);
        const int n = (k1 - k0 + atc::kKeys - 1) / atc::kKeys, TB = 128 / G;
        w.h = c.h;
        w.q_row = p.t0 + tk0;
        w.nt = min(tokens, p.n - tk0);
        w.k0 = k0;
        w.k1 = w.exist = k1;
        w.tiles = n;
        w.n[0] = ONE ? (n + 1) / 2 : n;
        w.n[1] = ONE ? n / 2 : (w.nt > TB ? n : 0);
        w.mask_from[0] = w.mask_from[1] = max(0, min(p.ctx, k1) - k0) / atc::kKeys;
        w.ctx = p.ctx;
        w.seq = p.row;
        w.tok0 = tk0;
        w.whole = c.whole();
        w.slot = 2 * blockIdx.x + (c.un0 > 0 ? 0 : 1);
        w.kind = p.prefix ? 2 : (p.joint ? 1 : 0);
        return true;
    }
    SFFN_DEV int page_of(const atc::Work &w, int key) const {
        return a.page_table[(size_t)w.seq * a.table_width + (key >> a.page_shift)];
    }
    // Row of the cache (head h's) that holds key `key`, on page pg; past the end if that is not one.
    SFFN_DEV long long cache_row(const atc::Work &w, int key, int pg) const {
        if (pg < 0 || pg >= a.n_pages) {
            record_error(a.err, SFFN_ERR_DEVICE);
            return ((long long)a.n_pages * a.n_kv_heads) << a.page_shift;
        }
        return (((long long)pg * a.n_kv_heads + w.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
    }
    // Page of this lane's part of key tile j, a box of `box` rows (16 boxes at most); looked up a
    // tile ahead of its use.
    SFFN_DEV int place(const atc::Work &w, int j, int lane) const {
        const int off = j * atc::kKeys + lane * box;
        return lane * box < atc::kKeys && off < w.k1 - w.k0 ? page_of(w, w.k0 + off) : 0;
    }
    SFFN_DEV void load_kv(const atc::Work &w, int j, int pg, const CUtensorMap *map, unsigned char *dst, uint64_t *bar,
                          int lane, uint64_t pol) const {
        constexpr int H = Cfg<D, ONE>::kHalves;
        const int kb = w.k0 + j * atc::kKeys, left = min(atc::kKeys, w.k1 - kb), boxes = (left + box - 1) / box;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * 128 * H));
        __syncwarp();
        if (lane < boxes) {
            const int row = (int)cache_row(w, kb + lane * box, pg);
            tc::tma_load_4d(dst + lane * box * 128 * H, map, 0, 0, 0, row >> 3, bar, pol);
        }
    }
    SFFN_DEV bool exists(const atc::Work &w, int j, int row) const { return w.k0 + j * atc::kKeys + row < w.exist; }
    SFFN_DEV RowInfo row_info(const atc::Work &w, int tok) const {
        return RowInfo{w.kind == 2 ? 0 : token_mask(a, w.q_row + tok, w.tok0 + tok)};  // (of a prefix every key is seen)
    }
    SFFN_DEV void visible(const atc::Work &w, const RowInfo &r, int j, uint32_t (&vis)[4]) const {
        const int kb = w.k0 + j * atc::kKeys;
        const int all = min(w.ctx, w.k1) - kb, end = w.k1 - kb, d0 = kb - w.ctx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int sh = d0 + 32 * i;  // new token of the word's first key
            uint32_t bits = 0;
            if (sh >= 0 && sh < 64) bits = (uint32_t)(r.mask >> sh);
            else if (sh < 0 && sh > -32) bits = (uint32_t)(r.mask << -sh);
            vis[i] = atc::low_bits(all - 32 * i) | (bits & atc::low_bits(end - 32 * i));
        }
    }
    SFFN_DEV const void *value_row(const atc::Work &w, const RowInfo &r, int key) const {
        if (key >= w.ctx && !((r.mask >> (key - w.ctx)) & 1)) return nullptr;
        const long long row = cache_row(w, key, page_of(w, key));
        if (row >= ((long long)a.n_pages * a.n_kv_heads) << a.page_shift) return nullptr;
        return static_cast<const uint16_t *>(a.cv) + (size_t)row * D;
    }
    SFFN_DEV bool partial(const atc::Work &w) const { return !w.whole || w.kind != 0; }
    SFFN_DEV unsigned char *begin_row(const atc::Work &w, int tok, int head, bool valid, float m, float l,
                                      float &inv) const {
        inv = l == 0.f ? 0.f : 1.f / l;
        if (!valid) return nullptr;
        const size_t row = (size_t)(w.q_row + tok) * a.n_heads + (size_t)w.h * G + head;
        if (!partial(w)) return reinterpret_cast<unsigned char *>(static_cast<uint16_t *>(a.out) + row * D);
        float *o, *sums;
        if (w.whole) {
            o = home_row(a, w.kind == 2, row, D);
            sums = home_sums(a, w.kind == 2, row, D);
        } else {
            // (a kernel's prefixes and own positions share its slots)
            float *slot = a.parts[0] + tree_slot_floats(a.rows_max[0], D) * (size_t)w.slot;
            o = slot + (size_t)(tok * G + head) * D;
            sums = slot + (size_t)a.rows_max[0] * D + 2 * (tok * G + head);
        }
        *reinterpret_cast<float2 *>(sums) = make_float2(m * a.scale, l);
        return reinterpret_cast<unsigned char *>(o);
    }
};

template <int D, bool ONE>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_shared_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const SharedArgs a, int which) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const Line line(a, smem_raw);
    SharedPolicy<D, ONE> policy(a, line, which);
    atc::attention_cta<Cfg<D, ONE>, D>(policy, map_q, map_k, map_v, map_q, a.scale, a.group, a.err,
                                       smem_raw + Line::bytes(a.n_groups, a.n_seq));
}

// ---------------------------------------------------------------------------
// Few rows: attn_few.cuh
// ---------------------------------------------------------------------------

template <typename T, int D>
struct FewPolicy {
    const SharedArgs &a;
    const Line &line;
    Walk walk;

    SFFN_DEV FewPolicy(const SharedArgs &args, const Line &l) : a(args), line(l) {}

    SFFN_DEV bool next(few::Work &w) {
        if (!walk.next(a, line)) return false;
        const Piece &c = walk.c;
        const Part &p = c.p;
        w.q_row = p.t0;
        w.r0 = c.tile * p.rows;
        w.rows = min(p.rows, p.n * a.group - w.r0);
        w.h = c.h;
        w.k0 = p.k0 + c.un0 * kTreeUnit;
        w.k1 = min(p.end, p.k0 + c.un1 * kTreeUnit);
        w.all = min(p.ctx, w.k1);
        w.ctx = p.ctx;
        w.seq = p.row;
        w.whole = c.whole();
        w.slot = 2 * walk.range + (c.un0 > 0 ? 0 : 1);
        w.kind = p.prefix ? 2 : (p.joint ? 1 : 0);
        return true;
    }
    SFFN_DEV int page_of(const few::Work &w, int key) const {
        const int pg = a.page_table[(size_t)w.seq * a.table_width + (key >> a.page_shift)];
        if (pg >= 0 && pg < a.n_pages) return pg;
        record_error(a.err, SFFN_ERR_DEVICE);
        return a.n_pages;
    }
    SFFN_DEV size_t row_of(const few::Work &w, int row) const {  // row of q and out, in heads
        return (size_t)(w.q_row + row / a.group) * a.n_heads + (size_t)w.h * a.group + row % a.group;
    }
    SFFN_DEV const T *query(const few::Work &w, int row) const {
        return static_cast<const T *>(a.q) + (size_t)(w.q_row + row / a.group) * a.q_stride +
               (size_t)(w.h * a.group + row % a.group) * D;
    }
    SFFN_DEV bool sees(const few::Work &w, int row, int key) const {
        const int i = row / a.group;
        return (token_mask(a, w.q_row + i, i) >> (key - w.ctx)) & 1;
    }
    SFFN_DEV T *out_row(const few::Work &w, int row) const {
        return static_cast<T *>(a.out) + row_of(w, row) * D;
    }
    SFFN_DEV bool partial(const few::Work &w) const { return !w.whole || w.kind != 0; }
    SFFN_DEV float *slot(const few::Work &w) const {
        const int kind = w.kind == 2 ? 0 : 1;
        return a.parts[kind] + tree_slot_floats(a.rows_max[kind], D) * (size_t)w.slot;
    }
    SFFN_DEV float *part_row(const few::Work &w, int row, int r) const {
        return w.whole ? home_row(a, w.kind == 2, row_of(w, row), D) : slot(w) + (size_t)r * D;
    }
    SFFN_DEV float2 *part_sums(const few::Work &w, int row, int r) const {
        return reinterpret_cast<float2 *>(w.whole ? home_sums(a, w.kind == 2, row_of(w, row), D)
                                                  : slot(w) + (size_t)a.rows_max[w.kind == 2 ? 0 : 1] * D + 2 * r);
    }
};

// which = kLineOwn: beside the kernel of the prefixes, which has waited for the inputs; this one waits for it
// before it ends, so that what follows follows both.
template <int D, int NT>
__global__ void __launch_bounds__(few::kThreads, 2)
    k_shared_few(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const SharedArgs a,
                 int which) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const Line line(a, smem_raw);
    if (which == kLineAll) griddep_wait();
    griddep_launch_dependents();
    line.build(a, which == kLineAll && blockIdx.x == 0);
    if (which == kLineAll) write_entries(a, line);
    FewPolicy<__nv_bfloat16, D> policy(a, line);
    policy.walk.start(a, line, stretch_of(a, line, which, kFewRanges), blockIdx.x * few::kWarps + (threadIdx.x >> 5));
    few::attention<D, NT>(policy, map_k, map_v, a.page_shift, a.n_kv_heads, a.scale, a.err,
                          smem_raw + Line::bytes(a.n_groups, a.n_seq));
    if (which != kLineAll) griddep_wait();
}

template <int D, int R>
__global__ void __launch_bounds__(few::kThreads, 2) k_shared_few32(const SharedArgs a, int which) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const Line line(a, smem_raw);
    if (which == kLineAll) griddep_wait();
    griddep_launch_dependents();
    line.build(a, which == kLineAll && blockIdx.x == 0);
    if (which == kLineAll) write_entries(a, line);
    FewPolicy<float, D> policy(a, line);
    policy.walk.start(a, line, stretch_of(a, line, which, kFewRanges), blockIdx.x * few::kWarps + (threadIdx.x >> 5));
    few::attention_f32<D, R>(policy, a.ck, a.cv, a.page_shift, a.n_pages, a.n_kv_heads, a.scale, a.err,
                             smem_raw + Line::bytes(a.n_groups, a.n_seq));
    if (which != kLineAll) griddep_wait();
}

// ---------------------------------------------------------------------------
// Join: half a warp a row.  What costs is latency, a row's own chain of loads (6 us) several times over: so the pieces of
// both parts are one list, and the rows of most calls are in flight at once.  6144 rows of 128 in 10 pieces: 13 us alone, 22 MB read.
// ---------------------------------------------------------------------------

constexpr int kJoinWarps = 4;

// The pieces of one part of a row: the first one's row and sums, and the others at equal distances.
struct Pieces {
    const float *row0, *sums0, *row, *sums;
    size_t step;
    int n;
    SFFN_DEV const float *row_at(int k) const { return k == 0 ? row0 : row + step * k; }
    SFFN_DEV const float *sums_at(int k) const { return k == 0 ? sums0 : sums + step * k; }
};
template <int D>
SFFN_DEV Pieces pieces_of(const SharedArgs &a, const Half &e, bool prefix, int t, int head, size_t row) {
    const int at = (t - e.t0) * a.group + head % a.group, tile = at / e.rows, r = at - tile * e.rows;
    const long long u = e.at + ((long long)(head / a.group) * e.tiles + tile) * (e.units + e.cost) + e.cost;
    int w0, w1;  // ranges of its pieces
    if ((u + e.units) * e.ranges < (1ll << 32) && e.length < (1ll << 32)) {  // (tree_owner)
        w0 = (int)(((uint32_t)(u + 1) * (uint32_t)e.ranges - 1u) / (uint32_t)e.length);
        w1 = (int)(((uint32_t)(u + e.units) * (uint32_t)e.ranges - 1u) / (uint32_t)e.length);
    } else {
        w0 = tree_owner(e.length, u, e.ranges);
        w1 = tree_owner(e.length, u + e.units - 1, e.ranges);
    }
    // the first piece lies in its range's second slot (or the whole in its home row), the others in the first
    const size_t sf = tree_slot_floats(e.rows_max, D);
    Pieces p;
    p.n = w1 - w0 + 1;
    p.step = 2 * sf;
    p.row = e.part + p.step * w0 + (size_t)r * D;
    p.sums = e.part + p.step * w0 + (size_t)e.rows_max * D + 2 * r;
    p.row0 = w0 == w1 ? home_row(a, prefix, row, D) : p.row + sf;
    p.sums0 = w0 == w1 ? home_sums(a, prefix, row, D) : p.sums + sf;
    return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 6) k_shared_join(const SharedArgs a) {
    constexpr int C = D / 16;  // columns of a lane
    const int lane = threadIdx.x & 15;
    const long long rows = (long long)a.T * a.n_heads, step = (long long)gridDim.x * kJoinWarps * 2;
    griddep_wait();
    griddep_launch_dependents();
    for (long long i0 = (long long)blockIdx.x * kJoinWarps * 2 + (threadIdx.x >> 5) * 2; i0 < rows; i0 += step) {
        const size_t row = i0 + ((threadIdx.x >> 4) & 1);
        Pieces own = {}, pre = {};
        if ((long long)row < rows) {
            const int t = (int)(row / a.n_heads), head = (int)(row - (size_t)t * a.n_heads), s = a.seq_of[t];
            const Entry &e = static_cast<const Entry *>(a.entries)[s >= 0 && s < a.n_seq ? s : 0];
            // (an old number, of a token that no sequence has, names a sequence without that token)
            if (s >= 0 && s < a.n_seq && t >= e.t0 && t < e.t0 + e.n) {
                own = pieces_of<D>(a, e.half[1], false, t, head, row);
                if (e.joint) pre = pieces_of<D>(a, e.half[0], true, t, head, row);
                else if (own.n == 1) own.n = 0;  // written at once
            }
        }
        const int all = pre.n + own.n, most = __reduce_max_sync(0xffffffffu, all);
        float o[C] = {}, l = 0.f, M = -INFINITY;
        for (int b = 0; b < most; b += 16) {  // 16 pieces at a time
            const int n = min(16, all - b);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) {
                const int k = b + lane;
                ml = __ldcg(reinterpret_cast<const float2 *>(k < pre.n ? pre.sums_at(k) : own.sums_at(k - pre.n)));
            }
            float Mn = ml.x;
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, x));
            Mn = fmaxf(Mn, M);
            const float ref = Mn == -INFINITY ? 0.f : Mn;
            // a piece without a key that this row sees has no weight
            const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : expf(ml.x - ref), keep = expf(M - ref);
            float sum = f * ml.y;
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l = l * keep + sum;
            M = Mn;
#pragma unroll
            for (int x = 0; x < C; ++x) o[x] *= keep;
            const int nk = min(16, most - b);
#pragma unroll 8
            for (int k = 0; k < nk; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k, 16);
                if (k >= n) continue;
                const float *p = (b + k < pre.n ? pre.row_at(b + k) : own.row_at(b + k - pre.n)) + lane * C;
#pragma unroll
                for (int x = 0; x < C; x += 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + x));
                    o[x] += fk * v.x, o[x + 1] += fk * v.y, o[x + 2] += fk * v.z, o[x + 3] += fk * v.w;
                }
            }
        }
        if (all == 0) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T *dst = static_cast<T *>(a.out) + row * D + lane * C;
#pragma unroll
        for (int x = 0; x < C; x += 4) {
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4 *>(dst + x) = make_float4(o[x] * inv, o[x + 1] * inv, o[x + 2] * inv, o[x + 3] * inv);
            else
                *reinterpret_cast<uint2 *>(dst + x) =
                    make_uint2(few::pack_bf16(o[x] * inv, o[x + 1] * inv), few::pack_bf16(o[x + 2] * inv, o[x + 3] * inv));
        }
    }
}

template <typename T, int D>
cudaError_t launch_join(const SharedArgs &a, cudaStream_t s) {
    const long long blocks = ((long long)a.T * a.n_heads + 2 * kJoinWarps - 1) / (2 * kJoinWarps), most = 8LL * a.sms;
    return launch_k(k_shared_join<T, D>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(32 * kJoinWarps), 0, s, a);
}

template <int D, int R>
cudaError_t launch_few32(const SharedArgs &a, int which, cudaStream_t s) {
    const size_t smem = few::Cfg32<D>::kSmem + Line::bytes(a.n_groups, a.n_seq);
    const cudaError_t e = set_max_smem((const void *)k_shared_few32<D, R>, (int)smem);
    return e == cudaSuccess ? launch_k(k_shared_few32<D, R>, dim3(2 * a.sms), dim3(few::kThreads), smem, s, a, which) : e;
}

template <int D>
cudaError_t launch_f32(SharedArgs a, cudaStream_t s) {
    const long long rows = (long long)a.T * a.group, per_group = rows / a.n_groups, per_seq = rows / a.n_seq;
    const bool few_own = per_seq <= kFew32Own, few_pre = few_own && per_group <= kFew32Pre;
    const long long most = few_pre ? per_group : per_seq;
    const int R = most <= 1 ? 1 : (most <= 2 ? 2 : (most <= 4 ? 4 : 8));
    const bool few_kind[2] = {few_pre, few_own};
    for (int k = 0; k < 2; ++k) {
        a.tile_rows[k] = few_kind[k] ? R : rows::kRows / a.group * a.group;
        a.cost[k] = few_kind[k] ? kCostFew : kCostRows;
        a.per[k] = few_kind[k] ? kFewRanges : 1;
        if (few_kind[k]) a.parts[k] = a.part_few, a.rows_max[k] = few::max_rows(D);
    }
    a.split = few_own && !few_pre;
    a.least = few_own ? 1 : kLeastFew;  // (16 sequences of 8 rows on 1024: 26.6 us, with 2 29.9; 5 of 19 rows 29.2 and 29.0)
    a.place[0] = kPlaceRows, a.place[1] = kPlaceFew32;
    cudaError_t e = cudaSuccess;
    if (!few_pre) {
        const size_t smem = sizeof(rows::Smem<D>) + Line::bytes(a.n_groups, a.n_seq);
        e = set_max_smem((const void *)k_shared_rows<D>, (int)smem);
        if (e == cudaSuccess) e = launch_k(k_shared_rows<D>, dim3(a.sms), dim3(rows::kThreads), smem, s, a, a.split ? kLinePrefixes : kLineAll);
    }
    if (e == cudaSuccess && few_own) {
        const int which = a.split ? kLineOwn : kLineAll;
        if (R == 1) e = launch_few32<D, 1>(a, which, s);
        else if (R == 2) e = launch_few32<D, 2>(a, which, s);
        else e = R == 4 ? launch_few32<D, 4>(a, which, s) : launch_few32<D, 8>(a, which, s);
    }
    return e == cudaSuccess ? launch_join<float, D>(a, s) : e;
}

// The cache as [8-row group][column block][row][64]: a box is a page's rows (`most` at most), all columns.
template <int D>
bool cache_maps(const SharedArgs &a, int most, CUtensorMap *mk, CUtensorMap *mv) {
    const int ps = 1 << a.page_shift;
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.n_pages * a.n_kv_heads * ps / 8}, sk[3] = {D * 2, 128, D * 16};
    const uint32_t bk[4] = {64, 8, D / 64, (uint32_t)(ps < most ? ps : most) / 8};
    return make_map_bf16(mk, a.ck, 4, dk, sk, bk) && make_map_bf16(mv, a.cv, 4, dk, sk, bk);
}

template <int D, bool ONE>
cudaError_t launch_tc(const SharedArgs &a, int which, cudaStream_t s) {
    const int G = a.group, TB = 128 / G;
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, sq[2] = {D * 2, (uint64_t)a.q_stride * 2};
    const uint32_t bq[3] = {64, (uint32_t)G, (uint32_t)TB};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !cache_maps<D>(a, 64, &mk, &mv)) return cudaErrorNotSupported;
    const size_t smem = Cfg<D, ONE>::kSmem + Line::bytes(a.n_groups, a.n_seq);
    const cudaError_t e = set_max_smem((const void *)k_shared_tc<D, ONE>, (int)smem);
    return e == cudaSuccess ? launch_k(k_shared_tc<D, ONE>, dim3(a.sms), dim3(atc::kThreads), smem, s, mq, mk, mv, a, which) : e;
}

template <int D, int NT>
cudaError_t launch_few(const SharedArgs &a, int which, cudaStream_t s) {
    CUtensorMap mk, mv;
    if (!cache_maps<D>(a, few::kKeys, &mk, &mv)) return cudaErrorNotSupported;
    const size_t smem = few::Cfg<D>::kSmem + Line::bytes(a.n_groups, a.n_seq);
    const cudaError_t e = set_max_smem((const void *)k_shared_few<D, NT>, (int)smem);
    return e == cudaSuccess ? launch_k(k_shared_few<D, NT>, dim3(2 * a.sms), dim3(few::kThreads), smem, s, mk, mv, a, which) : e;
}

template <int D>
cudaError_t launch_bf16(SharedArgs a, cudaStream_t s) {
    // Rows of the mean group and of the mean sequence.  Few-row warps for own positions: 96 sequences on 24576 shared positions
    // 126 us, all on the tensor cores 153; for a small group's prefix too: 4 sequences of one row on 1024 positions 18.6 us, the prefix on
    // the tensor cores 23.1.  One row tile an item: those 96 sequences' 768 rows 147 us, draft trees of 33 tokens 63 (two: 54); groups of 96 rows
    // on 16384 positions 40.0 us (two, the second empty: 40.9), of 84 on 30000 51.2 (52.6).
    const long long rows = (long long)a.T * a.group, per_group = rows / a.n_groups, per_seq = rows / a.n_seq;
    const bool one = per_group <= 128;
    constexpr int kFewRows = few::max_rows(D);
    const int few_rows = per_seq <= 8 ? 8 : (per_seq <= 16 ? 16 : kFewRows);
    const bool few_own = per_seq <= kFewRows, few_pre = few_own && per_group <= few_rows;
    const int tc_rows = (one ? 1 : 2) * (128 / a.group) * a.group;
    const bool few_kind[2] = {few_pre, few_own};
    for (int k = 0; k < 2; ++k) {
        a.tile_rows[k] = few_kind[k] ? few_rows : tc_rows;
        a.cost[k] = few_kind[k] ? kCostFew : kCostTc;
        a.per[k] = few_kind[k] ? kFewRanges : 1;
        if (few_kind[k]) a.parts[k] = a.part_few, a.rows_max[k] = kFewRows;
    }
    a.split = few_own && !few_pre;
    a.least = kLeastFew;
    a.place[0] = kPlaceTc, a.place[1] = kPlaceFew;
    cudaError_t e = cudaSuccess;
    if (!few_pre) {
        const int which = a.split ? kLinePrefixes : kLineAll;
        e = one ? launch_tc<D, true>(a, which, s) : launch_tc<D, false>(a, which, s);
    }
    if (e == cudaSuccess && few_own) {
        const int which = a.split ? kLineOwn : kLineAll;
        e = few_rows == 8 ? launch_few<D, 1>(a, which, s)
                          : (few_rows == 16 ? launch_few<D, 2>(a, which, s) : launch_few<D, kFewRows / 8>(a, which, s));
    }
    return e == cudaSuccess ? launch_join<__nv_bfloat16, D>(a, s) : e;
}

}  // namespace

SharedPlan make_shared_plan(int T, int n_heads, int n_kv_heads, int head_dim) {
    SharedPlan p = {};
    const int G = n_heads / n_kv_heads;
    p.sms = device_sm_count();
    p.rows_max = (T < 2 * (128 / G) ? T : 2 * (128 / G)) * G;
    size_t o = align_up(kControlBytes);
    p.off_part = o;
    o = align_up(o + sizeof(float) * 2 * (size_t)p.sms * tree_slot_floats(p.rows_max, head_dim));
    p.off_few = o;
    o = align_up(o + sizeof(float) * 2 * kFewRanges * (size_t)p.sms * tree_slot_floats(few::max_rows(head_dim), head_dim));
    p.off_home = o;
    o = align_up(o + sizeof(float) * 2 * home_floats(T, n_heads, head_dim));
    p.off_entries = o;
    o = align_up(o + sizeof(Entry) * kTreeMaxSeq);
    p.off_seq_of = o;
    o = align_up(o + sizeof(int32_t) * (size_t)T);
    p.total = o;
    return p;
}

sffn_status run_attn_shared(const SharedArgs &a, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16) e = head_dim == 128 ? launch_bf16<128>(a, s) : launch_bf16<64>(a, s);
    else e = head_dim == 128 ? launch_f32<128>(a, s) : launch_f32<64>(a, s);
    return e == cudaSuccess ? SFFN_OK : (e == cudaErrorNotSupported ? SFFN_ERR_UNSUPPORTED : SFFN_ERR_CUDA);
}

}  // namespace sffn
