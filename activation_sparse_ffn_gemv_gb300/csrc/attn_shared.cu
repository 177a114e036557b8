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
// own positions, cut evenly over the CTAs.  An item leaves its result in `home` rows (one set for prefixes, one for
// own positions), the pieces of a cut item in the CTA's slots; k_shared_join adds both parts of each
// row.  Rows of a sequence without a shared page that no cut touches are written at once.
#include "attn_rows.cuh"
#include "attn_tc.cuh"

namespace sffn {

namespace {

// An entry of the line: a group's prefix or a sequence's own positions.
struct Part {
    int t0, n;         // first token, tokens
    int k0, ctx, end;  // first position, end of those that every token sees, end of all
    int row;           // row of the page table
    int tiles, units;  // row tiles, units of each item
    bool prefix, joint;  // joint: its rows have another part too
    SFFN_DEV int span() const { return units + kTreeItemCost; }
};

// The groups' sequences and prefixes, in shared memory.
struct Groups {
    int seqs[kSharedMaxGroups + 1];
    int whole[kSharedMaxGroups];  // positions in whole pages; -1: the group breaks the contract
    int t0[kSharedMaxGroups], t1[kSharedMaxGroups];  // its tokens

    SFFN_DEV void load(const SharedArgs &a) {
        for (int g = threadIdx.x; g <= a.n_groups; g += blockDim.x) {
            const int s0 = a.group_seqs[g];
            seqs[g] = s0;
            if (g == a.n_groups) break;
            const int s1 = a.group_seqs[g + 1], p = a.prefix_lens[g];
            const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.n_seq && p >= 0 && (p >> a.page_shift) <= a.table_width &&
                            p <= kTreeMaxCtx;
            whole[g] = ok ? (p >> a.page_shift) << a.page_shift : -1;
            t0[g] = ok ? min(max(a.cu_tokens[s0], 0), a.T) : 0;
            t1[g] = ok ? min(max(a.cu_tokens[s1], 0), a.T) : 0;
        }
        __syncthreads();
    }
    SFFN_DEV int of(int s, int n_groups) const {  // the last group that begins at sequence s or before
        int lo = 0, hi = n_groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seqs[mid] <= s) lo = mid; else hi = mid;
        }
        return lo;
    }
};

SFFN_DEV Part prefix_part(const SharedArgs &a, const Groups &gr, int g) {
    Part p = {};
    p.prefix = p.joint = true;
    p.ctx = p.end = gr.whole[g];
    p.row = gr.seqs[g];
    p.t0 = gr.t0[g];
    if (p.end <= 0 || gr.t1[g] <= p.t0) return p;
    p.n = gr.t1[g] - p.t0;
    p.tiles = (p.n + a.tile_tokens - 1) / a.tile_tokens;
    p.units = (p.end + kTreeUnit - 1) / kTreeUnit;
    return p;
}

SFFN_DEV Part own_part(const SharedArgs &a, const Groups &gr, int s, bool record) {
    Part p = {};
    p.row = s;
    const TreeSeq q = tree_seq(a, s, record);
    const int g = gr.of(s, a.n_groups), whole = gr.whole[g];
    if (s < gr.seqs[g] || s >= gr.seqs[g + 1] || whole < 0 || a.ctx_lens[s] < whole ||
        (q.n > 0 && (q.t0 < gr.t0[g] || q.t0 + q.n > gr.t1[g]))) {
        if (record) record_error(a.err, SFFN_ERR_DEVICE);
        return p;
    }
    p.joint = whole > 0;
    p.t0 = q.t0;
    p.n = q.n;
    p.k0 = whole;
    p.ctx = q.ctx;
    p.end = q.ctx + q.n;
    p.tiles = q.tiles;
    p.units = (p.end - whole + kTreeUnit - 1) / kTreeUnit;
    return p;
}

SFFN_DEV Part part_of(const SharedArgs &a, const Groups &gr, int i, bool record) {
    return i < a.n_groups ? prefix_part(a, gr, i) : own_part(a, gr, i - a.n_groups, record);
}

// A CTA's place on the line, in shared memory.
struct Line {
    Groups groups;
    long long scratch[33];
    long long pre[kSharedMaxGroups + kTreeMaxSeq + 1];  // length before each entry, and of all

    SFFN_DEV void build(const SharedArgs &a, bool record) {
        groups.load(a);
        const int entries = a.n_groups + a.n_seq;
        line_prefix(entries, pre, scratch, [&](int i) {
            const Part p = part_of(a, groups, i, record);
            return (long long)p.tiles * a.n_kv_heads * p.span();
        });
    }
};

// The piece of an item at place u, in a range that ends at u1.
struct Piece {
    Part p;
    int h, tile;
    int un0, un1;    // units; none if the range ends before the first
    long long next;
};
SFFN_DEV Piece piece_at(const SharedArgs &a, const Line &line, long long u, long long u1) {
    Piece c;
    const int i = tree_find(line.pre, a.n_groups + a.n_seq, u);
    c.p = part_of(a, line.groups, i, false);
    const long long local = u - line.pre[i];
    const int span = c.p.span(), item = (int)(local / span), at = (int)(local - (long long)item * span);
    c.h = item / c.p.tiles;
    c.tile = item - c.h * c.p.tiles;
    const int end = (int)min((long long)span, at + (u1 - u));
    c.un0 = max(0, at - kTreeItemCost);
    c.un1 = max(0, end - kTreeItemCost);
    c.next = u + (end - at);
    return c;
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

// ---------------------------------------------------------------------------
// fp32: attn_rows.cuh
// ---------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(rows::kThreads, 1) k_shared_rows(const SharedArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rows::Smem<D> &sm = *reinterpret_cast<rows::Smem<D> *>(smem_raw);
    Line &line = *reinterpret_cast<Line *>(smem_raw + sizeof(rows::Smem<D>));
    __shared__ uint64_t mask[kTreeMaxTokens];
    griddep_wait();
    griddep_launch_dependents();
    line.build(a, blockIdx.x == 0);
    const int w = blockIdx.x, tid = threadIdx.x;
    const long long total = line.pre[a.n_groups + a.n_seq];
    const int W = tree_ctas(total, gridDim.x);
    if (w >= W) return;
    const long long u1 = tree_cut(total, w + 1, W);
    const int G = a.group, ps = 1 << a.page_shift;
    for (long long u = tree_cut(total, w, W); u < u1;) {
        const Piece c = piece_at(a, line, u, u1);
        u = c.next;
        if (c.un0 >= c.un1) continue;
        const Part &p = c.p;
        const int tk0 = c.tile * a.tile_tokens, nt = min(a.tile_tokens, p.n - tk0);
        const int32_t *table = a.page_table + (size_t)p.row * a.table_width;
        const int k0 = p.k0 + c.un0 * kTreeUnit, k1 = min(p.end, p.k0 + c.un1 * kTreeUnit);
        __syncthreads();
        if (tid < nt && !p.prefix)
            mask[tid] = a.tree_mask ? a.tree_mask[p.t0 + tk0 + tid]
                                    : (tk0 + tid == 63 ? ~0ull : (1ull << (tk0 + tid + 1)) - 1ull);
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
        const bool whole = c.un0 == 0 && c.un1 == p.units;
        float *slot = a.part + tree_slot_floats(a.rows_max, D) * (size_t)(2 * w + (c.un0 > 0 ? 0 : 1));
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
                    float *ml = whole ? home_sums(a, p.prefix, row, D) : slot + (size_t)a.rows_max * D + 2 * r;
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
    static constexpr bool kOneToken = false;
    const SharedArgs &a;
    Line &line;
    long long u, u1;  // this CTA's next place on the line, and the end of its range
    int G, box;       // box: cache rows of one copy (a page's, 64 at most)

    struct RowInfo {
        uint64_t mask;
    };

    SFFN_DEV SharedPolicy(const SharedArgs &args, Line &l)
        : a(args), line(l), G(args.group), box(min(64, 1 << args.page_shift)) {}

    SFFN_DEV void start() {
        line.build(a, blockIdx.x == 0);
        const long long total = line.pre[a.n_groups + a.n_seq];
        const int W = tree_ctas(total, gridDim.x), b = blockIdx.x;
        u = b < W ? tree_cut(total, b, W) : 0;
        u1 = b < W ? tree_cut(total, b + 1, W) : 0;
    }
    SFFN_DEV bool next(atc::Work &w) {
        Piece c;
        do {
            if (u >= u1) return false;
            c = piece_at(a, line, u, u1);
            u = c.next;
        } while (c.un0 >= c.un1);
        const Part &p = c.p;
        const int tk0 = c.tile * a.tile_tokens;
        const int k0 = p.k0 + c.un0 * kTreeUnit, k1 = min(p.end, p.k0 + c.un1 * kTreeUnit);
        const int n = (k1 - k0 + atc::kKeys - 1) / atc::kKeys, TB = 128 / G;
        w.h = c.h;
        w.q_row = p.t0 + tk0;
        w.nt = min(a.tile_tokens, p.n - tk0);
        w.k0 = k0;
        w.k1 = w.exist = k1;
        w.tiles = n;
        w.n[0] = ONE ? (n + 1) / 2 : n;
        w.n[1] = ONE ? n / 2 : (w.nt > TB ? n : 0);
        w.mask_from[0] = w.mask_from[1] = max(0, min(p.ctx, k1) - k0) / atc::kKeys;
        w.ctx = p.ctx;
        w.seq = p.row;
        w.tok0 = tk0;
        w.whole = c.un0 == 0 && c.un1 == p.units;
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
    SFFN_DEV RowInfo row_info(const atc::Work &w, int tok) const {
        const int i = w.tok0 + tok;
        if (w.kind == 2) return RowInfo{0};  // (of a prefix every key is seen)
        const uint64_t m = a.tree_mask ? a.tree_mask[w.q_row + tok] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
        return RowInfo{m};
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
            float *slot = a.part + tree_slot_floats(a.rows_max, D) * (size_t)w.slot;
            o = slot + (size_t)(tok * G + head) * D;
            sums = slot + (size_t)a.rows_max * D + 2 * (tok * G + head);
        }
        *reinterpret_cast<float2 *>(sums) = make_float2(m * a.scale, l);
        return reinterpret_cast<unsigned char *>(o);
    }
};

constexpr size_t kLineBytes = align16(sizeof(Line));

template <int D, bool ONE>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_shared_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const SharedArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SharedPolicy<D, ONE> policy(a, *reinterpret_cast<Line *>(smem_raw));
    atc::attention_cta<Cfg<D, ONE>, D>(policy, map_q, map_k, map_v, map_q, a.scale, a.group, a.err, smem_raw + kLineBytes);
}

// ---------------------------------------------------------------------------
// Join: a warp a row
// ---------------------------------------------------------------------------

constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_shared_join(const SharedArgs a, int grid) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Line &line = *reinterpret_cast<Line *>(smem_raw);
    line.build(a, false);  // of the inputs alone, which the pieces' kernel has waited for
    const long long total = line.pre[a.n_groups + a.n_seq];
    const int W = tree_ctas(total, grid), lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    const size_t sf = tree_slot_floats(a.rows_max, D);
    // (item by item of the sequences: a block takes a sequence's rows)
    for (int s = blockIdx.y; s < a.n_seq; s += gridDim.y) {
        const Part own = own_part(a, line.groups, s, false);
        const int g = line.groups.of(s, a.n_groups);
        const Part pre = own.joint ? prefix_part(a, line.groups, g) : Part{};
        for (int i = blockIdx.x * kJoinWarps + (threadIdx.x >> 5); i < own.n * a.n_heads; i += gridDim.x * kJoinWarps) {
            const int t = own.t0 + i / a.n_heads, head = i % a.n_heads, h = head / a.group;
            const size_t row = (size_t)t * a.n_heads + head;
            JoinedRow<D / 32> j;
            bool direct = true;
            auto add = [&](const Part &p, int entry) {
                const int tile = (t - p.t0) / a.tile_tokens, r = (t - p.t0 - tile * a.tile_tokens) * a.group + head % a.group;
                const long long i0 = line.pre[entry] + ((long long)h * p.tiles + tile) * p.span();
                const int w0 = tree_owner(total, i0 + kTreeItemCost, W), w1 = tree_owner(total, i0 + p.span() - 1, W);
                if (w0 == w1 && !p.joint) return;  // written at once
                direct = false;
                if (w0 == w1) {
                    j.add(1, lane, [&](int) { return home_sums(a, p.prefix, row, D); },
                          [&](int) { return home_row(a, p.prefix, row, D); });
                } else {
                    auto slot = [&](int k) { return a.part + sf * (size_t)(2 * (w0 + k) + (k == 0 ? 1 : 0)); };
                    j.add(w1 - w0 + 1, lane, [&](int k) { return slot(k) + (size_t)a.rows_max * D + 2 * r; },
                          [&](int k) { return slot(k) + (size_t)r * D; });
                }
            };
            if (pre.n > 0) add(pre, g);
            add(own, a.n_groups + s);
            if (!direct) j.write(static_cast<T *>(a.out) + row * D, lane);
        }
    }
}

template <typename T, int D>
cudaError_t launch_join(const SharedArgs &a, int grid, cudaStream_t s) {
    // about as many warps as rows, four a SM at the most blocks
    const int per = (int)(((long long)a.T * a.n_heads / a.n_seq + kJoinWarps - 1) / kJoinWarps);
    const int gx = per < 1 ? 1 : (per > 64 ? 64 : per), most = 8 * grid / gx, gy = most < 1 ? 1 : (most < a.n_seq ? most : a.n_seq);
    return launch_k(k_shared_join<T, D>, dim3(gx, gy), dim3(32 * kJoinWarps), sizeof(Line), s, a, grid);
}

template <int D>
sffn_status launch_f32(SharedArgs a, int grid, cudaStream_t s) {
    a.tile_tokens = rows::kRows / a.group;
    constexpr int smem = (int)(sizeof(rows::Smem<D>) + sizeof(Line));
    cudaError_t e = set_max_smem((const void *)k_shared_rows<D>, smem);
    if (e == cudaSuccess) e = launch_k(k_shared_rows<D>, dim3(grid), dim3(rows::kThreads), smem, s, a);
    if (e == cudaSuccess) e = launch_join<float, D>(a, grid, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

template <int D, bool ONE>
sffn_status launch_bf16(SharedArgs a, int grid, cudaStream_t s) {
    const int G = a.group, TB = 128 / G, ps = 1 << a.page_shift;
    a.tile_tokens = ONE ? TB : 2 * TB;
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, sq[2] = {D * 2, (uint64_t)a.q_stride * 2};
    // the cache as [8-row group][column block][row][64]: a box is a page's rows (64 at most), all columns
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.n_pages * a.n_kv_heads * ps / 8},
                   sk[3] = {D * 2, 128, D * 16};
    const uint32_t bq[3] = {64, (uint32_t)G, (uint32_t)TB}, bk[4] = {64, 8, D / 64, (uint32_t)(ps < 64 ? ps : 64) / 8};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !make_map_bf16(&mk, a.ck, 4, dk, sk, bk) ||
        !make_map_bf16(&mv, a.cv, 4, dk, sk, bk))
        return SFFN_ERR_UNSUPPORTED;
    constexpr int smem = Cfg<D, ONE>::kSmem + (int)kLineBytes;
    cudaError_t e = set_max_smem((const void *)k_shared_tc<D, ONE>, smem);
    if (e == cudaSuccess) e = launch_k(k_shared_tc<D, ONE>, dim3(grid), dim3(atc::kThreads), smem, s, mq, mk, mv, a);
    if (e == cudaSuccess) e = launch_join<__nv_bfloat16, D>(a, grid, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

template <int D>
sffn_status launch_bf16(const SharedArgs &a, int grid, cudaStream_t s) {
    // a second row tile where the groups' rows fill more than one in the mean
    return (long long)a.T * a.group <= 128LL * a.n_groups ? launch_bf16<D, true>(a, grid, s)
                                                          : launch_bf16<D, false>(a, grid, s);
}

}  // namespace

SharedPlan make_shared_plan(int T, int n_heads, int n_kv_heads, int head_dim) {
    SharedPlan p = {};
    const int G = n_heads / n_kv_heads;
    p.grid = device_sm_count();
    p.rows_max = (T < 2 * (128 / G) ? T : 2 * (128 / G)) * G;
    size_t o = align_up(kControlBytes);
    p.off_part = o;
    o = align_up(o + sizeof(float) * 2 * (size_t)p.grid * tree_slot_floats(p.rows_max, head_dim));
    p.off_home = o;
    o = align_up(o + sizeof(float) * 2 * home_floats(T, n_heads, head_dim));
    p.total = o;
    return p;
}

sffn_status run_attn_shared(const SharedArgs &a, const SharedPlan &p, int dtype, int head_dim, cudaStream_t s) {
    if (dtype == SFFN_BF16) return head_dim == 128 ? launch_bf16<128>(a, p.grid, s) : launch_bf16<64>(a, p.grid, s);
    return head_dim == 128 ? launch_f32<128>(a, p.grid, s) : launch_f32<64>(a, p.grid, s);
}

}  // namespace sffn
