// attn_tree.cu -- attention of drafted tokens (one: plain decode) over the paged
// cache (sm_103a).
//
// Bound: HBM, the cached keys and values, each read once for all the new tokens and
// all the query heads that share them.  Measured (a call among others, from Python): 8 tokens over 65531
// positions, 64/8 heads of 128, 55 us (4.9 TB/s, 0.72 of the measured copy rate); 48 ragged sequences of one token, 32/8
// heads, 65.5 us (4.6 TB/s); one token over 300 positions 13 us.  Over the contexts' lengths the first is 18 us and
// 7.2 TB/s, the second 21 us and 6.9 TB/s (pages of 16; of 128: 20 us and 7.2 TB/s): what is fixed, start, item
// boundaries, join and tail, keeps the calls from the copy rate, not the loads.
#include "attn_rows.cuh"
#include "attn_tc.cuh"

namespace sffn {

namespace {

template <int D>
__global__ void __launch_bounds__(rows::kThreads, 1) k_tree_rows(const TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rows::Smem<D> &sm = *reinterpret_cast<rows::Smem<D> *>(smem_raw);
    long long *pre = reinterpret_cast<long long *>(smem_raw + sizeof(rows::Smem<D>));
    __shared__ long long scratch[33];
    __shared__ uint64_t mask[kTreeMaxTokens];
    griddep_wait();
    griddep_launch_dependents();
    tree_prefix(a, pre, scratch, blockIdx.x == 0);
    const int w = blockIdx.x, tid = threadIdx.x;
    const long long total = pre[a.n_seq];
    const int W = tree_ctas(total, gridDim.x);
    if (w >= W) return;
    const long long u1 = tree_cut(total, w + 1, W);
    const int G = a.group, ps = 1 << a.page_shift;
    for (long long u = tree_cut(total, w, W); u < u1;) {
        TreeSeq q;
        const TreePiece pc = tree_piece(a, pre, u, u1, q);
        u = pc.next;
        if (pc.un0 >= pc.un1) continue;
        const int tk0 = pc.tile * a.tile_tokens, nt = min(a.tile_tokens, q.n - tk0);
        const int32_t *table = a.page_table + (size_t)pc.s * a.table_width;
        const int k0 = pc.un0 * kTreeUnit, k1 = min(q.ctx + q.n, pc.un1 * kTreeUnit);
        __syncthreads();
        if (tid < nt)
            mask[tid] = a.tree_mask ? a.tree_mask[q.t0 + tk0 + tid]
                                    : (tk0 + tid == 63 ? ~0ull : (1ull << (tk0 + tid + 1)) - 1ull);
        rows::Acc<D> acc;
        rows::attend<D>(
            sm, acc, nt * G, k0, k1, min(q.ctx, k1), a.scale,
            [&](int r) {
                return static_cast<const float *>(a.q) + (size_t)(q.t0 + tk0 + r / G) * a.q_stride +
                       (size_t)(pc.h * G + r % G) * D;
            },
            [&](int j, int which) -> const float * {
                const int pg = table[j >> a.page_shift];
                if (pg < 0 || pg >= a.n_pages) {
                    record_error(a.err, SFFN_ERR_DEVICE);
                    return nullptr;
                }
                return static_cast<const float *>(which ? a.cv : a.ck) +
                       ((((size_t)pg * a.n_kv_heads + pc.h) << a.page_shift) + (size_t)(j & (ps - 1))) * D;
            },
            [&](int r, int j) { return (mask[r / G] >> (j - q.ctx)) & 1; });
        const bool whole = pc.un0 == 0 && pc.un1 == q.units;
        float *slot = a.part + tree_slot_floats(a.rows_max, D) * (size_t)(2 * w + (pc.un0 > 0 ? 0 : 1));
        const int c = (tid % rows::Acc<D>::CT) * 4, g = (tid / rows::Acc<D>::CT) * rows::Acc<D>::RPT;
#pragma unroll
        for (int i = 0; i < rows::Acc<D>::RPT; ++i) {
            const int r = g + i;
            if (r < nt * G) {
                const float4 o = acc.o[i];
                if (whole) {
                    const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
                    float *dst = static_cast<float *>(a.out) +
                                 ((size_t)(q.t0 + tk0 + r / G) * a.n_heads + (size_t)(pc.h * G + r % G)) * D + c;
                    *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(slot + (size_t)r * D + c) = o;
                    if (c == 0) {
                        float *ml = slot + (size_t)a.rows_max * D + 2 * r;
                        ml[0] = sm.m[r];
                        ml[1] = sm.l[r];
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// bf16: attn_tc.cuh over the paged cache
// ---------------------------------------------------------------------------

template <int D>
using Cfg = atc::Cfg<D, D == 128 ? 5 : 10, true, true>;

template <int D>
struct TreePolicy {
    static constexpr bool kReread = false;
    const TreeArgs &a;
    long long *pre;         // length of the line before each sequence (shared memory)
    long long u, u1;        // this CTA's next place on the line, and the end of its range
    int G, TB, box;         // box: cache rows of one copy (a page's, 64 at most)

    struct RowInfo {
        uint64_t mask;
    };

    long long *scratch;

    SFFN_DEV TreePolicy(const TreeArgs &args, long long *prefix, long long *scan)
        : a(args), pre(prefix), G(args.group), TB(128 / args.group), box(min(64, 1 << args.page_shift)), scratch(scan) {}

    SFFN_DEV void start() {
        tree_prefix(a, pre, scratch, blockIdx.x == 0);
        const long long total = pre[a.n_seq];
        const int W = tree_ctas(total, gridDim.x), b = blockIdx.x;
        u = b < W ? tree_cut(total, b, W) : 0;
        u1 = b < W ? tree_cut(total, b + 1, W) : 0;
    }
    SFFN_DEV bool next(atc::Work &w) {
        TreeSeq q;
        TreePiece pc;
        do {
            if (u >= u1) return false;
            pc = tree_piece(a, pre, u, u1, q);
            u = pc.next;
        } while (pc.un0 >= pc.un1);
        const int un0 = pc.un0, un1 = pc.un1, s = pc.s, tk0 = pc.tile * a.tile_tokens;
        const int k0 = un0 * kTreeUnit, k1 = min(q.ctx + q.n, un1 * kTreeUnit);
        const int n = (k1 - k0 + atc::kKeys - 1) / atc::kKeys;
        w.h = pc.h;
        w.q_row = q.t0 + tk0;
        w.nt = min(a.tile_tokens, q.n - tk0);
        w.k0 = k0;
        w.k1 = w.exist = k1;
        w.tiles = n;
        w.n[0] = (n + 1) / 2;
        w.n[1] = n / 2;
        w.mask_from[0] = w.mask_from[1] = max(0, min(q.ctx, k1) - k0) / atc::kKeys;
        w.ctx = q.ctx;
        w.seq = s;
        w.tok0 = tk0;
        w.whole = un0 == 0 && un1 == q.units;
        w.slot = 2 * blockIdx.x + (un0 > 0 ? 0 : 1);
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
        constexpr int H = Cfg<D>::kHalves;
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
    SFFN_DEV bool partial(const atc::Work &w) const { return !w.whole; }
    SFFN_DEV unsigned char *begin_row(const atc::Work &w, int tok, int head, bool valid, float m, float l,
                                      float &inv) const {
        inv = l == 0.f ? 0.f : 1.f / l;
        if (!valid) return nullptr;
        if (w.whole)
            return reinterpret_cast<unsigned char *>(static_cast<uint16_t *>(a.out) +
                                                     ((size_t)(w.q_row + tok) * a.n_heads + (size_t)w.h * G + head) * D);
        float *slot = a.part + tree_slot_floats(a.rows_max, D) * (size_t)w.slot;
        const int row = tok * G + head;
        *reinterpret_cast<float2 *>(slot + (size_t)a.rows_max * D + 2 * row) = make_float2(m * a.scale, l);
        return reinterpret_cast<unsigned char *>(slot + (size_t)row * D);
    }
};

constexpr size_t kPrefixBytes = (kTreeMaxSeq + 1) * sizeof(long long);

template <int D>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ long long scratch[33];
    TreePolicy<D> policy(a, reinterpret_cast<long long *>(smem_raw), scratch);
    atc::attention_cta<Cfg<D>, D>(policy, map_q, map_k, map_v, map_q, a.scale, a.group, a.err, smem_raw + kPrefixBytes);
}

// Joins the pieces of cut items: for each row, M = max of the pieces' maxima,
// out = sum(exp(m_i - M) o_i) / sum(exp(m_i - M) l_i), the pieces in the order of
// their CTAs.
// There are `parts` blocks for each place between two CTAs' ranges; those of all the places that cut
// an item share its rows, a warp a row at a time (an item cut often has many
// pieces to read and as many more blocks).  What a block has to do depends on the call's inputs
// alone and is found before the wait for the pieces' kernel (which lets this one start once it has itself waited for the inputs; 128 threads of 40
// registers find room beside it); after the wait come one load of all maxima and sums and
// then the outputs, independent of one another.
constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 8;

template <typename T, int D>
SFFN_DEV void join_row(const TreeArgs &a, long long row, int w0, int w1, int r, int lane) {
    const size_t sf = tree_slot_floats(a.rows_max, D);
    auto slot = [&](int w) { return a.part + sf * (size_t)(2 * w + (w == w0 ? 1 : 0)); };
    constexpr int C = D / 32;  // columns of a lane
    float o[C], l = 0.f, M = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.f;
    for (int wb = w0; wb <= w1; wb += 32) {  // 32 pieces at a time
        const int n = min(32, w1 - wb + 1);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n) ml = __ldcg(reinterpret_cast<const float2 *>(slot(wb + lane) + (size_t)a.rows_max * D + 2 * r));
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
            const float *p = slot(wb + k) + (size_t)r * D + lane * C;
            if constexpr (C == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(p));
                o[0] += fk * x.x, o[1] += fk * x.y, o[2] += fk * x.z, o[3] += fk * x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(p));
                o[0] += fk * x.x, o[1] += fk * x.y;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(a.out) + (size_t)row * D + lane * C;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if constexpr (sizeof(T) == 4) dst[i] = o[i] * inv;
        else dst[i] = __float2bfloat16_rn(o[i] * inv);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 12) k_tree_join(const TreeArgs a, int grid, int parts) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    long long *pre = reinterpret_cast<long long *>(smem_raw);
    __shared__ long long scratch[33];
    tree_prefix(a, pre, scratch, false);
    const long long total = pre[a.n_seq];
    const int W = tree_ctas(total, grid), lane = threadIdx.x & 31;
    const int w = 1 + blockIdx.x / parts, part = blockIdx.x % parts;
    int w0 = 0, w1 = 0, nr = 0, tok = 0, head = 0;  // the item's CTAs, rows, first token and query head
    if (w < W) {
        const long long u = tree_cut(total, w, W);
        const int s = tree_find(pre, a.n_seq, u);
        const TreeSeq q = tree_seq(a, s, false);
        const long long local = u - pre[s];
        const int item = (int)(local / q.span());
        const long long i0 = pre[s] + (long long)item * q.span();
        const int h = item / q.tiles, tk0 = (item - h * q.tiles) * a.tile_tokens;
        w0 = tree_owner(total, i0 + kTreeItemCost, W);
        w1 = tree_owner(total, i0 + q.span() - 1, W);
        nr = min(a.tile_tokens, q.n - tk0) * a.group;
        tok = q.t0 + tk0;
        head = h * a.group;
    }
    griddep_wait();
    griddep_launch_dependents();
    if (w0 >= w || w > w1) return;  // no item is cut here
    const int blocks = (w1 - w0) * parts, b = (w - w0 - 1) * parts + part;
    for (int r = b * kJoinWarps + (threadIdx.x >> 5); r < nr; r += blocks * kJoinWarps)
        join_row<T, D>(a, (long long)(tok + r / a.group) * a.n_heads + head + r % a.group, w0, w1, r, lane);
}

template <typename T, int D>
cudaError_t launch_join(const TreeArgs &a, int grid, cudaStream_t s) {
    if (grid < 2) return cudaSuccess;  // one CTA: nothing is cut
    // two rows a warp where an item is cut once, as long as one wave of blocks takes them all
    int parts = (a.rows_max + kJoinRows - 1) / kJoinRows;
    if (parts > 12) parts = 12;
    return launch_k(k_tree_join<T, D>, dim3((unsigned)((grid - 1) * parts)), dim3(32 * kJoinWarps),
                    (size_t)(a.n_seq + 1) * sizeof(long long), s, a, grid, parts);
}

template <int D>
sffn_status launch_tree_f32(const TreeArgs &a, int grid, cudaStream_t s) {
    cudaError_t e = set_max_smem((const void *)k_tree_rows<D>, (int)(sizeof(rows::Smem<D>) + kPrefixBytes));
    if (e == cudaSuccess)
        e = launch_k(k_tree_rows<D>, dim3(grid), dim3(rows::kThreads),
                     sizeof(rows::Smem<D>) + (size_t)(a.n_seq + 1) * sizeof(long long), s, a);
    if (e == cudaSuccess) e = launch_join<float, D>(a, grid, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

template <int D>
sffn_status launch_tree_bf16(const TreeArgs &a, int grid, cudaStream_t s) {
    const int G = a.group, TB = 128 / G, ps = 1 << a.page_shift;
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, sq[2] = {D * 2, (uint64_t)a.q_stride * 2};
    // the cache as [8-row group][column block][row][64]: a box is a page's rows (64 at most), all columns
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.n_pages * a.n_kv_heads * ps / 8},
                   sk[3] = {D * 2, 128, D * 16};
    const uint32_t bq[3] = {64, (uint32_t)G, (uint32_t)TB}, bk[4] = {64, 8, D / 64, (uint32_t)(ps < 64 ? ps : 64) / 8};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !make_map_bf16(&mk, a.ck, 4, dk, sk, bk) ||
        !make_map_bf16(&mv, a.cv, 4, dk, sk, bk))
        return SFFN_ERR_UNSUPPORTED;
    constexpr int smem = Cfg<D>::kSmem + (int)kPrefixBytes;
    cudaError_t e = set_max_smem((const void *)k_tree_tc<D>, smem);
    if (e == cudaSuccess) e = launch_k(k_tree_tc<D>, dim3(grid), dim3(atc::kThreads), smem, s, mq, mk, mv, a);
    if (e == cudaSuccess) e = launch_join<__nv_bfloat16, D>(a, grid, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace

TreePlan make_tree_plan(int dtype, int T, int n_heads, int n_kv_heads, int head_dim) {
    TreePlan p = {};
    const int G = n_heads / n_kv_heads;
    p.grid = device_sm_count();
    p.tile_tokens = (dtype == SFFN_BF16 ? 128 : rows::kRows) / G;
    int tokens = T < kTreeMaxTokens ? T : kTreeMaxTokens;
    if (tokens > p.tile_tokens) tokens = p.tile_tokens;
    p.rows_max = tokens * G;
    size_t o = 0;
    o = align_up(o + kControlBytes);
    p.off_part = o;
    o = align_up(o + sizeof(float) * 2 * (size_t)p.grid * tree_slot_floats(p.rows_max, head_dim));
    p.total = o;
    return p;
}

sffn_status run_attn_tree(const TreeArgs &a, const TreePlan &p, int dtype, int head_dim, cudaStream_t s) {
    if (dtype == SFFN_BF16)
        return head_dim == 128 ? launch_tree_bf16<128>(a, p.grid, s) : launch_tree_bf16<64>(a, p.grid, s);
    return head_dim == 128 ? launch_tree_f32<128>(a, p.grid, s) : launch_tree_f32<64>(a, p.grid, s);
}

}  // namespace sffn
