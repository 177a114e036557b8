// attn_pages.cu -- attention of each token over its chosen pages of the paged cache (sm_103a).
//
// An item is a (token, key head): G rows against the n_sel chosen pages, taken one after the other as
// if they were consecutive positions.  The work of all items is one line as in attn.cuh (units of 64
// positions and kTreeItemCost more per item), token by token and head by head, cut evenly over the
// CTAs; items that lie in one CTA's range are finished there, the pieces of a cut item are joined by
// k_pages_join.
#include "attn_rows.cuh"
#include "attn_tc.cuh"

namespace sffn {

namespace {

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

SFFN_DEV int pages_units(const PagesArgs &a, int n) { return (int)((((long long)n << a.at.page_shift) + kTreeUnit - 1) / kTreeUnit); }
SFFN_DEV int pages_span(const PagesArgs &a, int n) { return n > 0 ? pages_units(a, n) + kTreeItemCost : 0; }

// A piece of an item.
struct PagesPiece {
    int t, h, n;   // token, key head, its pages
    int un0, un1;  // units
    bool whole;
};

// A CTA's walk along the line.
struct PagesWalk {
    const PagesArgs &a;
    long long u, u1;  // next place, end of the range
    long long at;     // where token t's items begin
    int t, n;         // token, its pages

    SFFN_DEV explicit PagesWalk(const PagesArgs &args) : a(args) {}

    // Every thread of the CTA: its range and the token at its beginning; rows of tokens without pages are
    // zeroed (dealt to the CTAs by token); tells the join which item the range's beginning cuts.
    template <typename T, int D>
    SFFN_DEV void start() {
        __shared__ long long s_scan[33], s_at;
        __shared__ int s_t;
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
        sum *= a.n_kv_heads;
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
        const int W = tree_ctas(total, gridDim.x), b = blockIdx.x;
        u = b < W ? tree_cut(total, b, W) : 0;
        u1 = b < W ? tree_cut(total, b + 1, W) : 0;
        if (b < W && before <= u && u < before + sum) {  // the token is one of this thread's
            int i = t0;
            for (;; ++i) {
                const long long len = (long long)pages_span(a, pages_of(a, i, false)) * a.n_kv_heads;
                if (u < before + len) break;
                before += len;
            }
            s_t = i;
            s_at = before;
        }
        __syncthreads();
        t = s_t;
        at = s_at;
        n = b < W ? pages_of(a, t, false) : 0;
        if (tid == 0) {
            int4 cut = make_int4(-1, 0, 0, 0);  // token, head, first and last CTA of the cut item
            if (b > 0 && b < W) {
                const int span = pages_span(a, n), h = (int)((u - at) / span);
                const long long i0 = at + (long long)h * span;
                const int w0 = tree_owner(total, i0 + kTreeItemCost, W), w1 = tree_owner(total, i0 + span - 1, W);
                if (w0 < b && b <= w1) cut = make_int4(t, h, w0, w1);
            }
            a.cuts[b] = cut;
        }
    }

    // The next piece with units (false: none is left).
    SFFN_DEV bool next(PagesPiece &p) {
        for (;;) {
            if (u >= u1) return false;
            int span = pages_span(a, n);
            while (u >= at + (long long)span * a.n_kv_heads) {  // on to the token that place u belongs to
                at += (long long)span * a.n_kv_heads;
                n = pages_of(a, ++t, false);
                span = pages_span(a, n);
            }
            const long long local = u - at;
            const int h = (int)(local / span), off = (int)(local - (long long)h * span);
            const int end = (int)min((long long)span, off + (u1 - u));
            u += end - off;
            p.t = t, p.h = h, p.n = n;
            p.un0 = max(0, off - kTreeItemCost), p.un1 = max(0, end - kTreeItemCost);
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

// Partial result slots as sffn_attn_tree's, of G rows.

// ---------------------------------------------------------------------------
// fp32: attn_rows.cuh
// ---------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(rows::kThreads, 1) k_pages_rows(const PagesArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rows::Smem<D> &sm = *reinterpret_cast<rows::Smem<D> *>(smem_raw);
    griddep_wait();
    griddep_launch_dependents();
    PagesWalk walk(a);
    walk.start<float, D>();
    const int tid = threadIdx.x, G = a.group, ps = 1 << a.at.page_shift;
    PagesPiece p;
    while (walk.next(p)) {
        const int k0 = p.un0 * kTreeUnit, k1 = min(seen(a, p.t, p.h, p.n), p.un1 * kTreeUnit);
        rows::Acc<D> acc;
        if (k0 < k1) {
            rows::attend<D>(
                sm, acc, G, k0, k1, k1, a.scale,
                [&](int r) { return static_cast<const float *>(a.q) + (size_t)p.t * a.q_stride + (size_t)(p.h * G + r) * D; },
                [&](int j, int which) -> const float * {
                    const int pg = cache_page(a, p.t, p.h, j);
                    if (pg < 0) return nullptr;
                    return static_cast<const float *>(which ? a.cv : a.ck) +
                           ((((size_t)pg * a.n_kv_heads + p.h) << a.at.page_shift) + (size_t)(j & (ps - 1))) * D;
                },
                [&](int, int) { return false; });
        } else {  // behind the last position that the token sees
            __syncthreads();
            if (tid < G) sm.m[tid] = -INFINITY, sm.l[tid] = 0.f;
#pragma unroll
            for (int i = 0; i < rows::Acc<D>::RPT; ++i) acc.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            __syncthreads();
        }
        float *slot = a.part + tree_slot_floats(G, D) * (size_t)(2 * blockIdx.x + (p.un0 > 0 ? 0 : 1));
        const int c = (tid % rows::Acc<D>::CT) * 4, g = (tid / rows::Acc<D>::CT) * rows::Acc<D>::RPT;
#pragma unroll
        for (int i = 0; i < rows::Acc<D>::RPT; ++i) {
            const int r = g + i;
            if (r >= G) continue;
            const float4 o = acc.o[i];
            if (p.whole) {
                const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
                float *dst = static_cast<float *>(a.out) + ((size_t)p.t * a.n_heads + (size_t)(p.h * G + r)) * D + c;
                *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            } else {
                *reinterpret_cast<float4 *>(slot + (size_t)r * D + c) = o;
                if (c == 0) *reinterpret_cast<float2 *>(slot + (size_t)G * D + 2 * r) = make_float2(sm.m[r], sm.l[r]);
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
struct PagesPolicy {
    static constexpr bool kReread = false;
    static constexpr bool kOneToken = true;
    const PagesArgs &a;
    PagesWalk walk;
    int G, box;  // box: cache rows of one copy (a page's, 64 at most)

    struct RowInfo {};

    SFFN_DEV explicit PagesPolicy(const PagesArgs &args) : a(args), walk(args), G(args.group), box(min(64, 1 << args.at.page_shift)) {}

    SFFN_DEV void start() { walk.template start<__nv_bfloat16, D>(); }
    SFFN_DEV bool next(atc::Work &w) {
        PagesPiece p;
        if (!walk.next(p)) return false;
        // (a piece behind the last position that the token sees has one key tile without keys)
        const int k0 = p.un0 * kTreeUnit, k1 = max(k0, min(seen(a, p.t, p.h, p.n), p.un1 * kTreeUnit));
        const int n = max(1, (k1 - k0 + atc::kKeys - 1) / atc::kKeys);
        w.h = p.h;
        w.q_row = p.t;
        w.nt = 1;
        w.k0 = k0;
        w.k1 = w.exist = k1;
        w.tiles = n;
        w.n[0] = (n + 1) / 2;
        w.n[1] = n / 2;
        w.mask_from[0] = w.mask_from[1] = (k1 - k0) / atc::kKeys;
        w.whole = p.whole;
        w.slot = 2 * blockIdx.x + (p.un0 > 0 ? 0 : 1);
        return true;
    }
    // Row of the cache (head h's) that holds place `j` of the token's pages, on page pg; past the end if that is not one.
    SFFN_DEV long long cache_row(const atc::Work &w, int j, int pg) const {
        return (((long long)(pg < 0 ? a.at.n_pages : pg) * a.n_kv_heads + (pg < 0 ? 0 : w.h)) << a.at.page_shift) +
               (pg < 0 ? 0 : j & ((1 << a.at.page_shift) - 1));
    }
    // Page of this lane's part of key tile j, a box of `box` rows (16 boxes at most); looked up a
    // tile ahead of its use.
    SFFN_DEV int place(const atc::Work &w, int j, int lane) const {
        const int off = j * atc::kKeys + lane * box;
        return lane * box < atc::kKeys && off < w.k1 - w.k0 ? cache_page(a, w.q_row, w.h, w.k0 + off) : 0;
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
    SFFN_DEV RowInfo row_info(const atc::Work &, int) const { return RowInfo{}; }
    SFFN_DEV void visible(const atc::Work &w, const RowInfo &, int j, uint32_t (&vis)[4]) const {
        const int n = w.k1 - w.k0 - j * atc::kKeys;
#pragma unroll
        for (int i = 0; i < 4; ++i) vis[i] = atc::low_bits(n - 32 * i);
    }
    SFFN_DEV const void *value_row(const atc::Work &w, const RowInfo &, int j) const {
        const int pg = cache_page(a, w.q_row, w.h, j);
        if (pg < 0) return nullptr;
        return static_cast<const uint16_t *>(a.cv) + (size_t)cache_row(w, j, pg) * D;
    }
    SFFN_DEV bool partial(const atc::Work &w) const { return !w.whole; }
    SFFN_DEV unsigned char *begin_row(const atc::Work &w, int, int head, bool valid, float m, float l, float &inv) const {
        inv = l == 0.f ? 0.f : 1.f / l;
        if (!valid) return nullptr;
        if (w.whole)
            return reinterpret_cast<unsigned char *>(static_cast<uint16_t *>(a.out) +
                                                     ((size_t)w.q_row * a.n_heads + (size_t)w.h * G + head) * D);
        float *slot = a.part + tree_slot_floats(G, D) * (size_t)w.slot;
        *reinterpret_cast<float2 *>(slot + (size_t)G * D + 2 * head) = make_float2(m * a.scale, l);
        return reinterpret_cast<unsigned char *>(slot + (size_t)head * D);
    }
};

template <int D>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_pages_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const PagesArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    PagesPolicy<D> policy(a);
    atc::attention_cta<Cfg<D>, D>(policy, map_q, map_k, map_v, map_q, a.scale, a.group, a.err, smem_raw);
}

// ---------------------------------------------------------------------------
// Join: `parts` blocks for each place between two CTAs' ranges; those of all the places that cut an
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
    const size_t sf = tree_slot_floats(a.group, D);
    auto slot = [&](int k) { return a.part + sf * (size_t)(2 * (w0 + k) + (k == 0 ? 1 : 0)); };
    for (int r = b * kJoinWarps + (threadIdx.x >> 5); r < a.group; r += blocks * kJoinWarps) {
        JoinedRow<D / 32> j;
        j.add(w1 - w0 + 1, lane, [&](int k) { return slot(k) + (size_t)a.group * D + 2 * r; },
              [&](int k) { return slot(k) + (size_t)r * D; });
        j.write(static_cast<T *>(a.out) + ((size_t)cut.x * a.n_heads + (size_t)cut.y * a.group + r) * D, lane);
    }
}

template <typename T, int D>
cudaError_t launch_join(const PagesArgs &a, int grid, cudaStream_t s) {
    if (grid < 2) return cudaSuccess;  // one CTA: nothing is cut
    const int parts = (a.group + 2 * kJoinWarps - 1) / (2 * kJoinWarps);
    return launch_k(k_pages_join<T, D>, dim3((unsigned)((grid - 1) * parts)), dim3(32 * kJoinWarps), 0, s, a, parts);
}

template <int D>
cudaError_t launch_f32(const PagesArgs &a, int grid, cudaStream_t s) {
    cudaError_t e = set_max_smem((const void *)k_pages_rows<D>, (int)sizeof(rows::Smem<D>));
    if (e == cudaSuccess) e = launch_k(k_pages_rows<D>, dim3(grid), dim3(rows::kThreads), sizeof(rows::Smem<D>), s, a);
    return e == cudaSuccess ? launch_join<float, D>(a, grid, s) : e;
}

template <int D>
cudaError_t launch_bf16(const PagesArgs &a, int grid, cudaStream_t s) {
    const int ps = 1 << a.at.page_shift;
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, sq[2] = {D * 2, (uint64_t)a.q_stride * 2};
    // the cache as [8-row group][column block][row][64]: a box is a page's rows (64 at most), all columns
    const uint64_t dk[4] = {64, 8, D / 64, (uint64_t)a.at.n_pages * a.n_kv_heads * ps / 8}, sk[3] = {D * 2, 128, D * 16};
    const uint32_t bq[3] = {64, (uint32_t)a.group, 1}, bk[4] = {64, 8, D / 64, (uint32_t)(ps < 64 ? ps : 64) / 8};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !make_map_bf16(&mk, a.ck, 4, dk, sk, bk) ||
        !make_map_bf16(&mv, a.cv, 4, dk, sk, bk))
        return cudaErrorNotSupported;
    cudaError_t e = set_max_smem((const void *)k_pages_tc<D>, Cfg<D>::kSmem);
    if (e == cudaSuccess) e = launch_k(k_pages_tc<D>, dim3(grid), dim3(atc::kThreads), Cfg<D>::kSmem, s, mq, mk, mv, a);
    return e == cudaSuccess ? launch_join<__nv_bfloat16, D>(a, grid, s) : e;
}

}  // namespace

PagesPlan make_pages_plan(int, int n_heads, int n_kv_heads, int head_dim) {
    PagesPlan p = {};
    p.grid = device_sm_count();
    size_t o = align_up(kControlBytes);
    p.off_cuts = o;
    o = align_up(o + sizeof(int4) * (size_t)p.grid);
    p.off_part = o;
    o = align_up(o + sizeof(float) * 2 * (size_t)p.grid * tree_slot_floats(n_heads / n_kv_heads, head_dim));
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
