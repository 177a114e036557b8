// attn_pages.cu -- attention of each token over its chosen pages of the paged cache (sm_103a).
//
// An item is a (token, key head, row tile): up to 32 (16 of 128 elements) of the G rows against the n_sel chosen pages, taken one after the
// other as if they were consecutive positions.  The work of all items is one line as in attn.cuh (units of 64
// positions and kItemCost more per item), token by token and head by head, cut evenly over the
// warps (fp32: the CTAs); items that lie in one range are finished there, the pieces of a cut item are joined by
// k_pages_join.
#include "attn_rows.cuh"
#include "attn_few.cuh"

namespace sffn {

namespace {

// Units (of 64 positions) that an item costs by itself (48 tokens of up to 2048 positions, 8 key heads: 55.5 us with 1,
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

SFFN_DEV int pages_units(const PagesArgs &a, int n) { return (int)((((long long)n << a.at.page_shift) + kTreeUnit - 1) / kTreeUnit); }
SFFN_DEV int pages_span(const PagesArgs &a, int n) { return n > 0 ? pages_units(a, n) + kItemCost : 0; }

// A piece of an item.
struct PagesPiece {
    int t, h, n;   // token, key head, its pages
    int tile;      // row tile
    int un0, un1;  // units
    bool whole;
};

// A CTA's (or a warp's) walk along the line.
struct PagesWalk {
    const PagesArgs &a;
    long long u, u1;  // next place, end of the range
    long long at;     // where the item of place u (or the one before it, all done) begins
    int t, n, span;   // token, its pages, length of its items
    int h, tile;      // the item
    int range;        // which range this is

    SFFN_DEV explicit PagesWalk(const PagesArgs &args) : a(args) {}

    // Every thread of the CTA: its range (RANGES = 1), or its warp's, and the token at the range's beginning; rows of
    // tokens without pages are zeroed (dealt to the CTAs by token); tells the join which item the beginning cuts.
    template <typename T, int D, int RANGES>
    SFFN_DEV void start() {
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
        const int r = RANGES == 1 ? 0 : warp, b = blockIdx.x * RANGES + r;
        range = b;
        u = u1 = 0;
        h = tile = 0;
        int4 cut = make_int4(-1, 0, 0, 0);  // token, its item, first and last range of the cut item
        if (b < W) {
            u = tree_cut(total, b, W);
            u1 = tree_cut(total, b + 1, W);
            t = s_t[r];
            n = pages_of(a, t, false);
            span = pages_span(a, n);
            const int item = (int)((u - s_at[r]) / span);
            at = s_at[r] + (long long)item * span;
            h = item / a.tiles;
            tile = item - h * a.tiles;
            const int w0 = tree_owner(total, at + kItemCost, W), w1 = tree_owner(total, at + span - 1, W);
            if (w0 < b && b <= w1) cut = make_int4(t, item, w0, w1);
        }
        if (RANGES == 1 ? tid == 0 : lane == 0) a.cuts[b] = cut;
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
    walk.start<float, D, 1>();
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
        float *slot = a.part + tree_slot_floats(a.row_tile, D) * (size_t)(2 * blockIdx.x + (p.un0 > 0 ? 0 : 1));
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
                if (c == 0) *reinterpret_cast<float2 *>(slot + (size_t)a.row_tile * D + 2 * r) = make_float2(sm.m[r], sm.l[r]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// bf16: attn_few.cuh over the paged cache
// ---------------------------------------------------------------------------

template <int D>
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
        w.k0 = p.un0 * kTreeUnit;
        w.k1 = w.all = max(w.k0, min(seen(a, p.t, p.h, p.n), p.un1 * kTreeUnit));  // (none behind the last that it sees)
        w.whole = p.whole;
        w.slot = 2 * walk.range + (p.un0 > 0 ? 0 : 1);
        return true;
    }
    SFFN_DEV int page_of(const few::Work &w, int j) const {
        const int pg = cache_page(a, w.q_row, w.h, j);
        return pg < 0 ? a.at.n_pages : pg;
    }
    SFFN_DEV const __nv_bfloat16 *query(const few::Work &w, int row) const {
        return static_cast<const __nv_bfloat16 *>(a.q) + (size_t)w.q_row * a.q_stride + (size_t)(w.h * a.group + row) * D;
    }
    SFFN_DEV bool sees(const few::Work &, int, int) const { return false; }
    SFFN_DEV __nv_bfloat16 *out_row(const few::Work &w, int row) const {
        return static_cast<__nv_bfloat16 *>(a.out) + ((size_t)w.q_row * a.n_heads + (size_t)w.h * a.group + row) * D;
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
    PagesPolicy<D> policy(a);
    policy.walk.template start<__nv_bfloat16, D, few::kWarps>();
    few::attention<D, NT>(policy, map_k, map_v, a.at.page_shift, a.n_kv_heads, a.scale, a.err, smem_raw);
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
    auto slot = [&](int k) { return a.part + sf * (size_t)(2 * (w0 + k) + (k == 0 ? 1 : 0)); };
    for (int r = b * kJoinWarps + (threadIdx.x >> 5); r < rows; r += blocks * kJoinWarps) {
        JoinedRow<D / 32> j;
        j.add(w1 - w0 + 1, lane, [&](int k) { return slot(k) + (size_t)a.row_tile * D + 2 * r; },
              [&](int k) { return slot(k) + (size_t)r * D; });
        j.write(static_cast<T *>(a.out) + ((size_t)cut.x * a.n_heads + (size_t)h * a.group + r0 + r) * D, lane);
    }
}

template <typename T, int D>
cudaError_t launch_join(const PagesArgs &a, int ranges, cudaStream_t s) {
    if (ranges < 2) return cudaSuccess;  // one: nothing is cut
    const int parts = (a.row_tile + 2 * kJoinWarps - 1) / (2 * kJoinWarps);
    return launch_k(k_pages_join<T, D>, dim3((unsigned)((ranges - 1) * parts)), dim3(32 * kJoinWarps), 0, s, a, parts);
}

template <int D>
cudaError_t launch_f32(PagesArgs a, int grid, cudaStream_t s) {
    a.row_tile = a.group;
    a.tiles = 1;
    cudaError_t e = set_max_smem((const void *)k_pages_rows<D>, (int)sizeof(rows::Smem<D>));
    if (e == cudaSuccess) e = launch_k(k_pages_rows<D>, dim3(grid), dim3(rows::kThreads), sizeof(rows::Smem<D>), s, a);
    return e == cudaSuccess ? launch_join<float, D>(a, grid, s) : e;
}

template <int D, int NT>
cudaError_t launch_few(PagesArgs a, int grid, cudaStream_t s) {
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

template <int D>
cudaError_t launch_bf16(const PagesArgs &a, int grid, cudaStream_t s) {
    if (a.group <= 8) return launch_few<D, 1>(a, grid, s);
    return a.group <= 16 ? launch_few<D, 2>(a, grid, s) : launch_few<D, few::max_rows(D) / 8>(a, grid, s);
}

}  // namespace

PagesPlan make_pages_plan(int, int n_heads, int n_kv_heads, int head_dim) {
    PagesPlan p = {};
    p.grid = device_sm_count();
    size_t o = align_up(kControlBytes);
    p.off_cuts = o;
    const size_t ranges = 2 * few::kWarps * (size_t)p.grid;
    o = align_up(o + sizeof(int4) * ranges);
    p.off_part = o;
    // bf16: a slot pair a warp, of a row tile; fp32: a CTA, of all rows
    const int G = n_heads / n_kv_heads, most = few::max_rows(head_dim);
    const size_t b = ranges * tree_slot_floats(G < most ? G : most, head_dim), f = p.grid * tree_slot_floats(G, head_dim);
    o = align_up(o + sizeof(float) * 2 * (b > f ? b : f));
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
