// attn_tree.cu -- attention of drafted tokens (one: plain decode) over the paged
// cache (sm_103a).
//
// Bound: HBM, the cached keys and values, each read once for all the new tokens and
// all the query heads that share them.
#include "attn_rows.cuh"

namespace sffn {

namespace {

template <typename T, int D>
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
        const int s = tree_find(pre, a.n_seq, u);
        const TreeSeq q = tree_seq(a, s, false);
        const long long local = u - pre[s];
        const int item = (int)(local / q.units), un0 = (int)(local - (long long)item * q.units);
        const int un1 = (int)min((long long)q.units, un0 + (u1 - u));
        const int tile = item / a.n_kv_heads, h = item - tile * a.n_kv_heads;
        const int tk0 = tile * a.tile_tokens, nt = min(a.tile_tokens, q.n - tk0);
        const int32_t *table = a.page_table + (size_t)s * a.table_width;
        const long long keys = (long long)q.ctx + q.n;
        const long long k0 = (long long)un0 * kTreeUnit, k1 = min(keys, (long long)un1 * kTreeUnit);
        __syncthreads();
        if (tid < nt)
            mask[tid] = a.tree_mask ? a.tree_mask[q.t0 + tk0 + tid]
                                    : (tk0 + tid == 63 ? ~0ull : (1ull << (tk0 + tid + 1)) - 1ull);
        rows::Acc<D> acc;
        rows::attend<T, D>(
            sm, acc, nt * G, k0, k1, a.scale,
            [&](int r) {
                return static_cast<const T *>(a.q) + (size_t)(q.t0 + tk0 + r / G) * a.q_stride +
                       (size_t)(h * G + r % G) * D;
            },
            [&](long long j, int which) -> const T * {
                const int pg = table[j >> a.page_shift];
                if (pg < 0 || pg >= a.n_pages) {
                    record_error(a.err, SFFN_ERR_DEVICE);
                    return nullptr;
                }
                return static_cast<const T *>(which ? a.cv : a.ck) +
                       ((((size_t)pg * a.n_kv_heads + h) << a.page_shift) + (size_t)(j & (ps - 1))) * D;
            },
            [&](int r, long long j) { return j < q.ctx || ((mask[r / G] >> (j - q.ctx)) & 1); });
        const bool whole = un0 == 0 && un1 == q.units;
        float *slot = a.part + tree_slot_floats(a.rows_max, D) * (size_t)(2 * w + (un0 > 0 ? 0 : 1));
        const int c = (tid % rows::Acc<D>::CT) * 4, g = tid / rows::Acc<D>::CT;
#pragma unroll
        for (int i = 0; i < rows::Acc<D>::RPT; ++i) {
            const int r = g + i * rows::Acc<D>::RG;
            if (r < nt * G) {
                float4 o = acc.o[i];
                if (whole) {
                    const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
                    T *dst = static_cast<T *>(a.out) +
                             ((size_t)(q.t0 + tk0 + r / G) * a.n_heads + (size_t)(h * G + r % G)) * D + c;
                    rows::store4<T>(dst, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
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
        u += un1 - un0;
    }
}

// Joins the pieces of cut items: for each row, M = max of the pieces' maxima,
// out = sum(exp(m_i - M) o_i) / sum(exp(m_i - M) l_i), the pieces in the order of
// their CTAs.  One warp a row (token, query head).
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_tree_join(const TreeArgs a, int grid) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    long long *pre = reinterpret_cast<long long *>(smem_raw);
    __shared__ long long scratch[33];
    griddep_wait();
    griddep_launch_dependents();
    tree_prefix(a, pre, scratch, false);
    const long long total = pre[a.n_seq];
    const int W = tree_ctas(total, grid);
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (row >= (long long)a.T * a.n_heads) return;
    const int t = (int)(row / a.n_heads), hq = (int)(row - (long long)t * a.n_heads);
    // the sequence of token t: the last one that starts at or before it
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_tokens[mid] <= t) lo = mid; else hi = mid;
    }
    const TreeSeq q = tree_seq(a, lo, false);
    if (t < q.t0 || t >= q.t0 + q.n) return;
    const int G = a.group, h = hq / G, tile = (t - q.t0) / a.tile_tokens;
    const int r = (t - q.t0 - tile * a.tile_tokens) * G + hq - h * G;
    const long long i0 = pre[lo] + ((long long)tile * a.n_kv_heads + h) * q.units, i1 = i0 + q.units;
    const int w0 = tree_owner(total, i0, W), w1 = tree_owner(total, i1 - 1, W);
    if (w0 == w1) return;  // finished by its one CTA
    const size_t sf = tree_slot_floats(a.rows_max, D);
    auto slot = [&](int w) { return a.part + sf * (size_t)(2 * w + (w == w0 ? 1 : 0)); };
    float M = -INFINITY;
    for (int w = w0 + lane; w <= w1; w += 32) M = fmaxf(M, slot(w)[(size_t)a.rows_max * D + 2 * r]);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float o[D / 32], l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    for (int w = w0; w <= w1; ++w) {
        const float *p = slot(w), *ml = p + (size_t)a.rows_max * D + 2 * r;
        const float m = ml[0], f = expf(m - ref);
        if (m == -INFINITY && ml[1] == 0.f) continue;  // a piece without a key that this row sees
        l += f * ml[1];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] += f * p[(size_t)r * D + lane * (D / 32) + i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(a.out) + (size_t)row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        if constexpr (sizeof(T) == 4) dst[i] = o[i] * inv;
        else dst[i] = __float2bfloat16_rn(o[i] * inv);
    }
}

template <typename T, int D>
sffn_status launch_tree(const TreeArgs &a, int W, cudaStream_t s) {
    const size_t pre = (size_t)(a.n_seq + 1) * sizeof(long long);
    const size_t smem = sizeof(rows::Smem<D>) + pre;
    cudaError_t e = set_max_smem((const void *)k_tree_rows<T, D>, (int)(sizeof(rows::Smem<D>) + (kTreeMaxSeq + 1) * 8));
    if (e == cudaSuccess) e = launch_k(k_tree_rows<T, D>, dim3(W), dim3(rows::kThreads), smem, s, a);
    const long long rows = (long long)a.T * a.n_heads;
    if (e == cudaSuccess)
        e = launch_k(k_tree_join<T, D>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(32 * kJoinWarps),
                     pre, s, a, W);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace

TreePlan make_tree_plan(int T, int n_heads, int n_kv_heads, int head_dim) {
    TreePlan p = {};
    const int G = n_heads / n_kv_heads;
    p.grid = device_sm_count();
    p.tile_tokens = rows::kRows / G;
    p.rows_max = (T < p.tile_tokens ? T : p.tile_tokens) * G;
    size_t o = 0;
    o = align_up(o + kControlBytes);
    p.off_part = o;
    o = align_up(o + sizeof(float) * 2 * (size_t)p.grid * tree_slot_floats(p.rows_max, head_dim));
    p.total = o;
    return p;
}

sffn_status run_attn_tree(const TreeArgs &a, const TreePlan &p, int dtype, int head_dim, cudaStream_t s) {
    if (dtype == SFFN_BF16)
        return head_dim == 128 ? launch_tree<__nv_bfloat16, 128>(a, p.grid, s)
                               : launch_tree<__nv_bfloat16, 64>(a, p.grid, s);
    return head_dim == 128 ? launch_tree<float, 128>(a, p.grid, s) : launch_tree<float, 64>(a, p.grid, s);
}

}  // namespace sffn
