// attn_shared.cu -- attention of new tokens over the paged cache for sequences that share prefixes (sm_103a).
#include "attn_warp.cuh"

namespace sffn {

namespace {

constexpr int kWarps = 4;

// A warp: one token and query head, over its sequence's own table row.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) k_shared_warp(const SharedArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, s = blockIdx.y;
    const TreeSeq q = tree_seq(a, s, blockIdx.x == 0 && threadIdx.x == 0);
    int g = 0;
    while (g + 1 < a.n_groups && a.group_seqs[g + 1] <= s) ++g;
    const int p = a.prefix_lens[g];
    if (s < a.group_seqs[g] || s >= a.group_seqs[g + 1] || p < 0 || (p >> a.page_shift) > a.table_width ||
        ((p >> a.page_shift) << a.page_shift) > a.ctx_lens[s]) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, SFFN_ERR_DEVICE);
        return;
    }
    for (int row = blockIdx.x * kWarps + (threadIdx.x >> 5); row < q.n * a.n_heads; row += gridDim.x * kWarps) {
        const int i = row / a.n_heads, head = row - i * a.n_heads, h = head / a.group, t = q.t0 + i;
        const uint64_t mask = a.tree_mask ? a.tree_mask[t] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
        WarpRow<T, D> r;
        r.begin(static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)head * D, a.scale, lane);
        for (int j = 0; j < q.ctx + q.n; ++j) {
            if (j >= q.ctx && !((mask >> (j - q.ctx)) & 1)) continue;
            const int pg = a.page_table[(size_t)s * a.table_width + (j >> a.page_shift)];
            const bool there = pg >= 0 && pg < a.n_pages;
            if (!there && lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
            const size_t at = ((((size_t)(there ? pg : 0) * a.n_kv_heads + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
            r.add(there ? static_cast<const T *>(a.ck) + at : nullptr, there ? static_cast<const T *>(a.cv) + at : nullptr, lane);
        }
        r.end(static_cast<T *>(a.out) + ((size_t)t * a.n_heads + head) * D, lane);
    }
}

template <typename T, int D>
cudaError_t launch_shared(const SharedArgs &a, cudaStream_t s) {
    return launch_k(k_shared_warp<T, D>, dim3((unsigned)((a.n_heads + kWarps - 1) / kWarps), (unsigned)a.n_seq),
                    dim3(32 * kWarps), 0, s, a);
}

}  // namespace

SharedPlan make_shared_plan(int, int, int, int) { return SharedPlan{kAlign}; }

sffn_status run_attn_shared(const SharedArgs &a, const SharedPlan &, int dtype, int head_dim, cudaStream_t s) {
    SharedArgs b = a;
    b.tile_tokens = 1;
    cudaError_t e;
    if (dtype == SFFN_BF16)
        e = head_dim == 128 ? launch_shared<__nv_bfloat16, 128>(b, s) : launch_shared<__nv_bfloat16, 64>(b, s);
    else
        e = head_dim == 128 ? launch_shared<float, 128>(b, s) : launch_shared<float, 64>(b, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace sffn
