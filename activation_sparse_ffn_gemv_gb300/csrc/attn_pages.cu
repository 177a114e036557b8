// attn_pages.cu -- attention of each token over its chosen pages of the paged cache (sm_103a).
#include "attn_warp.cuh"

namespace sffn {

namespace {

constexpr int kWarps = 4;

// A warp: one token and query head.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) k_pages_warp(const PagesArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (long long)a.T * a.n_heads) return;
    const int t = (int)(row / a.n_heads), head = (int)(row - (long long)t * a.n_heads), h = head / a.group;
    const int pos = a.at.positions[t], seq = a.at.seqs[t], n = a.n_sel[t];
    if (pos < 0) return;
    if (seq < 0 || seq >= a.at.n_seq || (pos >> a.at.page_shift) >= a.at.table_width || n < 0 || n > a.n_keep) {
        if (lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
        return;
    }
    const int ps = 1 << a.at.page_shift, mine = pos >> a.at.page_shift;
    const int32_t *sel = a.sel + ((size_t)t * a.n_kv_heads + h) * a.n_keep;
    WarpRow<T, D> r;
    r.begin(static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)head * D, a.scale, lane);
    for (int i = 0; i < n; ++i) {
        const int page = sel[i], pg = page < 0 || page > mine ? -1 : a.at.page_table[(size_t)seq * a.at.table_width + page];
        const bool there = pg >= 0 && pg < a.at.n_pages;
        if (!there && lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
        const int end = page == mine ? (pos & (ps - 1)) + 1 : ps;
        const size_t at = (((size_t)(there ? pg : 0) * a.n_kv_heads + h) << a.at.page_shift) * D;
        const T *k = there ? static_cast<const T *>(a.ck) + at : nullptr, *v = there ? static_cast<const T *>(a.cv) + at : nullptr;
        for (int j = 0; j < end; ++j) r.add(k ? k + (size_t)j * D : nullptr, v ? v + (size_t)j * D : nullptr, lane);
    }
    r.end(static_cast<T *>(a.out) + (size_t)row * D, lane);
}

template <typename T, int D>
cudaError_t launch_pages(const PagesArgs &a, cudaStream_t s) {
    const long long rows = (long long)a.T * a.n_heads;
    return launch_k(k_pages_warp<T, D>, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, s, a);
}

}  // namespace

PagesPlan make_pages_plan(int, int, int, int) { return PagesPlan{kAlign}; }

sffn_status run_attn_pages(const PagesArgs &a, const PagesPlan &, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16)
        e = head_dim == 128 ? launch_pages<__nv_bfloat16, 128>(a, s) : launch_pages<__nv_bfloat16, 64>(a, s);
    else
        e = head_dim == 128 ? launch_pages<float, 128>(a, s) : launch_pages<float, 64>(a, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace sffn
