// attn_prompt.cu -- causal attention over packed prompts (sm_103a).
#include "attn_rows.cuh"

namespace sffn {

namespace {

// One CTA: a row tile (64 / G tokens, every query head of a key head) of one sequence.
template <int D>
__global__ void __launch_bounds__(rows::kThreads, 1) k_prompt_rows(const PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rows::Smem<D> &sm = *reinterpret_cast<rows::Smem<D> *>(smem_raw);
    typedef __nv_bfloat16 T;
    griddep_wait();
    griddep_launch_dependents();
    const int G = a.group, TT = rows::kRows / G;
    const int h = blockIdx.y;
    // tile number -> sequence (a walk: this is the plain kernel)
    int left = blockIdx.x, t0 = 0, n = 0, s = 0;
    for (; s < a.n_seq; ++s) {
        t0 = a.cu_seqlens[s];
        n = a.cu_seqlens[s + 1] - t0;
        if (t0 < 0 || n < 0 || t0 + n > a.T) {
            if (h == 0 && threadIdx.x == 0) record_error(a.err, SFFN_ERR_DEVICE);
            n = 0;
        }
        const int tiles = (n + TT - 1) / TT;
        if (left < tiles) break;
        left -= tiles;
    }
    if (s == a.n_seq) return;
    const int i0 = left * TT, nt = min(TT, n - i0);
    rows::Acc<D> acc;
    rows::attend<T, D>(
        sm, acc, nt * G, 0, i0 + nt, a.scale,
        [&](int r) {
            return static_cast<const T *>(a.q) + (size_t)(t0 + i0 + r / G) * a.q_stride + (size_t)(h * G + r % G) * D;
        },
        [&](long long j, int which) -> const T * {
            return which ? static_cast<const T *>(a.v) + (size_t)(t0 + j) * a.v_stride + (size_t)h * D
                         : static_cast<const T *>(a.k) + (size_t)(t0 + j) * a.k_stride + (size_t)h * D;
        },
        [&](int r, long long j) { return j <= i0 + r / G; });
    const int tid = threadIdx.x, c = (tid % rows::Acc<D>::CT) * 4, g = tid / rows::Acc<D>::CT;
#pragma unroll
    for (int i = 0; i < rows::Acc<D>::RPT; ++i) {
        const int r = g + i * rows::Acc<D>::RG;
        if (r < nt * G) {
            const float inv = 1.f / sm.l[r];
            const float4 o = acc.o[i];
            rows::store4<T>(static_cast<T *>(a.out) +
                                ((size_t)(t0 + i0 + r / G) * a.n_heads + (size_t)(h * G + r % G)) * D + c,
                            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        }
    }
}

template <int D>
sffn_status launch_prompt(const PromptArgs &a, cudaStream_t s) {
    const int TT = rows::kRows / a.group;
    const long long tiles = (long long)a.T / TT + a.n_seq;  // at most: a partial tile per sequence
    cudaError_t e = set_max_smem((const void *)k_prompt_rows<D>, (int)sizeof(rows::Smem<D>));
    if (e == cudaSuccess)
        e = launch_k(k_prompt_rows<D>, dim3((unsigned)tiles, a.n_kv_heads), dim3(rows::kThreads),
                     sizeof(rows::Smem<D>), s, a);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace

sffn_status run_attn_prompt(const PromptArgs &a, int head_dim, cudaStream_t s) {
    return head_dim == 128 ? launch_prompt<128>(a, s) : launch_prompt<64>(a, s);
}

}  // namespace sffn
