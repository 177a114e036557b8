// The tensor-core attention kernels with a loading warp that leaves out one load: the wait for it runs
// out, and the kernel has to report that and end.  PAGED selects the draft-tree kernel's source.
#ifdef PAGED
#include "attn_tree.cu"
#else
#include "attn_prompt.cu"
#endif

namespace sffn {
namespace {

// The policy P without a CTA's load number `skip` (from 0).
template <typename P>
struct LeavesOut : P {
    int left;
    template <typename... A>
    SFFN_DEV explicit LeavesOut(int skip, A &&...args) : P(args...), left(skip) {}
    template <typename... A>
    SFFN_DEV void load_kv(A &&...args) {
        if (left-- != 0) P::load_kv(args...);
    }
};

constexpr int kD = 128;

template <typename K, typename... A>
int launch(K *kernel, int grid, int smem, cudaStream_t s, A... args) {
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_k(kernel, dim3(grid), dim3(atc::kThreads), smem, s, args...);
    return (int)e;
}

#ifndef PAGED
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_prompt(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
             const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const PromptArgs a, int skip) {
    extern __shared__ unsigned char smem_raw[];
    LeavesOut<PromptPolicy<kD>> policy(skip, a);
    atc::attention_cta<Cfg<kD>, kD>(policy, mq, mk, mv, mo, a.scale, a.group, a.err, smem_raw);
}
#else
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_tree(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
           const __grid_constant__ CUtensorMap mv, const TreeArgs a, int skip) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ long long scratch[33];
    LeavesOut<TreePolicy<kD>> policy(skip, a, reinterpret_cast<long long *>(smem_raw), scratch);
    atc::attention_cta<Cfg<kD>, kD>(policy, mq, mk, mv, mq, a.scale, a.group, a.err, smem_raw + kPrefixBytes);
}
#endif

}  // namespace
}  // namespace sffn

using namespace sffn;

#ifndef PAGED
// q, k, v and out contiguous, heads of 128.
extern "C" int run_leaving_out(const void *q, const void *k, const void *v, int T, int hq, int hkv, const int32_t *cu,
                               int n_seq, float scale, void *out, int32_t *err, int skip, void *stream) {
    PromptArgs a = {};
    a.q = q, a.k = k, a.v = v, a.out = out, a.cu_seqlens = cu, a.err = err;
    a.q_stride = hq * kD, a.k_stride = a.v_stride = hkv * kD;
    a.T = T, a.n_heads = hq, a.n_kv_heads = hkv, a.group = hq / hkv, a.n_seq = n_seq, a.scale = scale;
    const uint64_t dq[3] = {kD, (uint64_t)hq, (uint64_t)T}, dk[3] = {kD, (uint64_t)hkv, (uint64_t)T};
    const uint64_t sq[2] = {kD * 2, (uint64_t)hq * kD * 2}, sk[2] = {kD * 2, (uint64_t)hkv * kD * 2};
    const uint32_t bq[3] = {64, (uint32_t)a.group, (uint32_t)(128 / a.group)}, bk[3] = {64, 1, atc::kKeys};
    CUtensorMap mq, mk, mv, mo;
    if (!make_map_bf16(&mq, q, 3, dq, sq, bq) || !make_map_bf16(&mk, k, 3, dk, sk, bk) ||
        !make_map_bf16(&mv, v, 3, dk, sk, bk) || !make_map_bf16(&mo, out, 3, dq, sq, bq))
        return -1;
    return launch(k_prompt, device_sm_count(), Cfg<kD>::kSmem, (cudaStream_t)stream, mq, mk, mv, mo, a, skip);
}
#else
// q and out contiguous, heads of 128; part: the workspace's place for partial results.
extern "C" int run_leaving_out(const void *q, const void *ck, const void *cv, int T, int hq, int hkv, int page_shift,
                               int n_pages, const int32_t *table, int width, const int32_t *ctx, const int32_t *cu,
                               int n_seq, float scale, void *out, float *part, int32_t *err, int skip, void *stream) {
    const TreePlan p = make_tree_plan(SFFN_BF16, T, hq, hkv, kD);
    TreeArgs a = {};
    a.q = q, a.ck = ck, a.cv = cv, a.out = out, a.page_table = table, a.ctx_lens = ctx, a.cu_tokens = cu, a.err = err;
    a.q_stride = hq * kD, a.T = T, a.n_heads = hq, a.n_kv_heads = hkv, a.group = hq / hkv, a.n_seq = n_seq;
    a.page_shift = page_shift, a.n_pages = n_pages, a.table_width = width, a.scale = scale, a.part = part;
    a.tile_tokens = p.tile_tokens, a.rows_max = p.rows_max;
    const int ps = 1 << page_shift;
    const uint64_t dq[3] = {kD, (uint64_t)hq, (uint64_t)T}, sq[2] = {kD * 2, (uint64_t)hq * kD * 2};
    const uint64_t dk[4] = {64, 8, kD / 64, (uint64_t)n_pages * hkv * ps / 8}, sk[3] = {kD * 2, 128, kD * 16};
    const uint32_t bq[3] = {64, (uint32_t)a.group, (uint32_t)(128 / a.group)},
                   bk[4] = {64, 8, kD / 64, (uint32_t)(ps < 64 ? ps : 64) / 8};
    CUtensorMap mq, mk, mv;
    if (!make_map_bf16(&mq, q, 3, dq, sq, bq) || !make_map_bf16(&mk, ck, 4, dk, sk, bk) ||
        !make_map_bf16(&mv, cv, 4, dk, sk, bk))
        return -1;
    return launch(k_tree, p.grid, Cfg<kD>::kSmem + (int)kPrefixBytes, (cudaStream_t)stream, mq, mk, mv, a, skip);
}
#endif
