// attn_prompt.cu -- causal attention over packed prompts (sm_103a): attn_tc.cuh over
// contiguous keys.
//
// Bound: the tensor cores for long prompts (4 D operations a visible (query, key)
// pair), latency for short ones.  Measured (a call among others, from Python): one prompt of 16384, 64/8
// heads of 128: 2.87 ms, 1.53 PFLOP/s (0.81 of cuBLAS's measured burst); 13 ragged prompts of 9075 tokens, 28/4
// heads: 84.5 us; prompts of 2048, 1777 and 1, 32 heads of 64: 55 us; prompts of 1 to 130 tokens: 9.9 us.
//
// Work.  An item is 2 TB tokens (TB = 128 / G) of one sequence with every query head
// of one key head; it runs over the keys up to its last token.  The longest items go
// first: a sequence's tokens form blocks 0, 1, ... of growing cost, and the items are
// taken by falling block number over all sequences, dealt to the CTAs in turn,
// forwards and backwards alternately (two successive rounds cancel the difference
// between the first and the last CTA of a round).  The order needs no sort: the number of
// blocks at or above a number is known from the lengths, and a warp walks down the
// distinct block counts (PromptPolicy::next).  It keeps its place among the sequences from item to item, so it
// reads the lengths once for each distinct block count and once at most for each block number, 256 lengths at a
// time: 16384 prompts of 16 tokens, 16/8 heads of 128, 3.6 ms (with a search from the first sequence for every item 68 ms,
// and fifteen times that for four times the prompts).
#include "attn_tc.cuh"

namespace sffn {

namespace {

template <int D>
using Cfg = atc::Cfg<D, D == 128 ? 4 : 8, false, false>;  // 224 KB and 192 KB of shared memory

template <int D>
struct PromptPolicy {
    static constexpr bool kReread = true;
    const PromptArgs &a;
    int G, TB;
    // The walk's place: blocks [nxt, top] of the `cnt` sequences that have them; `before` pairs
    // (sequence, block) come ahead of this stretch, and `rank0` of the `cnt` sequences lie before sequence `s0`.
    // Items stay below 2^30: T <= 2^20, 1024 heads.
    int before, round, top, nxt, cnt, s0, rank0;

    SFFN_DEV PromptPolicy(const PromptArgs &args) : a(args), G(args.group), TB(128 / args.group) {}

    // Sequence s's first row, and its tokens (none if it breaks the contract or is past the last).
    SFFN_DEV int tokens(int s, int &t0) const {
        t0 = 0;
        if (s >= a.n_seq) return 0;
        t0 = a.cu_seqlens[s];
        const int t1 = a.cu_seqlens[s + 1];
        return t0 < 0 || t1 > a.T || t1 < t0 ? 0 : t1 - t0;
    }
    SFFN_DEV int tokens(int s) const {
        int t0;
        return tokens(s, t0);
    }
    // Sequences with `limit` blocks or more, and the largest count below it.
    SFFN_DEV void stretch(int limit) {
        int above = 0, below = 0;
#pragma unroll 8
        for (int s = threadIdx.x & 31; s < a.n_seq; s += 32) {
            const int b = (tokens(s) + 2 * TB - 1) / (2 * TB);
            if (b >= limit) ++above;
            else below = max(below, b);
        }
        cnt = __reduce_add_sync(0xffffffffu, above);
        nxt = __reduce_max_sync(0xffffffffu, below);
        s0 = rank0 = 0;
    }
    SFFN_DEV void start() {
        before = round = 0;
        top = -1;
        if (threadIdx.x >= 32) return;
        if (blockIdx.x == 0)
            for (int s = threadIdx.x; s < a.n_seq; s += 32) {
                const int t0 = a.cu_seqlens[s], t1 = a.cu_seqlens[s + 1];
                if (t0 < 0 || t1 > a.T || t1 < t0) record_error(a.err, SFFN_ERR_DEVICE);
            }
        stretch(0x7fffffff);  // nxt: the largest count
        top = nxt - 1;
        if (top >= 0) stretch(top + 1);
    }
    // The sequence of rank `rank` among those that have the stretch's blocks.
    SFFN_DEV int find(int rank) {
        constexpr int kWords = 8;
        const int lane = threadIdx.x & 31, least = top * 2 * TB;
        if (rank < rank0) s0 = rank0 = 0;  // the next lower block number begins with the first sequence again
        for (; s0 < a.n_seq; s0 += 32 * kWords) {
            int n[kWords], all = 0;
            uint32_t m[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) n[i] = tokens(s0 + 32 * i + lane);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                m[i] = __ballot_sync(0xffffffffu, n[i] > least);
                all += __popc(m[i]);
            }
            if (rank < rank0 + all) {
                int left = rank - rank0;
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int c = __popc(m[i]);
                    if (left < c) {
                        uint32_t x = m[i];
                        for (; left > 0; --left) x &= x - 1;
                        return s0 + 32 * i + __ffs(x) - 1;
                    }
                    left -= c;
                }
            }
            rank0 += all;
        }
        return 0;  // not reached: the stretch has more than `rank` sequences
    }
    SFFN_DEV bool next(atc::Work &w) {
        const int W = gridDim.x, idx = round * W + ((round & 1) ? W - 1 - (int)blockIdx.x : (int)blockIdx.x);
        const int pair = idx / a.n_kv_heads;
        ++round;
        while (top >= 0 && pair - before >= cnt * (top - nxt + 1)) {
            before += cnt * (top - nxt + 1);
            top = nxt - 1;
            if (top >= 0) stretch(top + 1);
        }
        if (top < 0) return false;
        const int off = pair - before, down = off / cnt, block = top - down;
        int t0;
        const int n = tokens(find(off - down * cnt), t0);
        const int i0 = block * 2 * TB, nt = min(2 * TB, n - i0), k1 = i0 + nt;
        w.h = idx - pair * a.n_kv_heads;
        w.i0 = i0;
        w.base = t0;
        w.q_row = t0 + i0;
        w.nt = nt;
        w.k0 = 0;
        w.k1 = k1;
        w.exist = n;
        w.tiles = (k1 + atc::kKeys - 1) / atc::kKeys;
        w.n[0] = (min(i0 + TB, n) + atc::kKeys - 1) / atc::kKeys;
        w.n[1] = nt > TB ? w.tiles : 0;
        w.mask_from[0] = (i0 + 1) / atc::kKeys;
        w.mask_from[1] = (i0 + TB + 1) / atc::kKeys;
        return true;
    }
    // Row of a key tile's first key.
    SFFN_DEV int place(const atc::Work &w, int j, int) const { return w.base + j * atc::kKeys; }
    SFFN_DEV void load_kv(const atc::Work &w, int, int row, const CUtensorMap *map, unsigned char *dst, uint64_t *bar,
                          int lane, uint64_t pol) const {
        if (lane != 0) return;
        mbar_arrive_expect_tx(bar, Cfg<D>::kTile);
        for (int c = 0; c < Cfg<D>::kHalves; ++c)
            tc::tma_load_3d(dst + c * Cfg<D>::kBlock, map, c * 64, w.h, row, bar, pol);
    }

    struct RowInfo {
        int pos;  // the row's position
    };
    SFFN_DEV RowInfo row_info(const atc::Work &w, int tok) const { return RowInfo{w.i0 + tok}; }
    SFFN_DEV void visible(const atc::Work &, const RowInfo &r, int j, uint32_t (&vis)[4]) const {
        const int n = r.pos + 1 - j * atc::kKeys;
#pragma unroll
        for (int i = 0; i < 4; ++i) vis[i] = atc::low_bits(n - 32 * i);
    }
    SFFN_DEV const void *value_row(const atc::Work &w, const RowInfo &r, int key) const {
        if (key > r.pos) return nullptr;
        return static_cast<const uint16_t *>(a.v) + (size_t)(w.base + key) * a.v_stride + (size_t)w.h * D;
    }
    SFFN_DEV bool partial(const atc::Work &) const { return false; }
    SFFN_DEV unsigned char *begin_row(const atc::Work &w, int tok, int head, bool valid, float, float l,
                                      float &inv) const {
        inv = 1.f / l;
        if (!valid) return nullptr;
        return reinterpret_cast<unsigned char *>(static_cast<uint16_t *>(a.out) +
                                                 ((size_t)(w.q_row + tok) * a.n_heads + (size_t)w.h * G + head) * D);
    }
};

template <int D>
__global__ void __launch_bounds__(atc::kThreads, 1)
    k_attn_prompt(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const PromptArgs a) {
    extern __shared__ unsigned char smem_raw[];
    PromptPolicy<D> policy(a);
    atc::attention_cta<Cfg<D>, D>(policy, map_q, map_k, map_v, map_o, a.scale, a.group, a.err, smem_raw);
}

template <int D>
sffn_status launch_prompt(const PromptArgs &a, cudaStream_t s) {
    const int G = a.group, TB = 128 / G;
    CUtensorMap mq, mk, mv, mo;
    const uint64_t dq[3] = {D, (uint64_t)a.n_heads, (uint64_t)a.T}, dk[3] = {D, (uint64_t)a.n_kv_heads, (uint64_t)a.T};
    const uint64_t sq[2] = {D * 2, (uint64_t)a.q_stride * 2}, sk[2] = {D * 2, (uint64_t)a.k_stride * 2},
                   sv[2] = {D * 2, (uint64_t)a.v_stride * 2}, so[2] = {D * 2, (uint64_t)a.n_heads * D * 2};
    const uint32_t bq[3] = {64, (uint32_t)G, (uint32_t)TB}, bk[3] = {64, 1, atc::kKeys};
    if (!make_map_bf16(&mq, a.q, 3, dq, sq, bq) || !make_map_bf16(&mk, a.k, 3, dk, sk, bk) ||
        !make_map_bf16(&mv, a.v, 3, dk, sv, bk) || !make_map_bf16(&mo, a.out, 3, dq, so, bq))
        return SFFN_ERR_UNSUPPORTED;
    // at most one partial block per sequence
    const long long items = ((long long)a.T / (2 * TB) + a.n_seq) * a.n_kv_heads;
    const int grid = (int)(items < device_sm_count() ? items : device_sm_count());
    cudaError_t e = set_max_smem((const void *)k_attn_prompt<D>, Cfg<D>::kSmem);
    if (e == cudaSuccess)
        e = launch_k(k_attn_prompt<D>, dim3(grid), dim3(atc::kThreads), Cfg<D>::kSmem, s, mq, mk, mv, mo, a);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace

sffn_status run_attn_prompt(const PromptArgs &a, int head_dim, cudaStream_t s) {
    return head_dim == 128 ? launch_prompt<128>(a, s) : launch_prompt<64>(a, s);
}

}  // namespace sffn
