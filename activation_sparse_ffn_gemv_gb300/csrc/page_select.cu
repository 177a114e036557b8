// page_select.cu -- which pages of a long context a token reads: the pages' key bounds,
// the score of its queries against them and the choice of the best (sm_103a).
//
// Bounds of a page, per key head and column: hi >= every key >= lo, on a grid of whole
// multiples of one power of two (at most 127 of them on either side of zero).  A query is
// rounded to such a grid likewise (c, in units of its step), and
//   score(page) = max over the key head's query heads of sum_d max(c_d, 0) hi_d + min(c_d, 0) lo_d.
// Every term is a whole multiple, of at most 127 * 127, of the page's step, and there are at most 128
// that are not zero: below 2^21 of them, so any sum of terms is exact in 32 bits.  The choice
// therefore does not depend on the order in which a kernel adds, and equal scores are equal.
#include "common.cuh"
#include "internal.h"

namespace sffn {

namespace {

constexpr float kTop = 1.2676506002282294e30f;  // 2^100: larger magnitudes count as this
constexpr int kLeast = -100;                    // least exponent of a step

// e of the least step 2^e, e >= kLeast, with a <= 127 * 2^e (a finite, >= 0): with a = 1.m 2^E that is
// E - 6, and one more where 1.m > 127 / 64.
SFFN_DEV int step_exponent(float a) {
    const uint32_t b = __float_as_uint(a);
    return max(kLeast, (int)(b >> 23) - 127 - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0));
}
SFFN_DEV float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

SFFN_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
SFFN_DEV float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Into [-2^100, 2^100]; NaN to `nan`.
SFFN_DEV float within(float x, float nan) { return x != x ? nan : fminf(fmaxf(x, -kTop), kTop); }

// Eight consecutive elements as floats.
SFFN_DEV void load8(const __nv_bfloat16 *p, float (&f)[8]) {
    const uint4 u = ldg_stream(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16lo(w[i]), f[2 * i + 1] = bf16hi(w[i]);
}
SFFN_DEV void load8(const float *p, float (&f)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 u = ldg_stream(p + 4 * h);
        f[4 * h] = __uint_as_float(u.x), f[4 * h + 1] = __uint_as_float(u.y);
        f[4 * h + 2] = __uint_as_float(u.z), f[4 * h + 3] = __uint_as_float(u.w);
    }
}

// ---------------------------------------------------------------------------
// Bounds.  Bound: HBM, the pages' keys, read once.  A warp takes a page's keys of one
// head, D / 8 lanes a key.
// ---------------------------------------------------------------------------

constexpr int kBoundsWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kBoundsWarps) k_page_bounds(const BoundsArgs a) {
    constexpr int LPK = D / 8, KPW = 32 / LPK;  // lanes of a key, keys of a warp at a time
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    if (item >= (long long)a.n * a.n_kv_heads) return;
    const int i = (int)(item / a.n_kv_heads), h = (int)(item - (long long)i * a.n_kv_heads), pg = a.pages[i];
    if (pg < 0 || pg >= a.n_pages) {
        if (pg != -1 && lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
        return;
    }
    const int ps = 1 << a.page_shift, col = (lane % LPK) * 8;
    const T *k = static_cast<const T *>(a.ck) + ((((size_t)pg * a.n_kv_heads + h) << a.page_shift) + lane / LPK) * D + col;
    float hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
#pragma unroll 4
    for (int j = 0; j < ps; j += KPW) {
        float x[8];
        load8(k + (size_t)j * D, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) hi[e] = max_nan(hi[e], x[e]), lo[e] = min_nan(lo[e], x[e]);
    }
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) {
            hi[e] = max_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
            lo[e] = min_nan(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
        }
        hi[e] = within(hi[e], kTop);
        lo[e] = within(lo[e], -kTop);
        most = fmaxf(most, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
    }
    const int ex = step_exponent(warp_max(most));
    const float step = pow2(ex), inv = pow2(-ex);
    if (lane < LPK) {
        uint32_t w[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 u = __floats2bfloat162_rn(ceilf(hi[2 * e] * inv) * step, ceilf(hi[2 * e + 1] * inv) * step),
                           d = __floats2bfloat162_rn(floorf(lo[2 * e] * inv) * step, floorf(lo[2 * e + 1] * inv) * step);
            w[0][e] = *reinterpret_cast<uint32_t *>(&u);
            w[1][e] = *reinterpret_cast<uint32_t *>(&d);
        }
        uint16_t *dst = static_cast<uint16_t *>(a.bounds) + ((size_t)pg * a.n_kv_heads + h) * 2 * D + col;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
        *reinterpret_cast<uint4 *>(dst + D) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
    }
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------

// A token's pages: its own (the last), and whether the choice needs scores.
struct Token {
    int seq, mine;  // row of the page table; own page, -1: no pages
};
SFFN_DEV Token token_of(const Places &p, int t, int32_t *err) {
    Token k{p.seqs[t], -1};
    const int pos = p.positions[t];
    if (pos < 0) return k;  // padding
    if (k.seq < 0 || k.seq >= p.n_seq || (pos >> p.page_shift) >= p.table_width) {
        if (err) record_error(err, SFFN_ERR_DEVICE);
        return k;
    }
    k.mine = pos >> p.page_shift;
    return k;
}

constexpr int kScoreThreads = 128;

// A CTA: one token and key head, 128 pages, one a thread.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads) k_page_scores(const SelectPagesArgs a) {
    __shared__ float c[64][D];  // the query heads' codes
    __shared__ float s_most[kScoreThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x, h = blockIdx.z, p0 = blockIdx.y * kScoreThreads, tid = threadIdx.x;
    const Token k = token_of(a.at, t, nullptr);
    const int last = k.mine - a.n_recent;  // the last page that a score decides about
    if (k.mine + 1 <= a.n_keep || p0 > last) return;
    const T *q = static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)h * a.group * D;
    float most = 0.f;
    for (int i = tid; i < a.group * D; i += kScoreThreads) {
        const float x = within((float)q[i], 0.f);
        c[i / D][i % D] = x;
        most = fmaxf(most, fabsf(x));
    }
    most = warp_max(most);
    if ((tid & 31) == 0) s_most[tid >> 5] = most;
    __syncthreads();
    for (int w = 0; w < kScoreThreads / 32; ++w) most = fmaxf(most, s_most[w]);
    const float inv = pow2(-step_exponent(most));
    for (int i = tid; i < a.group * D; i += kScoreThreads) c[i / D][i % D] = rintf(c[i / D][i % D] * inv);
    __syncthreads();
    const int page = p0 + tid;
    if (page > last) return;
    const int pg = a.at.page_table[(size_t)k.seq * a.at.table_width + page];
    float score = 0.f;
    if (pg < 0 || pg >= a.at.n_pages) {
        record_error(a.err, SFFN_ERR_DEVICE);
    } else {
        score = -INFINITY;
        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(a.bounds) + ((size_t)pg * a.n_kv_heads + h) * 2 * D;
        for (int g = 0; g < a.group; ++g) {
            float s = 0.f;
            for (int d = 0; d < D; ++d) {
                const float x = c[g][d];
                s += x * bf16_to_f32(b[x > 0.f ? d : D + d]);
            }
            score = fmaxf(score, s);
        }
    }
    a.scores[((size_t)t * a.n_kv_heads + h) * a.at.table_width + page] = score;
}

// ---------------------------------------------------------------------------
// Choice: one CTA a token and key head, its scores in registers.  The cut (the `need`-th largest key)
// is found bit by bit: the largest value that at least `need` keys reach.  Each warp holds
// consecutive pages, 32 at a time, so ballots give the ascending order.
// ---------------------------------------------------------------------------

template <int NT, int R>
__global__ void __launch_bounds__(NT) k_page_choose(const SelectPagesArgs a) {
    constexpr int NW = NT / 32;
    __shared__ int s_count[32], s_above[NW], s_equal[NW];
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x / a.n_kv_heads, h = blockIdx.x - t * a.n_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Token k = token_of(a.at, t, h == 0 && tid == 0 ? a.err : nullptr);
    const int n = min(k.mine + 1, a.n_keep);
    int32_t *sel = a.sel + (size_t)blockIdx.x * a.n_keep;
    if (h == 0 && tid == 0) a.n_sel[t] = n;
    for (int i = n + tid; i < a.n_keep; i += NT) sel[i] = -1;
    if (k.mine + 1 <= a.n_keep) {
        for (int i = tid; i < n; i += NT) sel[i] = i;
        return;
    }
    const int need = a.n_keep - a.n_first - a.n_recent;
    const int c0 = a.n_first, c1 = k.mine - a.n_recent + 1;  // candidates [c0, c1)
    const float *score = a.scores + (size_t)blockIdx.x * a.at.table_width;
    uint32_t key[R];  // in the order of the scores; 0: not a candidate
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int page = (warp * R + r) * 32 + lane;
        key[r] = 0;
        if (page >= c0 && page < c1) {
            const uint32_t b = __float_as_uint(__ldcg(score + page) + 0.f);  // (-0 is 0)
            key[r] = b & 0x80000000u ? ~b : b | 0x80000000u;
        }
    }
    if (tid < 32) s_count[tid] = 0;
    __syncthreads();
    uint32_t cut = 0;
    if (need > 0) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t v = cut | (1u << bit);
            int m = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) m += key[r] >= v;
            m = __reduce_add_sync(0xffffffffu, m);
            if (lane == 0 && m) atomicAdd(&s_count[bit], m);
            __syncthreads();
            if (s_count[bit] >= need) cut = v;
        }
    } else {
        cut = 0xffffffffu;  // above every key
    }
    int above = 0, equal = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) above += key[r] > cut, equal += key[r] == cut;
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
    __syncthreads();
    int before = 0, ties = 0, all = 0;  // above the cut and at it, in the warps before this one; above in all
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += s_above[w], ties += s_equal[w];
        all += s_above[w];
    }
    const int spare = need - all;  // of those at the cut, the first `spare` are taken
    for (int i = tid; i < a.n_first; i += NT) sel[i] = i;
    for (int i = tid; i < a.n_recent; i += NT) sel[a.n_keep - a.n_recent + i] = c1 + i;
    int at = a.n_first + before + min(ties, spare);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t up = __ballot_sync(0xffffffffu, key[r] > cut), eq = __ballot_sync(0xffffffffu, key[r] == cut);
        const uint32_t below = (1u << lane) - 1u;
        const int my_tie = ties + __popc(eq & below);
        const bool tie = key[r] == cut && my_tie < spare;
        const uint32_t take = up | __ballot_sync(0xffffffffu, tie);
        if ((take >> lane) & 1u) sel[at + __popc(take & below)] = (warp * R + r) * 32 + lane;
        at += __popc(take);
        ties += __popc(eq);
    }
}

template <typename T, int D>
cudaError_t launch_bounds_k(const BoundsArgs &a, cudaStream_t s) {
    const long long items = (long long)a.n * a.n_kv_heads;
    return launch_k(k_page_bounds<T, D>, dim3((unsigned)((items + kBoundsWarps - 1) / kBoundsWarps)),
                    dim3(32 * kBoundsWarps), 0, s, a);
}

template <typename T, int D>
cudaError_t launch_select(const SelectPagesArgs &a, cudaStream_t s) {
    const int width = a.at.table_width;
    cudaError_t e = launch_k(k_page_scores<T, D>,
                             dim3((unsigned)a.T, (unsigned)((width + kScoreThreads - 1) / kScoreThreads), (unsigned)a.n_kv_heads),
                             dim3(kScoreThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const dim3 rows((unsigned)a.T * (unsigned)a.n_kv_heads);
    if (width <= 256 * 4) return launch_k(k_page_choose<256, 4>, rows, dim3(256), 0, s, a);
    if (width <= 256 * 16) return launch_k(k_page_choose<256, 16>, rows, dim3(256), 0, s, a);
    return launch_k(k_page_choose<1024, 32>, rows, dim3(1024), 0, s, a);
}

}  // namespace

sffn_status run_page_bounds(const BoundsArgs &a, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16)
        e = head_dim == 128 ? launch_bounds_k<__nv_bfloat16, 128>(a, s) : launch_bounds_k<__nv_bfloat16, 64>(a, s);
    else
        e = head_dim == 128 ? launch_bounds_k<float, 128>(a, s) : launch_bounds_k<float, 64>(a, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

size_t page_select_workspace(int T, int n_kv_heads, int table_width) {
    return kAlign + align_up(sizeof(float) * (size_t)T * n_kv_heads * table_width);
}

sffn_status run_page_select(const SelectPagesArgs &a, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16)
        e = head_dim == 128 ? launch_select<__nv_bfloat16, 128>(a, s) : launch_select<__nv_bfloat16, 64>(a, s);
    else
        e = head_dim == 128 ? launch_select<float, 128>(a, s) : launch_select<float, 64>(a, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace sffn
