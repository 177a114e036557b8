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
//
// What the 8 bits cost: one step for all columns of a page and head (and for all query heads of a key head) is coarse
// where a few columns are much larger than the others.  Of 123 chosen among 1000 pages of 16 keys (8 query heads of 128,
// random keys) 0.97 are those that the same score without rounding chooses, 0.76 with two columns of 10 times the
// size, 0.93 with two of 30 times, 0.95 with one of 100 times; the softmax weight of the chosen pages was as large in each
// (0.165 and 0.165, 0.31 and 0.30, 0.66 and 0.63, 0.78 and 0.77): rounding outwards leans to pages of large keys.
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
// head, D / 8 lanes a key: 1024 pages of 64 keys, 8 heads of 128, bf16: 22.2 us = 6.2 TB/s, 0.93 of a copy's rate.
// ---------------------------------------------------------------------------

constexpr int kBoundsWarps = 4;

// Largest and least of eight columns, NaN once one is: bf16 stays packed (half the registers, a quarter of the instructions).
template <typename T>
struct Extremes;

template <>
struct Extremes<float> {
    float hi[8], lo[8];
    SFFN_DEV void clear() {
#pragma unroll
        for (int e = 0; e < 8; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
    }
    SFFN_DEV void add(const float *p) {
        float x[8];
        load8(p, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) hi[e] = max_nan(hi[e], x[e]), lo[e] = min_nan(lo[e], x[e]);
    }
    SFFN_DEV void get(float (&h)[8], float (&l)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = hi[e], l[e] = lo[e];
    }
};

template <>
struct Extremes<__nv_bfloat16> {
    uint32_t hi[4], lo[4];
    SFFN_DEV void clear() {
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[e] = 0xff80ff80u, lo[e] = 0x7f807f80u;
    }
    SFFN_DEV void add(const __nv_bfloat16 *p) {
        const uint4 u = ldg_stream(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi[e]) : "r"(w[e]));
            asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo[e]) : "r"(w[e]));
        }
    }
    SFFN_DEV void get(float (&h)[8], float (&l)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[2 * e] = bf16lo(hi[e]), h[2 * e + 1] = bf16hi(hi[e]);
            l[2 * e] = bf16lo(lo[e]), l[2 * e + 1] = bf16hi(lo[e]);
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kBoundsWarps, sizeof(T) == 2 ? 16 : 10) k_page_bounds(const BoundsArgs a) {
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
    Extremes<T> x;
    x.clear();
#pragma unroll 4
    for (int j = 0; j < ps; j += KPW) x.add(k + (size_t)j * D);
    float hi[8], lo[8];
    x.get(hi, lo);
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

// Scores are a matrix product: pages (bounds hi | lo, 2 D columns) times query rows (max(c, 0) | min(c, 0)), then the
// maximum over a token's rows.  The codes are whole numbers of at most 127 and the bounds multiples of one
// step, so bf16 holds both and the tensor cores' fp32 sums are exact.
//
// A CTA has a tile of tokens, one key head and a stretch of pages.  The tokens' rows (`rows` each: the
// group's heads, some twice so that they fill columns evenly) lie in shared memory; a warp holds 16 pages' bounds in
// registers as the 16 x 16 operand and runs all rows past them, 8 at a time.  The order of the columns is free
// in such a sum: lane c of four takes columns 8 c .. 8 c + 7 of each 32, so operands are read 16 bytes at a
// time, straight from the bounds.  (mma.sync: a decode step has 8 rows a token, where the bound is the
// bounds' bytes and not the product.)
// Consecutive tokens of one sequence (a run) read its bounds once.
// Two pieces of 1045 tokens of 28/4 heads of 128 over 560 pages: 38 us of scores (30 % of the tensor rate of an SM's cycles, 26 % of its
// issue slots: latency of the operands), 12 of choice; on the CUDA cores, a thread a page, 5.9 ms.
constexpr int kScoreWarps = 4;
constexpr int kScorePages = 16 * kScoreWarps;  // pages of a CTA at a time
constexpr int kScoreRows = 64;                 // rows of a CTA at most

SFFN_DEV void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// tile: tokens of a CTA (tile * rows <= kScoreRows, or one token); rows: of a token, 1, 2, 4 or a multiple of 8;
// stretch: pages of a CTA.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kScoreWarps) k_page_scores(const SelectPagesArgs a, int tile, int rows, int stretch) {
    constexpr int NB = 4;                // products of 8 rows at a time (chains of sums for the tensor cores to work on)
    constexpr int kStride = 2 * D + 32;  // elements of a row (64 bytes apart mod 128: no bank conflicts)
    constexpr int KB = 2 * D / 32;       // blocks of 32 columns
    __shared__ __align__(16) __nv_bfloat16 s_code[kScoreRows][kStride];
    __shared__ int s_seq[kScoreRows], s_last[kScoreRows];  // a token's sequence, and its last page with a score
    griddep_wait();
    griddep_launch_dependents();
    const int t0 = blockIdx.x * tile, nt = min(tile, a.T - t0), h = blockIdx.z, p0 = blockIdx.y * stretch;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < tile) {
        Token k{0, -1};
        if (tid < nt) k = token_of(a.at, t0 + tid, nullptr);
        s_seq[tid] = k.seq;
        s_last[tid] = k.mine + 1 <= a.n_keep ? -1 : k.mine - a.n_recent;  // with fewer pages all are taken
    }
    __syncthreads();
    bool any = false;
    for (int i = 0; i < nt; ++i) any |= s_last[i] >= p0;
    if (!any) return;
    // codes: a warp a token
    for (int i = warp; i < nt; i += kScoreWarps) {
        const T *q = static_cast<const T *>(a.q) + (size_t)(t0 + i) * a.q_stride + (size_t)h * a.group * D;
        const int units = a.group * D / 8;  // of 8 elements
        float most = 0.f;
        for (int u = lane; u < units; u += 32) {
            float x[8];
            load8(q + u * 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(within(x[e], 0.f)));
        }
        const float inv = pow2(-step_exponent(warp_max(most)));
        for (int u = lane; u < rows * D / 8; u += 32) {
            const int r = u * 8 / D, d = u * 8 % D;
            float x[8];
            load8(q + (r % a.group) * D + d, x);
            uint32_t up[4], dn[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = rintf(within(x[2 * e], 0.f) * inv), x1 = rintf(within(x[2 * e + 1], 0.f) * inv);
                __nv_bfloat162 pu = __floats2bfloat162_rn(fmaxf(x0, 0.f), fmaxf(x1, 0.f)),
                               pd = __floats2bfloat162_rn(fminf(x0, 0.f), fminf(x1, 0.f));
                up[e] = *reinterpret_cast<uint32_t *>(&pu);
                dn[e] = *reinterpret_cast<uint32_t *>(&pd);
            }
            *reinterpret_cast<uint4 *>(&s_code[i * rows + r][d]) = make_uint4(up[0], up[1], up[2], up[3]);
            *reinterpret_cast<uint4 *>(&s_code[i * rows + r][D + d]) = make_uint4(dn[0], dn[1], dn[2], dn[3]);
        }
    }
    __syncthreads();
    const int g = lane >> 2, c = lane & 3;  // row of the operands, and which columns
    const int reduce = rows >= 8 ? 4 : rows / 2;  // lanes that hold a token's columns (0: each its own two)
    for (int r0 = 0, r1; r0 < nt; r0 = r1) {  // runs
        int last = s_last[r0];
        for (r1 = r0 + 1; r1 < nt && s_seq[r1] == s_seq[r0]; ++r1) last = max(last, s_last[r1]);
        const int end = min(p0 + stretch, last + 1);
        for (int pb = p0 + warp * 16; pb < end; pb += kScorePages) {
            uint4 x[KB], y[KB];  // the bounds of pages pb + g and pb + g + 8
            const int32_t *table = a.at.page_table + (size_t)s_seq[r0] * a.at.table_width + pb + g;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int pg = pb + g + 8 * half < end ? table[8 * half] : -1;
                const bool there = pg >= 0 && pg < a.at.n_pages;
                if (!there && c == 0 && pb + g + 8 * half < end) record_error(a.err, SFFN_ERR_DEVICE);
                const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(a.bounds) +
                                         ((size_t)(there ? pg : 0) * a.n_kv_heads + h) * 2 * D + c * 8;
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (there) v = ldg_v4(b + k * 32);
                    (half ? y : x)[k] = v;
                }
            }
            float *dst = a.scores + ((size_t)t0 * a.n_kv_heads + h) * a.at.table_width + pb + g;
            const int step = a.n_kv_heads * a.at.table_width;  // (64 tokens of it at most: below 2^31)
            auto put = [&](int i, int half, float v) {  // token i of the tile
                const int page = pb + g + 8 * half;
                if (i >= r0 && i < r1 && page <= s_last[i] && page < end) dst[i * step + 8 * half] = v;
            };
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const int n0 = r0 * rows / 8, n1 = (r1 * rows + 7) / 8;
            for (int nb = n0; nb < n1; nb += NB) {
                float d[NB][4];
#pragma unroll
                for (int j = 0; j < NB; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    uint4 z[NB];
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        z[j] = *reinterpret_cast<const uint4 *>(&s_code[min(nb + j, n1 - 1) * 8 + g][c * 8 + k * 32]);
#pragma unroll
                    for (int j = 0; j < NB; ++j) mma_16x8x16(d[j], x[k].x, y[k].x, x[k].y, y[k].y, z[j].x, z[j].y);
#pragma unroll
                    for (int j = 0; j < NB; ++j) mma_16x8x16(d[j], x[k].z, y[k].z, x[k].w, y[k].w, z[j].z, z[j].w);
                }
                // Tokens of 8 or 4 rows: the four lanes of a page share the maxima of the four products out among
                // them (each sends what another keeps), so that every lane writes.
                auto best = [&](int half, float (&u)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[j] = fmaxf(d[j][2 * half], d[j][2 * half + 1]);
                    // lane c keeps products j of its own parity
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, c & 1 ? u[j] : u[j + 1], 1);
                        u[j / 2] = fmaxf(c & 1 ? u[j + 1] : u[j], other);
                    }
                };
                if (rows == 8) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float u[4];
                        best(half, u);
                        const float other = __shfl_xor_sync(0xffffffffu, c & 2 ? u[0] : u[1], 2);
                        put(nb + c, half, fmaxf(c & 2 ? u[1] : u[0], other));  // product c: its parity, and its half
                    }
                    continue;
                }
                if (rows == 4) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float u[4];
                        best(half, u);
                        put((nb + (c & 1)) * 2 + (c >> 1), half, u[0]);
                        put((nb + 2 + (c & 1)) * 2 + (c >> 1), half, u[1]);
                    }
                    continue;
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int n = nb + j;
                    if (n >= n1) break;
                    float (&f)[4] = d[j];
                    // f[0], f[1]: page g, rows 2 c and 2 c + 1; f[2], f[3]: page g + 8
                    if (rows > 8) {  // several products a token
#pragma unroll
                        for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], f[e]);
                        if ((n + 1) * 8 % rows) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = m[e], m[e] = -INFINITY;
                    }
                    if (rows == 1) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) put(n * 8 + 2 * c + (e & 1), e >> 1, f[e]);
                        continue;
                    }
                    float u = fmaxf(f[0], f[1]), v = fmaxf(f[2], f[3]);
                    for (int o = 1; o < reduce; o <<= 1) {
                        u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                    }
                    const int i = (n * 8 + 2 * c) / rows;
                    if (c % reduce == 0) {
                        put(i, 0, u);
                        put(i, 1, v);
                    }
                }
            }
        }
    }
}

// One token and a group of at most 8 heads: a warp makes the codes that its lanes need in registers (row g, columns 8 c and
// on of each 32, for both bounds), while its pages' bounds are on their way; no warp waits for another.  One token of 64/8 heads over
// 1024 pages 8.3 us a call (by k_page_scores 11.1), 48 tokens of up to 1000 pages, 32/8 heads, 20.8 (28.3): 70 MB of bounds in
// 17 us = 4.1 TB/s, then 8 of choice.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kScoreWarps) k_page_scores_one(const SelectPagesArgs a, int stretch) {
    constexpr int KB = D / 32;  // blocks of 32 columns of a bound
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x, h = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int p0 = blockIdx.y * stretch + warp * 16;
    float q[KB][8];
    const T *src = static_cast<const T *>(a.q) + (size_t)t * a.q_stride + ((size_t)h * a.group + min(g, a.group - 1)) * D + c * 8;
#pragma unroll
    for (int k = 0; k < KB; ++k) load8(src + k * 32, q[k]);
    const Token tok = token_of(a.at, t, nullptr);
    const int last = tok.mine + 1 <= a.n_keep ? -1 : tok.mine - a.n_recent;  // with fewer pages all are taken
    const int end = min((int)(blockIdx.y + 1) * stretch, last + 1);
    if (p0 >= end) return;
    const int32_t *table = a.at.page_table + (size_t)tok.seq * a.at.table_width;
    uint4 x[2 * KB], y[2 * KB];  // the bounds of pages pb + g and pb + g + 8
    auto load = [&](int pb) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int page = pb + g + 8 * half, pg = page < end ? table[page] : -1;
            const bool there = pg >= 0 && pg < a.at.n_pages;
            if (!there && c == 0 && page < end) record_error(a.err, SFFN_ERR_DEVICE);
            const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(a.bounds) +
                                     ((size_t)(there ? pg : 0) * a.n_kv_heads + h) * 2 * D + c * 8;
#pragma unroll
            for (int k = 0; k < 2 * KB; ++k) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (there) v = ldg_stream(b + k * 32);
                (half ? y : x)[k] = v;
            }
        }
    };
    load(p0);
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[k][e] = within(q[k][e], 0.f), most = fmaxf(most, fabsf(q[k][e]));
    const float inv = pow2(-step_exponent(warp_max(most)));
    uint32_t z[2 * KB][4];  // codes against the upper bounds, then the lower
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = rintf(q[k][2 * e] * inv), v = rintf(q[k][2 * e + 1] * inv);
            __nv_bfloat162 up = __floats2bfloat162_rn(fmaxf(u, 0.f), fmaxf(v, 0.f)), dn = __floats2bfloat162_rn(fminf(u, 0.f), fminf(v, 0.f));
            z[k][e] = *reinterpret_cast<uint32_t *>(&up);
            z[KB + k][e] = *reinterpret_cast<uint32_t *>(&dn);
        }
    float *dst = a.scores + ((size_t)t * a.n_kv_heads + h) * a.at.table_width + g;
    for (int pb = p0; pb < end; pb += kScorePages) {
        if (pb != p0) load(pb);
        float d[2][4] = {};
#pragma unroll
        for (int k = 0; k < 2 * KB; ++k) {
            mma_16x8x16(d[0], x[k].x, y[k].x, x[k].y, y[k].y, z[k][0], z[k][1]);
            mma_16x8x16(d[1], x[k].z, y[k].z, x[k].w, y[k].w, z[k][2], z[k][3]);
        }
        // (the sum of two exact sums is exact, too)
        float u = fmaxf(d[0][0] + d[1][0], d[0][1] + d[1][1]), v = fmaxf(d[0][2] + d[1][2], d[0][3] + d[1][3]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        }
        if (c == 0 && pb + g < end) dst[pb] = u;
        if (c == 1 && pb + g + 8 < end) dst[pb + 8] = v;
    }
}

// ---------------------------------------------------------------------------
// Choice: NW warps a token and key head, the scores in registers.  The cut (the `need`-th largest key) is found bit
// by bit from the highest that differs: the largest value that at least `need` keys reach; when exactly
// `need` do, that is the choice.  Each warp holds consecutive pages, 32 at a time, so ballots give the ascending
// order.
// ---------------------------------------------------------------------------

// Rows of a CTA.
template <int NW>
struct ChooseRows {
    static constexpr int value = NW == 1 ? 4 : 1;
};

template <int NW, int R>
__global__ void __launch_bounds__(32 * NW * ChooseRows<NW>::value) k_page_choose(const SelectPagesArgs a) {
    constexpr int NT = 32 * NW;
    __shared__ int s_count[32], s_above[NW], s_equal[NW];
    __shared__ uint32_t s_most[NW], s_least[NW];
    griddep_wait();
    griddep_launch_dependents();
    const unsigned row = NW == 1 ? blockIdx.x * ChooseRows<NW>::value + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= (unsigned)a.T * (unsigned)a.n_kv_heads) return;
    const int t = (int)(row / (unsigned)a.n_kv_heads), h = (int)(row - (unsigned)t * (unsigned)a.n_kv_heads);
    const int tid = NW == 1 ? threadIdx.x & 31 : threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Token k = token_of(a.at, t, h == 0 && tid == 0 ? a.err : nullptr);
    const int n = min(k.mine + 1, a.n_keep);
    int32_t *sel = a.sel + (size_t)row * a.n_keep;
    if (h == 0 && tid == 0) a.n_sel[t] = n;
    for (int i = n + tid; i < a.n_keep; i += NT) sel[i] = -1;
    if (k.mine + 1 <= a.n_keep) {
        for (int i = tid; i < n; i += NT) sel[i] = i;
        return;
    }
    const int need = a.n_keep - a.n_first - a.n_recent;
    const int c0 = a.n_first, c1 = k.mine - a.n_recent + 1;  // candidates [c0, c1), more than `need`
    for (int i = tid; i < a.n_first; i += NT) sel[i] = i;
    for (int i = tid; i < a.n_recent; i += NT) sel[a.n_keep - a.n_recent + i] = c1 + i;
    if (need == 0) return;
    const float *score = a.scores + (size_t)row * a.at.table_width;
    uint32_t key[R], most = 1, least = 0xffffffffu;  // in the order of the scores; 0: not a candidate
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int page = (warp * R + r) * 32 + lane;
        key[r] = 0;
        if (page >= c0 && page < c1) {
            const uint32_t b = __float_as_uint(__ldcg(score + page) + 0.f);  // (-0 is 0)
            key[r] = max(1u, b & 0x80000000u ? ~b : b | 0x80000000u);
            most = max(most, key[r]);
            least = min(least, key[r]);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if constexpr (NW > 1) {
        if (tid < 32) s_count[tid] = 0;
        if (lane == 0) s_most[warp] = most, s_least[warp] = least;
        __syncthreads();
        for (int w = 0; w < NW; ++w) most = max(most, s_most[w]), least = min(least, s_least[w]);
    }
    // every candidate has the bits of `least` above the highest that differs
    int bit = most == least ? -1 : 31 - __clz(most ^ least);
    uint32_t cut = bit < 0 ? least : least & ~((2u << bit) - 1u);
    bool exact = false;  // those that reach `cut` are the choice
    for (; bit >= 0 && !exact; --bit) {
        const uint32_t v = cut | (1u << bit);
        int m = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) m += key[r] >= v;
        m = __reduce_add_sync(0xffffffffu, m);
        if constexpr (NW > 1) {
            if (lane == 0 && m) atomicAdd(&s_count[bit], m);
            __syncthreads();
            m = s_count[bit];
        }
        if (m >= need) cut = v;
        exact = m == need;
    }
    if (exact) --cut;  // nothing at the cut is taken: all above it is
    int before = 0, ties = 0, spare = 0;  // above the cut and at it in the warps before this one; of the latter, how many are taken
    if constexpr (NW > 1) {
        int above = 0, equal = 0, all = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) above += key[r] > cut, equal += key[r] == cut;
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
        __syncthreads();
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += s_above[w], ties += s_equal[w];
            all += s_above[w];
        }
        spare = need - all;
    } else if (!exact) {
        int above = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) above += key[r] > cut;
        spare = need - __reduce_add_sync(0xffffffffu, above);
    }
    int at = a.n_first + before + min(ties, spare);
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t up = __ballot_sync(0xffffffffu, key[r] > cut), eq = __ballot_sync(0xffffffffu, key[r] == cut);
        // the first of those at the cut
        const bool tie = key[r] == cut && ties + __popc(eq & below) < spare;
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
    const int width = a.at.table_width, G = a.group;
    int rows = G > 4 ? (G + 7) / 8 * 8 : (G > 2 ? 4 : G);
    int tile = 1;  // as many tokens as a sequence has in the mean, as far as their rows go
    while (2 * tile * rows <= kScoreRows && 2 * tile * a.at.n_seq <= a.T) tile *= 2;
    const bool alone = tile == 1 && G <= 8;
    // Stretches of pages so that every SM has several CTAs: many where a token is alone (its sequence may be short, and
    // most of them empty; 48 tokens: 20.8 us with 24 an SM, 21.2 with 8, 21.7 with 72), fewer where the codes of many tokens are made
    // for each (1045 tokens: 51.6 us with 2, 55.1 with 4).
    const long long tiles = ((long long)a.T + tile - 1) / tile * a.n_kv_heads, fill = (tile == 1 ? 24LL : 2LL) * device_sm_count();
    long long cut = (fill + tiles - 1) / tiles;
    const int most = (width + kScorePages - 1) / kScorePages;
    if (cut > most) cut = most;
    const int stretch = (most + (int)cut - 1) / (int)cut * kScorePages;
    const dim3 grid((unsigned)((a.T + tile - 1) / tile), (unsigned)((width + stretch - 1) / stretch), (unsigned)a.n_kv_heads);
    cudaError_t e = alone ? launch_k(k_page_scores_one<T, D>, grid, dim3(32 * kScoreWarps), 0, s, a, stretch)
                          : launch_k(k_page_scores<T, D>, grid, dim3(32 * kScoreWarps), 0, s, a, tile, rows, stretch);
    if (e != cudaSuccess) return e;
    const unsigned lists = (unsigned)a.T * (unsigned)a.n_kv_heads;
    if (width <= 1024) {  // a warp a list where there are enough of them (4180 lists: 51.6 us, with eight 64.9; 384: 22.0 and 20.8)
        if (lists >= 16u * (unsigned)device_sm_count())
            return launch_k(width <= 512 ? k_page_choose<1, 16> : k_page_choose<1, 32>, dim3((lists + 3) / 4), dim3(128), 0, s, a);
        return launch_k(k_page_choose<8, 4>, dim3(lists), dim3(256), 0, s, a);
    }
    if (width <= 4096) return launch_k(k_page_choose<16, 8>, dim3(lists), dim3(512), 0, s, a);
    return launch_k(k_page_choose<32, 32>, dim3(lists), dim3(1024), 0, s, a);
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
