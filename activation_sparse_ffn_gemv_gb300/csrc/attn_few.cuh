// attn_few.cuh -- attention of few query rows (a token's query heads, a few drafted tokens) over a
// long run of cached keys, bf16.
//
//   o_r = sum_j w_rj v_j / sum_j w_rj,  w_rj = exp(scale q_r . k_j - m_r)
//
// With 8 rows a key the bound is HBM, the keys and values read once, and what keeps a kernel from it is
// latency: where an item begins (its pages are looked up, its first keys come), where it ends (the
// parts are joined and written).  So each warp works on its own: it has a ring of 16-key tiles that it fills by
// TMA from one lane, and goes on loading the next item while it finishes one; two CTAs of four warps share an SM.
//
// The products are mma.sync with the keys as the 16-row operand and the rows as the 8 columns (tcgen05 tiles
// have 128 rows; 8 of them would be used): S^T = K Q^T, then O^T += V^T P^T, V's operand read transposed by
// ldmatrix and P^T made of S^T's registers by two 8 x 8 transpositions.  A tile of 16 keys costs a warp
// 16 products of D = 128 for every 8 rows.  The four warps of a CTA take the tiles of a piece in turn and join
// their results (maximum, sum, row) in shared memory at its end.
//
// A weight of zero times an infinite or NaN value would be NaN: where a tile has keys that some row does not see and
// V holds such a value, its product is made value by value, leaving out what a row does not see.
#pragma once

#include "attn.cuh"
#include "tcgen05.cuh"

namespace sffn {
namespace few {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;           // keys of a tile
constexpr float kLazyLog2 = 8.f;    // the running maximum moves when passed by 2^8

template <int D>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;               // bytes of K or V
    static constexpr int kStages = D == 128 ? 3 : 6;          // K and V pairs of a warp's ring
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kPad = 68;                           // floats of a row of 64 columns in the join
    static constexpr int kJoin = kWarps * 8 * kPad * 4;
    static constexpr int kSmem = kRing + kJoin + 1024 /*alignment*/;
};

// A piece of an item: `nt` tokens' rows of key head h against the keys at places [k0, k1).
struct Work {
    int q_row, nt;    // first token, tokens
    int r0, rows;     // first row (token * G + query head) of the row tile, rows
    int h;
    int k0, k1, all;  // keys below `all` are seen by every row
    int seq, tok0;    // the policy's own
    int whole, slot, kind;
};

SFFN_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
SFFN_DEV uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}
SFFN_DEV void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
SFFN_DEV void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
SFFN_DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
SFFN_DEV void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SFFN_DEV bool nonfinite2(uint32_t w) { return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0; }

// P: the policy.  It gives
//   bool next(Work &)          the CTA's pieces in turn (every warp walks by itself)
//   int page_of(w, key)        the cache's page behind a place; n_pages or more: none (zeros)
//   const bf16 *query(w, row)  a row's query
//   bool sees(w, row, key)     of a key at or past `all`
//   T *out_row / float *part   where a row goes (null: the other one does)
// NT: products of 8 rows; rows of a tile: 8 NT at most.
template <int D, int NT, typename P>
SFFN_DEV void attention(P &policy, const CUtensorMap &map_k, const CUtensorMap &map_v, int page_shift, int n_kv_heads,
                        float scale, int32_t *err, unsigned char *smem_raw) {
    using C = Cfg<D>;
    constexpr int NS = C::kStages, KB = D / 16;
    __shared__ uint64_t full[kWarps][NS];
    __shared__ float2 s_ml[kWarps][8 * NT];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t raw_addr = smem_u32(smem_raw), base = (raw_addr + 1023u) & ~1023u;
    unsigned char *ring = smem_raw + (base - raw_addr) + warp * NS * 2 * C::kTile;
    const uint32_t ring_addr = base + (uint32_t)(warp * NS * 2 * C::kTile);
    float *join = reinterpret_cast<float *>(smem_raw + (base - raw_addr) + C::kRing);
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < NS; ++i) mbar_init(&full[w][i], 1);
        s_abort = 0;
        mbar_fence_init();
        tc::prefetch_tensormap(&map_k);
        tc::prefetch_tensormap(&map_v);
    }
    __syncthreads();

    // ---- loads: this warp's tiles, one after the other through the pieces, NS ahead at most ----
    P ahead = policy;                    // a walk of its own
    const int box = min(kKeys, 1 << page_shift), boxes = kKeys / box;  // rows of a copy, copies of a tile
    const uint64_t keep = l2_evict_first_policy();
    Work lw;
    int li = 0, ln = 0, issued = 0;      // tile of the piece, tiles of it (for this warp), tiles issued
    int pages[2] = {0, 0};               // this lane's pages of 32 tiles from li on: tile li + lane, both halves
    bool more = true;
    auto tiles_of = [&](const Work &w) { return max(0, ((w.k1 - w.k0 + kKeys - 1) / kKeys - warp + kWarps - 1) / kWarps); };
    auto key_of = [&](const Work &w, int i) { return w.k0 + (i * kWarps + warp) * kKeys; };
    auto given_up = [&]() { return __any_sync(0xffffffffu, s_abort != 0); };
    auto issue = [&]() {
        while (more && li == ln) {
            more = ahead.next(lw);
            li = 0;
            ln = more ? tiles_of(lw) : 0;
        }
        if (!more || given_up()) return;
        if ((li & 31) == 0) {
            const int i = li + lane, key = key_of(lw, i);
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (b < boxes && i < ln && key + b * box < lw.k1) pages[b] = ahead.page_of(lw, key + b * box);
        }
        const int s = issued % NS, key = key_of(lw, li), src = li & 31;
        int n = 0;
        int row[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int pg = __shfl_sync(0xffffffffu, pages[b], src);
            if (b < boxes && key + b * box < lw.k1) {
                ++n;
                row[b] = (int)((((long long)pg * n_kv_heads + lw.h) << page_shift) + ((key + b * box) & ((1 << page_shift) - 1)));
            }
        }
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[warp][s], (uint32_t)(n * box * D * 4));
            unsigned char *dst = ring + s * 2 * C::kTile;
            for (int b = 0; b < n; ++b) {
                tc::tma_load_4d(dst + b * box * D * 2, &map_k, 0, 0, 0, row[b] >> 3, &full[warp][s], keep);
                tc::tma_load_4d(dst + C::kTile + b * box * D * 2, &map_v, 0, 0, 0, row[b] >> 3, &full[warp][s], keep);
            }
        }
        ++li;
        ++issued;
    };
    for (int i = 0; i < NS; ++i) issue();

    // Lane addresses inside a tile (8-row groups, column blocks of 64, rows of 128 bytes, chunks swizzled by the row):
    // K by rows (keys) and columns, V transposed.
    const int mi = lane >> 3, l8 = lane & 7;
    const int k_row = l8 + (mi & 1) * 8, k_col = (mi >> 1) * 8, v_row = l8 + (mi >> 1) * 8, v_col = (mi & 1) * 8;
    auto at = [&](int r, int col) {
        return (uint32_t)((r >> 3) * (D / 64) * 1024 + (col >> 6) * 1024 + (r & 7) * 128 + ((((col & 63) >> 3) ^ (r & 7)) << 4));
    };
    const float cf = scale * 1.44269504088896341f;  // the exponent in powers of two
    int used = 0, landed = 0;  // tiles taken, and those that came
    Work w;
    while (policy.next(w)) {
        uint32_t q[NT][KB][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = n * 8 + g;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(policy.query(w, w.r0 + min(row, w.rows - 1)));
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                q[n][k][0] = __ldg(src + k * 8 + c);
                q[n][k][1] = __ldg(src + k * 8 + c + 4);
            }
        }
        float o[NT][KB][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < KB; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        const int tiles = tiles_of(w);
        for (int i = 0; i < tiles; ++i, ++used) {
            const int st = used % NS, kb = key_of(w, i);
            // (once a wait has run out nothing is loaded or written any more, and the loops come to their end)
            if (!given_up()) {
                if (__all_sync(0xffffffffu, mbar_wait(&full[warp][st], (uint32_t)((used / NS) & 1)))) {
                    ++landed;
                } else if (lane == 0) {
                    s_abort = 1;
                    record_error(err, SFFN_ERR_TIMEOUT);
                }
            }
            __syncwarp();
            const uint32_t kt = ring_addr + (uint32_t)(st * 2 * C::kTile), vt = kt + C::kTile;
            float s[NT][4];
            {
                float s2[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    uint32_t a[4];
                    ldmatrix4(kt + at(k_row, k * 16 + k_col), a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(NT == 1 && (k & 1) ? s2[n] : s[n], a, q[n][k][0], q[n][k][1]);
                }
                if constexpr (NT == 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[0][e] += s2[0][e];
                }
            }
            // s[n][0], s[n][1]: key kb + g, rows 8 n + 2 c and + 1; s[n][2], s[n][3]: key kb + g + 8
            const bool masked = kb + kKeys > w.all;
            uint32_t seen = 0xffffffffu;  // bit 4 n + e
            if (masked) {
                seen = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = kb + g + (e >> 1) * 8, row = n * 8 + 2 * c + (e & 1);
                        const bool v = key < w.k1 && (key < w.all || (row < w.rows && policy.sees(w, w.r0 + row, key)));
                        if (v) seen |= 1u << (4 * n + e);
                        else s[n][e] = -INFINITY;
                    }
            }
            bool up = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) up |= (s[n][e] - m[n][e & 1]) * cf > kLazyLog2;
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                        for (int f = 4; f < 32; f <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, f));
                        if ((x - m[n][e]) * cf > kLazyLog2) {
                            const float f = ex2((m[n][e] - x) * cf);
                            m[n][e] = x;
                            l[n][e] *= f;
#pragma unroll
                            for (int k = 0; k < KB; ++k) o[n][k][e] *= f, o[n][k][e + 2] *= f;
                        }
                    }
            }
            // The weights are rounded to bf16 because the second product takes both operands in one type and V
            // is bf16 (as in the tensor-core kernels: an output is off by 2^-8 of sum w|v| at most); the sums
            // are of the unrounded ones.
            float p[NT][4];
            uint32_t pt[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float me = m[n][e & 1];
                    p[n][e] = ex2(fmaf(s[n][e], cf, me == -INFINITY ? 0.f : -me * cf));
                    l[n][e & 1] += p[n][e];
                }
                pt[n][0] = transpose8(pack_bf16(p[n][0], p[n][1]));
                pt[n][1] = transpose8(pack_bf16(p[n][2], p[n][3]));
            }
            bool plain = true;
            if (masked) {
                bool bad = false;
                const uint4 *v = reinterpret_cast<const uint4 *>(ring + st * 2 * C::kTile + C::kTile);
                for (int e = lane; e < C::kTile / 16; e += 32) {
                    const uint4 x = v[e];
                    bad |= nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
                }
                plain = !__any_sync(0xffffffffu, bad);
            }
            if (plain) {
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    uint32_t a[4];
                    ldmatrix4_trans(vt + at(v_row, k * 16 + v_col), a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(o[n][k], a, pt[n][0], pt[n][1]);
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < kKeys; ++j) {
                    const int src = (j & 7) * 4 + c;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const bool hi = j >= 8;
                        const float x0 = __shfl_sync(0xffffffffu, hi ? p[n][2] : p[n][0], src),
                                    x1 = __shfl_sync(0xffffffffu, hi ? p[n][3] : p[n][1], src);
                        const uint32_t vis = __shfl_sync(0xffffffffu, seen, src) >> (4 * n + (hi ? 2 : 0));
                        const float w0 = __bfloat162float(__float2bfloat16_rn(x0)), w1 = __bfloat162float(__float2bfloat16_rn(x1));
#pragma unroll
                        for (int k = 0; k < KB; ++k)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int d = k * 16 + g + half * 8;
                                const uint16_t b = *reinterpret_cast<const uint16_t *>(ring + st * 2 * C::kTile + C::kTile +
                                                                                       at(j, d & ~7) + (d & 7) * 2);
                                const float v = __uint_as_float((uint32_t)b << 16);
                                if (vis & 1) o[n][k][half * 2] += w0 * v;
                                if (vis & 2) o[n][k][half * 2 + 1] += w1 * v;
                            }
                    }
                }
            }
            __syncwarp();  // every lane has read the tile
            issue();
        }
        // ---- join the warps' results ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[n][e];
#pragma unroll
                for (int f = 4; f < 32; f <<= 1) x += __shfl_xor_sync(0xffffffffu, x, f);
                if (g == 0) s_ml[warp][n * 8 + 2 * c + e] = make_float2(m[n][e], x);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n * 8 >= w.rows) break;
#pragma unroll
            for (int dh = 0; dh < D / 64; ++dh) {
                float *mine = join + warp * 8 * C::kPad;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mine[(2 * c + (e & 1)) * C::kPad + k * 16 + g + (e >> 1) * 8] = o[n][dh * 4 + k][e];
                __syncthreads();
                const int row = tid >> 4, col = (tid & 15) * 4;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) M = fmaxf(M, s_ml[x][n * 8 + row].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float2 ml = s_ml[x][n * 8 + row];
                    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2((ml.x - ref) * cf);  // (no key: no weight)
                    const float4 y = *reinterpret_cast<const float4 *>(join + (x * 8 + row) * C::kPad + col);
                    L += f * ml.y;
                    v.x += f * y.x, v.y += f * y.y, v.z += f * y.z, v.w += f * y.w;
                }
                if (n * 8 + row < w.rows && !s_abort) {
                    float *part = policy.part_row(w, w.r0 + n * 8 + row, n * 8 + row, M * scale, L, dh == 0 && col == 0);
                    if (part) {
                        *reinterpret_cast<float4 *>(part + dh * 64 + col) = v;
                    } else {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        *reinterpret_cast<uint2 *>(policy.out_row(w, w.r0 + n * 8 + row) + dh * 64 + col) =
                            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
                    }
                }
                __syncthreads();
            }
        }
    }
    // no copy is in flight when the CTA exits, whoever gave up
    for (int i = landed; i < issued; ++i) mbar_wait(&full[warp][i % NS], (uint32_t)((i / NS) & 1));
}

}  // namespace few
}  // namespace sffn
