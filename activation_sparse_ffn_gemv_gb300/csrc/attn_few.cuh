// attn_few.cuh -- attention of few query rows (a token's query heads, a few drafted tokens) over a
// long run of cached keys, bf16.
//
//   o_r = sum_j w_rj v_j / sum_j w_rj,  w_rj = exp(scale q_r . k_j - m_r)
//
// With 8 rows a key the bound is HBM, the keys and values read once, and what keeps a kernel from it is
// latency: where an item begins (its pages are looked up, its first keys come), where it ends (its rows
// are written).  So each warp works by itself, on a stretch of the line of work of its own: it has a ring of 16-key
// tiles that it fills by TMA from one lane, and goes on loading the next item while it finishes one; two CTAs
// of four warps share an SM.  (Four warps an item, joined in shared memory at its end: 3000 cycles an item for the join
// alone.)
//
// The products are mma.sync with the keys as the 16-row operand and the rows as the 8 columns (tcgen05 tiles
// have 128 rows; 8 of them would be used): S^T = K Q^T, then O^T += V^T P^T, V's operand read transposed by
// ldmatrix and P^T made of S^T's registers by two 8 x 8 transpositions.  A tile of 16 keys costs a warp
// 16 products of D = 128 for every 8 rows.  48 tokens of up to 2048 chosen positions, 32/8 heads of 128: 298 MB in 54 us with the
// join, 5.5 TB/s, 0.82 of a copy's rate (a tcgen05 tile an item: 68); 14 % of the issue slots.
//
// A weight of zero times an infinite or NaN value would be NaN: where a tile has keys that some row does not see, such
// values become zeros before the product and are added by themselves to the rows that see them.  The sums of a row
// are then the same whatever lies in places that it does not see, or in the half of a tile that a lone page of 8 leaves as it was.
#pragma once

#include "attn.cuh"
#include "tma_warp.cuh"

namespace sffn {
namespace few {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;           // keys of a tile
constexpr float kLazyLog2 = 8.f;    // the running maximum moves when passed by 2^8
constexpr uint32_t kHoldNs = 1000000;  // the hardware may hold a waiting warp for 1 ms at a time

template <int D>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;               // bytes of K or V
    static constexpr int kStages = D == 128 ? 3 : 6;          // K and V pairs of a warp's ring
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kSmem = kRing + 1024 /*alignment*/;
};

// Rows of the largest row tile (registers: 4 results a lane for every row and 64 columns).
constexpr int max_rows(int D) { return D == 128 ? 16 : 32; }

// A piece of an item: rows of key head h against the keys at places [k0, k1).
struct Work {
    int q_row;        // first token
    int r0, rows;     // first row (token * G + query head) of the row tile, rows
    int h;
    int k0, k1, all;  // keys below `all` are seen by every row
    int seq, ctx, whole, slot, kind;  // the policy's own
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
// The halves of two bf16 that are infinite or NaN (their sign bits), whether there is one, and zeros in their place.
SFFN_DEV uint32_t nonfinite_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
SFFN_DEV bool nonfinite2(uint32_t w) { return nonfinite_bits(w) != 0; }
SFFN_DEV uint32_t finite2(uint32_t w) { return w & ~((nonfinite_bits(w) >> 15) * 0xffffu); }

// At a warp's end: where it gave up, copies of its own may be in flight, and the CTA waits for those before it exits (one more
// second for all of them, in equal shares).  A wait that runs out ends its own warp's loads and stores; the other warps have rings and
// waits of their own.
template <int NS>
SFFN_DEV void drain(uint64_t (&full)[NS], int landed, int issued) {
    for (int i = landed; i < issued; ++i) mbar_wait(&full[i % NS], (uint32_t)((i / NS) & 1), kWaitLimitNs / NS);
}

// P: the policy.  It gives
//   bool next(Work &)          the warp's pieces in turn
//   int page_of(w, key)        the cache's page behind a place; n_pages or more: none (zeros)
//   const bf16 *query(w, row)  a row's query
//   bool sees(w, row, key)     of a key at or past `all`
//   bool partial(w)            whether the result is a partial one
//   bf16 *out_row(w, row)      where a row goes
//   float *part_row, part_sums where a row (`r` of the tile) of a partial result goes, and its (maximum, sum)
// NT: products of 8 rows; rows of a tile: 8 NT at most.
template <int D, int NT, typename P>
SFFN_DEV void attention(P &policy, const CUtensorMap &map_k, const CUtensorMap &map_v, int page_shift, int n_kv_heads,
                        float scale, int32_t *err, unsigned char *smem_raw) {
    using C = Cfg<D>;
    constexpr int NS = C::kStages, KB = D / 16;
    __shared__ uint64_t full[kWarps][NS];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t raw_addr = smem_u32(smem_raw), base = (raw_addr + 1023u) & ~1023u;
    unsigned char *ring = smem_raw + (base - raw_addr) + warp * NS * 2 * C::kTile;
    const uint32_t ring_addr = base + (uint32_t)(warp * NS * 2 * C::kTile);
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < NS; ++i) mbar_init(&full[w][i], 1);
        mbar_fence_init();
        tc::prefetch_tensormap(&map_k);
        tc::prefetch_tensormap(&map_v);
    }
    __syncthreads();

    // ---- loads: this warp's tiles, one after the other through the pieces, NS ahead at most ----
    P ahead = policy;                    // a walk of its own
    const int box = min(kKeys, 1 << page_shift);  // rows of a copy: a tile is one, or two of 8
    const uint64_t keep = l2_evict_first_policy();
    Work lw, nw;                         // the piece whose tiles are loaded, and the one after it
    int li = 0, ln = 0, issued = 0, islot = 0;  // tile of the piece, tiles of it, tiles issued, ring position
    int pages[2] = {0, 0}, npages[2] = {0, 0};  // this lane's pages of 32 tiles: tile (li & ~31) + lane, both halves
    int nn;                              // the next piece's tiles (-1: there is none)
    bool dead = false;                   // a wait has run out, nothing is loaded or written any more
    auto tiles_of = [&](const Work &w) { return (w.k1 - w.k0 + kKeys - 1) / kKeys; };
    auto key_of = [&](const Work &w, int i) { return w.k0 + i * kKeys; };
    auto look_up = [&](const Work &w, int i, int (&pg)[2]) {  // pages of tiles i + lane
        const int key = key_of(w, i + lane);
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (b * box < kKeys && key + b * box < w.k1) pg[b] = ahead.page_of(w, key + b * box);
    };
    auto fetch = [&]() {  // the next piece, and its first pages, a piece ahead of their use
        nn = ahead.next(nw) ? tiles_of(nw) : -1;
        if (nn > 0) look_up(nw, 0, npages);
    };
    fetch();
    auto issue = [&]() {
        while (li == ln && nn >= 0) {
            lw = nw, li = 0, ln = nn;
            pages[0] = npages[0], pages[1] = npages[1];
            fetch();
        }
        if (li == ln || dead) return;
        const int key = key_of(lw, li);
        if ((li & 31) == 0 && li > 0) look_up(lw, li, pages);
        // 8-row groups of the cache: below 2^28
        auto group = [&](int pg, int k) {
            return ((pg * n_kv_heads + lw.h) << (page_shift - 3)) + ((k & ((1 << page_shift) - 1)) >> 3);
        };
        const int g0 = group(__shfl_sync(0xffffffffu, pages[0], li & 31), key), two = box < kKeys && key + box < lw.k1;
        const int g1 = two ? group(__shfl_sync(0xffffffffu, pages[1], li & 31), key + box) : 0;
        const uint32_t bar = smem_u32(&full[warp][islot]), dst = ring_addr + (uint32_t)(islot * 2 * C::kTile);
        tc::mbar_expect_tx_warp(bar, (uint32_t)((1 + two) * box * D * 4));
        tc::tma_load_rows_warp(dst, &map_k, g0, bar, keep);
        tc::tma_load_rows_warp(dst + C::kTile, &map_v, g0, bar, keep);
        if (two) {
            tc::tma_load_rows_warp(dst + box * D * 2, &map_k, g1, bar, keep);
            tc::tma_load_rows_warp(dst + C::kTile + box * D * 2, &map_v, g1, bar, keep);
        }
        ++li;
        ++issued;
        if (++islot == NS) islot = 0;
    };
    for (int i = 0; i < NS; ++i) issue();

    // Lane addresses inside a tile (8-row groups, column blocks of 64, rows of 128 bytes, chunks swizzled by the row):
    // K by rows (keys) and columns, V transposed.
    const int mi = lane >> 3, l8 = lane & 7;
    const int k_row = l8 + (mi & 1) * 8, k_col = (mi >> 1) * 8, v_row = l8 + (mi >> 1) * 8, v_col = (mi & 1) * 8;
    // (a chunk's place is its number and the row's, exclusive-or: along a row the even chunks differ in bits 5 and 6)
    auto at = [&](int r, int col) {
        return (uint32_t)((r >> 3) * (D / 64) * 1024 + (col >> 6) * 1024 + (r & 7) * 128 + ((((col & 63) >> 3) ^ (r & 7)) << 4));
    };
    const float cf = scale * 1.44269504088896341f;  // the exponent in powers of two
    const uint32_t k_lane = at(k_row, k_col), v_lane = at(v_row, v_col);
    int landed = 0, slot = 0;  // tiles that came, ring position and its parity
    uint32_t par = 0;
    uint32_t q[NT][KB][2];
    auto load_q = [&](const Work &w) {
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
    };
    Work w, w2;
    bool have = policy.next(w);
    if (have) load_q(w);
    for (; have; w = w2) {
        float o[NT][KB][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < KB; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        const int tiles = tiles_of(w);
        for (int i = 0; i < tiles; ++i) {
            const int st = slot, kb = key_of(w, i);
            if (!dead) {
                bool came = __all_sync(0xffffffffu, mbar_try_wait(&full[warp][st], par));
                if (!came) {
                    const uint64_t t0 = globaltimer_ns();
                    while (!came && !__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs))
                        came = __all_sync(0xffffffffu, mbar_try_wait_for(&full[warp][st], par, kHoldNs));
                }
                if (came) {
                    ++landed;
                } else {
                    dead = true;
                    if (lane == 0) record_error(err, SFFN_ERR_TIMEOUT);
                }
            }
            if (++slot == NS) slot = 0, par ^= 1;
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
                    ldmatrix4(((kt + k_lane) ^ ((k & 3) << 5)) + (k >> 2) * 1024, a);
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
            if (masked) {
                // One product, whatever a row does not see: non-finite values become zeros in the tile, and are added by
                // themselves to the rows that see them.
                uint4 *v = reinterpret_cast<uint4 *>(ring + st * 2 * C::kTile + C::kTile);
                bool bad = false;
                for (int e = lane; e < C::kTile / 16; e += 32) {
                    const uint4 x = v[e];
                    bad |= nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
                }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                    for (int j = 0; j < kKeys; ++j) {
                        const int src = (j & 7) * 4 + c;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t vis = __shfl_sync(0xffffffffu, seen, src) >> (4 * n + (j >> 3) * 2);
#pragma unroll
                            for (int k = 0; k < KB; ++k)
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const int d = k * 16 + g + half * 8;
                                    const uint16_t b = *reinterpret_cast<const uint16_t *>(
                                        reinterpret_cast<const unsigned char *>(v) + at(j, d & ~7) + (d & 7) * 2);
                                    if ((b & 0x7f80u) != 0x7f80u) continue;
                                    const float x = __uint_as_float((uint32_t)b << 16);
                                    if (vis & 1) o[n][k][half * 2] += x;
                                    if (vis & 2) o[n][k][half * 2 + 1] += x;
                                }
                        }
                    }
                    __syncwarp();
                    for (int e = lane; e < C::kTile / 16; e += 32) {
                        const uint4 x = v[e];
                        v[e] = make_uint4(finite2(x.x), finite2(x.y), finite2(x.z), finite2(x.w));
                    }
                    fence_proxy_async_smem();  // (before a later copy into the slot)
                    __syncwarp();
                }
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                uint32_t a[4];
                ldmatrix4_trans(((vt + v_lane) ^ ((k & 3) << 5)) + (k >> 2) * 1024, a);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma(o[n][k], a, pt[n][0], pt[n][1]);
            }
            __syncwarp();  // every lane has read the tile
            issue();
        }
        // the next piece's queries come while this one's rows are written
        have = policy.next(w2);
        if (have) load_q(w2);
        if (dead) continue;
        const bool partial = policy.partial(w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = n * 8 + 2 * c;  // and the one after it
            if (n * 8 >= w.rows) break;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int f = 4; f < 32; f <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], f);
            if (partial) {  // 32 bytes of four rows at a time
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (row + e >= w.rows) continue;
                    float *dst = policy.part_row(w, w.r0 + row + e, row + e) + g;
#pragma unroll
                    for (int k = 0; k < KB; ++k) dst[k * 16] = o[n][k][e], dst[k * 16 + 8] = o[n][k][2 + e];
                    if (g == 0) *policy.part_sums(w, w.r0 + row + e, row + e) = make_float2(m[n][e] * scale, l[n][e]);
                }
            } else {  // pairs of columns of row g, by the transpose of pairs of rows
                const float i0 = l[n][0] == 0.f ? 0.f : 1.f / l[n][0], i1 = l[n][1] == 0.f ? 0.f : 1.f / l[n][1];
                const bool there = n * 8 + g < w.rows;
                uint32_t *dst = reinterpret_cast<uint32_t *>(policy.out_row(w, w.r0 + (there ? n * 8 + g : 0))) + c;
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t v = transpose8(pack_bf16(o[n][k][2 * half] * i0, o[n][k][2 * half + 1] * i1));
                        if (there) dst[k * 8 + half * 4] = v;
                    }
            }
        }
    }
    drain<NS>(full[warp], landed, issued);
}

// ---------------------------------------------------------------------------
// fp32, on the CUDA cores: the same walk and ring, tiles of 8 keys (one bulk copy each of K and V: 8 rows of a page lie
// together).  Scores: eight lanes a key, D / 8 columns of every row each, then the lanes share the rows out
// among them; values: a lane has D / 32 columns of every row, the weights through shared memory.  Every product and
// sum is fp32.  Bound: HBM for a row or two, the
// multiply-adds (64 a key and lane for 8 rows of 128) beyond.  24 tokens of 1344 positions, 32/32 heads of 128, each of a sequence
// of its own: 165 us = 6.4 TB/s, 0.96 of a copy's rate; all of one sequence, its keys from L2: 89 us.
// ---------------------------------------------------------------------------

template <int D>
struct Cfg32 {
    static constexpr int kKeys = 8;
    static constexpr int kTile = kKeys * D * 4;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kSmem = kWarps * kStages * 2 * kTile;
};

// R: rows of a tile at most: 1, 2, 4 or 8.  ck, cv: the cache.
template <int D, int R, typename P>
SFFN_DEV void attention_f32(P &policy, const void *ck, const void *cv, int page_shift, int n_pages, int n_kv_heads, float scale,
                            int32_t *err, unsigned char *smem_raw) {
    using C = Cfg32<D>;
    constexpr int NS = C::kStages, KB = D / 32, K = C::kKeys, V = D / 32;
    __shared__ uint64_t full[kWarps][NS];
    __shared__ __align__(16) float s_p[kWarps][K][R < 4 ? 4 : R];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, kg = lane >> 3, sub = lane & 7;
    unsigned char *ring = smem_raw + warp * NS * 2 * C::kTile;
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < NS; ++i) mbar_init(&full[w][i], 1);
        mbar_fence_init();
    }
    __syncthreads();

    // ---- loads, as in attention() ----
    P ahead = policy;
    const uint64_t keep = l2_evict_first_policy();
    Work lw, nw;
    int li = 0, ln = 0, issued = 0, islot = 0, nn, page = 0, npage = 0;
    bool dead = false;
    auto tiles_of = [&](const Work &w) { return (w.k1 - w.k0 + K - 1) / K; };
    auto look_up = [&](const Work &w, int i, int &pg) {
        const int key = w.k0 + (i + lane) * K;
        if (key < w.k1) pg = ahead.page_of(w, key);
    };
    auto fetch = [&]() {
        nn = ahead.next(nw) ? tiles_of(nw) : -1;
        if (nn > 0) look_up(nw, 0, npage);
    };
    fetch();
    auto issue = [&]() {
        while (li == ln && nn >= 0) {
            lw = nw, li = 0, ln = nn, page = npage;
            fetch();
        }
        if (li == ln || dead) return;
        if ((li & 31) == 0 && li > 0) look_up(lw, li, page);
        const int pg = __shfl_sync(0xffffffffu, page, li & 31), key = lw.k0 + li * K;
        unsigned char *dst = ring + islot * 2 * C::kTile;
        if (pg < n_pages) {
            const size_t at = ((((size_t)pg * n_kv_heads + lw.h) << page_shift) + (key & ((1 << page_shift) - 1))) * (D * 4);
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[warp][islot], 2 * C::kTile);
                bulk_load(dst, static_cast<const char *>(ck) + at, C::kTile, &full[warp][islot], keep);
                bulk_load(dst + C::kTile, static_cast<const char *>(cv) + at, C::kTile, &full[warp][islot], keep);
            }
        } else {  // no page of the cache: zeros
            for (int i = lane; i < 2 * C::kTile / 16; i += 32) reinterpret_cast<uint4 *>(dst)[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();  // (before a later copy into the slot)
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[warp][islot]);
        }
        ++li;
        ++issued;
        if (++islot == NS) islot = 0;
    };
    for (int i = 0; i < NS; ++i) issue();

    const float cf = scale * 1.44269504088896341f;
    int landed = 0, slot = 0;
    uint32_t par = 0;
    float4 q[R][KB];
    auto load_q = [&](const Work &w) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 *src = reinterpret_cast<const float4 *>(policy.query(w, w.r0 + min(r, w.rows - 1)));
#pragma unroll
            for (int k = 0; k < KB; ++k) q[r][k] = __ldg(src + k * 8 + sub);
        }
    };
    const int my = sub & (R - 1);  // the row whose scores this lane has
    Work w, w2;
    bool have = policy.next(w);
    if (have) load_q(w);
    for (; have; w = w2) {
        float o[R][V], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int x = 0; x < V; ++x) o[r][x] = 0.f;
        const int tiles = tiles_of(w);
        for (int i = 0; i < tiles; ++i) {
            const int kb = w.k0 + i * K;
            if (!dead) {
                bool came = __all_sync(0xffffffffu, mbar_try_wait(&full[warp][slot], par));
                if (!came) {
                    const uint64_t t0 = globaltimer_ns();
                    while (!came && !__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs))
                        came = __all_sync(0xffffffffu, mbar_try_wait_for(&full[warp][slot], par, kHoldNs));
                }
                if (came) {
                    ++landed;
                } else {
                    dead = true;
                    if (lane == 0) record_error(err, SFFN_ERR_TIMEOUT);
                }
            }
            const float4 *kt = reinterpret_cast<const float4 *>(ring + slot * 2 * C::kTile);
            const float *vt = reinterpret_cast<const float *>(ring + slot * 2 * C::kTile + C::kTile) + lane * V;
            if (++slot == NS) slot = 0, par ^= 1;
            float s[2];
            const bool masked = kb + K > w.all;
            bool seen[2] = {true, true};
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // key 4 j + kg
                float a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) a[r] = 0.f;
#pragma unroll
                for (int k = 0; k < KB; ++k) {
                    const float4 x = kt[(4 * j + kg) * (D / 4) + k * 8 + sub];
#pragma unroll
                    for (int r = 0; r < R; ++r) a[r] += x.x * q[r][k].x + x.y * q[r][k].y + x.z * q[r][k].z + x.w * q[r][k].w;
                }
                // sums over the eight lanes, lane `sub` ending with row sub % R: while there are several rows the lanes of
                // a pair keep half of them each
#pragma unroll
                for (int f = 4, n = R; f > 0; f >>= 1) {
                    if (n > f) {
                        n >>= 1;
#pragma unroll
                        for (int r = 0; r < R / 2; ++r)
                            if (r < n) {
                                const bool up = sub & f;
                                const float other = __shfl_xor_sync(0xffffffffu, up ? a[r] : a[r + n], f);
                                a[r] = (up ? a[r + n] : a[r]) + other;
                            }
                    } else {
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (r < n) a[r] += __shfl_xor_sync(0xffffffffu, a[r], f);
                    }
                }
                s[j] = a[0];
                if (masked) {
                    const int key = kb + 4 * j + kg;
                    seen[j] = key < w.k1 && (key < w.all || (my < w.rows && policy.sees(w, w.r0 + my, key)));
                    if (!seen[j]) s[j] = -INFINITY;
                }
            }
            float x = fmaxf(s[0], s[1]);
            const bool up = (x - m) * cf > kLazyLog2;
            if (__any_sync(0xffffffffu, up)) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                float f = 1.f;
                if ((x - m) * cf > kLazyLog2) {
                    f = ex2((m - x) * cf);
                    m = x;
                    l *= f;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float fr = __shfl_sync(0xffffffffu, f, r);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[r][e] *= fr;
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = ex2((s[j] - ref) * cf);
                l += p;
                // -1: a key that the row does not see, whose value is left out
                if (sub < R) s_p[warp][4 * j + kg][my] = seen[j] ? p : -1.f;
            }
            __syncwarp();
#pragma unroll
            for (int key = 0; key < K; ++key) {
                float v[V], p[R];
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(vt + key * D);
                    v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2 *>(vt + key * D);
                    v[0] = y.x, v[1] = y.y;
                }
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(&s_p[warp][key][r]);
                    p[r] = y.x;
                    if (R > 1) p[(r + 1) % R] = y.y;
                    if (R > 2) p[(r + 2) % R] = y.z, p[(r + 3) % R] = y.w;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (masked && p[r] < 0.f) continue;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[r][e] += p[r] * v[e];
                }
            }
            __syncwarp();  // every lane has read the tile
            issue();
        }
        have = policy.next(w2);
        if (have) load_q(w2);
        if (dead) continue;
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const bool partial = policy.partial(w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float lr = __shfl_sync(0xffffffffu, l, r), mr = __shfl_sync(0xffffffffu, m, r);
            if (r >= w.rows) continue;
            const float inv = partial ? 1.f : (lr == 0.f ? 0.f : 1.f / lr);
            float *dst = (partial ? policy.part_row(w, w.r0 + r, r) : policy.out_row(w, w.r0 + r)) + lane * V;
            if constexpr (V == 4)
                *reinterpret_cast<float4 *>(dst) = make_float4(o[r][0] * inv, o[r][1] * inv, o[r][2] * inv, o[r][3] * inv);
            else
                *reinterpret_cast<float2 *>(dst) = make_float2(o[r][0] * inv, o[r][1] * inv);
            if (partial && lane == 0) *policy.part_sums(w, w.r0 + r, r) = make_float2(mr * scale, lr);
        }
    }
    drain<NS>(full[warp], landed, issued);
}

}  // namespace few
}  // namespace sffn
