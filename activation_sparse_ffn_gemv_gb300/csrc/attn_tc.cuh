// attn_tc.cuh -- softmax attention of bf16 queries on the tensor cores (tcgen05,
// TMEM, TMA), shared by the packed prompts and the paged cache.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j - m_i)
//
// for any m_i that keeps the exponentials in range; the running maximum is used and
// moved only when a row's scores pass it by more than 2^8, so the accumulator is
// rarely rescaled (the sums stay exact in either case: both carry the same m_i).
//
// Rows.  The G query heads of a key head read the same keys, so a row is a (token,
// query head) pair and a 128-row tile holds TB = 128 / G tokens (one TMA box of TB
// tokens x G heads x 64 elements lays them out as rows).  An item has two such tiles (or one).
//
// One CTA per SM, ten warps, no CTA-wide barrier between items:
//   warp 0      loads: queries, then the ring of 128-key K and V tiles
//   warp 1      issues the tcgen05.mma: S_t = Q_t K^T into TMEM (fp32), later O_t += P_t V
//   warps 2-5   softmax of tile 0 (6-9: of tile 1): a thread owns a row; S_t from TMEM, weights
//               P_t (bf16) back to TMEM over S_t, where the second product reads them as its
//               A operand; at the end O_t / sum to global memory
// While one tile's softmax runs, the tensor cores work on the other tile.  Where every item has
// one row tile (ONE: few new tokens over a long cache) its key tiles are dealt to the two
// pipelines instead, and at the end the first one joins both results, reading the
// other's accumulator from TMEM (the same rows are the same lanes).
//
// A weight of zero times an infinite or NaN value would be NaN, so in a tile with
// masked keys the softmax warps look through V in shared memory before the second
// product: non-finite elements become zero, and where they belong to existing keys the
// rows that do see them get them added at the end.  Rows that do not see them come out bit
// for bit as without them.
#pragma once

#include "attn.cuh"
#include "tcgen05.cuh"

namespace sffn {
namespace atc {

constexpr int kThreads = 320;
constexpr int kKeys = 128;                   // keys of a tile
constexpr int kItems = 3;                    // items that the loading warp has described, at most
constexpr uint32_t kHoldNs = 10000000;       // the hardware may hold a waiting warp for 10 ms at a time,
constexpr uint64_t kGiveUpNs = 2000000000;   // and a wait gives up after 2 s
constexpr float kLazyLog2 = 8.f;             // the running maximum moves when passed by 2^8

// GROUPED: layout of the K and V tiles in shared memory.  false: column block by column block
// (a TMA box is 128 rows of one block).  true: by groups of 8 rows, each with its column blocks in
// turn, so that any multiple of 8 rows with all its columns is one box (a page).
// ONE: every item has one row tile (both pipelines read the same Q_0; the memory goes to the ring).
// TMA_OUT: whole row tiles leave by TMA.
template <int D, int STAGES, bool GROUPED, bool ONE, bool TMA_OUT = !ONE>
struct Cfg {
    static constexpr int kHalves = D / 64;                      // 64-element (128-byte) column blocks
    static constexpr int kBlock = 128 * 128;                    // bytes of a column block: 128 rows x 128 bytes
    static constexpr int kTile = kHalves * kBlock;              // Q, K or V tile
    static constexpr int kStages = STAGES;                      // K and V tiles of the ring
    static constexpr bool kOne = ONE;
    static constexpr int kQ = ONE ? 1 : 2;
    static constexpr bool kGrouped = GROUPED;
    static constexpr int kRows8 = GROUPED ? kHalves * 1024 : 1024;  // bytes from 8 rows to the next 8
    static constexpr int kColBlock = GROUPED ? 1024 : kBlock;       // bytes from a column block to the next
    // Row of a K or V tile that its i-th 16-byte chunk belongs to.
    SFFN_DEV static int row_of(int i) { return GROUPED ? (i / (64 * kHalves)) * 8 + ((i >> 3) & 7) : (i >> 3) & 127; }
    static constexpr int kColO = 256;                           // TMEM columns: S_0, S_1 (128 each), O_0, O_1
    static constexpr bool kTmaOut = TMA_OUT;
    static constexpr int kOut = TMA_OUT ? 4096 : 2048;          // a softmax warp's: 64 (128) bytes of its 32 output rows
    static constexpr int kSmem = (kQ + kStages) * kTile + (ONE ? 4 : 8) * kOut + 1024 /*alignment*/;
};

// One item.  The loading warp finds the items and describes them in a small ring.
struct Work {
    int more;           // 0: no further item
    int q_row;          // first token (row of q and out)
    int nt;             // tokens
    int h;              // key head
    int tiles;          // key tiles
    int n[2];           // those of each pipeline
    int mask_from[2];   // first key tile with masked keys
    int k0, k1;         // keys [k0, k1) (logical positions)
    int exist;          // keys below this one exist
    int i0;             // prompt: position of the first token; pages: least own page of the tokens
    int base;           // prompt: row of key 0; pages: key tiles of the items before
    int ctx;            // tree: committed positions
    int seq, tok0;      // tree: sequence, first token of the item within its new tokens
    bool whole;         // tree: the item's every key (else a partial result)
    int slot;           // tree: partial result slot
    int kind;           // shared prefixes: which part of its rows' keys the item has
};

// 2^x, good to about 2^-22 of it (a bf16 weight needs 2^-9); weights below 2^-126 are zero.
SFFN_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 at a time: (a.x b.x + c.x, a.y b.y + c.y), and the sum.
SFFN_DEV uint64_t f32x2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
SFFN_DEV void split(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
SFFN_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
SFFN_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Maximum of three (NaNs are passed over, as in fmaxf).
SFFN_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

SFFN_DEV uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

// The bf16 halves of w that are infinite or NaN (their sign bits), as a mask of 0x8000s.
SFFN_DEV uint32_t nonfinite_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// 0 * w + sum, of two bf16: NaN once a factor was infinite or NaN.
SFFN_DEV uint32_t zero_times(uint32_t w, uint32_t sum) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(sum));
    return r;
}

// Low 32 bits with the first n set (n clamped to 0 .. 32).
SFFN_DEV uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// P: the policy (prompts, tree, shared prefixes or chosen pages).  It gives
//   start                  before the first item (every warp calls it)
//   kWordMasks             whether masks often cover 32 keys alike
//   kReread                whether other CTAs read the same keys again (the L2 hint of the loads)
//   bool next(Work &)      the CTA's items in turn (the loading warp alone)
//   place, load_kv         where a key tile lies, looked up a tile ahead; the load of its K or V
//   row_info, visible      a row's own data; which keys of a masked tile it sees, as four words
//   exists                 whether there is a key at a row of a masked tile
//   value_row              a key's value row in memory (null: the row does not see the key)
//   begin_row, partial     where a row's output goes; whether as fp32 partial result
template <typename C, int D, typename P>
SFFN_DEV void attention_cta(P &policy, const CUtensorMap &map_q, const CUtensorMap &map_k, const CUtensorMap &map_v,
                            const CUtensorMap &map_o, float scale, int G, int32_t *err, unsigned char *smem_raw) {
    const uint32_t raw_addr = smem_u32(smem_raw), q_addr = (raw_addr + 1023u) & ~1023u, kv_addr = q_addr + C::kQ * C::kTile;
    unsigned char *sm_q = smem_raw + (q_addr - raw_addr), *sm_kv = sm_q + C::kQ * C::kTile,
                  *sm_out = sm_kv + C::kStages * C::kTile;
    constexpr int NS = C::kStages;
    __shared__ uint64_t kv_full[NS], kv_empty[NS], q_full[2], q_empty[2], s_full[2], p_ready[2], o_full[2], mdone,
        i_full[kItems], i_empty[kItems], x_full, x_empty, g_met[2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort, s_bad;
    __shared__ float2 s_x[128];  // maximum and sum of the second pipeline's rows (keys dealt to both)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&kv_full[i], 1), mbar_init(&kv_empty[i], 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_empty[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_ready[t], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&g_met[t], 4);
        }
        mbar_init(&mdone, 1);
        mbar_init(&x_full, 4);
        mbar_init(&x_empty, 4);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 9);  // the issuing warp and the eight softmax warps
        }
        s_abort = 0;
        s_bad = 0;
        mbar_fence_init();
        tc::prefetch_tensormap(&map_q);
        tc::prefetch_tensormap(&map_k);
        tc::prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0;  // the CTA owns all 512 columns, so they start at 0
    if (tid == 0 && tmem_slot != tmem) {
        s_abort = 1;
        record_error(err, SFFN_ERR_DEVICE);
    }

    // Bounded wait of a whole warp: true once the phase has come.  One that runs out records the error and
    // gives up, and so does every other wait of the CTA whose phase has not come by then.  A warp that gets
    // false leaves its loops at once: nothing is loaded, issued or stored on behalf of a phase that never
    // came.  The answer is the same in every lane.
    auto wait_slow = [&](uint64_t *bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!__any_sync(0xffffffffu, s_abort || globaltimer_ns() - t0 > kGiveUpNs))
            if (__all_sync(0xffffffffu, mbar_try_wait_for(bar, parity, kHoldNs))) return true;
        if (lane == 0) {
            s_abort = 1;
            record_error(err, SFFN_ERR_TIMEOUT);
        }
        return false;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait_for(bar, parity, kHoldNs)) || wait_slow(bar, parity);
    };

    griddep_wait();
    const int TB = 128 / G;
    __shared__ Work s_work[kItems];
    policy.start();
    griddep_launch_dependents();
    int item = 0;  // items taken so far
    // The other warps' next item (null: none, or a wait gave up), and its return.
    auto take = [&]() -> const Work * {
        const int i = item % kItems;
        return wait(&i_full[i], (uint32_t)((item / kItems) & 1)) && s_work[i].more ? &s_work[i] : nullptr;
    };
    auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[item % kItems]);
        ++item;
    };

    if (warp == 0) {
        // ---------------- loads ----------------
        int it = 0, qn[2] = {0, 0};
        const uint64_t keep = P::kReread ? tc::l2_evict_last_policy() : l2_evict_first_policy();
        auto load = [&](const Work &w) {  // an item's tiles; false: gave up
            const int tiles = w.tiles;
            int place = policy.place(w, 0, lane);
            for (int j = 0; j < tiles; ++j) {
                const int nxt = j + 1 < tiles ? policy.place(w, j + 1, lane) : 0;  // a tile ahead
                for (int part = 0; part < 2; ++part) {
                    // the item's queries: the first tile's before the first K, the second's after it
                    if (j == 0 && w.n[part] > 0 && part < C::kQ) {
                        if (!wait(&q_empty[part], (uint32_t)((qn[part] & 1) ^ 1))) return false;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&q_full[part], (uint32_t)(TB * G * 128 * C::kHalves));
                            for (int c = 0; c < C::kHalves; ++c)
                                tc::tma_load_3d(sm_q + part * C::kTile + c * C::kBlock, &map_q, c * 64, w.h * G,
                                                w.q_row + part * TB, &q_full[part], keep);
                        }
                        ++qn[part];
                    }
                    const int s = it % NS;
                    if (!wait(&kv_empty[s], (uint32_t)(((it / NS) & 1) ^ 1))) return false;
                    policy.load_kv(w, j, place, part ? &map_v : &map_k, sm_kv + s * C::kTile, &kv_full[s], lane, keep);
                    ++it;
                }
                place = nxt;
            }
            return true;
        };
        for (;; ++item) {
            Work &w = s_work[item % kItems];
            if (!wait(&i_empty[item % kItems], (uint32_t)(((item / kItems) & 1) ^ 1))) break;
            const bool more = policy.next(w);
            __syncwarp();
            if (lane == 0) {
                w.more = more;
                mbar_arrive(&i_full[item % kItems]);
            }
            __syncwarp();
            if (!more || !load(w)) break;
        }
        if (lane == 0) {  // no copy is in flight when the CTA exits, whoever gave up (one more second for all, in equal shares)
            constexpr uint64_t share = kWaitLimitNs / (NS + 2);
            for (int j = max(0, it - NS); j < it; ++j) mbar_wait(&kv_full[j % NS], (uint32_t)((j / NS) & 1), share);
            for (int t = 0; t < 2; ++t)
                if (qn[t]) mbar_wait(&q_full[t], (uint32_t)((qn[t] - 1) & 1), share);
        }
    } else if (warp == 1) {
        // ---------------- tensor cores ----------------
        constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128, false);
        constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D, true);
        // The whole warp runs this code, uniformly; one lane issues each instruction.
        const uint64_t hi_q = tc::smem_desc_sw128(0, 16, 1024), hi_k = tc::smem_desc_sw128(0, 16, C::kRows8),
                       hi_v = tc::smem_desc_sw128(0, C::kColBlock, C::kRows8);
        auto scores = [&](int t, uint32_t tile) {  // S_t = Q_t K^T
            const uint64_t a = hi_q | ((q_addr + (C::kOne ? 0 : t) * C::kTile) >> 4), b = hi_k | (tile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_bf16_warp(tmem + t * 128, a + (((kk >> 2) * C::kBlock + (kk & 3) * 32) >> 4),
                                  b + (((kk >> 2) * C::kColBlock + (kk & 3) * 32) >> 4), idesc_s, kk != 0);
            tc::mma_commit_warp(&s_full[t]);
        };
        auto values = [&](int t, uint32_t tile, bool acc) {  // O_t (+)= P_t V
            const uint64_t b = hi_v | (tile >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                tc::mma_bf16_ts_warp(tmem + C::kColO + t * D, tmem + t * 128 + kk * 8, b + kk * (2 * C::kRows8 >> 4), idesc_o,
                                     acc || kk != 0);
        };
        int slot = 0;                                        // ring position and its parity
        uint32_t par = 0, q_par[2] = {0, 0}, p_par[2] = {0, 0};
        auto step = [&]() {
            if (++slot == NS) slot = 0, par ^= 1;
        };
        auto tile_of = [&](int s) { return kv_addr + (uint32_t)s * C::kTile; };
        // (each of these: false if a wait gave up)
        auto first_scores = [&](int t) {
            if (t < C::kQ) {
                if (!wait(&q_full[t], q_par[t])) return false;
                q_par[t] ^= 1;
            }
            tc::fence_after_sync();
            scores(t, tile_of(slot));
            return true;
        };
        auto weigh = [&](int t, uint32_t v, bool acc) {  // once the weights are there
            if (!wait(&p_ready[t], p_par[t])) return false;
            p_par[t] ^= 1;
            tc::fence_after_sync();
            values(t, v, acc);
            return true;
        };
        // Two row tiles (or the first alone) over the same key tiles.
        auto both = [&](const int n0, const int n1) {
            const int n[2] = {n0, n1}, nmax = max(n0, n1);
            if (!wait(&kv_full[slot], par)) return false;
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (n[t] > 0 && !first_scores(t)) return false;
            step();
            for (int j = 0; j < nmax; ++j) {
                const int vs = slot;
                if (!wait(&kv_full[vs], par)) return false;
                step();
                const bool more = j + 1 < nmax;
                if (more && !wait(&kv_full[slot], par)) return false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < n[t]) {
                        if (!weigh(t, tile_of(vs), j > 0)) return false;
                        if (j + 1 == n[t]) tc::mma_commit_warp(&o_full[t]);
                    }
                    if (j + 1 < n[t]) scores(t, tile_of(slot));
                }
                if (more) step();
            }
            return true;
        };
        // One row tile: pipeline t takes every other key tile.
        auto dealt = [&](const int tiles) {
            if (!wait(&kv_full[slot], par) || !first_scores(0)) return false;
            step();
            // V of tile i lies at the position of step i; K of tile i + 1 follows it
            int v_slot = slot;
            uint32_t v_par = par;
            step();
            if (tiles > 1) {
                if (!wait(&kv_full[slot], par) || !first_scores(1)) return false;
                step();
            }
            if (C::kOne && tiles <= 2) tc::mma_commit_warp(&q_empty[0]);
            for (int i = 0; i < tiles; i += 2) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (i + t < tiles) {
                        if (!wait(&kv_full[v_slot], v_par) || !weigh(t, tile_of(v_slot), i > 0)) return false;
                        // given back at once: S_t(i + 2) would say so too, but only after the next K's load
                        tc::mma_commit_warp(&kv_empty[v_slot]);
                        // on to the next tile's V; position `slot` is that of tile i + t + 1's V
                        v_slot = slot;
                        v_par = par;
                        if (i + t + 1 < tiles) step();
                        if (i + t + 2 < tiles) {
                            if (!wait(&kv_full[slot], par)) return false;
                            tc::fence_after_sync();
                            scores(t, tile_of(slot));
                            step();
                            if (C::kOne && i + t + 3 == tiles) tc::mma_commit_warp(&q_empty[0]);
                        } else {
                            tc::mma_commit_warp(&o_full[t]);
                        }
                    }
                }
            }
            return true;
        };
        // The ring's tiles are given back by the softmax warps, which see S_t(j) arrive after their last
        // reader, with no more commits here (V of a dealt tile excepted).
        for (;; give_back()) {
            const Work *w = take();
            if (!w) break;
            // uniform by construction; the reductions tell the compiler so
            const int n0 = __reduce_max_sync(0xffffffffu, w->n[0]), n1 = __reduce_max_sync(0xffffffffu, w->n[1]);
            if constexpr (C::kOne) {
                if (!dealt(n0 + n1)) break;
            } else {
                if (!both(n0, n1)) break;
            }
        }
        // Every product of this CTA has completed before teardown.  A commit covers its own thread's products, so
        // it is issued as they are, by the elected lane of the whole warp.
        tc::mma_commit_warp(&mdone);
        mbar_wait(&mdone, 0);
    } else {
        // ---------------- softmax of row tile t ----------------
        const int t = (warp - 2) >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const int tok = row / G, head = row - tok * G;  // token of the tile, query head of the group
        const uint32_t ts = tmem + ((uint32_t)(quad * 32) << 16) + t * 128;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + C::kColO + t * D;
        const float c = scale * 1.44269504088896341f;  // the exponent in powers of two
        int sn = 0, on = 0, xn = 0, gn = 0, base = 0;
        // The four warps of the group meet (their writes to shared memory are seen after it); false: gave up.
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&g_met[t]);
            return wait(&g_met[t], (uint32_t)(gn++ & 1));
        };
        // Whether this warp knows that the fill before V_0 in its ring slot (V of the next to last key tile before this
        // item, or an older one) has landed: it does after the product with that tile or a later one.
        bool seen = true;
        for (;;) {
            const Work *next = take();
            if (!next) break;
            const Work &w = *next;
            const int n = w.n[t], tiles = w.tiles;
            constexpr bool dealt = C::kOne;
            const int item_tok = (dealt ? 0 : t * TB) + tok;  // token of the item
            const bool valid = tok < TB && item_tok < w.nt;
            typename P::RowInfo ri = policy.row_info(w, valid ? item_tok : 0);
            // of two row tiles' pipelines the second is the last reader of a key tile
            const bool releases = dealt || t == (w.n[1] > 0 ? 1 : 0);
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                const int kt = dealt ? 2 * j + t : j, k_at = base + 2 * kt;  // key tile, ring index of its K
                const bool masked = kt >= w.mask_from[t];
                // The look through V comes before S_t(j) (it costs nothing there), except where the slot's
                // fill before V has not been seen by then (a wait tells only successive fills apart)
                // or is given back with S_t(j).
                const bool late = dealt || (j == 0 && !seen);
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    if (masked && pass == (late ? 1 : 0)) {
                        // Non-finite values of this tile: zero (and noted, if their keys exist)
                        const int iv = k_at + 1, vs = iv % NS;
                        if (!wait(&kv_full[vs], (uint32_t)((iv / NS) & 1))) goto done;
                        uint4 *v = reinterpret_cast<uint4 *>(sm_kv + vs * C::kTile);
#pragma unroll 1
                        for (int i0 = quad * 32 + lane; i0 < C::kTile / 16; i0 += 512) {
                            uint4 x[4];
                            uint32_t any[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int u = 0; u < 4; ++u) x[u] = v[i0 + u * 128];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {  // zero times it is NaN (one instruction a pair)
                                any[0] = zero_times(x[u].x, any[0]);
                                any[1] = zero_times(x[u].y, any[1]);
                                any[2] = zero_times(x[u].z, any[2]);
                                any[3] = zero_times(x[u].w, any[3]);
                            }
                            if (nonfinite_bits(any[0]) | nonfinite_bits(any[1]) | nonfinite_bits(any[2]) | nonfinite_bits(any[3])) {
#pragma unroll 1
                                for (int i = i0; i < i0 + 512; i += 128) {
                                    uint4 y = v[i];
                                    const uint32_t b0 = nonfinite_bits(y.x), b1 = nonfinite_bits(y.y),
                                                   b2 = nonfinite_bits(y.z), b3 = nonfinite_bits(y.w);
                                    if (!(b0 | b1 | b2 | b3)) continue;
                                    if (policy.exists(w, kt, C::row_of(i))) {
                                        s_bad = 1;
                                        __threadfence_block();
                                    }
                                    // (bit >> 15) * 0xffff: the whole half
                                    y.x &= ~((b0 >> 15) * 0xffffu);
                                    y.y &= ~((b1 >> 15) * 0xffffu);
                                    y.z &= ~((b2 >> 15) * 0xffffu);
                                    y.w &= ~((b3 >> 15) * 0xffffu);
                                    v[i] = y;
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    if (pass == 0) {
                        if (!wait(&s_full[t], (uint32_t)(sn & 1))) goto done;
                        ++sn;
                        if (lane == 0 && quad == 0) {
                            // S_t(j) is there: Q_t is free after the last tile; K of this tile and V of the one
                            // before it are, once the later row tile's products are through
                            if (!C::kOne && j + 1 == n) mbar_arrive_relaxed(&q_empty[t]);
                            if (releases) {
                                mbar_arrive_relaxed(&kv_empty[k_at % NS]);
                                if (j > 0 && !dealt) mbar_arrive_relaxed(&kv_empty[(k_at - 1) % NS]);
                            }
                        }
                        tc::fence_after_sync();
                    }
                }
                uint32_t s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32(ts + q * 32, s[q]);
                tc::tmem_wait_ld();
                if (masked) {
                    uint32_t vis[4];
                    policy.visible(w, ri, kt, vis);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (P::kWordMasks && __all_sync(0xffffffffu, vis[q] == 0 || vis[q] == 0xffffffffu)) {
                            const bool on = vis[q] != 0;  // one test for the word
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[q][i] = on ? s[q][i] : 0xff800000u;  // -inf
                        } else if (__any_sync(0xffffffffu, vis[q] != 0xffffffffu)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                s[q][i] = (vis[q] >> i) & 1u ? s[q][i] : 0xff800000u;  // -inf
                        }
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
                    for (int i = 2; i < 32; i += 2)
                        mx[q] = max3(mx[q], __uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1]));
                }
                const float mnew = max3(m, fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool up = (mnew - m) * c > kLazyLog2;
                if (__any_sync(0xffffffffu, up)) {
                    const float alpha = up ? ex2((m - mnew) * c) : 1.f;
                    // (a row that has seen nothing yet has an accumulator of zeros)
                    const bool rescale = __any_sync(0xffffffffu, up && m != -INFINITY);
                    if (up) m = mnew;
                    l *= alpha;
                    if (j > 0 && rescale) {
                        // the product of tile j - 1 is complete: it was issued before S_t(j)
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            tc::tmem_ld16(to + q * 16, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tc::tmem_st16(to + q * 16, o);
                        }
                    }
                }
                const float mc = (m == -INFINITY ? 0.f : m) * c;  // nothing seen yet: every weight is 2^-inf = 0
                const uint64_t c2 = f32x2(__float_as_uint(c), __float_as_uint(c)),
                               mc2 = f32x2(__float_as_uint(-mc), __float_as_uint(-mc));
                // The weights are rounded to bf16 because the second product takes both operands in one type and V
                // is bf16; the sum is of the unrounded ones.  A weight is off by 2^-8 of itself at most, which
                // adds to the output about what the output's own rounding does: against 64 bits the norm of the
                // error goes from 0.0016 of the output's to 0.0018 (short prompts), 0.0020 (long ones), 0.0023 (a long context).
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        split(fma2(f32x2(s[q][2 * i], s[q][2 * i + 1]), c2, mc2), x0, x1);
                        const float e0 = ex2(x0), e1 = ex2(x1);
                        sum[i & 1] = add2(sum[i & 1], f32x2(__float_as_uint(e0), __float_as_uint(e1)));
                        p[i] = pack_bf16(e0, e1);
                    }
                    tc::tmem_st16(ts + q * 16, p);
                }
                // (handing over the first 64 keys' weights early cost the issuing warp a second look at
                // a barrier and gained nothing: 190 against 187 us for 8192 tokens of 16 heads)
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[t]);
                float l0, l1;
                split(add2(sum[0], sum[1]), l0, l1);
                l += l0 + l1;
            }
            if (n > 0) {
                if (!wait(&o_full[t], (uint32_t)(on & 1))) goto done;
                ++on;
                if (releases && !dealt && lane == 0 && quad == 0) mbar_arrive_relaxed(&kv_empty[(base + 2 * n - 1) % NS]);
                tc::fence_after_sync();
            }
            float f0 = 1.f, f1 = 0.f;  // factors of O_0 and O_1 in a joint result
            const bool join = dealt && w.n[1] > 0;
            if (join) {
                if (t == 1) {  // hand over; O_1 stays as it is until it has been read
                    s_x[row] = make_float2(m, l);
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full);
                    if (!wait(&x_empty, (uint32_t)(xn & 1))) goto done;
                } else {
                    if (!wait(&x_full, (uint32_t)(xn & 1))) goto done;
                    tc::fence_after_sync();
                    const float2 o = s_x[row];
                    const float mj = fmaxf(m, o.x), ref = mj == -INFINITY ? 0.f : mj;
                    f0 = ex2((m - ref) * c);
                    f1 = ex2((o.x - ref) * c);
                    l = l * f0 + o.y * f1;
                    m = mj;
                }
                ++xn;
            }
            if (n > 0 && !(join && t == 1)) {
                const bool bad = s_bad != 0;
                // this lane's row of the output (null: not a row), and a factor
                float inv;
                unsigned char *dst = policy.begin_row(w, item_tok, head, valid, m, l, inv);
                if (join) {
                    // O_0 <- f0 O_0 + f1 O_1
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t x[16], y[16];
                        tc::tmem_ld16(to + q * 16, x);
                        tc::tmem_ld16(to + D + q * 16, y);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * f0 + __uint_as_float(y[i]) * f1);
                        tc::tmem_st16(to + q * 16, x);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_empty);
                }
                const bool f32 = policy.partial(w);
                unsigned char *stage = sm_out + (C::kOne ? quad : warp - 2) * C::kOut;
                if (__any_sync(0xffffffffu, bad && valid)) {
                    // the masked tiles' non-finite values that this row sees
                    const int from = w.k0 + min(w.mask_from[0], w.mask_from[1]) * kKeys;
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tc::tmem_ld16(to + q * 16, o);
                        tc::tmem_wait_ld();
                        for (int key = from; valid && key < w.k1; ++key) {
                            const uint4 *vr = reinterpret_cast<const uint4 *>(policy.value_row(w, ri, key));
                            if (!vr) continue;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint4 x = vr[q * 2 + i];
                                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t nb = nonfinite_bits(xs[e]);
                                    uint32_t &lo = o[i * 8 + e * 2], &hi = o[i * 8 + e * 2 + 1];
                                    if (nb & 0x8000u) lo = __float_as_uint(__uint_as_float(lo) + bf16lo(xs[e]));
                                    if (nb & 0x80000000u) hi = __float_as_uint(__uint_as_float(hi) + bf16hi(xs[e]));
                                }
                            }
                        }
                        __syncwarp();
                        tc::tmem_st16(to + q * 16, o);
                    }
                    tc::tmem_wait_st();
                }
                const int o_h = w.h * G, o_row = w.q_row + t * TB;
                const bool full = C::kTmaOut && w.nt >= (t + 1) * TB;
                give_back();  // before the stores, which the release would wait for
                if constexpr (C::kTmaOut) {
                    // A whole row tile leaves by TMA, 64 columns at a time: the warps go on while it is
                    // written (their own stores took 4000 cycles an item, stalling the loads after them).
                    unsigned char *buf = sm_out + t * 4 * C::kOut;
                    const bool issues = quad == 0 && lane == 0;
                    if (full) {
#pragma unroll 1
                        for (int q2 = 0; q2 < D / 64; ++q2) {
                            if (issues) tc::bulk_wait_read();
                            if (!meet()) goto done;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t o[32];
                                tc::tmem_ld32(to + q2 * 64 + h * 32, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    uint32_t p[4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        p[e] = pack_bf16(__uint_as_float(o[i * 8 + 2 * e]) * inv,
                                                         __uint_as_float(o[i * 8 + 2 * e + 1]) * inv);
                                    *reinterpret_cast<uint4 *>(buf + row * 128 + (((h * 4 + i) ^ (row & 7)) << 4)) =
                                        make_uint4(p[0], p[1], p[2], p[3]);
                                }
                            }
                            fence_proxy_async_smem();
                            if (!meet()) goto done;
                            if (issues) {
                                tc::tma_store_3d(&map_o, q2 * 64, o_h, o_row, buf);
                                tc::bulk_commit();
                            }
                        }
                    } else {
                        if (issues) tc::bulk_wait_read();
                        if (!meet()) goto done;
                    }
                }
                // 64 bytes of every row at a time through shared memory, the 16-byte chunks swizzled by
                // the row: a store then covers 64 bytes of eight rows instead of 16 of 32
                auto flush = [&](const uint32_t (&x)[16], int seg) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = i * 8 + (lane >> 2), ch = lane & 3;
                        unsigned char *d = reinterpret_cast<unsigned char *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
                        if (d) *reinterpret_cast<uint4 *>(d + (size_t)seg * 64 + ch * 16) = v;
                    }
                };
                if (full) {
                    // on its way
                } else if (f32) {
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tc::tmem_ld16(to + q * 16, o);
                        tc::tmem_wait_ld();
                        flush(o, q);
                    }
                } else {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32], pk[16];
                        tc::tmem_ld32(to + q * 32, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            pk[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        flush(pk, q);
                    }
                }
                tc::fence_before_sync();  // O_t has been read: the next item's product may overwrite it
            } else {
                give_back();
            }
            base += 2 * tiles;
            seen = !dealt && n > 0 && n >= tiles - 1;  // (an item without work for this group tells it nothing)
        }
    done:
        if (C::kTmaOut && quad == 0 && lane == 0) tc::bulk_wait();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

}  // namespace atc
}  // namespace sffn
