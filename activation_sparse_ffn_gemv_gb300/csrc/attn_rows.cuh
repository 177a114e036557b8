// attn_rows.cuh -- attention of up to 64 query rows over a range of keys on the CUDA
// cores, fp32 (the fp32 cache's path: fp32 has no tensor-core product of its precision).
//
// One CTA of 256 threads keeps the rows' queries in shared memory and takes 64 keys at a
// time: scores (thread: one key, 16 rows), the running maximum and sum (thread: one row,
// 16 keys), the product with the values (thread: four columns, D / 16 rows; the weights lie
// key by key, so a thread reads four rows' at once).  The next keys' rows are copied
// meanwhile (cp.async, two buffers).  Bound: shared-memory reads of the two products,
// about 5 a 16 multiply-adds.  Measured: 4 sequences of up to 4000 positions, 1 to 8 tokens, 16/2
// heads of 64, 27.5 us with the join (latency: a CTA has one or two tiles).
#pragma once

#include "attn.cuh"

namespace sffn {
namespace rows {

constexpr int kThreads = 256;
constexpr int kRows = 64;   // rows of a CTA
constexpr int kKeys = 64;   // keys of a tile

template <int D>
struct Smem {
    float q[kRows][D];
    float k[2][kKeys][D + 4];
    float v[2][kKeys][D];
    float p[kKeys][kRows + 4];
    float part[4][kRows];
    float m[kRows], l[kRows], alpha[kRows];
};

// 16 bytes global -> shared, asynchronously; zeros instead if `src` is null.
SFFN_DEV void copy16(void *dst, const float *src, const float *any) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src ? src : any),
                 "r"(src ? 16 : 0)
                 : "memory");
}

template <int D>
struct Acc {
    static constexpr int CT = D / 4;              // threads of a row
    static constexpr int RG = kThreads / CT;      // row groups
    static constexpr int RPT = kRows / RG;        // rows of a thread: group * RPT + i
    float4 o[RPT];
};

// Attention of rows [0, nr) over keys [k0, k1): leaves the unnormalised output in acc,
// maximum and sum in sm.m / sm.l.  q_row(r): the row's D elements; key(j, which): key
// or value row j (null: zeros); keys below `all` are seen by every row, of the others sees(r, j)
// tells.  A key that a row does not see has weight zero and its value is not
// multiplied, whatever it holds.
template <int D, typename QRow, typename Key, typename Sees>
SFFN_DEV void attend(Smem<D> &sm, Acc<D> &acc, int nr, int k0, int k1, int all, float scale, QRow q_row, Key key,
                     Sees sees) {
    constexpr int CT = Acc<D>::CT, RPT = Acc<D>::RPT;
    const int tid = threadIdx.x;
    auto load = [&](int j0, int buf) {
#pragma unroll 4
        for (int i = tid; i < kKeys * CT; i += kThreads) {
            const int j = i / CT, c = (i % CT) * 4;
            const float *kp = nullptr, *vp = nullptr;
            if (j0 + j < k1) {
                kp = key(j0 + j, 0);
                vp = key(j0 + j, 1);
            }
            const float *any = q_row(0);
            copy16(&sm.k[buf][j][c], kp ? kp + c : nullptr, any);
            copy16(&sm.v[buf][j][c], vp ? vp + c : nullptr, any);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();
    load(k0, 0);
    for (int i = tid; i < kRows * CT; i += kThreads) {
        const int r = i / CT, c = (i % CT) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nr) x = *reinterpret_cast<const float4 *>(q_row(r) + c);
        *reinterpret_cast<float4 *>(&sm.q[r][c]) = make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
    }
    if (tid < kRows) sm.m[tid] = -INFINITY, sm.l[tid] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) acc.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    int buf = 0;
    for (int j0 = k0; j0 < k1; j0 += kKeys, buf ^= 1) {
        const bool masked = j0 + kKeys > all;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // this tile is there, and nobody reads the other buffer any more
        if (j0 + kKeys < k1) load(j0 + kKeys, buf ^ 1);
        {
            const int j = tid & 63, g = tid >> 6;  // rows g * 16 .. + 15
            if (g * 16 < nr) {
                float s[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll 2
                for (int c = 0; c < D; c += 4) {
                    const float4 kx = *reinterpret_cast<const float4 *>(&sm.k[buf][j][c]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 qx = *reinterpret_cast<const float4 *>(&sm.q[g * 16 + i][c]);
                        s[i] += qx.x * kx.x + qx.y * kx.y + qx.z * kx.z + qx.w * kx.w;
                    }
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = g * 16 + i;
                        if (!(r < nr && j0 + j < k1 && (j0 + j < all || sees(r, j0 + j)))) s[i] = -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(&sm.p[j][g * 16 + i]) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
            }
        }
        __syncthreads();
        {
            const int r = tid & 63, part = tid >> 6;  // keys part * 16 .. + 15
            float s[16], mx = -INFINITY;
            if (r < nr) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[i] = sm.p[part * 16 + i][r];
                    mx = fmaxf(mx, s[i]);
                }
                sm.part[part][r] = mx;
            }
            __syncthreads();
            float sum = 0.f, mo = 0.f, mn = 0.f;
            if (r < nr) {
                mo = sm.m[r];
                mn = fmaxf(fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r])), mo);
                const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is exp(-inf) = 0
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = expf(s[i] - ref);
                    sum += p;
                    // -1 marks a key that the row does not see: its value is left out, not multiplied by zero
                    sm.p[part * 16 + i][r] = masked && s[i] == -INFINITY ? -1.f : p;
                }
                if (part == 0) sm.alpha[r] = expf(mo - ref);
            }
            __syncthreads();  // everyone has read m and the maxima
            if (r < nr) {
                sm.part[part][r] = sum;
                if (part == 0) sm.m[r] = mn;
            }
        }
        __syncthreads();
        if (tid < nr)
            sm.l[tid] = sm.l[tid] * sm.alpha[tid] + ((sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]));
        const int c = (tid % CT) * 4, g = (tid / CT) * RPT;
        if (g < nr) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float al = g + i < nr ? sm.alpha[g + i] : 0.f;
                acc.o[i].x *= al, acc.o[i].y *= al, acc.o[i].z *= al, acc.o[i].w *= al;
            }
#pragma unroll 4
            for (int j = 0; j < kKeys; ++j) {
                const float4 vx = *reinterpret_cast<const float4 *>(&sm.v[buf][j][c]);
#pragma unroll
                for (int i = 0; i < RPT; i += 4) {
                    const float4 p4 = *reinterpret_cast<const float4 *>(&sm.p[j][g + i]);
                    const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (masked && p[e] == -1.f) continue;
                        float4 &o = acc.o[i + e];
                        o.x += p[e] * vx.x, o.y += p[e] * vx.y, o.z += p[e] * vx.z, o.w += p[e] * vx.w;
                    }
                }
            }
        }
    }
    __syncthreads();
}

}  // namespace rows
}  // namespace sffn
