// attn_rows.cuh -- attention of up to 64 query rows over a range of keys on the CUDA
// cores, fp32 arithmetic throughout.
//
// One CTA of 256 threads keeps the rows' queries in shared memory and takes 64 keys
// at a time: scores (thread: one key, every fourth group of 16 rows), the running
// maximum and sum of the softmax (a warp per row), then the product with the values
// (thread: four output columns of D / 16 rows).
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
    float k[kKeys][D + 4];
    float v[kKeys][D];
    float p[kRows][kKeys + 4];
    float m[kRows], l[kRows], alpha[kRows];
};

template <typename T>
SFFN_DEV float4 load4(const T *p);
template <>
SFFN_DEV float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <>
SFFN_DEV float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
template <typename T>
SFFN_DEV void store4(T *p, float4 v);
template <>
SFFN_DEV void store4<float>(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
template <>
SFFN_DEV void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2((uint32_t)f32_to_bf16_bits(v.x) | ((uint32_t)f32_to_bf16_bits(v.y) << 16),
                   (uint32_t)f32_to_bf16_bits(v.z) | ((uint32_t)f32_to_bf16_bits(v.w) << 16));
}

template <int D>
struct Acc {
    static constexpr int CT = D / 4;              // threads of a row
    static constexpr int RG = kThreads / CT;      // row groups
    static constexpr int RPT = kRows / RG;        // rows of a thread: row = group + i * RG
    float4 o[RPT];
};

// Attention of rows [0, nr) over keys [k0, k1): leaves the unnormalised output in acc,
// maximum and sum in sm.m / sm.l.  q_row(r): the row's D elements; key(j, which): key
// or value row j (null: zeros); sees(r, j).  A key that a row does not see has weight
// zero and its value is not multiplied, whatever it holds.
template <typename T, int D, typename QRow, typename Key, typename Sees>
SFFN_DEV void attend(Smem<D> &sm, Acc<D> &acc, int nr, long long k0, long long k1, float scale, QRow q_row, Key key,
                     Sees sees) {
    constexpr int CT = Acc<D>::CT, RG = Acc<D>::RG, RPT = Acc<D>::RPT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    for (int i = tid; i < kRows * CT; i += kThreads) {
        const int r = i / CT, c = (i % CT) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nr) x = load4<T>(q_row(r) + c);
        *reinterpret_cast<float4 *>(&sm.q[r][c]) = make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
    }
    if (tid < kRows) sm.m[tid] = -INFINITY, sm.l[tid] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) acc.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long j0 = k0; j0 < k1; j0 += kKeys) {
        const int nk = (int)min((long long)kKeys, k1 - j0);
        for (int i = tid; i < kKeys * CT; i += kThreads) {
            const int j = i / CT, c = (i % CT) * 4;
            float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
            if (j < nk) {
                const T *kp = key(j0 + j, 0), *vp = key(j0 + j, 1);
                if (kp) kx = load4<T>(kp + c), vx = load4<T>(vp + c);
            }
            *reinterpret_cast<float4 *>(&sm.k[j][c]) = kx;
            *reinterpret_cast<float4 *>(&sm.v[j][c]) = vx;
        }
        __syncthreads();
        {
            const int j = tid & 63, g = tid >> 6;  // rows g * 16 .. + 15
            if (g * 16 < nr) {
                float s[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.f;
                for (int c = 0; c < D; c += 4) {
                    const float4 kx = *reinterpret_cast<const float4 *>(&sm.k[j][c]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 qx = *reinterpret_cast<const float4 *>(&sm.q[g * 16 + i][c]);
                        s[i] += qx.x * kx.x + qx.y * kx.y + qx.z * kx.z + qx.w * kx.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sm.p[g * 16 + i][j] = (g * 16 + i < nr && j < nk && sees(g * 16 + i, j0 + j)) ? s[i] : -INFINITY;
            }
        }
        __syncthreads();
        for (int r = warp; r < nr; r += kThreads / 32) {
            const float a0 = sm.p[r][lane], a1 = sm.p[r][lane + 32];
            const float mo = sm.m[r], mn = fmaxf(mo, warp_max(fmaxf(a0, a1)));
            const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is exp(-inf) = 0
            const float p0 = expf(a0 - ref), p1 = expf(a1 - ref);
            const float sum = warp_sum(p0 + p1);
            __syncwarp();
            // -1 marks a key that the row does not see: its value is left out, not multiplied by zero
            sm.p[r][lane] = a0 == -INFINITY ? -1.f : p0;
            sm.p[r][lane + 32] = a1 == -INFINITY ? -1.f : p1;
            if (lane == 0) {
                const float al = expf(mo - ref);
                sm.alpha[r] = al;
                sm.l[r] = sm.l[r] * al + sum;
                sm.m[r] = mn;
            }
        }
        __syncthreads();
        const int c = (tid % CT) * 4, g = tid / CT;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = g + i * RG;
            if (r < nr) {
                const float al = sm.alpha[r];
                float4 o = acc.o[i];
                o.x *= al, o.y *= al, o.z *= al, o.w *= al;
                for (int j = 0; j < nk; ++j) {
                    const float p = sm.p[r][j];
                    if (p >= 0.f || p != p) {
                        const float4 vx = *reinterpret_cast<const float4 *>(&sm.v[j][c]);
                        o.x += p * vx.x, o.y += p * vx.y, o.z += p * vx.z, o.w += p * vx.w;
                    }
                }
                acc.o[i] = o;
            }
        }
        __syncthreads();
    }
    __syncthreads();
}

}  // namespace rows
}  // namespace sffn
