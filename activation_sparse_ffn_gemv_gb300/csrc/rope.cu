// rope.cu -- per-head RMS norm of queries and keys, the position rotation and the
// paged cache's new key and value rows, in one pass (sm_103a).
//
// For a head row x of D elements: y = x w / sqrt(mean(x^2) + eps), then every pair
// (a, b) of the first rot elements turns by its position's angle:
// (a cos - b sin, b cos + a sin).  Everything between the load and the one rounding
// at the store is fp32.
//
// Bound: HBM (each row is read and written once; about 8 flops an element).  A lane
// holds 8 consecutive elements of a row, so a row of D takes D / 8 lanes and a warp
// D = 128: 2, D = 64: 4 rows at a time.  The norm's sum and, with half-split pairs, the
// partner elements cross lanes by shuffles; interleaved pairs stay in a lane.  A
// warp takes U rows of one token per lane group, all loads first, so that the
// token's table row is read once for them and U 16-byte loads are in flight a lane.
#include "common.cuh"
#include "internal.h"

namespace sffn {

namespace {

constexpr int kRopeWarps = 4;

template <typename T>
struct Row8;  // 8 elements of a lane

template <>
struct Row8<__nv_bfloat16> {
    uint4 u;
    SFFN_DEV void load(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    SFFN_DEV void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = u; }
    SFFN_DEV void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16lo(w[i]), f[2 * i + 1] = bf16hi(w[i]);
    }
    SFFN_DEV void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)f32_to_bf16_bits(f[2 * i]) | ((uint32_t)f32_to_bf16_bits(f[2 * i + 1]) << 16);
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    SFFN_DEV void zero() { u = make_uint4(0, 0, 0, 0); }
};

template <>
struct Row8<float> {
    float4 a, b;
    SFFN_DEV void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    SFFN_DEV void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    SFFN_DEV void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    SFFN_DEV void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    SFFN_DEV void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};

SFFN_DEV void load8(const float *p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(32 * kRopeWarps, 6) k_qk_norm_rope(const RopeArgs a) {
    constexpr int LPH = D / 8;       // lanes of a row
    constexpr int RPW = 32 / LPH;    // rows of a warp at a time
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, l = lane % LPH, grp = lane / LPH;
    const int hkv = a.hkv, hqk = a.hq + hkv;
    const int rows = hqk + (a.ck ? hkv : 0);  // rows of a token: q, k, and v for the cache
    const int chunks = (rows + RPW * U - 1) / (RPW * U);
    // below 2^31: at most 2^20 tokens of 1536 chunks
    const unsigned items = (unsigned)a.T * (unsigned)chunks, stride = gridDim.x * kRopeWarps;
    unsigned item = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);

    // Rows, position and slot of an item; the next item's are on their way while this one is worked
    // on (in an in-place call too: no warp writes another's rows).
    struct In {
        Row8<T> x[U];
        int t, c, p, slot;
    };
    auto fetch = [&](unsigned it, In &in) {
        const int t = (int)(it / (unsigned)chunks), c = (int)(it - (unsigned)t * (unsigned)chunks);
        in.t = t;
        in.c = c;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (c * U + u) * RPW + grp;
            const T *src = nullptr;
            if (r < a.hq)
                src = static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)r * D;
            else if (r < hqk)
                src = static_cast<const T *>(a.k) + (size_t)t * a.k_stride + (size_t)(r - a.hq) * D;
            else if (r < rows)
                src = static_cast<const T *>(a.v) + (size_t)t * a.v_stride + (size_t)(r - hqk) * D;
            if (src)
                in.x[u].load(src + l * 8);
            else
                in.x[u].zero();
        }
        in.p = a.rot ? a.positions[t] : 0;
        in.slot = a.ck ? a.slots[t] : -1;
    };
    In in;
    if (item < items) fetch(item, in);
    for (; item < items; item += stride) {
        Row8<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = in.x[u];
        const int t = in.t, c = in.c, p = in.p, slot = in.slot;
        if (item + stride < items) fetch(item + stride, in);
        if (a.rot && (p < 0 || p >= a.max_pos)) {
            if (lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
            continue;
        }
        // this lane's cosines and sines (of 8 pairs with half-split, of 4 with interleaved pairs)
        float cs[8], sn[8];
        const bool turns = l * 8 < a.rot;
        const bool low = l * 16 < a.rot;  // half-split: this lane holds the pairs' first elements
        const int half = a.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
        if (turns) {
            const float *row = a.table + (size_t)p * a.rot;
            if (a.style == SFFN_ROPE_HALF) {
                const int i0 = low ? l * 8 : l * 8 - half;
                load8(row + i0, cs);
                load8(row + half + i0, sn);
                if (low) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sn[i] = -sn[i];  // first element: a cos - b sin
                }
            } else {
                const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + l * 4));
                const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + l * 4));
                cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
                sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
            }
        }
        // lane of the pair's other half (half-split); itself when nothing turns
        const int partner = !turns ? lane : (low ? lane + a.rot / 16 : lane - a.rot / 16);

        // where the token's cache rows go
        long long crow = -1;  // row index of head 0 at this token's slot
        if (a.ck) {
            const int pg = slot >> a.page_shift;
            if (slot >= 0 && pg < a.n_pages)
                crow = (((long long)pg * hkv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
            else if (slot != -1 && lane == 0)
                record_error(a.err, SFFN_ERR_DEVICE);
        }

#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (c * U + u) * RPW + grp;
            float f[8];
            x[u].get(f);
            const void *w = r < a.hq ? a.q_weight : a.k_weight;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w && r < hqk) {
                Row8<T> wr;
                wr.load(static_cast<const T *>(w) + l * 8);
                float wf[8];
                wr.get(wf);
                const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * wf[i];
            }
            float y[8];
            if (a.style == SFFN_ROPE_HALF) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float o = __shfl_sync(0xffffffffu, f[i], partner);
                    y[i] = turns ? f[i] * cs[i] + o * sn[i] : f[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e0 = f[2 * i], e1 = f[2 * i + 1];
                    y[2 * i] = turns ? e0 * cs[i] - e1 * sn[i] : e0;
                    y[2 * i + 1] = turns ? e1 * cs[i] + e0 * sn[i] : e1;
                }
            }
            if (r < hqk) x[u].set(y);  // a value row goes on as it came
            if (r < a.hq) {
                x[u].store(static_cast<T *>(a.q_out) + ((size_t)t * a.hq + r) * D + l * 8);
            } else if (r < rows) {
                const bool is_k = r < hqk;
                const int h = is_k ? r - a.hq : r - hqk;
                if (is_k && a.k_out) x[u].store(static_cast<T *>(a.k_out) + ((size_t)t * hkv + h) * D + l * 8);
                if (crow >= 0)
                    x[u].store(static_cast<T *>(is_k ? a.ck : a.cv) + (size_t)(crow + ((long long)h << a.page_shift)) * D +
                               l * 8);
            }
        }
    }
}

template <typename T, int D, int U>
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s) {
    constexpr int per = (32 / (D / 8)) * U;
    const int rows = a.hq + a.hkv + (a.ck ? a.hkv : 0);
    const long long items = (long long)a.T * ((rows + per - 1) / per);
    long long grid = (items + kRopeWarps - 1) / kRopeWarps;
    const long long resident = 6LL * device_sm_count();
    if (grid > resident) grid = resident;
    return launch_k(k_qk_norm_rope<T, D, U>, dim3((unsigned)grid), dim3(32 * kRopeWarps), 0, s, a);
}

template <typename T, int D>
cudaError_t launch_rope_u(const RopeArgs &a, cudaStream_t s) {
    // Several rows a lane (64 bytes) once that still leaves every SM several warps; one row below
    // (the smallest calls: more warps, each with one load to wait for).
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const long long rows = (long long)a.T * (a.hq + 2 * a.hkv);
    return rows >= 64LL * device_sm_count() ? launch_rope<T, D, U>(a, s) : launch_rope<T, D, 1>(a, s);
}

}  // namespace

sffn_status run_qk_norm_rope(const RopeArgs &a, int dtype, int head_dim, cudaStream_t s) {
    cudaError_t e;
    if (dtype == SFFN_BF16)
        e = head_dim == 128 ? launch_rope_u<__nv_bfloat16, 128>(a, s) : launch_rope_u<__nv_bfloat16, 64>(a, s);
    else
        e = head_dim == 128 ? launch_rope_u<float, 128>(a, s) : launch_rope_u<float, 64>(a, s);
    return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA;
}

}  // namespace sffn
