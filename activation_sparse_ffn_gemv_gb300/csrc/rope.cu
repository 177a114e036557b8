// rope.cu -- per-head RMS norm of queries and keys, the position rotation and the
// paged cache's new key and value rows, in one pass (sm_103a).
//
// For a head row x of D elements: y = x w / sqrt(mean(x^2) + eps), then every pair
// (a, b) of the first rot elements turns by its position's angle:
// (a cos - b sin, b cos + a sin).  Everything between the load and the one rounding
// at the store is fp32.
//
// Bound: HBM (each row is read and written once; about 8 flops an element).  A lane
// holds four pairs of a row, so a row takes D / 8 lanes and a warp D = 128: 2, D = 64: 4 rows
// at a time.  With half-split pairs that is 4 elements at i and 4 at i + rot / 2, in two
// loads: both elements of a pair are in one lane and only the norm's sum crosses lanes (8
// consecutive elements and a shuffle of every partner: 183 us for 16384 tokens of
// 64 + 8 heads).  A warp takes U rows per lane group, all of one token and one kind (query, key
// or value), so that addresses, weights, cosines and sines are found once for them and
// all its loads are in flight together: 124 us there, 5.75 TB/s (0.85 of the measured copy
// rate); one token of 32 + 32 heads 1.8 us.
#include "common.cuh"
#include "internal.h"

namespace sffn {

namespace {

constexpr int kRopeWarps = 4;

// Four consecutive elements.
template <typename T>
struct Quad;

template <>
struct Quad<__nv_bfloat16> {
    uint2 u;
    SFFN_DEV void load(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    SFFN_DEV void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = u; }
    SFFN_DEV void get(float (&f)[4]) const { f[0] = bf16lo(u.x), f[1] = bf16hi(u.x), f[2] = bf16lo(u.y), f[3] = bf16hi(u.y); }
    SFFN_DEV void set(const float (&f)[4]) {
        __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        u = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
    }
    SFFN_DEV void zero() { u = make_uint2(0, 0); }
};

template <>
struct Quad<float> {
    float4 u;
    SFFN_DEV void load(const float *p) { u = __ldcs(reinterpret_cast<const float4 *>(p)); }
    SFFN_DEV void store(float *p) const { *reinterpret_cast<float4 *>(p) = u; }
    SFFN_DEV void get(float (&f)[4]) const { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
    SFFN_DEV void set(const float (&f)[4]) { u = make_float4(f[0], f[1], f[2], f[3]); }
    SFFN_DEV void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
};

template <typename T, int D, int U, bool HALF>
__global__ void __launch_bounds__(32 * kRopeWarps, 8) k_qk_norm_rope(const RopeArgs a, int cq, int ck) {
    constexpr int LPH = D / 8;       // lanes of a row
    constexpr int RPW = 32 / LPH;    // rows of a warp at a time
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, l = lane % LPH, grp = lane / LPH;
    // an item: up to RPW * U rows of one token, all queries, all keys or all values
    const int chunks = cq + (a.ck ? 2 : 1) * ck;
    // below 2^31: at most 2^20 tokens of 1536 chunks
    const unsigned item = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    if (item >= (unsigned)a.T * (unsigned)chunks) return;
    const int t = (int)(item / (unsigned)chunks), c = (int)(item - (unsigned)t * (unsigned)chunks);
    const int kind = c < cq ? 0 : (c < cq + ck ? 1 : 2);  // q, k, v
    const int r0 = (c - (kind == 0 ? 0 : (kind == 1 ? cq : cq + ck))) * (RPW * U) + grp, heads = kind == 0 ? a.hq : a.hkv;

    // this lane's elements: o0 .. o0 + 3 and o1 .. o1 + 3
    const bool turns = l * 8 < a.rot;
    const int o0 = turns && HALF ? l * 4 : l * 8, o1 = turns && HALF ? a.rot / 2 + l * 4 : l * 8 + 4;
    const T *src = static_cast<const T *>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) +
                   (size_t)t * (kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride)) + (size_t)r0 * D;
    Quad<T> x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (r0 + u * RPW < heads) {
            x[u][0].load(src + u * RPW * D + o0);
            x[u][1].load(src + u * RPW * D + o1);
        } else {
            x[u][0].zero();
            x[u][1].zero();
        }
    }
    int p = 0, slot = -1;
    if (a.rot) p = a.positions[t];
    if (a.ck && kind > 0) slot = a.slots[t];
    const T *w = static_cast<const T *>(kind == 0 ? a.q_weight : a.k_weight);
    float wf[2][4];
    if (kind < 2 && w) {
        Quad<T> wx;
        wx.load(w + o0);
        wx.get(wf[0]);
        wx.load(w + o1);
        wx.get(wf[1]);
    }
    if (a.rot && (p < 0 || p >= a.max_pos)) {
        if (lane == 0) record_error(a.err, SFFN_ERR_DEVICE);
        return;
    }
    T *out = nullptr;      // packed rows of the kind, if any
    if (kind == 0)
        out = static_cast<T *>(a.q_out) + ((size_t)t * a.hq + r0) * D;
    else if (kind == 1 && a.k_out)
        out = static_cast<T *>(a.k_out) + ((size_t)t * a.hkv + r0) * D;
    T *cache = nullptr;    // the token's row of head r0 in the cache, if it has one; heads lie `step` apart
    const size_t step = (size_t)D << a.page_shift;
    if (a.ck && kind > 0) {
        const int pg = slot >> a.page_shift;
        if (slot >= 0 && pg < a.n_pages)
            cache = static_cast<T *>(kind == 1 ? a.ck : a.cv) + ((size_t)pg * a.hkv + r0) * step +
                    (size_t)(slot & ((1 << a.page_shift) - 1)) * D;
        else if (slot != -1 && lane == 0)
            record_error(a.err, SFFN_ERR_DEVICE);
    }
    if (kind < 2) {  // a value row goes on as it came
        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns) {
            const float *row = a.table + (size_t)p * a.rot + l * 4;
            cs = __ldg(reinterpret_cast<const float4 *>(row));
            sn = __ldg(reinterpret_cast<const float4 *>(row + a.rot / 2));
        }
        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[2][4];
            x[u][0].get(f[0]);
            x[u][1].get(f[1]);
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss += f[i >> 2][i & 3] * f[i >> 2][i & 3];
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i >> 2][i & 3] *= inv * wf[i >> 2][i & 3];
            }
            if (turns) {
                float y[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // half-split: pair i is (f[0][i], f[1][i]); interleaved: (f[i / 2][2 (i % 2)], its neighbour)
                    const float ea = HALF ? f[0][i] : f[i >> 1][(i & 1) * 2];
                    const float eb = HALF ? f[1][i] : f[i >> 1][(i & 1) * 2 + 1];
                    y[0][i] = ea * cv[i] - eb * sv[i];
                    y[1][i] = eb * cv[i] + ea * sv[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[0][i] = HALF ? y[0][i] : y[i & 1][i >> 1];
                    f[1][i] = HALF ? y[1][i] : y[i & 1][2 + (i >> 1)];
                }
            }
            x[u][0].set(f[0]);
            x[u][1].set(f[1]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (r0 + u * RPW < heads) {
            if (out) {
                x[u][0].store(out + u * RPW * D + o0);
                x[u][1].store(out + u * RPW * D + o1);
            }
            if (cache) {
                T *d = cache + (size_t)(u * RPW) * step;
                x[u][0].store(d + o0);
                x[u][1].store(d + o1);
            }
        }
    }
}

template <typename T, int D, int U>
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s) {
    constexpr int per = (32 / (D / 8)) * U;
    const int cq = (a.hq + per - 1) / per, ck = (a.hkv + per - 1) / per;
    const long long items = (long long)a.T * (cq + (a.ck ? 2 : 1) * ck);
    const long long grid = (items + kRopeWarps - 1) / kRopeWarps;
    auto k = a.style == SFFN_ROPE_HALF ? k_qk_norm_rope<T, D, U, true> : k_qk_norm_rope<T, D, U, false>;
    return launch_k(k, dim3((unsigned)grid), dim3(32 * kRopeWarps), 0, s, a, cq, ck);
}

template <typename T, int D>
cudaError_t launch_rope_u(const RopeArgs &a, cudaStream_t s) {
    // Several rows a lane (64 bytes) once that still leaves every SM several warps; one row below
    // (the smallest calls: more warps, each with one row to wait for).
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
