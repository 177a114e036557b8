// attn_warp.cuh -- attention of one (token, query head) row by one warp, fp32 arithmetic: the plain form
// of the kernels over the paged cache.
#pragma once

#include "attn.cuh"

namespace sffn {

// D / 32 consecutive elements a lane.
template <int C>
SFFN_DEV void lane_load(const __nv_bfloat16 *p, float (&f)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) f[i] = bf16_to_f32(p[i]);
}
template <int C>
SFFN_DEV void lane_load(const float *p, float (&f)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) f[i] = p[i];
}
SFFN_DEV void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
SFFN_DEV void put(float *p, float x) { *p = x; }

template <typename T, int D>
struct WarpRow {
    static constexpr int C = D / 32;
    float q[C], o[C], m, l;
    SFFN_DEV void begin(const T *row, float scale, int lane) {
        lane_load<C>(row + lane * C, q);
#pragma unroll
        for (int i = 0; i < C; ++i) q[i] *= scale, o[i] = 0.f;
        m = -INFINITY, l = 0.f;
    }
    // One key and its value (null: zeros).
    SFFN_DEV void add(const T *k, const T *v, int lane) {
        float x[C] = {}, y[C] = {}, s = 0.f;
        if (k) {
            lane_load<C>(k + lane * C, x);
            lane_load<C>(v + lane * C, y);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) s += q[i] * x[i];
        s = warp_sum(s);
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn, f = expf(m - ref), p = expf(s - ref);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = o[i] * f + p * y[i];
        m = mn;
    }
    SFFN_DEV void end(T *row, int lane) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < C; ++i) put(row + lane * C + i, o[i] * inv);
    }
};

}  // namespace sffn
