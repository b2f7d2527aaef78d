// Top-k selection and softmax over the selected, by one warp (shared by the router kernels and the
// MXFP4 layer).
#pragma once

#include <math.h>

#include "moe_common.cuh"

// (v, id) ordering of the selection: larger logit first, then lower id.
__device__ __forceinline__ bool better(float v1, int i1, float v2, int i2) {
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

// Top-k of one token's logits held by a warp (lane l holds experts l, l+32, ...; -inf
// beyond E), larger first and ties to the lower id, then the softmax over the k selected;
// lanes 0..k-1 write ids/weights of row `row`.
__device__ __forceinline__ void select_topk_softmax(const float (&v)[MOE_MAX_E / 32], int E, int k, int lane,
                                                    size_t row, int32_t *__restrict__ ids,
                                                    float *__restrict__ weights, float min_w) {
    constexpr int NPL = MOE_MAX_E / 32;
    unsigned taken = 0;
    float sel_v[MOE_MAX_K];
    int sel_i[MOE_MAX_K];
    for (int j = 0; j < k; ++j) {
        float bv = -INFINITY;
        int bi = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < E && !(taken >> i & 1u) && better(v[i], e, bv, bi)) {
                bv = v[i];
                bi = e;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
            if (better(ov, oi, bv, bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
        sel_v[j] = bv;
        sel_i[j] = bi;
    }
    float denom = 0.f;
    for (int j = 0; j < k; ++j) denom += expf(sel_v[j] - sel_v[0]);
    if (lane < k) {
        float myv = sel_v[0];
        int myi = sel_i[0];
        for (int j = 1; j < k; ++j)
            if (j == lane) {
                myv = sel_v[j];
                myi = sel_i[j];
            }
        // a route whose weight is below the load threshold is dropped: id -1, weight 0
        const float w = expf(myv - sel_v[0]) / denom;
        const bool drop = w < min_w;
        ids[row * k + lane] = drop ? -1 : myi;
        weights[row * k + lane] = drop ? 0.f : w;
    }
}
