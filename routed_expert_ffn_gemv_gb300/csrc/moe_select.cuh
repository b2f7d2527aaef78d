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

#ifdef __CUDACC__
// The same selection where its latency counts: logits lg[0 .. E) in shared memory (no NaN: those are
// -inf), one warp.  A logit is an unsigned key that orders like it; each step is one warp maximum of the
// keys and one warp minimum of the ids that hold it, and only the lane that lost its best looks for
// another.  Lanes 0 .. k-1 write ids / weights of row `row`.  (Measured on the decode layer: 0.6 us for 8
// of 128 where the shuffle selection took 3 to 5 us.)
__device__ __forceinline__ void select_topk_keys(const float *lg, int E, int k, int lane, size_t row,
                                                 int32_t *__restrict__ ids, float *__restrict__ weights) {
    auto key_of = [](float v) {
        const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and 0 are equal logits
        return b & 0x80000000u ? ~b : b | 0x80000000u;
    };
    unsigned taken = 0;
    uint32_t best = 0;
    int best_e = 0x7FFFFFFF;
    auto look = [&]() {
        best = 0;
        best_e = 0x7FFFFFFF;
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (!(taken >> (e >> 5) & 1u)) {
                const uint32_t q = key_of(lg[e]);
                if (best_e == 0x7FFFFFFF || q > best) {
                    best = q;
                    best_e = e;
                }
            }
    };
    look();
    int my_id = 0;
    float my_v = 0.f, top = 0.f;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        const int e = (int)__reduce_min_sync(0xffffffffu, best == m ? (unsigned)best_e : 0x7FFFFFFFu);
        const float v = lg[e];
        if (j == 0) top = v;
        if (lane == j) {
            my_id = e;
            my_v = v;
        }
        if ((e & 31) == lane) {
            taken |= 1u << (e >> 5);
            look();
        }
        __syncwarp();
    }
    const float x = lane < k ? expf(my_v - top) : 0.f;
    float sum = x;
#pragma unroll
    for (int o = 1; o < MOE_MAX_K; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < k) {
        ids[row * k + lane] = my_id;
        weights[row * k + lane] = x / sum;
    }
}
static_assert(MOE_MAX_K == 8, "the sum over the selected takes three exchanges");
#endif
