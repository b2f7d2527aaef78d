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
// The same selection where its latency counts, by a block of 256 threads: key[0 .. E) in shared memory
// (16-byte aligned, zeros up to a multiple of 4) holds select_key of the logits.  An expert's rank is the
// number of experts before it, counted by all threads at once, several to an expert; no step waits for
// another.  `sel`: 2 * MOE_MAX_K words.  Syncs the block once; after that the first warp writes ids /
// weights of row `row` and the others return.  (Measured on the decode layer, 8 of 128: the shuffle
// selection took 3 to 5 us.)
__device__ __forceinline__ uint32_t select_key(float v) {
    const uint32_t b = __float_as_uint((v != v ? -INFINITY : v) + 0.0f);  // NaN never wins; -0 equals 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float select_value(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ void select_topk_block(const uint32_t *key, int E, int k, uint32_t *sel, size_t row,
                                                  int32_t *__restrict__ ids, float *__restrict__ weights) {
    const int tid = threadIdx.x;
    int lg = 0;  // log2 of the experts' power of two: 256 >> lg threads (1 to 32) to an expert
    while ((1 << lg) < E) ++lg;
    const int lp = min(5, 8 - lg), part = tid & ((1 << lp) - 1), e = tid >> lp;
    const uint32_t mine = e < E ? key[e] : 0;
    int rank = 0;
#pragma unroll 4
    for (int j = 4 * part; j < E; j += 4 << lp) {
        const uint4 v = *(const uint4 *)(key + j);
        rank += (v.x > mine || (v.x == mine && j < e)) + (v.y > mine || (v.y == mine && j + 1 < e)) +
                (v.z > mine || (v.z == mine && j + 2 < e)) + (v.w > mine || (v.w == mine && j + 3 < e));
    }
    for (int o = 1; o < 1 << lp; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (e < E && part == 0 && rank < k) {
        sel[2 * rank] = (uint32_t)e;
        sel[2 * rank + 1] = mine;
    }
    __syncthreads();
    if (tid < 32) {
        const bool on = tid < k;
        const float x = on ? expf(select_value(sel[2 * tid + 1]) - select_value(sel[1])) : 0.f;
        float sum = x;
#pragma unroll
        for (int o = 1; o < MOE_MAX_K; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (on) {
            ids[row * k + tid] = (int32_t)sel[2 * tid];
            weights[row * k + tid] = x / sum;
        }
    }
}
static_assert(MOE_MAX_K == 8 && MOE_MAX_E == 256, "three exchanges over the selected, a thread per expert at least");
#endif
