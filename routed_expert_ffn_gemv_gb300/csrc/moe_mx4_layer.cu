// A whole MoE layer for a few tokens over resident MXFP4 experts (moe_mx4_layer).
#include "moe_mx4_gemm.cuh"

namespace {

// One warp per output element pair: lanes walk the 32-column blocks of K.
template <int IN>  // MOE_MXFP4: codes + scales rows; MOE_F32 + 16 / MOE_BF16 + 16: plain rows
struct Act {
    const void *p;
    const uint8_t *scales;
    int K;
    __device__ void block(size_t row, int b, float (&v)[32]) const {
        if (IN == MOE_MXFP4) {
            const uint8_t *c = (const uint8_t *)p + row * (K / 2) + 16 * b;
            const float m = e8m0_value(scales[row * (K / 32) + b]);
            for (int i = 0; i < 16; ++i) {
                v[2 * i] = e2m1_value(c[i] & 15) * m;
                v[2 * i + 1] = e2m1_value(c[i] >> 4) * m;
            }
        } else if (IN == MOE_BF16 + 16) {
            for (int i = 0; i < 32; ++i) v[i] = __bfloat162float(((const __nv_bfloat16 *)p)[row * K + 32 * b + i]);
        } else {
            for (int i = 0; i < 32; ++i) v[i] = ((const float *)p)[row * K + 32 * b + i];
        }
    }
};

__device__ float weight_dot(const uint8_t *m, int B, int row, int b, const float (&v)[32]) {
    const uint8_t *c = m + mx4_code_offset(B, row, 32 * b);
    float s = 0.f;
    for (int i = 0; i < 16; ++i)
        s += e2m1_value(c[i] & 15) * v[2 * i] + e2m1_value(c[i] >> 4) * v[2 * i + 1];
    return s * e8m0_value(m[mx4_scale_offset(B, row, 32 * b)]);
}

__device__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ const uint8_t *image_of(int e, int E, const int32_t *table, int n_slots, const void *pool,
                                   size_t slot_bytes, int *status) {
    if (e == -1) return nullptr;
    int slot = -1;
    if (e >= 0 && e < E) slot = table ? table[e] : e;
    if (slot < 0 || slot >= n_slots) {
        moe_set_status(status, MOE_ERR_INVALID);
        return nullptr;
    }
    return (const uint8_t *)pool + (size_t)slot * slot_bytes;
}

template <int IN, int OUT>
__global__ void gateup_simple(Act<IN> x, int k, int H, int F, int E, const int32_t *ids, const int32_t *table,
                              int n_slots, const void *pool, size_t slot_bytes, void *h, int *status) {
    const int r = blockIdx.x, lane = threadIdx.x & 31;
    const uint8_t *m = image_of(ids[r], E, table, n_slots, pool, slot_bytes, status);
    if (!m) return;
    const int B = (H + 127) / 128;
    for (int f = blockIdx.y * 8 + threadIdx.x / 32; f < F; f += gridDim.y * 8) {
        float g = 0.f, u = 0.f;
        for (int b = lane; b < H / 32; b += 32) {
            float v[32];
            x.block(r / k, b, v);
            g += weight_dot(m, B, mx4_gate_row(f), b, v);
            u += weight_dot(m, B, mx4_gate_row(f) + 64, b, v);
        }
        g = warp_sum(g);
        u = warp_sum(u);
        const float y = g / (1.0f + expf(-g)) * u;
        if (lane == 0) {
            if (OUT == MOE_BF16) ((__nv_bfloat16 *)h)[(size_t)r * F + f] = __float2bfloat16(y);
            else ((float *)h)[(size_t)r * F + f] = y;
        }
    }
}

template <int IN>
__global__ void down_simple(Act<IN> hq, int H, int F, int E, const int32_t *ids, const float *weights,
                            const int32_t *table, int n_slots, const void *pool, size_t slot_bytes, float *partial,
                            int *status) {
    const int r = blockIdx.x, lane = threadIdx.x & 31;
    const uint8_t *m = image_of(ids[r], E, table, n_slots, pool, slot_bytes, status);
    if (!m) return;
    m += mx4_gu_bytes(H, F);
    const int B = (F + 127) / 128;
    const float w = weights[r];
    for (int o = blockIdx.y * 8 + threadIdx.x / 32; o < H; o += gridDim.y * 8) {
        float y = 0.f;
        for (int b = lane; b < F / 32; b += 32) {
            float v[32];
            hq.block(r, b, v);
            y += weight_dot(m, B, o, b, v);
        }
        y = warp_sum(y);
        if (lane == 0) partial[(size_t)r * H + o] = w * y;
    }
}

}  // namespace

static int mx4_simple_gateup_plain(const void *x, int xtype, int T, int H, int F, int E, int k, const int32_t *ids,
                            const int32_t *table, int n_slots, const void *pool, size_t slot_bytes, float *h,
                            cudaStream_t s) {
    int *status = moe_status_word_device_ptr();
    const dim3 g(T * k, (F + 7) / 8);
    if (xtype == MOE_BF16)
        gateup_simple<MOE_BF16 + 16, MOE_F32><<<g, 256, 0, s>>>({x, nullptr, H}, k, H, F, E, ids, table, n_slots, pool,
                                                                slot_bytes, h, status);
    else
        gateup_simple<MOE_F32 + 16, MOE_F32><<<g, 256, 0, s>>>({x, nullptr, H}, k, H, F, E, ids, table, n_slots, pool,
                                                               slot_bytes, h, status);
    MOE_TRY_CUDA(cudaGetLastError());
    return MOE_OK;
}

static int mx4_simple_down_plain(const float *h, int T, int H, int F, int E, int k, const int32_t *ids, const float *weights,
                          const int32_t *table, int n_slots, const void *pool, size_t slot_bytes, float *partial,
                          cudaStream_t s) {
    down_simple<MOE_F32 + 16><<<dim3(T * k, (H + 7) / 8), 256, 0, s>>>({h, nullptr, F}, H, F, E, ids, weights, table,
                                                                       n_slots, pool, slot_bytes, partial,
                                                                       moe_status_word_device_ptr());
    MOE_TRY_CUDA(cudaGetLastError());
    return MOE_OK;
}


namespace {

struct LayerWs {
    size_t ids, weights, h, partial, total;
};

LayerWs layer_ws(int T, int H, int F, int k) {
    LayerWs L;
    const size_t R = (size_t)T * k;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o += (n + 255) / 256 * 256;
        return at;
    };
    L.ids = take(R * 4);
    L.weights = take(R * 4);
    L.h = take(R * F * 4);
    L.partial = take(R * H * 4);
    L.total = o;
    return L;
}

}  // namespace

extern "C" int moe_mx4_layer_workspace(int T, int H, int F, int E, int k, size_t *bytes) {
    MOE_CHECK(bytes);
    const int rc = mx4_ffn_check(T, H, F, E, k);
    if (rc != MOE_OK) return rc;
    MOE_CHECK(T <= MOE_DECODE_MAX_T);
    *bytes = layer_ws(T, H, F, k).total;
    return MOE_OK;
}

extern "C" int moe_mx4_layer(const void *x, int xtype, int T, int H, int F, int E, int k, const uint16_t *w_router,
                             const float *bias, const int32_t *d_slot_table, int n_slots, const void *pool,
                             size_t slot_bytes, const float *extra, float *y, int32_t *ids, float *weights,
                             void *workspace, size_t ws_bytes, moe_stream_t s) {
    size_t need = 0;
    int rc = moe_mx4_layer_workspace(T, H, F, E, k, &need);
    if (rc != MOE_OK) return rc;
    MOE_CHECK(xtype == MOE_F32 || xtype == MOE_BF16);
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && w_router && y && workspace && ws_bytes >= need && ((uintptr_t)workspace & 255) == 0);
    if ((rc = mx4_pool_check(H, F, n_slots, pool, slot_bytes)) != MOE_OK) return rc;
    const LayerWs L = layer_ws(T, H, F, k);
    uint8_t *w = (uint8_t *)workspace;
    if (!ids) ids = (int32_t *)(w + L.ids);
    if (!weights) weights = (float *)(w + L.weights);
    float *h = (float *)(w + L.h), *partial = (float *)(w + L.partial);
    cudaStream_t st = moe_cuda_stream(s);
    if ((rc = moe_router_topk(x, xtype, T, H, w_router, bias, E, k, ids, weights, nullptr, s)) != MOE_OK) return rc;
    MOE_TRY_CUDA(cudaMemsetAsync(partial, 0, (size_t)T * k * H * 4, st));
    if ((rc = mx4_simple_gateup_plain(x, xtype, T, H, F, E, k, ids, d_slot_table, n_slots, pool, slot_bytes, h, st)) !=
        MOE_OK)
        return rc;
    if ((rc = mx4_simple_down_plain(h, T, H, F, E, k, ids, weights, d_slot_table, n_slots, pool, slot_bytes, partial,
                                    st)) != MOE_OK)
        return rc;
    return moe_combine(partial, T, k, H, extra, y, s);
}
