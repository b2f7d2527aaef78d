// A whole MoE layer for a few tokens over resident MXFP4 experts (moe_mx4_layer).
#include "moe_mx4_gemm.cuh"

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
