// moe_grouped_matmul and moe_grouped_weight_grad: checks, tensor maps and launches of the kernel in moe_grouped.cuh.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "moe_grouped.cuh"

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    });
    return fn;
}

bool type16(int t) { return t == MOE_BF16 || t == MOE_F16; }
size_t type_bytes(int t) { return t == MOE_F32 ? 4 : 2; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// What both calls check of their groups and of a matrix of rows (of 16-bit elements).
int check_groups(int G, int R) {
    MOE_CHECK(G >= 1 && G <= MOE_MAX_GROUPS && R >= 0 && R <= 1 << 24);
    return MOE_OK;
}
int check_sizes(int N, int K) {
    MOE_CHECK(N >= 1 && K >= 1);
    if (N % 8 || K % 8 || N > 1 << 16 || K > 1 << 16) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
int check_rows(int rows, int cols, size_t ld) {
    MOE_CHECK(rows >= 0 && ld >= (size_t)cols && ld % 8 == 0 && ld <= (size_t)1 << 32);
    return MOE_OK;
}

// Rows in boxes of 64 elements of `box` rows.
int rows_map(CUtensorMap *map, int type, const void *x, int rows, int cols, size_t ld, int box) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
    const uint32_t b[2] = {64, (uint32_t)box};
    return grouped_map(map, type, 2, x, dims, strides, b, 128);
}

}  // namespace

int grouped_sms() {
    static std::atomic<int> sms[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = sms[dev].load();
    if (!n && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) sms[dev].store(n);
    return n;
}

int grouped_map(CUtensorMap *map, int type, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box, int swizzle_bytes) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return MOE_ERR_UNSUPPORTED;
    cuuint64_t d[4], st[3];
    cuuint32_t b[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i + 1 < rank) st[i] = strides[i];
    }
    if (enc(map,
            type == MOE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
            : type == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            (cuuint32_t)rank, (void *)base, d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
            : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

extern "C" int moe_grouped_matmul(const void *x, int type, int x_rows, size_t ldx, const int32_t *x_index, int x_share,
                                  const int32_t *offsets, int G, int R, const void *w, int w_order, int N, int K, int act,
                                  const float *scale, const int32_t *y_index, void *y, int ytype, int y_rows, size_t ldy,
                                  moe_stream_t s) {
    MOE_CHECK(type16(type) && (ytype == MOE_F32 || type16(ytype)) && (w_order == MOE_ORDER_NK || w_order == MOE_ORDER_KN));
    MOE_CHECK(act == MOE_ACT_NONE || act == MOE_ACT_SWIGLU);
    int rc = check_groups(G, R);
    if (rc != MOE_OK || (rc = check_sizes(N, K)) != MOE_OK) return rc;
    if ((rc = check_rows(x_rows, K, ldx)) != MOE_OK || (rc = check_rows(y_rows, N, ldy)) != MOE_OK) return rc;
    MOE_CHECK(!x_index || x_share >= 1);
    if (act == MOE_ACT_SWIGLU && w_order != MOE_ORDER_NK) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    MOE_CHECK(x && offsets && w && y && x_rows >= 1 && y_rows >= 1);
    MOE_CHECK(aligned16(x) && aligned16(w) && aligned16(y) && ((uintptr_t)scale & 3) == 0);

    const bool swiglu = act == MOE_ACT_SWIGLU;
    const int mode = swiglu ? GP_SWIGLU : w_order == MOE_ORDER_NK ? GP_NK : GP_KN;
    // few rows, and no more rows of the matrices than CTAs run at once (one row, N = 1536: 7.9 -> 5.5 us by the kernel for few
    // rows; eight rows of eight groups 12.8 -> 14.7)
    if (mode != GP_KN && R <= 8 && (long long)std::min(R, G) * ((N + 15) / 16) <= 2LL * grouped_sms()) {
        GroupedFewParams f = {};
        f.x = (const uint16_t *)x;
        f.w = (const uint16_t *)w;
        f.ldx = ldx;
        f.offsets = offsets;
        f.G = G;
        f.R = R;
        f.x_index = x_index;
        f.x_share = x_share;
        f.x_rows = x_rows;
        f.y_index = y_index;
        f.y_rows = y_rows;
        f.scale = scale;
        f.y = y;
        f.ldy = ldy;
        f.ytype = ytype;
        f.M = N;
        f.K = K;
        f.status = moe_status_word_device_ptr();
        return grouped_few_launch(f, mode, type == MOE_BF16, moe_cuda_stream(s));
    }
    GroupedParams p = {};
    if (swiglu) {
        const uint64_t dims[4] = {(uint64_t)K, (uint64_t)N, 2, (uint64_t)G};
        const uint64_t strides[3] = {(uint64_t)K * 2, (uint64_t)N * K * 2, (uint64_t)N * K * 4};
        const uint32_t box[4] = {64, 16, 2, 1};
        rc = grouped_map(&p.a, type, 4, w, dims, strides, box, 128);
    } else {
        const uint64_t in = mode == GP_NK ? K : N, out = mode == GP_NK ? N : K;
        const uint64_t dims[3] = {in, out, (uint64_t)G}, strides[2] = {in * 2, in * out * 2};
        const uint32_t box[3] = {64, mode == GP_NK ? 128u : 64u, 1};
        rc = grouped_map(&p.a, type, 3, w, dims, strides, box, 128);
    }
    if (rc != MOE_OK || (rc = rows_map(&p.b, type, x, x_rows, K, ldx, 16)) != MOE_OK) return rc;
    if ((rc = rows_map(&p.b64, type, x, x_rows, K, ldx, 64)) != MOE_OK) return rc;
    p.rows = (const uint16_t *)x;
    p.ld = ldx;
    p.offsets = offsets;
    p.G = G;
    p.R = R;
    p.x_index = x_index;
    p.x_share = x_share;
    p.x_rows = x_rows;
    p.y_index = y_index;
    p.y_rows = y_rows;
    p.scale = scale;
    p.y = y;
    p.ldy = ldy;
    p.M = N;
    p.K = K;
    p.fmt = type == MOE_BF16;
    p.status = moe_status_word_device_ptr();
    // few rows to a group: narrow tiles, one CTA each (gate/up, 32 experts of 2 x 512 x 1024: 8 rows an expert 13.5 us against 15.8
    // by pairs, 32 rows 18.3 against 16.0; 128 experts of 2 x 768 x 2048, 8 rows 126 against 134, 64 rows 233 against 138)
    const bool wide = R > 16LL * G;
    const int nt = !wide ? 32 : ytype != MOE_F32 ? 256 : 128, mrows = (swiglu ? 64 : 128) * (wide ? 2 : 1);
    const long long row_tiles = (long long)R / nt + std::min(G, R);
    return grouped_launch(p, ytype, mode, wide, row_tiles * ((N + mrows - 1) / mrows), (K + 63) / 64, moe_cuda_stream(s));
}

extern "C" int moe_grouped_weight_grad(const void *x, int type, int x_rows, size_t ldx, const int32_t *x_index,
                                       int x_share, const void *dy, int dy_rows, size_t lddy, const int32_t *dy_index,
                                       const int32_t *offsets, int G, int R, int N, int K, int accumulate, void *dw,
                                       int wtype, moe_stream_t s) {
    MOE_CHECK(type16(type) && (wtype == MOE_F32 || type16(wtype)) && (accumulate == 0 || accumulate == 1));
    int rc = check_groups(G, R);
    if (rc != MOE_OK || (rc = check_sizes(N, K)) != MOE_OK) return rc;
    if ((rc = check_rows(x_rows, K, ldx)) != MOE_OK || (rc = check_rows(dy_rows, N, lddy)) != MOE_OK) return rc;
    MOE_CHECK(!x_index || x_share >= 1);
    MOE_CHECK(dw && aligned16(dw));
    if (R == 0) {
        // (no rows: nothing to add)
        if (!accumulate)
            MOE_TRY_CUDA(cudaMemsetAsync(dw, 0, (size_t)G * N * K * type_bytes(wtype), moe_cuda_stream(s)));
        return MOE_OK;
    }
    MOE_CHECK(x && dy && offsets && x_rows >= 1 && dy_rows >= 1 && aligned16(x) && aligned16(dy));

    GroupedParams p = {};
    if ((rc = rows_map(&p.a, type, x, x_rows, K, ldx, 64)) != MOE_OK) return rc;
    if ((rc = rows_map(&p.b, type, dy, dy_rows, N, lddy, 64)) != MOE_OK) return rc;
    {
        const uint64_t size = type_bytes(wtype), dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)G};
        const uint64_t strides[2] = {K * size, (uint64_t)N * K * size};
        const uint32_t box[3] = {32, wtype == MOE_F32 ? 16u : 32u, 1};
        if ((rc = grouped_map(&p.yt, wtype, 3, dw, dims, strides, box, wtype == MOE_F32 ? 0 : 64)) != MOE_OK) return rc;
    }
    p.rows = (const uint16_t *)x;
    p.ld = ldx;
    p.dy = (const uint16_t *)dy;
    p.lddy = lddy;
    p.offsets = offsets;
    p.G = G;
    p.R = R;
    p.x_index = x_index;
    p.x_share = x_share;
    p.x_rows = x_rows;
    p.y_index = dy_index;
    p.y_rows = dy_rows;
    p.y = dw;
    p.ldy = K;
    p.M = K;
    p.N = N;
    p.accumulate = accumulate;
    p.fmt = type == MOE_BF16;
    p.status = moe_status_word_device_ptr();
    const int nt = wtype == MOE_F32 && !grouped_grad_short(R, G) ? 128 : 256;
    const long long items = (long long)G * ((N + nt - 1) / nt) * ((K + 255) / 256);
    return grouped_launch(p, wtype, GP_GRAD, true, items, 0, moe_cuda_stream(s));
}
