// moe_lora_matmul: a shared projection and each token's low-rank adapter in one product.
//
//   y[t] = W x_t + B_a u_t,   u_t = scale[a] A_a x_t,   a = adapter[t]
// Two kernels.  lora_shrink_kernel computes u in fp32 and leaves it as two 16-bit halves (the nearest, and the nearest of what
// is left: 16 bits of bf16, 22 of fp16), 32 ranks to a 128-byte row piece, upper halves first.  The product's kernel (moe_grouped.cuh, GP_LORA) runs K on into the ranks: for each adapter that has tokens in
// its tile, 32 ranks at a time, B_a's tile against the tokens' rows of u, zeros for the tokens of other adapters.  So y
// is rounded once and W's part and the adapters' share an accumulator.  The product starts beside the first kernel and waits
// for u only where it loads it.
#include <algorithm>

#include "moe_grouped.cuh"

namespace {

#define LS_RANKS 4  // ranks of a warp

template <bool BF>
__device__ __forceinline__ float2 pair_value(uint32_t w) {
    if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*(const __half2 *)&w);
}
template <bool BF>
__device__ __forceinline__ void split16(float v, uint16_t &hi, uint16_t &lo) {
    if (BF) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v), l = __float2bfloat16_rn(v - __bfloat162float(h));
        hi = __bfloat16_as_ushort(h);
        lo = __bfloat16_as_ushort(l);
    } else {
        const __half h = __float2half_rn(v), l = __float2half_rn(v - __half2float(h));
        hi = __half_as_ushort(h);
        lo = __half_as_ushort(l);
    }
}

// A warp: LS_RANKS ranks of one token.  u: [T][chunks][64].
template <bool BF>
__global__ void __launch_bounds__(256) lora_shrink_kernel(const uint16_t *x, size_t ldx, int T, int K, const int32_t *adapter,
                                                          int n_adapters, const uint16_t *a, int rank, const float *scale,
                                                          uint16_t *u) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % 32, chunks = (rank + 31) / 32, groups = chunks * 32 / LS_RANKS;
    const long long job = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    const int t = (int)(job / groups), j0 = (int)(job % groups) * LS_RANKS;
    if (t >= T) return;
    const int ad = adapter[t];
    if (ad < 0 || ad >= n_adapters) return;  // (no product reads this row)
    float v[LS_RANKS] = {};
    if (j0 < rank) {
        const uint16_t *xr = x + (size_t)t * ldx, *ar = a + ((size_t)ad * rank + j0) * K;
        for (int k = 8 * lane; k < K; k += 256) {
            const uint4 xv = *(const uint4 *)(xr + k);
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int j = 0; j < LS_RANKS; ++j) {  // (the rank is a multiple of 8)
                const uint4 av = *(const uint4 *)(ar + (size_t)j * K + k);
                const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = pair_value<BF>(xw[i]), q = pair_value<BF>(aw[i]);
                    v[j] = fmaf(p.x, q.x, v[j]);
                    v[j] = fmaf(p.y, q.y, v[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < LS_RANKS; ++j)
#pragma unroll
            for (int d = 16; d > 0; d /= 2) v[j] += __shfl_xor_sync(0xffffffffu, v[j], d);
    }
    if (lane < LS_RANKS) {
        float r = 0.f;
#pragma unroll
        for (int j = 0; j < LS_RANKS; ++j)
            if (j == lane) r = v[j];
        if (scale) r *= scale[ad];
        if (j0 >= rank) r = 0.f;
        uint16_t hi, lo;
        split16<BF>(r, hi, lo);
        const int j = j0 + lane;
        uint16_t *row = u + ((size_t)t * chunks + j / 32) * 64 + j % 32;
        row[0] = hi;
        row[32] = lo;
    }
}

int check(int T, int rank) {
    MOE_CHECK(T >= 0 && T <= 1 << 24 && rank >= 1);
    if (rank % 8 || rank > MOE_MAX_RANK) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" int moe_lora_workspace(int T, int rank, size_t *bytes) {
    MOE_CHECK(bytes);
    const int rc = check(T, rank);
    if (rc != MOE_OK) return rc;
    *bytes = (size_t)T * ((rank + 31) / 32) * 128;
    return MOE_OK;
}

extern "C" int moe_lora_matmul(const void *x, int type, int T, size_t ldx, const void *w, int N, int K,
                               const int32_t *adapter, int n_adapters, const void *a, const void *b, int rank,
                               const float *scale, void *y, int ytype, size_t ldy, void *workspace, size_t ws_bytes,
                               moe_stream_t s) {
    size_t need = 0;
    int rc = moe_lora_workspace(T, rank, &need);
    if (rc != MOE_OK) return rc;
    MOE_CHECK((type == MOE_BF16 || type == MOE_F16) && (ytype == MOE_F32 || ytype == MOE_BF16 || ytype == MOE_F16));
    MOE_CHECK(N >= 1 && K >= 1 && n_adapters >= 1);
    if (N % 8 || K % 8 || N > 1 << 16 || K > 1 << 16) return MOE_ERR_UNSUPPORTED;
    MOE_CHECK(ldx >= (size_t)K && ldx % 8 == 0 && ldx <= (size_t)1 << 32 && ldy >= (size_t)N && ldy % 8 == 0);
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && w && adapter && a && b && y && workspace && ws_bytes >= need);
    MOE_CHECK((((uintptr_t)x | (uintptr_t)w | (uintptr_t)a | (uintptr_t)b | (uintptr_t)y) & 15) == 0);
    MOE_CHECK(((uintptr_t)workspace & 255) == 0);

    const int chunks = (rank + 31) / 32;
    GroupedParams p = {};
    {
        const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, 1}, strides[2] = {(uint64_t)K * 2, (uint64_t)N * K * 2};
        const uint32_t box[3] = {64, 128, 1};
        if ((rc = grouped_map(&p.a, type, 3, w, dims, strides, box, 128)) != MOE_OK) return rc;
    }
    {
        const uint64_t dims[2] = {(uint64_t)K, (uint64_t)T}, strides[1] = {(uint64_t)ldx * 2};
        const uint32_t box[2] = {64, 16}, box64[2] = {64, 64};
        if ((rc = grouped_map(&p.b, type, 2, x, dims, strides, box, 128)) != MOE_OK) return rc;
        if ((rc = grouped_map(&p.b64, type, 2, x, dims, strides, box64, 128)) != MOE_OK) return rc;
    }
    {
        const uint64_t dims[3] = {(uint64_t)rank, (uint64_t)N, (uint64_t)n_adapters};
        const uint64_t strides[2] = {(uint64_t)rank * 2, (uint64_t)N * rank * 2};
        const uint32_t box[3] = {32, 128, 1};
        if ((rc = grouped_map(&p.ab, type, 3, b, dims, strides, box, 64)) != MOE_OK) return rc;
    }
    p.rows = (const uint16_t *)workspace;
    p.ld = (size_t)chunks * 64;
    p.G = 1;
    p.R = T;
    p.x_rows = T;
    p.y_rows = T;
    p.x_share = 1;
    p.y = y;
    p.ldy = ldy;
    p.M = N;
    p.K = K;
    p.adapter = adapter;
    p.n_adapters = n_adapters;
    p.rank = rank;
    p.fmt = type == MOE_BF16;
    p.status = moe_status_word_device_ptr();

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const long long jobs = (long long)T * (chunks * 32 / LS_RANKS);
    moe_pdl_config(&cfg, attr, dim3((unsigned)((jobs + 7) / 8)), dim3(256), 0, moe_cuda_stream(s));
    const uint16_t *xa = (const uint16_t *)x, *aa = (const uint16_t *)a;
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, type == MOE_BF16 ? lora_shrink_kernel<true> : lora_shrink_kernel<false>, xa, ldx, T,
                                    K, adapter, n_adapters, aa, rank, scale, (uint16_t *)workspace));
    const bool wide = T > 32;
    const long long tiles = wide ? (T + 255) / 256 : (T + 31) / 32;
    return grouped_launch(p, ytype, GP_LORA, wide, tiles * ((N + 127) / 128), (K + 63) / 64 + std::min(T, n_adapters) * chunks,
                          moe_cuda_stream(s));
}
