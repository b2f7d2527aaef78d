// MXFP4 quantisation and its inverse: rows of activations, and whole experts to slot images.
//
// Per 32 elements: s = max(0, exponent field of max|x| - 2), codes = round_e2m1(x * 2^(127 - s)).
// The scale is a power of two, so the product is exact and the codes are the same bits on every
// path.  Bound by HBM: a row element costs its own bytes in and 17/32 of a byte out.
#include <algorithm>

#include "moe_mx4.cuh"

#define MXQ_THREADS 256

namespace {

// Rows: a thread takes eight consecutive columns (one 16-byte load of bf16, two of fp32) and
// writes their four code bytes; the four threads of a block share its scale by two shuffles.  IPT such
// groups a thread, MXQ_THREADS apart, every load first: several where there are blocks enough to fill the
// GPU (4096 x 2048 bf16 and back: 11.1 us with one, 9.5 with four), one where latency counts.  I: the index
// type (32 bits wherever the rows have fewer than 2^31 groups: the division by the row length is what an
// element costs most).
template <int XT, int IPT, typename I>
__global__ void __launch_bounds__(MXQ_THREADS)
mx4_rows_kernel(const void *__restrict__ x, I n, I per, size_t ld, int wide, uint8_t *__restrict__ codes,
                uint8_t *__restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    for (I i0 = (I)blockIdx.x * (MXQ_THREADS * IPT); i0 < n; i0 += (I)gridDim.x * (MXQ_THREADS * IPT)) {
        Raw8<XT> v[IPT];
        I c[IPT];
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const I i = i0 + k * MXQ_THREADS + threadIdx.x, r = i / per;
            c[k] = i - r * per;
            v[k] = {};
            if (i < n) v[k] = load_raw8<XT>(x, (size_t)r * ld + (size_t)c[k] * 8, wide);
        }
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const I i = i0 + k * MXQ_THREADS + threadIdx.x;
            int s;
            const uint32_t q = mx4_quant8<XT>(v[k], s);
            if (i < n) {
                ((uint32_t *)codes)[i] = q;
                if ((c[k] & 3) == 0) scales[i >> 2] = (uint8_t)s;
            }
        }
    }
}

template <int YT, int IPT, typename I>
__global__ void __launch_bounds__(MXQ_THREADS)
mx4_rows_back_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, I n, I per, size_t ld,
                     int wide, void *__restrict__ y) {
    pdl_wait();
    pdl_trigger();
    for (I i0 = (I)blockIdx.x * (MXQ_THREADS * IPT); i0 < n; i0 += (I)gridDim.x * (MXQ_THREADS * IPT)) {
        uint32_t q[IPT];
        int s[IPT];
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const I i = i0 + k * MXQ_THREADS + threadIdx.x;
            q[k] = 0;
            s[k] = 0;
            if (i < n) {
                q[k] = ((const uint32_t *)codes)[i];
                s[k] = scales[i >> 2];
            }
        }
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const I i = i0 + k * MXQ_THREADS + threadIdx.x, r = i / per, c = i - r * per;
            float v[8];
            mx4_dequant8(q[k], s[k], v);
            if (i < n) store8<YT>(y, (size_t)r * ld + (size_t)c * 8, wide, v);
        }
    }
}

// Experts: one CTA per tile block (128 rows x 128 columns of one of an expert's two matrices).
// A half-warp reads one row's 128 columns; the tile block is put together in shared memory in
// its final order and leaves as one contiguous run.
struct Mx4Tile {
    const void *src[2];  // rows 0..63 and 64..127 (gate, up) or both halves of down
    int row0[2];         // their first source row
    int nrow[2];         // rows that exist
    int col0, K;         // first column, columns of the matrix
};

template <int XT>
__device__ __forceinline__ Mx4Tile mx4_tile_of(const void *gate, const void *up, const void *down, int i, int H, int F,
                                               int tile) {
    const size_t es = XT == MOE_BF16 ? 2 : 4;
    const int HB = (H - 1) / 128 + 1, FB = (F - 1) / 128 + 1, gu = ((F - 1) / 64 + 1) * HB;
    Mx4Tile t;
    const size_t base = (size_t)i * H * F * es;
    if (tile < gu) {
        const int g = tile / HB;
        t.col0 = tile % HB * 128;
        t.K = H;
        t.src[0] = (const char *)gate + base;
        t.src[1] = (const char *)up + base;
        t.row0[0] = t.row0[1] = 64 * g;
        t.nrow[0] = t.nrow[1] = min(64, F - 64 * g);
    } else {
        const int g = (tile - gu) / FB;
        t.col0 = (tile - gu) % FB * 128;
        t.K = F;
        t.src[0] = t.src[1] = (const char *)down + base;
        for (int h = 0; h < 2; ++h) {
            t.row0[h] = 128 * g + 64 * h;
            t.nrow[h] = max(0, min(64, H - t.row0[h]));
        }
    }
    return t;
}

template <int XT>
__global__ void __launch_bounds__(MXQ_THREADS)
mx4_experts_kernel(const void *__restrict__ gate, const void *__restrict__ up, const void *__restrict__ down, int H,
                   int F, int wide, int tiles, uint8_t *__restrict__ pool, size_t slot_bytes,
                   const int32_t *__restrict__ slots, int n_slots, int *status) {
    __shared__ __align__(16) uint8_t tb[MX4_TB];
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int slot = slots ? slots[i] : i;
    if (slot < 0 || slot >= n_slots) {
        if (threadIdx.x == 0) moe_set_status(status, MOE_ERR_INVALID);
        return;
    }
    const Mx4Tile t = mx4_tile_of<XT>(gate, up, down, i, H, F, tile);
    const int c = (threadIdx.x & 15) * 8;  // the half-warp's row takes 16 threads of 8 columns
    Raw8<XT> v[8];  // every load first
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = threadIdx.x / 16 + 16 * j, h = j >> 2, r = row & 63;
        v[j] = {};
        if (r < t.nrow[h] && t.col0 + c < t.K)
            v[j] = load_raw8<XT>(t.src[h], (size_t)(t.row0[h] + r) * t.K + t.col0 + c, wide);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = threadIdx.x / 16 + 16 * j;
        int s;
        const uint32_t q = mx4_quant8<XT>(v[j], s);
        *(uint32_t *)(tb + mx4_code_offset(1, row, c)) = q;
        if ((c & 31) == 0) tb[mx4_scale_offset(1, row, c)] = (uint8_t)s;
    }
    __syncthreads();
    uint4 *dst = (uint4 *)(pool + (size_t)slot * slot_bytes + (size_t)tile * MX4_TB);
    for (int k = threadIdx.x; k < MX4_TB / 16; k += MXQ_THREADS) dst[k] = ((const uint4 *)tb)[k];
}

template <int YT>
__global__ void __launch_bounds__(MXQ_THREADS)
mx4_experts_back_kernel(const uint8_t *__restrict__ pool, size_t slot_bytes, const int32_t *__restrict__ slots,
                        int n_slots, int H, int F, int wide, int tiles, void *gate, void *up, void *down,
                        int *status) {
    __shared__ __align__(16) uint8_t tb[MX4_TB];
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int slot = slots ? slots[i] : i;
    if (slot < 0 || slot >= n_slots) {
        if (threadIdx.x == 0) moe_set_status(status, MOE_ERR_INVALID);
        return;
    }
    const uint4 *src = (const uint4 *)(pool + (size_t)slot * slot_bytes + (size_t)tile * MX4_TB);
    for (int k = threadIdx.x; k < MX4_TB / 16; k += MXQ_THREADS) ((uint4 *)tb)[k] = src[k];
    const Mx4Tile t = mx4_tile_of<YT>(gate, up, down, i, H, F, tile);
    __syncthreads();
    const int c = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = threadIdx.x / 16 + 16 * j, h = j >> 2, r = row & 63;
        if (r >= t.nrow[h] || t.col0 + c >= t.K) continue;
        float v[8];
        mx4_dequant8(*(const uint32_t *)(tb + mx4_code_offset(1, row, c)), tb[mx4_scale_offset(1, row, c)], v);
        store8<YT>((void *)t.src[h], (size_t)(t.row0[h] + r) * t.K + t.col0 + c, wide, v);
    }
}

bool type_ok(int t) { return t == MOE_F32 || t == MOE_BF16; }

// Whether eight-element groups of rows `ld` apart are 16-byte aligned.
int wide_rows(const void *p, size_t ld, int type) {
    const size_t es = type == MOE_BF16 ? 2 : 4;
    return ((uintptr_t)p & 15) == 0 && (ld * es & 15) == 0;
}

// A launch with the programmatic dependency on the stream's previous kernel.
template <typename... K, typename... A>
int launch(void (*kernel)(K...), size_t blocks, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    moe_pdl_config(&cfg, attr, dim3((unsigned)std::min<size_t>(blocks, 0x7FFFFFFFu)), dim3(MXQ_THREADS), 0, s);
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, (K)args...));
    return MOE_OK;
}

// Groups of a pass from which on a thread takes four (a block's worth for every multiprocessor, eight times).
#define MXQ_MANY (8u * 152 * MXQ_THREADS)

template <int XT>
int launch_rows(const void *x, int rows, int cols, size_t ld, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const size_t per = (size_t)cols / 8, n = per * rows, g1 = (n + MXQ_THREADS - 1) / MXQ_THREADS, g4 = (g1 + 3) / 4;
    const int wide = wide_rows(x, ld, XT);
    if (n < MXQ_MANY) return launch(mx4_rows_kernel<XT, 1, uint32_t>, g1, s, x, n, per, ld, wide, codes, scales);
    return n < (1u << 31) ? launch(mx4_rows_kernel<XT, 4, uint32_t>, g4, s, x, n, per, ld, wide, codes, scales)
                          : launch(mx4_rows_kernel<XT, 4, size_t>, 1u << 20, s, x, n, per, ld, wide, codes, scales);
}

template <int YT>
int launch_rows_back(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y, size_t ld, cudaStream_t s) {
    const size_t per = (size_t)cols / 8, n = per * rows, g1 = (n + MXQ_THREADS - 1) / MXQ_THREADS, g4 = (g1 + 3) / 4;
    const int wide = wide_rows(y, ld, YT);
    if (n < MXQ_MANY) return launch(mx4_rows_back_kernel<YT, 1, uint32_t>, g1, s, codes, scales, n, per, ld, wide, y);
    return n < (1u << 31) ? launch(mx4_rows_back_kernel<YT, 4, uint32_t>, g4, s, codes, scales, n, per, ld, wide, y)
                          : launch(mx4_rows_back_kernel<YT, 4, size_t>, 1u << 20, s, codes, scales, n, per, ld, wide, y);
}

// Checks of the expert calls; tiles of one image.
int experts_check(int wtype, int n, int H, int F, size_t slot_bytes, int n_slots, const int32_t *slots, int *tiles) {
    MOE_CHECK(type_ok(wtype) && n >= 0 && H > 0 && F > 0 && H % 32 == 0 && F % 32 == 0);
    MOE_CHECK(n_slots >= 1 && (slots || n <= n_slots));
    MOE_CHECK(slot_bytes % 256 == 0 && slot_bytes >= moe_expert_image_bytes(MOE_MXFP4, H, F));
    const size_t t = moe_expert_image_bytes(MOE_MXFP4, H, F) / MX4_TB;
    if (t * (size_t)std::max(n, 1) > 0x7FFFFFFFu) return MOE_ERR_UNSUPPORTED;
    *tiles = (int)t;
    return MOE_OK;
}

}  // namespace

extern "C" int moe_mx4_quantize(const void *x, int xtype, int rows, int cols, size_t ld, uint8_t *codes,
                                uint8_t *scales, moe_stream_t s) {
    MOE_CHECK(type_ok(xtype) && rows >= 0 && cols > 0 && cols % 32 == 0 && ld >= (size_t)cols);
    if (rows == 0) return MOE_OK;
    MOE_CHECK(x && codes && scales);
    MOE_CHECK(((uintptr_t)x & (xtype == MOE_BF16 ? 1 : 3)) == 0 && ((uintptr_t)codes & 15) == 0);
    cudaStream_t st = moe_cuda_stream(s);
    return xtype == MOE_BF16 ? launch_rows<MOE_BF16>(x, rows, cols, ld, codes, scales, st)
                             : launch_rows<MOE_F32>(x, rows, cols, ld, codes, scales, st);
}

extern "C" int moe_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y, int ytype,
                                  size_t ld, moe_stream_t s) {
    MOE_CHECK(type_ok(ytype) && rows >= 0 && cols > 0 && cols % 32 == 0 && ld >= (size_t)cols);
    if (rows == 0) return MOE_OK;
    MOE_CHECK(y && codes && scales);
    MOE_CHECK(((uintptr_t)y & (ytype == MOE_BF16 ? 1 : 3)) == 0 && ((uintptr_t)codes & 15) == 0);
    cudaStream_t st = moe_cuda_stream(s);
    return ytype == MOE_BF16 ? launch_rows_back<MOE_BF16>(codes, scales, rows, cols, y, ld, st)
                             : launch_rows_back<MOE_F32>(codes, scales, rows, cols, y, ld, st);
}

extern "C" int moe_mx4_quantize_experts(const void *gate, const void *up, const void *down, int wtype, int n, int H,
                                        int F, void *pool, size_t slot_bytes, const int32_t *slots, int n_slots,
                                        moe_stream_t s) {
    int tiles = 0;
    const int rc = experts_check(wtype, n, H, F, slot_bytes, n_slots, slots, &tiles);
    if (rc != MOE_OK || n == 0) return rc;
    MOE_CHECK(gate && up && down && pool && ((uintptr_t)pool & 255) == 0);
    const uintptr_t any = (uintptr_t)gate | (uintptr_t)up | (uintptr_t)down;
    MOE_CHECK((any & (wtype == MOE_BF16 ? 1 : 3)) == 0);
    const int wide = (any & 15) == 0;
    int *status = moe_status_word_device_ptr();
    cudaStream_t st = moe_cuda_stream(s);
    const size_t g = (size_t)tiles * n;
    return wtype == MOE_BF16 ? launch(mx4_experts_kernel<MOE_BF16>, g, st, gate, up, down, H, F, wide, tiles,
                                      (uint8_t *)pool, slot_bytes, slots, n_slots, status)
                             : launch(mx4_experts_kernel<MOE_F32>, g, st, gate, up, down, H, F, wide, tiles,
                                      (uint8_t *)pool, slot_bytes, slots, n_slots, status);
}

extern "C" int moe_mx4_dequantize_experts(const void *pool, size_t slot_bytes, const int32_t *slots, int n_slots,
                                          int n, int H, int F, void *gate, void *up, void *down, int wtype,
                                          moe_stream_t s) {
    int tiles = 0;
    const int rc = experts_check(wtype, n, H, F, slot_bytes, n_slots, slots, &tiles);
    if (rc != MOE_OK || n == 0) return rc;
    MOE_CHECK(gate && up && down && pool && ((uintptr_t)pool & 255) == 0);
    const uintptr_t any = (uintptr_t)gate | (uintptr_t)up | (uintptr_t)down;
    MOE_CHECK((any & (wtype == MOE_BF16 ? 1 : 3)) == 0);
    const int wide = (any & 15) == 0;
    int *status = moe_status_word_device_ptr();
    cudaStream_t st = moe_cuda_stream(s);
    const size_t g = (size_t)tiles * n;
    return wtype == MOE_BF16 ? launch(mx4_experts_back_kernel<MOE_BF16>, g, st, (const uint8_t *)pool, slot_bytes, slots,
                                      n_slots, H, F, wide, tiles, gate, up, down, status)
                             : launch(mx4_experts_back_kernel<MOE_F32>, g, st, (const uint8_t *)pool, slot_bytes, slots,
                                      n_slots, H, F, wide, tiles, gate, up, down, status);
}
