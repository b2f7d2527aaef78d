// A whole MoE layer for a few tokens over resident MXFP4 experts (moe_mx4_layer): two kernels.
//
// The 4-bit tensor cores multiply E2M1 by E2M1.  To keep 23 bits of the activations they are
// written in radix 8: an activation is a 24-bit fixed-point number under a common scale, and its
// eight digits -4 .. 3 are all E2M1 values, so a token becomes eight exact 4-bit columns and
//     w . x = scale * sum_p 8^p (w . digit_p),
// each term an exact product of 4-bit operands summed in fp32 by the MMA.  Eight columns are the
// narrowest MMA there is, so one token's digits cost nothing over a single 4-bit column, the weights
// go from HBM through shared memory to the tensor core untouched, and no thread dequantises.
// x and h have one power of two per 32 columns, the MMA's own E8M0 scale: the largest magnitude of the 32
// becomes a number of 1.71 * 2^21 to 1.71 * 2^22 (the largest symmetric 8-digit one), so that an element is off
// by at most 2^-22.7 of it, and columns of another block by nothing.
//
//  * mx4_prep_kernel, 8-CTA clusters of 1 or 2 tokens: the router (a CTA sums its eighth of H, the
//    partial logits meet over distributed shared memory, one CTA per token ranks the experts), the tokens'
//    digits and scales in operand order, and the counters of the second kernel.
//  * mx4_layer_kernel: persistent.  Units: (chunk of at most NR routes of one expert, 128-row weight
//    tile) of gate/up, then of down, then (tile of H, eight tokens) of the combine.  CTAs take units in order from a counter, so a down unit only
//    ever waits for gate/up units that running CTAs hold: no co-residency is needed, and other work
//    on the GPU cannot deadlock it.  Roles as in the grouped product, with
//      warp 0      claims units, copies the weights (17 KB a stage: bound by HBM),
//      warp 1      copies the digits of h once the chunk's gate/up units are all done (and x's, where
//                  they do not stay in shared memory),
//      warp 2      the MMAs, warps 4-7 the scales,
//      warps 8-11  gate/up: sum_p, SwiGLU, the digits and scales of h (a block of 32 columns is a
//                  warp: one reduction; an 8x8 nibble transpose by three shuffles); down: sum_p, the
//                  router weight, partial rows.  Units after the last down unit add the partial rows of
//                  a tile of H in route order onto extra;
//      warp 3      publishes finished units to the other CTAs.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "moe_mx4_gemm.cuh"
#include "moe_select.cuh"
#include "moe_tc.cuh"

#define MXL_CLUSTER 8
#define MXL_MAX_CLUSTERS 16   // of the first kernel, 1 or 2 tokens each
#define MXL_PREP_THREADS 256
#define MXL_THREADS 384
#define MXL_Q 4               // claimed units in flight in a CTA
#define MXL_PUB (2 * MXL_Q)   // the epilogue may be MXL_Q units ahead of warp 3 and of a queue slot's reuse
#define MXL_MAX_R (MOE_DECODE_MAX_T * MOE_MAX_K)
#define MXL_BIAS 9586980u     // 4 (8^8 - 1) / 7: turns digits -4 .. 3 into 0 .. 7
#define MXL_SC 16             // bytes of a row's scales in a stage: a word for each 128 columns, and padding
#define MXL_ROW (1024 + MXL_SC)  // a row's digits and scales
#define MXL_WBYTES (2 * MX4_TB)

static_assert(MXL_PREP_THREADS == MOE_MAX_E, "a thread per expert");

namespace {

// (a chunk holds a route at least)
typedef Mx4Chunks<MXL_MAX_R, MXL_MAX_R> LayerChunks;

// Most routes of a chunk (NR of the second kernel).
int chunk_routes(int T) { return T <= 8 ? 8 : 16; }

struct LayerWs {
    size_t ctr, ids, weights, xq, hq, partial, total;
    size_t ctr_ints;
};

LayerWs layer_ws(int T, int H, int F, int k) {
    LayerWs L;
    const size_t R = (size_t)T * k, HB = (H + 127) / 128, FB = (F + 127) / 128;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o += (n + 511) / 512 * 512;
        return at;
    };
    L.ctr_ints = 4 + R + HB;  // ticket, (pad), ready[chunk], done[tile of H]
    L.ctr = take(L.ctr_ints * 4);
    L.ids = take(R * 4);
    L.weights = take(R * 4);
    L.xq = take((HB + 1) / 2 * T * MXL_ROW);  // every stage's digits, then every stage's scales
    L.hq = take(R * ((FB + 1) / 2) * (1024 + chunk_routes(T) * MXL_SC));  // (at most a chunk per route)
    L.partial = take(R * H * 4);
    L.total = o;
    return L;
}

// Code of the radix-8 digit d (0 .. 7 for -4 .. 3).
__device__ __forceinline__ uint32_t digit_code(uint32_t d) { return (0x5420ACDEu >> (4 * d)) & 15u; }

// The scale byte of a block whose largest magnitude has these bits: the power of two that makes it a number
// of at most 7190000 < 3 (8^8 - 1) / 7 = 1.7142.. * 2^22, the largest symmetric one of eight digits; at least
// 2^-127 (blocks below 2^-105 keep fewer digits); 255 for an infinity or a NaN.  A mantissa beyond
// 7190000 / 2^22 (0x5B6BE0 steps above 1) carries into the exponent.
__device__ __forceinline__ int digit_scale(uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? 255 : max(0, (int)((amax_bits + 0x24941Fu) >> 23) - 22);
}
// A block's digits under that scale, a column's value to a lane, transposed: lane 8a + b gets digit b of columns
// 8a .. 8a + 7 (zeros under 255).
__device__ __forceinline__ uint32_t digit_word(float v, int scale, int lane) {
    uint32_t u = MXL_BIAS, w = 0;
    if (scale != 255) u += (uint32_t)__float2int_rn(v * e8m0_inverse(scale));
#pragma unroll
    for (int p = 0; p < 8; ++p) w |= digit_code((u >> (3 * p)) & 7u) << (4 * p);
    uint32_t y = __shfl_xor_sync(0xffffffffu, w, 4);
    w = lane & 4 ? (w & 0xFFFF0000u) | (y >> 16) : (w & 0x0000FFFFu) | (y << 16);
    y = __shfl_xor_sync(0xffffffffu, w, 2);
    w = lane & 2 ? (w & 0xFF00FF00u) | ((y >> 8) & 0x00FF00FFu) : (w & 0x00FF00FFu) | ((y & 0x00FF00FFu) << 8);
    y = __shfl_xor_sync(0xffffffffu, w, 1);
    return lane & 1 ? (w & 0xF0F0F0F0u) | ((y >> 4) & 0x0F0F0F0Fu) : (w & 0x0F0F0F0Fu) | ((y & 0x0F0F0F0Fu) << 4);
}

// ------------------------------------------------------------------ router, digits of x

struct PrepParams {
    const void *x;
    const uint16_t *w_router;
    const float *bias;
    int T, H, E, k;
    int32_t *ids;
    float *weights;
    uint8_t *xq, *xsc;  // [stage][token] of 1024, of MXL_SC bytes
    int *ctr;
    int n_ctr;
    int w_elems;  // elements of w_router that a pass holds in shared memory
    int *status;
};

// Most dynamic shared memory of the first kernel (its static arrays, about 1 KB, come on top) for tokens and sums,
// and with the router's weights where they go through it (the rest of a block's, 24 KB at least).
#define MXL_PREP_SMEM (200 * 1024)
#define MXL_PREP_SMEM_W (225 * 1024)

size_t prep_smem(int H, int E, int TT) {
    const int E8 = (E + 7) / 8 * 8;
    return ((size_t)H / MXL_CLUSTER * TT + (size_t)(MXL_PREP_THREADS / 32 + 1) * TT * E8) * 4;
}

__device__ __forceinline__ void half8(const uint4 &u, float (&w)[8]) {
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*(const __half2 *)&q[j]);
        w[2 * j] = f.x;
        w[2 * j + 1] = f.y;
    }
}

// TT: tokens of a cluster (the last one may hold fewer).  Few tokens to a cluster and up to 16 clusters:
// the router's sums, not its reads of w_router from L2, take the time.  The kernel is a chain of
// latencies, instruction fetches among them: loops are kept rolled.  WIDE: rows of w_router in 16-byte loads
// (E a multiple of 8, 16-byte aligned).  Otherwise the rows, one run of bytes, come to shared memory by a bulk copy,
// as many at a time as there is room for, and a lane sums one expert's column: no two lanes share a bank.  (18
// tokens, H 1760, 73 experts, in graphs: 26.6 us; eight experts a thread, as in WIDE, 28.2; element loads straight
// to registers one after the other 30.0.)
template <int XT, int TT, bool WIDE>
__global__ void __launch_bounds__(MXL_PREP_THREADS) mx4_prep_kernel(const __grid_constant__ PrepParams p) {
    extern __shared__ __align__(16) float sm[];
    __shared__ __align__(16) uint32_t key[MOE_MAX_E];
    __shared__ uint32_t sel[2 * MOE_MAX_K];
    __shared__ uint64_t w_bar;
    constexpr int NW = MXL_PREP_THREADS / 32, PRE = 8;  // rows of w_router a thread reads at a time
    const int rank = (int)cluster_ctarank(), tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int HS = p.H / MXL_CLUSTER, h0 = rank * HS, E8 = (p.E + 7) & ~7;
    const int t0 = blockIdx.y * TT, nt = min(TT, p.T - t0);
    float *xs = sm;                   // [HS][TT]
    float *red = xs + HS * TT;        // [NW][TT][E8]
    float *part = red + NW * TT * E8; // [TT][E8]
    // logits: thread (cg, hsub) takes experts 8 cg .. 8 cg + 7 of rows hsub, hsub + NH, ...
    int ncl = 0;  // log2 of the column groups, a power of two of them
    while ((8 << ncl) < E8) ++ncl;
    const int cg = tid & ((1 << ncl) - 1), hsub = tid >> ncl, NH = MXL_PREP_THREADS >> ncl;
    const uint16_t *wr = p.w_router + (size_t)h0 * p.E + 8 * cg;
    const int ne = p.E - 8 * cg;
    auto load_rows = [&](int h, uint4 (&a)[PRE]) {
#pragma unroll
        for (int i = 0; i < PRE; ++i, h += NH) {
            a[i] = make_uint4(0, 0, 0, 0);
            if (h < HS && ne > 0) a[i] = *(const uint4 *)(wr + (size_t)h * p.E);
        }
    };
    // the router's weights, too, may come from the kernel before: ahead of the wait they are only brought to L2
    // (this CTA's rows are one run of bytes)
    if (tid == 0 && blockIdx.y == 0) {
        const uintptr_t w0 = (uintptr_t)(p.w_router + (size_t)h0 * p.E), w1 = w0 + (size_t)HS * p.E * 2;
        const uintptr_t a0 = (w0 + 15) & ~(uintptr_t)15, a1 = w1 & ~(uintptr_t)15;
        if (a1 > a0) bulk_prefetch_l2((const void *)a0, (uint32_t)(a1 - a0));
    }
    if (!WIDE && tid == 0) {
        mbar_init(&w_bar, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();  // not before: the next kernel reads its slot table before its own wait
    uint4 wa[PRE], wb[PRE];
    // a pass of the rows in shared memory, as far from a 16-byte boundary there as here: whole pieces by one copy,
    // the ends by elements
    uint16_t *ws = (uint16_t *)(part + TT * E8);
    const int pass_rows = p.w_elems / p.E & ~3;
    auto fetch = [&](int r0) -> const uint16_t * {
        const uint16_t *src = p.w_router + (size_t)(h0 + r0) * p.E;
        const int n = min(pass_rows, HS - r0) * p.E, off = (int)((uintptr_t)src & 15) >> 1;
        const int head = min(n, (8 - off) & 7), whole = (n - head) & ~7, tail = head + whole;
        if (tid == 0) {
            mbar_arrive_expect_tx(&w_bar, (uint32_t)whole * 2u);
            if (whole) bulk_g2s(ws + off + head, src + head, (uint32_t)whole * 2u, &w_bar);
        }
        if (tid < head) ws[off + tid] = src[tid];
        if (tid < n - tail) ws[off + tail + tid] = src[tail + tid];
        return ws + off;
    };
    const uint16_t *w_rows = nullptr;
    if (WIDE) {
        load_rows(hsub, wa);
        load_rows(hsub + PRE * NH, wb);
    } else {
        w_rows = fetch(0);
    }
    // this CTA's eighth of the tokens
    for (int h = tid; h < HS; h += MXL_PREP_THREADS)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float v = 0.f;
            if (t < nt) {
                const size_t at = (size_t)(t0 + t) * p.H + h0 + h;
                v = XT == MOE_BF16 ? __bfloat162float(((const __nv_bfloat16 *)p.x)[at]) : ((const float *)p.x)[at];
            }
            xs[h * TT + t] = v;
        }
    const float bias = p.bias && tid < p.E ? p.bias[tid] : 0.f;
    if (blockIdx.y == 0)
        for (int i = rank * MXL_PREP_THREADS + tid; i < p.n_ctr; i += MXL_CLUSTER * MXL_PREP_THREADS) p.ctr[i] = 0;
    __syncthreads();
    float acc[TT][8];
    int sums = NW;  // partial sums of a logit
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = 0.f;
    auto add_row = [&](const float (&w)[8], const float *xh) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float xv = xh[t];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(xv, w[j], acc[t][j]);
        }
    };
    if (WIDE) {
#pragma unroll 1
        for (int h = hsub; h < HS; h += PRE * NH) {
#pragma unroll
            for (int i = 0; i < PRE; ++i) {
                float w[8];
                half8(wa[i], w);
                add_row(w, xs + min(h + i * NH, HS - 1) * TT);  // (rows past the slice are zeros)
                wa[i] = wb[i];
            }
            if (h + 2 * PRE * NH < HS) load_rows(h + 2 * PRE * NH, wb);
        }
    } else {
        // a lane per expert: consecutive elements of a row; the rows in `ng` runs
        const int el = (p.E + 31) & ~31, ng = MXL_PREP_THREADS / el, grp = tid / el, e_mine = tid - grp * el;
        sums = ng;
#pragma unroll 1
        for (int r0 = 0, pass = 0; r0 < HS; r0 += pass_rows, ++pass) {
            if (r0) {
                fence_proxy_async_smem();  // the ends' elements were ordinary stores
                __syncthreads();
                w_rows = fetch(r0);
                __syncthreads();
            }
            if (!mbar_wait_bounded(&w_bar, pass & 1, p.status)) break;
            const int nr = min(pass_rows, HS - r0), q = ((nr + ng - 1) / ng + 3) & ~3;  // (multiples of 4 all)
            const uint16_t *col = w_rows + e_mine;
            if (grp < ng && e_mine < p.E)
#pragma unroll 2
                for (int h = grp * q; h < min(nr, grp * q + q); h += 4) {
                    float w[4], xv[4 * TT];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = __half2float(__ushort_as_half(col[(h + i) * p.E]));
#pragma unroll
                    for (int i = 0; i < TT; ++i) *(float4 *)(xv + 4 * i) = *(const float4 *)(xs + (r0 + h) * TT + 4 * i);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int t = 0; t < TT; ++t) acc[t][0] = fmaf(xv[TT * i + t], w[i], acc[t][0]);
                }
        }
        if (grp < ng && e_mine < p.E)
#pragma unroll
            for (int t = 0; t < TT; ++t) red[(grp * TT + t) * E8 + e_mine] = acc[t][0];
    }
    if (WIDE) {
#pragma unroll 1
        for (int o = 1 << ncl; o < 32; o <<= 1)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[t][j] += __shfl_xor_sync(0xffffffffu, acc[t][j], o);
        if (lane < (1 << ncl) && ne > 0)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) red[(warp * TT + t) * E8 + 8 * cg + j] = acc[t][j];
    }
    __syncthreads();
    for (int i = tid; i < TT * E8; i += MXL_PREP_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            if (WIDE || w < sums) s += red[w * TT * E8 + i];
        part[i] = s;
    }
    cluster_sync_all();
    // a thread per expert sums token t0 + rank's logit
    if (rank < nt && tid < p.E) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < MXL_CLUSTER; ++r) s += ld_cluster_f32(cluster_map(&part[rank * E8 + tid], r));
        key[tid] = select_key(s + bias);
    } else {
        key[tid] = 0;
    }
    __syncthreads();
    // nothing of another CTA is read after this; a CTA's own shared memory stays until all have come here
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank < nt) select_topk_block(key, p.E, p.k, sel, (size_t)(t0 + rank), p.ids, p.weights);
    if (warp > 0) {
        // digits and scales, by the other warps: a block of 32 columns of one token to a warp; of this CTA's eighth
        // of H where it is whole blocks, else of the tokens' blocks in turn
        const bool own = HS % 32 == 0;
        const int per = (own ? HS : p.H) / 32, step = (NW - 1) * (own ? 1 : MXL_CLUSTER);
        const int d = lane & 7;  // this lane's digit after the transpose
#pragma unroll 1
        for (int i = own ? warp - 1 : (warp - 1) * MXL_CLUSTER + rank; i < nt * per; i += step) {
            const int t = i / per, col = (i - t * per) * 32 + (own ? h0 : 0), c = (col >> 5) & 3;
            const size_t in = (size_t)(t0 + t) * p.H + col + lane;
            const float v = own ? xs[(col - h0 + lane) * TT + t]
                          : XT == MOE_BF16 ? __bfloat162float(((const __nv_bfloat16 *)p.x)[in]) : ((const float *)p.x)[in];
            const int sc = digit_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
            const size_t at = (size_t)(col >> 8) * p.T + t0 + t;
            uint8_t *atom = p.xq + at * 1024 + ((col >> 7) & 1) * 512;
            *(uint32_t *)(atom + d * 64 + ((c ^ ((d >> 1) & 3)) << 4) + 4 * (lane >> 3)) = digit_word(v, sc, lane);
            if (lane == 0) {
                uint8_t *dst = p.xsc + at * MXL_SC + ((col >> 7) & 1) * 4 + c;
                dst[0] = (uint8_t)sc;
                // the MMA's last 64 columns may be 32 columns and 32 past H, against weights of zero: any scale but NaN
                if (col + 32 == p.H && (c & 1) == 0) dst[1] = 0;
            }
        }
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ experts and combine

struct FfnParams {
    int T, H, F, E, k;
    const int32_t *ids, *table;
    const float *weights, *extra;
    int n_slots;
    const uint8_t *pool;
    size_t slot_bytes;
    const uint8_t *xq, *xsc;
    uint8_t *hq;
    float *partial, *y;
    int *ticket, *ready, *done;
    int *status;
    int res, xsr; // bytes of resident digits and of x's resident scales (0: copied by stage)
    int S, stage; // ring stages, bytes of one
};

// Shared memory: control, the tokens' digits (resident: T <= NR = 8) and their scales (resident where, like the
// digits, they leave four stages of the ring), then S stages of two weight blocks and `cap` routes' digits (1024
// bytes each: two 512-byte atoms of 8 rows x 128 columns) followed by their scales.  (Scales copied a row at a
// time with each stage: 32 tokens, Qwen-shaped, 61.7 us against 59.8.)
template <int NR>
struct LayerGeom {
    static constexpr int N = NR * 8;
    static constexpr int SFCOL = 2 * N;      // scales after the two accumulators, 16 columns a stage
    static constexpr int MAXS = 10;
    static constexpr int CTRL = (1024 + 2 * 4 * NR * 32 * 4 + (int)sizeof(LayerChunks) + 2 * MXL_MAX_R * 4 +
                                 MOE_MAX_E * 4 + 1023) / 1024 * 1024;
    static_assert(SFCOL + MAXS * 16 <= 512, "tensor memory");
    static_assert(sizeof(LayerChunks) % 16 == 0 && 2 * 4 * NR * 32 * 4 % 16 == 0 && MXL_MAX_R * 4 % 16 == 0,
                  "the control block's arrays follow one another on 16-byte boundaries");
};

__device__ __forceinline__ int ld_acquire_gpu(const int *a) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
    return v;
}
__device__ __forceinline__ void red_release_gpu(int *a) {
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Digits of h of stage kc of a chunk of n routes (n * 1024 bytes, then its scales; on 128-byte boundaries).
template <int NR>
__device__ __forceinline__ size_t hq_offset(int chunk, int pos, int n, int stages, int kc) {
    return (size_t)stages * (pos * 1024 + chunk * NR * MXL_SC) + (size_t)kc * (n * 1024 + NR * MXL_SC);
}

// A unit: gate/up or down tile m of a chunk, or (last) tile m of y for tokens 8 c .. 8 c + 7.
enum { MXL_UP = 0, MXL_DOWN = 1, MXL_COMBINE = 2, MXL_NONE = 3, MXL_ABORT = 4 };
struct Unit {
    int kind, c, m;
};
__device__ __forceinline__ Unit unit_of(int u, int nch, int FT, int HT) {
    Unit r;
    r.kind = u < nch * FT ? MXL_UP : u < nch * (FT + HT) ? MXL_DOWN : MXL_COMBINE;
    const int v = r.kind == MXL_UP ? u : r.kind == MXL_DOWN ? u - nch * FT : u - nch * (FT + HT);
    const int per = r.kind == MXL_UP ? FT : HT;
    r.c = v / per;
    r.m = v - r.c * per;
    return r;
}

// A unit in one word (chunks: 8 bits, tiles: 20), as it travels to the CTA's roles; -1: none left.
__device__ __forceinline__ int unit_pack(const Unit &u) { return u.kind << 28 | u.c << 20 | u.m; }
__device__ __forceinline__ Unit unit_unpack(int v) {
    return v < 0 ? Unit{MXL_NONE, 0, 0} : Unit{v >> 28, (v >> 20) & 0xFF, v & 0xFFFFF};
}

// y[t][columns of tile m] = extra + the partial rows of token t's routes, in route order (`on`: routes
// that were computed), for eight tokens by 128 threads: four columns of a token to a thread.
__device__ __forceinline__ void combine_tile(const FfnParams &p, int m, int t0, int thr, const int *on) {
    const int o = 128 * m + 4 * (thr & 31);
    if (o >= p.H) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = t0 + (thr >> 5) + 4 * i;
        if (t >= p.T) break;
        float4 v[MOE_MAX_K];
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            v[j] = j < p.k && on[t * p.k + j] ? __ldcg((const float4 *)(p.partial + (size_t)(t * p.k + j) * p.H + o))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const size_t at = (size_t)t * p.H + o;
        if (p.extra)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] = p.extra[at + q];
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            if (j < p.k) {
                s[0] += v[j].x;
                s[1] += v[j].y;
                s[2] += v[j].z;
                s[3] += v[j].w;
            }
#pragma unroll
        for (int q = 0; q < 4; ++q) p.y[at + q] = s[q];
    }
}

// Bounded wait of a warp until *a >= want (counted up by other CTAs that are running).
__device__ __forceinline__ bool wait_count(const int *a, int want, int *status, volatile int *abort_flag) {
    bool ok = false;
    for (uint32_t it = 0; it < MOE_SPIN_LIMIT; ++it) {
        if ((ok = ld_acquire_gpu(a) >= want) || *abort_flag) break;
    }
    if (!ok && !*abort_flag) {
        moe_set_status(status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
    }
    return __all_sync(0xffffffffu, ok);
}

template <int NR>
__global__ void __launch_bounds__(MXL_THREADS, 1) mx4_layer_kernel(const __grid_constant__ FfnParams p) {
    using G = LayerGeom<NR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint64_t *s_full = (uint64_t *)smem;       // weights and digits of a stage
    uint64_t *s_empty = s_full + G::MAXS;
    uint64_t *sf_full = s_empty + G::MAXS;
    uint64_t *acc_full = sf_full + G::MAXS;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *q_full = acc_empty + 2;
    uint64_t *q_empty = q_full + MXL_Q;
    uint64_t *pub = q_empty + MXL_Q;           // a unit's outputs are written (4 epilogue warps)
    uint64_t *x_full = pub + MXL_PUB;          // resident digits
    uint64_t *xs_full = x_full + 1;            // and their scales
    uint64_t *mma_done = xs_full + 1;
    uint32_t *tmem_slot = (uint32_t *)(mma_done + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    volatile int *q_unit = (volatile int *)(tmem_slot + 2);  // [MXL_Q]
    static_assert((3 * G::MAXS + 4 + 2 * MXL_Q + MXL_PUB + 3) * 8 + (2 + MXL_Q) * 4 <= 1024, "barriers");
    float *xch = (float *)(smem + 1024);                     // [2 buffers][2 pairs][gate, up][NR][32]
    LayerChunks &ch = *(LayerChunks *)(xch + 2 * 4 * NR * 32);
    int *s_on = (int *)(&ch + 1);                            // [MXL_MAX_R] whether a route is computed
    float *s_w = (float *)(s_on + MXL_MAX_R);                // [MXL_MAX_R] router weights
    int *s_table = (int *)(s_w + MXL_MAX_R);                 // [MOE_MAX_E]
    uint8_t *xres = smem + G::CTRL;
    const uint8_t *xsres = xres + p.res;
    uint8_t *ring = xres + p.res + (p.xsr + 511) / 512 * 512;
    const int S = p.S, STAGE = p.stage;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 1);
            mbar_init(&sf_full[s], 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        for (int q = 0; q < MXL_Q; ++q) {
            mbar_init(&q_full[q], 1);
            mbar_init(&q_empty[q], 11);  // every warp but warp 0
        }
        for (int q = 0; q < MXL_PUB; ++q) mbar_init(&pub[q], 4);
        mbar_init(x_full, 1);
        mbar_init(xs_full, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // (the first kernel lets this one start after everything before it is complete)
    if (p.table && tid < p.E) s_table[tid] = p.table[tid];
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    // the first unit is claimed, and the resident digits are fetched, while the chunks are put together
    int claim = 0;
    if (tid == 0) {
        claim = atomicAdd(p.ticket, 1);
        if (p.xsr) {
            mbar_arrive_expect_tx(xs_full, (uint32_t)p.xsr);
            bulk_g2s(xres + p.res, p.xsc, (uint32_t)p.xsr, xs_full);
        }
        if (p.res) {
            mbar_arrive_expect_tx(x_full, (uint32_t)p.res);
            bulk_g2s(xres, p.xq, (uint32_t)p.res, x_full);
        }
    }
    const int R = p.T * p.k;
    if (tid < R) s_w[tid] = p.weights[tid];
    tc_fence_before();
    mx4_local_chunks<MXL_THREADS>(ch, (uint16_t *)ring, p.ids, R, p.E, p.table ? s_table : nullptr, p.n_slots, NR, s_on,
                                  p.status);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int nch = ch.nch;
    const int HB = (p.H + 127) / 128, FB = (p.F + 127) / 128, FT = (p.F + 63) / 64, HT = HB;
    const int n_units = nch * (FT + HT) + HT * ((p.T + 7) / 8);
    const size_t down_off = mx4_gu_bytes(p.H, p.F);

    // a consumer's next unit
    auto next_unit = [&](int i) -> Unit {
        const int q = i % MXL_Q;
        if (!mbar_wait_warp(&q_full[q], (i / MXL_Q) & 1, p.status, abort_flag)) return Unit{MXL_ABORT, 0, 0};
        const int v = __shfl_sync(0xffffffffu, q_unit[q], 0);
        if (lane == 0) mbar_arrive1(&q_empty[q]);
        return unit_unpack(v);
    };
    // ring position: stage index and the parity of its current fill
    int s = 0;
    uint32_t ph = 0;
    auto advance = [&]() {
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
    };

    if (nch == 0) {
        // no expert is resident: the layer is its extra
        if (tid == 0 && (!p.xsr || mbar_wait_role(xs_full, 0, p.status, abort_flag)) && p.res)
            mbar_wait_role(x_full, 0, p.status, abort_flag);
        for (int m = blockIdx.x; m < HT; m += gridDim.x)
            if (tid < 128)
                for (int t = 0; t < p.T; t += 8) combine_tile(p, m, t, tid, s_on);
    } else if (warp == 0) {
        // ---------------- claims and weights; a stage's barrier expects its digits' bytes too
        {
            bool ok = true;
            int fills = 0;
            const uint64_t once = l2_evict_first();
            for (int i = 0; ok; ++i) {
                const int q = i % MXL_Q, u = __shfl_sync(0xffffffffu, claim, 0);
                if (i >= MXL_Q && !(ok = mbar_wait_warp(&q_empty[q], ((i / MXL_Q) & 1) ^ 1, p.status, abort_flag))) break;
                const Unit un = unit_of(u, nch, FT, HT);
                if (lane == 0) {
                    q_unit[q] = u < n_units ? unit_pack(un) : -1;
                    mbar_arrive1(&q_full[q]);
                    if (u < n_units) claim = atomicAdd(p.ticket, 1);
                }
                if (u >= n_units) break;
                if (un.kind == MXL_COMBINE) continue;
                const bool down = un.kind == MXL_DOWN;
                const int KB = down ? FB : HB, NKS = (KB + 1) / 2, n = __shfl_sync(0xffffffffu, ch.n[un.c], 0);
                const uint32_t nb = (uint32_t)n * (down ? MXL_ROW : (p.res ? 0 : 1024) + (p.xsr ? 0 : MXL_SC));
                const uint8_t *w = p.pool + (size_t)__shfl_sync(0xffffffffu, ch.slot[un.c], 0) * p.slot_bytes +
                                   (down ? down_off : 0) + (size_t)un.m * KB * MX4_TB;
                for (int kc = 0; kc < NKS; ++kc, advance(), ++fills, w += MXL_WBYTES) {
                    if (fills >= S && !(ok = mbar_wait_warp(&s_empty[s], ph ^ 1u, p.status, abort_flag))) break;
                    const uint32_t wb = 2 * kc + 1 < KB ? MXL_WBYTES : MX4_TB;
                    mbar_arrive_expect_tx_elect(&s_full[s], wb + nb);
                    bulk_g2s_elect_hint(ring + (size_t)s * STAGE, w, wb, &s_full[s], once);
                }
            }
            // never leave with copies in flight: the last fill of every stage
            if (ok && p.xsr) ok = mbar_wait_role(xs_full, 0, p.status, abort_flag);
            if (ok && p.res) ok = mbar_wait_role(x_full, 0, p.status, abort_flag);
            for (int i = 0; ok && i < S && i < fills; ++i) {
                if (--s < 0) {
                    s = S - 1;
                    ph ^= 1u;
                }
                ok = mbar_wait_role(&s_full[s], ph, p.status, abort_flag);
            }
            if (!ok) settle_after_abort();
        }
    } else if (warp == 1) {
        // ---------------- digits (it keeps step with the ring through the units that need none)
        bool ok = true;
        int fills = 0;
        uint32_t ready = 0;  // bit b: chunk 32 b + lane has all its rows of h
        for (int i = 0; ok; ++i) {
            const Unit un = next_unit(i);
            if (un.kind >= MXL_COMBINE) {
                if (un.kind == MXL_COMBINE) continue;
                ok = un.kind != MXL_ABORT;
                break;
            }
            const bool down = un.kind == MXL_DOWN;
            const int NKS = ((down ? FB : HB) + 1) / 2;
            const int n = __shfl_sync(0xffffffffu, ch.n[un.c], 0), pos = __shfl_sync(0xffffffffu, ch.pos[un.c], 0);
            if (down) {
                // every gate/up unit of the chunk is done, its digits and scales written.  One look covers 32
                // chunks, so a chunk seen ready costs no more looks.
                const int b = un.c >> 5, mine = 32 * b + lane;
                bool looked = false;
                for (uint32_t it = 0; !(__shfl_sync(0xffffffffu, ready, un.c & 31) >> b & 1u); ++it) {
                    looked = true;
                    if (mine < nch && ld_acquire_gpu(&p.ready[mine]) >= FT) ready |= 1u << b;
                    if (it >= MOE_SPIN_LIMIT && lane == 0) {
                        moe_set_status(p.status, MOE_ERR_TIMEOUT);
                        *abort_flag = 1;
                    }
                    if (!(ok = __all_sync(0xffffffffu, !*abort_flag))) break;
                }
                if (!ok) break;
                // the rows were written as ordinary stores; from here on they are read by bulk copies, by
                // whichever lane is elected (hence the warp's barrier after the looking lane's acquire)
                if (looked) {
                    __syncwarp();
                    fence_proxy_async_all();
                }
            }
            const int tok = !down && lane < n ? ch.rows[pos + lane] / p.k : 0;
            for (int kc = 0; kc < NKS; ++kc, advance(), ++fills) {
                if (fills >= S && !(ok = mbar_wait_warp(&s_empty[s], ph ^ 1u, p.status, abort_flag))) break;
                uint8_t *st = ring + (size_t)s * STAGE;
                if (down) {
                    bulk_g2s_elect(st + MXL_WBYTES, p.hq + hq_offset<NR>(un.c, pos, n, NKS, kc), (uint32_t)n * MXL_ROW, &s_full[s]);
                } else if (!p.res && lane < n) {
                    const size_t at = (size_t)kc * p.T + tok;
                    bulk_g2s(st + MXL_WBYTES + lane * 1024, p.xq + at * 1024, 1024, &s_full[s]);
                    if (!p.xsr)
                        bulk_g2s(st + MXL_WBYTES + n * 1024 + lane * MXL_SC, p.xsc + at * MXL_SC, MXL_SC, &s_full[s]);
                }
                __syncwarp();
            }
        }
        if (!ok) settle_after_abort();
    } else if (warp == 2) {
        // ---------------- MMA issuer.  Resident digits: gate/up multiplies every token's (the width is
        // free, and the chunk's tokens need not be adjacent)
        bool ok = true, xok = !p.res;
        for (int i = 0; ok; ++i) {
            const Unit un = next_unit(i);
            if (un.kind >= MXL_COMBINE) {  // combines come last: units before them keep their numbering
                if (un.kind == MXL_COMBINE) continue;
                break;
            }
            const bool down = un.kind == MXL_DOWN, all = !down && p.res;
            if (all && !xok) ok = xok = mbar_wait_warp(x_full, 0, p.status, abort_flag);
            const int K = down ? p.F : p.H, NKS = (K + 255) / 256;
            const int N = 8 * (all ? p.T : __shfl_sync(0xffffffffu, ch.n[un.c], 0));
            const uint32_t id0 = umma_idesc_mxf4(128, N, 0), id2 = umma_idesc_mxf4(128, N, 2);
            const int buf = i & 1;
            if (ok && i >= 2) ok = mbar_wait_warp(&acc_empty[buf], ((i / 2) - 1) & 1, p.status, abort_flag);
            tc_fence_after();
            const uint32_t d = tmem + buf * G::N;
            for (int kc = 0; kc < NKS && ok; ++kc, advance()) {
                // (the scale warps saw the stage land before they arrived)
                if (!(ok = mbar_wait_warp(&sf_full[s], ph, p.status, abort_flag))) break;
                tc_fence_after();
                const uint32_t st = smem_u32(ring) + (uint32_t)(s * STAGE);
                const uint64_t a = umma_desc_sw64(st);
                const uint64_t b = umma_desc_sw64_rows1024(all ? smem_u32(xres) + kc * p.T * 1024 : st + MXL_WBYTES);
                const uint32_t sf = tmem + G::SFCOL + 16 * s;
                const int steps = (K - 256 * kc + 63) / 64;
                constexpr int A1 = MX4_TB >> 4, B1 = 512 >> 4;
                umma_mxf4(d, a, b, id0, sf, sf + 8, kc > 0);
                if (steps > 1) umma_mxf4(d, a + 2, b + 2, id2, sf, sf + 8, 1);
                if (steps > 2) umma_mxf4(d, a + A1, b + B1, id0, sf + 4, sf + 12, 1);
                if (steps > 3) umma_mxf4(d, a + A1 + 2, b + B1 + 2, id2, sf + 4, sf + 12, 1);
                umma_commit_elect(&s_empty[s]);
            }
            if (ok) umma_commit_elect(&acc_full[buf]);
        }
        umma_commit_elect(mma_done);
        mbar_wait_bounded(mma_done, 0, p.status);
    } else if (warp == 3) {
        // ---------------- publishes finished units: rows of h for the chunk's down units, partial rows
        // for the tile's combine
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const Unit un = next_unit(i);
            if (un.kind == MXL_COMBINE) continue;
            if (un.kind > MXL_COMBINE) break;
            if (!(ok = mbar_wait_warp(&pub[i % MXL_PUB], (i / MXL_PUB) & 1, p.status, abort_flag))) break;
            if (lane == 0) {
                red_release_gpu(un.kind == MXL_UP ? &p.ready[un.c] : &p.done[un.m]);
            }
            __syncwarp();
        }
    } else if (warp >= 4 && warp < 8) {
        // ---------------- scales: the weights' rows lane, lane + 32, ..; a route's (a resident token's) for its 8
        // columns
        const uint32_t t0 = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + G::SFCOL;
        bool ok = true, xok = false;
        for (int i = 0; ok; ++i) {
            const Unit un = next_unit(i);
            if (un.kind == MXL_COMBINE) continue;
            if (un.kind > MXL_COMBINE) break;
            const bool down = un.kind == MXL_DOWN;
            const int KB = down ? FB : HB, NKS = (KB + 1) / 2, n = ch.n[un.c];
            const bool resident = !down && p.xsr;
            if (resident && !xok && !(ok = xok = mbar_wait_warp(xs_full, 0, p.status, abort_flag))) break;
            // (rows past the chunk's or the tokens: unused columns, any scale)
            int row[NR / 4];
#pragma unroll
            for (int c = 0; c < NR / 4; ++c) {
                const int r = 4 * c + (lane >> 3);
                row[c] = MXL_SC * (!resident ? r : p.res ? min(r, p.T - 1) : r < n ? ch.rows[ch.pos[un.c] + r] / p.k : 0);
            }
            for (int kc = 0; kc < NKS; ++kc, advance()) {
                const uint8_t *st = ring + (size_t)s * STAGE;
                uint2 w[NR / 4];
                auto row_scales = [&](const uint8_t *rs) {
#pragma unroll
                    for (int c = 0; c < NR / 4; ++c) w[c] = *(const uint2 *)(rs + row[c]);
                };
                if (resident) row_scales(xsres + kc * p.T * MXL_SC);
                if (!(ok = mbar_wait_warp(&s_full[s], ph, p.status, abort_flag))) break;
                tc_fence_after();
                if (!resident) row_scales(st + MXL_WBYTES + n * 1024);
                const bool two = 2 * kc + 1 < KB;
                const uint4 a = *(const uint4 *)(st + 8192 + 16 * lane);
                uint4 b = make_uint4(0, 0, 0, 0);
                if (two) b = *(const uint4 *)(st + MX4_TB + 8192 + 16 * lane);
                const uint32_t va[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                uint32_t vb[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < NR / 4; ++c) {
                    vb[c] = w[c].x;
                    vb[4 + c] = w[c].y;
                }
                tmem_st8(t0 + 16 * s, va);
                tmem_st8(t0 + 16 * s + 8, vb);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sf_full[s]);
            }
        }
    } else if (warp >= 8) {
        // ---------------- epilogue
        const int q = warp & 3, ew = tid - 256;
        const float pow8[8] = {1.f, 8.f, 64.f, 512.f, 4096.f, 32768.f, 262144.f, 2097152.f};
        // sum_p 8^p (eight columns), smallest first
        auto digit_sum = [&](const uint32_t (&v)[8]) {
            float a = __uint_as_float(v[0]);
#pragma unroll
            for (int d = 1; d < 8; ++d) a = fmaf(__uint_as_float(v[d]), pow8[d], a);
            return a;
        };
        for (int i = 0;; ++i) {
            const Unit un = next_unit(i);
            bool ok = un.kind != MXL_ABORT;
            if (un.kind == MXL_COMBINE) ok = wait_count(&p.done[un.m], nch, p.status, abort_flag);
            else if (un.kind < MXL_COMBINE) ok = mbar_wait_role(&acc_full[i & 1], (i / 2) & 1, p.status, abort_flag);
            if (!bar_and_n(1, 128, ok) || un.kind == MXL_NONE) break;
            if (un.kind == MXL_COMBINE) {
                combine_tile(p, un.m, 8 * un.c, ew, s_on);
                continue;
            }
            tc_fence_after();
            const int buf = i & 1, n = ch.n[un.c], pos = ch.pos[un.c];
            const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + buf * G::N;
            if (un.kind == MXL_UP) {
                // route r's gate (lane quarters 0, 1) and up (2, 3) values meet in shared memory; the gate warps
                // finish the even routes, the up warps the odd ones.  (Loops, not unrolled code: the first
                // unit of a CTA runs at the speed of instruction fetches from memory.)
                float *xg = xch + (size_t)(buf * 2 + (q & 1)) * 2 * NR * 32 + lane, *xu = xg + NR * 32;
                float *own = q < 2 ? xg : xu;
#pragma unroll 1
                for (int r = 0; r < n; ++r) {
                    uint32_t v[8];
                    tmem_ld8(tb + 8 * (p.res ? ch.rows[pos + r] / p.k : r), v);
                    tmem_ld_wait();
                    own[32 * r] = digit_sum(v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&acc_empty[buf]);
                bar_sync_n(2 + (q & 1), 64);
                const int f0 = 64 * un.m + 32 * (q & 1), kb = f0 >> 7, cb = (f0 >> 5) & 3;
                uint8_t *hq = p.hq + hq_offset<NR>(un.c, pos, n, (FB + 1) / 2, kb >> 1);
                const int d = lane & 7;  // this lane's digit after the transpose
                uint8_t *dst = hq + (kb & 1) * 512 + d * 64 + ((cb ^ ((d >> 1) & 3)) << 4) + 4 * (lane >> 3);
#pragma unroll 1
                for (int r = q >> 1; r < n; r += 2) {
                    const float gv = xg[32 * r], uv = xu[32 * r];
                    const float h = mx4_swiglu<true>(gv, uv);
                    const int sc = digit_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu));
                    *(uint32_t *)(dst + r * 1024) = digit_word(h, sc, lane);
                    if (lane == 0) hq[n * 1024 + r * MXL_SC + (kb & 1) * 4 + cb] = (uint8_t)sc;
                }
            } else {
                const int o = 128 * un.m + 32 * q + lane;
#pragma unroll 1
                for (int i2 = 0; i2 < n; ++i2) {
                    uint32_t v[8];
                    tmem_ld8(tb + 8 * i2, v);
                    tmem_ld_wait();
                    const int r = ch.rows[pos + i2];
                    const float a = s_w[r] * digit_sum(v);
                    if (o < p.H) p.partial[(size_t)r * p.H + o] = a;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&acc_empty[buf]);
            }
            // warp 3 publishes the unit (its fence does not hold the epilogue up)
            __syncwarp();
            if (lane == 0) mbar_arrive1(&pub[i % MXL_PUB]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host

template <int XT, int TT, bool WIDE>
int launch_prep_t(const PrepParams &p, cudaStream_t s) {
    PrepParams a = p;
    size_t smem = prep_smem(p.H, p.E, TT);
    if (!WIDE) {
        // an offset of up to 7 elements in front, the end of a last group behind
        const size_t room = (MXL_PREP_SMEM_W - smem) / 2 - 16, all = (size_t)p.H / MXL_CLUSTER * p.E;
        a.w_elems = (int)std::min(room, all);
        smem += ((size_t)a.w_elems + 16) * 2;
    }
    // the limit is raised once, to the most: another thread's call may come between this and the launch
    static std::mutex mu;
    static bool raised[64] = {false};
    int dev = -1;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!raised[dev]) {
            MOE_TRY_CUDA(cudaFuncSetAttribute(mx4_prep_kernel<XT, TT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              WIDE ? MXL_PREP_SMEM : MXL_PREP_SMEM_W));
            raised[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    moe_pdl_config(&cfg, attr, dim3(MXL_CLUSTER, (p.T + TT - 1) / TT), dim3(MXL_PREP_THREADS), smem, s);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = MXL_CLUSTER;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, mx4_prep_kernel<XT, TT, WIDE>, a));
    return MOE_OK;
}

static_assert(MOE_DECODE_MAX_T <= 2 * MXL_MAX_CLUSTERS, "two tokens a cluster at most");
int cluster_tokens(int T) { return T <= MXL_MAX_CLUSTERS ? 1 : 2; }

template <int XT>
int launch_prep(const PrepParams &p, cudaStream_t s) {
    const bool wide = p.E % 8 == 0 && ((uintptr_t)p.w_router & 15) == 0;
    if (cluster_tokens(p.T) == 1) return wide ? launch_prep_t<XT, 1, true>(p, s) : launch_prep_t<XT, 1, false>(p, s);
    return wide ? launch_prep_t<XT, 2, true>(p, s) : launch_prep_t<XT, 2, false>(p, s);
}

// Shared memory of a block, less the alignment of its start.
#define MXL_SMEM (227 * 1024 - 1024)

template <int NR>
int launch_layer_t(FfnParams &p, cudaStream_t s) {
    using G = LayerGeom<NR>;
    const int HK = ((p.H + 127) / 128 + 1) / 2, cap = std::min(p.T, NR);
    p.stage = (MXL_WBYTES + cap * MXL_ROW + 511) / 512 * 512;
    // what stays resident leaves four ring stages: digits and scales, else the scales alone, else nothing
    int front = 0;
    for (int what = p.T <= 8 ? 2 : 1; what >= 0; --what) {
        p.res = what == 2 ? HK * p.T * 1024 : 0;
        p.xsr = what >= 1 ? HK * p.T * MXL_SC : 0;
        front = G::CTRL + p.res + (p.xsr + 511) / 512 * 512;
        if (front + 4 * p.stage <= MXL_SMEM) break;
    }
    p.S = std::min<int>(G::MAXS, (MXL_SMEM - front) / p.stage);
    static_assert((MXL_SMEM - G::CTRL) / (MXL_WBYTES + NR * MXL_ROW + 511) >= 4, "a ring");
    static std::mutex mu;
    static int sms[64] = {0};
    int dev = -1, n = 0;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!sms[dev]) {
            MOE_TRY_CUDA(cudaFuncSetAttribute(mx4_layer_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              MXL_SMEM + 1024));
            MOE_TRY_CUDA(cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev));
        }
        n = sms[dev];
    }
    const long chunks = (long)p.T * p.k;
    const long units = chunks * ((p.F + 63) / 64 + (p.H + 127) / 128);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    moe_pdl_config(&cfg, attr, dim3((unsigned)std::min<long>(units, n)), dim3(MXL_THREADS),
                   1024 + front + (size_t)p.S * p.stage, s);
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, mx4_layer_kernel<NR>, p));
    return MOE_OK;
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
    MOE_CHECK(((uintptr_t)x & (xtype == MOE_BF16 ? 1 : 3)) == 0);
    if ((rc = mx4_pool_check(H, F, n_slots, pool, slot_bytes)) != MOE_OK) return rc;
    // a unit travels in a word with 20 bits for its tile (H stays far below by the router's shared memory)
    if ((F + 63L) / 64 > 1 << 20) return MOE_ERR_UNSUPPORTED;
    if (prep_smem(H, E, cluster_tokens(T)) > MXL_PREP_SMEM) return MOE_ERR_UNSUPPORTED;
    const LayerWs L = layer_ws(T, H, F, k);
    uint8_t *w = (uint8_t *)workspace;
    cudaStream_t st = moe_cuda_stream(s);
    PrepParams a;
    a.x = x;
    a.w_router = w_router;
    a.bias = bias;
    a.T = T; a.H = H; a.E = E; a.k = k;
    a.ids = ids ? ids : (int32_t *)(w + L.ids);
    a.weights = weights ? weights : (float *)(w + L.weights);
    a.xq = w + L.xq;
    a.xsc = a.xq + (size_t)((H + 127) / 128 + 1) / 2 * T * 1024;
    a.ctr = (int *)(w + L.ctr);
    a.n_ctr = (int)L.ctr_ints;
    a.status = moe_status_word_device_ptr();
    FfnParams b;
    b.T = T; b.H = H; b.F = F; b.E = E; b.k = k;
    b.ids = a.ids;
    b.table = d_slot_table;
    b.weights = a.weights;
    b.extra = extra;
    b.n_slots = n_slots;
    b.pool = (const uint8_t *)pool;
    b.slot_bytes = slot_bytes;
    b.xq = a.xq;
    b.xsc = a.xsc;
    b.hq = w + L.hq;
    b.partial = (float *)(w + L.partial);
    b.y = y;
    b.ticket = a.ctr;
    b.ready = a.ctr + 4;
    b.done = b.ready + (size_t)T * k;
    b.status = a.status;
    rc = xtype == MOE_BF16 ? launch_prep<MOE_BF16>(a, st) : launch_prep<MOE_F32>(a, st);
    if (rc != MOE_OK) return rc;
    return chunk_routes(T) == 8 ? launch_layer_t<8>(b, st) : launch_layer_t<16>(b, st);
}
