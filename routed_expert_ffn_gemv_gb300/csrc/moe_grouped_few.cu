// The products of moe_grouped.cuh for few rows (GP_NK, GP_SWIGLU, GP_LORA): decode.
//
// What such a call waits for is latency: a tile of the tensor-core kernel passes its prologue, a ring of copies, 4 MMAs a
// stage of at least 80 clocks each and an epilogue.  Here nothing is staged: a warp loads 16 rows of the matrix straight into
// the fragments of mma.sync m16n8k16 (the reduction's order is free: a lane's 16 bytes of a row, eight consecutive
// elements, are its share of two steps, and the same eight of its token's row the other side's), for up to 32 rows of the
// group.  A CTA's eight warps share the reduction in turns of 32 elements and add their sums up in shared memory in
// the order of the warps (a warp's own of more than eight turns as well: its MMAs' sums truncate, see moe_grouped.cuh).  HBM bounds it: every matrix element is read once, coalesced in 64-byte pieces, 16 rows of them
// in flight per warp and instruction.
#include <algorithm>
#include <cfloat>

#include "moe_grouped.cuh"

#define GF_WARPS 8
#define GF_THREADS (32 * GF_WARPS)
#define GF_ROWS 16                       // of the matrix: M of the MMA
#define GF_PITCH 18                      // floats of a token's sums (padded)

namespace {

// Sixteen bytes that are read once.
__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
template <bool BF>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 elements of the reduction: rows g and g + 8 of the matrix (lo, hi) by the token's row.
template <bool BF>
__device__ __forceinline__ void mma32(float (&c)[4], const uint4 &lo, const uint4 &hi, const uint4 &x) {
    mma16<BF>(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
    mma16<BF>(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

template <bool BF>
__device__ __forceinline__ float value16(uint16_t h) {
    return BF ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// An fp32 number as two of tf32, the nearest and the nearest of what is left (22 bits).
__device__ __forceinline__ uint32_t nearest_tf32(float v) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 elements of the reduction as in mma32, of fp16 (which tf32 holds) by fp32: a lane's eight are its share of four steps.
__device__ __forceinline__ void mma32_f32(float (&c)[4], const uint4 &lo, const uint4 &hi, const float4 &x, const float4 &y) {
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    float left[4] = {};  // (two short chains of MMAs)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*(const __half2 *)&l[i]), q = __half22float2(*(const __half2 *)&h[i]);
        const uint32_t u0 = nearest_tf32(v[2 * i]), u1 = nearest_tf32(v[2 * i + 1]);
        const uint32_t a0 = __float_as_uint(p.x), a1 = __float_as_uint(q.x), a2 = __float_as_uint(p.y), a3 = __float_as_uint(q.y);
        mma8(c, a0, a1, a2, a3, u0, u1);
        mma8(left, a0, a1, a2, a3, nearest_tf32(v[2 * i] - __uint_as_float(u0)), nearest_tf32(v[2 * i + 1] - __uint_as_float(u1)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += left[i];
}

// An output's weights (those of up to 128 ranks from k0 on) by u of token t.
template <bool BF>
__device__ __forceinline__ float whole_sum(const uint16_t *w, const GroupedFewParams &p, int t, int k0) {
    const int chunks = (p.rank + 31) / 32;
    float s = 0.f;
    for (int j = k0; j < min(p.rank, k0 + 128); ++j) {
        const size_t piece = (size_t)t * chunks + j / 32;
        const uint16_t *u = p.u + piece * p.parts * 64 + j % 32;
        const float v = BF ? value16<BF>(u[0]) + value16<BF>(u[32]) + (p.parts == 2 ? value16<BF>(u[64]) : 0.f)
                           : ((const float *)p.u)[piece * 32 + j % 32];
        s = fmaf(value16<BF>(w[j]), v, s);
    }
    return s;
}

struct FewTile {
    int g, row0, n;
};

// NB: blocks of eight rows of the group in a tile
template <int MODE, bool BF, int NB>
__global__ void __launch_bounds__(GF_THREADS, 2) grouped_few_kernel(const __grid_constant__ GroupedFewParams p) {
    constexpr int MATS = MODE == GP_SWIGLU ? 2 : 1, NT = 8 * NB;
    __shared__ FewTile tiles[GF_MAX_TILES];
    __shared__ int sums[GF_WARPS], n_tiles_s;
    __shared__ alignas(16) float red[GF_WARPS][MATS][NT][GF_PITCH];  // (read two at a time)
    __shared__ uint8_t *s_y[NT];
    __shared__ float s_scale[NT];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t4 = lane & 3;
    // (GP_LORA: see grouped_kernel)
    if (MODE != GP_LORA) pdl_wait();
    pdl_trigger();
    // ---------------- tiles of at most NT rows of a group
    {
        int base = 0, taken = 0;  // tiles so far; where offsets descend: the end of the rows that earlier groups have
        bool descend = false;
        for (int g0 = 0; g0 < p.G; g0 += GF_THREADS) {
            const int i = g0 + tid;
            int begin = 0, end = 0;
            if (i < p.G) {
                begin = p.offsets ? p.offsets[i] : 0;
                end = p.offsets ? p.offsets[i + 1] : p.R;
            }
            const bool bad = begin < 0 || end < begin || end > p.R;
            if (bad) moe_set_status(p.status, MOE_ERR_INVALID);
            if (!descend && g0) taken = p.offsets[g0];
            descend |= __syncthreads_or(bad) != 0;
            if (descend) {  // (see grouped_kernel)
                int top = bad ? 0 : end;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int v = __shfl_up_sync(0xffffffffu, top, d);
                    if (lane >= d) top = max(top, v);
                }
                if (lane == 31) sums[warp] = top;
                const int before = __shfl_up_sync(0xffffffffu, top, 1);
                __syncthreads();
                const int in_front = (int)__reduce_max_sync(0xffffffffu, (unsigned)(lane < warp ? sums[lane] : 0));
                begin = max(begin, max(max(in_front, taken), lane ? before : 0));
                taken = max(taken, (int)__reduce_max_sync(0xffffffffu, (unsigned)(lane < GF_WARPS ? sums[lane] : 0)));
                __syncthreads();
            }
            const int cnt = bad ? 0 : max(0, end - begin);
            const int mine = (cnt + NT - 1) / NT;
            int inc = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += v;
            }
            if (lane == 31) sums[warp] = inc;
            __syncthreads();
            const int before = base + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) + inc - mine;
            base += __reduce_add_sync(0xffffffffu, lane < GF_WARPS ? sums[lane] : 0);
            for (int t = 0; t < mine; ++t)
                if (before + t < GF_MAX_TILES) tiles[before + t] = FewTile{i, begin + t * NT, min(NT, cnt - t * NT)};
            __syncthreads();
        }
        if (tid == 0) n_tiles_s = min(base, GF_MAX_TILES);
    }
    __syncthreads();
    const int blocks = (p.M + GF_ROWS - 1) / GF_ROWS, n_items = n_tiles_s * blocks;
    // the matrix, PF turns of the warp ahead and across items: rows m0 + g and m0 + g + 8 (past the last one: that one again, not
    // stored), elements 32 (warp + 8 i) + 8 t4 .. + 7 of turn i
    constexpr int PF = NB > 1 ? 4 : MATS == 2 ? 5 : 8;
    uint4 a[PF][MATS][2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint16_t *w[MATS][2];
    auto aim = [&](int item) {
        const int g0 = tiles[item / blocks].g, m0 = item % blocks * GF_ROWS;
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[m][h] = p.w + ((size_t)g0 * MATS * p.M + (size_t)m * p.M + min(m0 + g + 8 * h, p.M - 1)) * p.K + 32 * warp + 8 * t4;
    };
    auto fetch = [&](uint4 (&v)[MATS][2], int turn) {
        const int k = 32 * GF_WARPS * turn;
        const bool in = 32 * warp + 8 * t4 + k < p.K;
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[m][h] = in ? ld_once(w[m][h] + k) : zero;
    };
    const int turns = max(0, (p.K - 32 * warp + 32 * GF_WARPS - 1) / (32 * GF_WARPS));
    if ((int)blockIdx.x < n_items) {
        aim(blockIdx.x);
#pragma unroll
        for (int i = 0; i < PF; ++i) fetch(a[i], i);
    }
    bool waited = false;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        const FewTile tile = tiles[item / blocks];
        const int m0 = item % blocks * GF_ROWS;
        // the tile's rows: this lane's of each block, and (threads 0 .. NT-1) where they go
        const uint16_t *x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int c = 8 * b + g;
            int r = -1;
            if (c < tile.n) {
                r = tile.row0 + c;
                if (p.x_index) {
                    const int v = p.x_index[r];
                    r = v < 0 ? -1 : v / p.x_share;
                }
            }
            x[b] = r >= 0 && r < p.x_rows ? p.x + (size_t)r * p.ldx : nullptr;
        }
        if (tid < NT) {
            uint8_t *y = nullptr;
            float scale = 1.f;
            if (tid < tile.n) {
                const int i = tile.row0 + tid;
                const int s = p.x_index ? p.x_index[i] : i, d = p.y_index ? p.y_index[i] : i;
                if (s >= 0 && s / (p.x_index ? p.x_share : 1) < p.x_rows && d >= 0 && d < p.y_rows) {
                    y = (uint8_t *)p.y + (size_t)d * p.ldy * (p.ytype == MOE_F32 ? 4 : 2);
                    if (p.scale) scale = p.scale[d];
                } else {
                    moe_set_status(p.status, MOE_ERR_INVALID);
                }
            }
            s_y[tid] = y;
            s_scale[tid] = scale;
        }
        float acc[MATS][NB][4] = {};
        auto sum_at = [&](int m, int b, int i) -> float & { return red[warp][m][8 * b + 2 * t4 + (i & 1)][g + 4 * (i & 2)]; };
        bool kept = false;  // sums of turns so far are there
        auto total = [&](int m, int b, int i) -> float { return kept ? sum_at(m, b, i) + acc[m][b][i] : acc[m][b][i]; };
        // ---------------- the matrix by the tile's rows
        for (int i0 = 0; i0 < turns; i0 += PF) {
#pragma unroll
            for (int i = 0; i < PF; ++i) {
                const int k = 32 * (warp + GF_WARPS * (i0 + i)) + 8 * t4;  // (turns past the last one: zeros)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint4 v = k < p.K && x[b] ? *(const uint4 *)(x[b] + k) : zero;
#pragma unroll
                    for (int m = 0; m < MATS; ++m) mma32<BF>(acc[m][b], a[i][m][0], a[i][m][1], v);
                }
                if (i0 + PF < turns) fetch(a[i], i0 + PF + i);
            }
            constexpr int BATCHES = (8 + PF - 1) / PF;
            if (i0 + PF < turns && i0 / PF % BATCHES == BATCHES - 1) {
#pragma unroll
                for (int m = 0; m < MATS; ++m)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sum_at(m, b, i) = total(m, b, i);
                            acc[m][b][i] = 0.f;
                        }
                kept = true;
            }
        }
        if (item + (int)gridDim.x < n_items) {
            aim(item + gridDim.x);
#pragma unroll
            for (int i = 0; i < PF; ++i) fetch(a[i], i);
        }
        if (MODE == GP_LORA) {
            // ---------------- the adapters of the tile's tokens, the warps in turns; u's upper halves, then the rest of u (its parts)
            int id = lane < tile.n ? p.adapter[tile.row0 + lane] : -1;  // token `lane` of the tile
            if (!waited) pdl_wait();
            waited = true;
            if (id < -1 || id >= p.n_adapters) {
                moe_set_status(p.status, MOE_ERR_INVALID);
                id = -1;
            }
            const int chunks = (p.rank + 31) / 32;
            int turn = 0;
            for (int last = -1;; ++turn) {
                const unsigned left = __reduce_min_sync(0xffffffffu, id > last ? (unsigned)id : 0x7FFFFFFFu);
                if (left == 0x7FFFFFFFu) break;
                const int ad = last = (int)left;
                if (turn % GF_WARPS != warp) continue;
                const unsigned who = __ballot_sync(0xffffffffu, id == ad);
                const uint16_t *w0 = p.b + ((size_t)ad * p.M + min(m0 + g, p.M - 1)) * p.rank;
                const uint16_t *w1 = p.b + ((size_t)ad * p.M + min(m0 + g + 8, p.M - 1)) * p.rank;
                for (int c0 = 0; c0 < chunks; c0 += 4) {  // (128 ranks: the MMAs' sums truncate, see moe_grouped.cuh)
                    // sums of their own: an infinity or a NaN in b, times the zeros of the other tokens, stays out of theirs
                    float part[NB][4] = {};
                    for (int c = c0; c < min(chunks, c0 + 4); ++c) {
                        const int k = 32 * c + 8 * t4;
                        const bool in = k < p.rank;
                        const uint4 lo = in ? ld_once(w0 + k) : zero, hi = in ? ld_once(w1 + k) : zero;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            if (!(who >> (8 * b) & 0xFF)) continue;
                            const bool mine = who >> (8 * b + g) & 1;
                            const uint16_t *u = p.u + ((size_t)(tile.row0 + 8 * b + g) * chunks + c) * p.parts * 64 + 8 * t4;
                            if (BF) {
                                mma32<BF>(part[b], lo, hi, mine ? *(const uint4 *)u : zero);
                                mma32<BF>(part[b], lo, hi, mine ? *(const uint4 *)(u + 32) : zero);
                            } else {
                                const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
                                const float4 *v = (const float4 *)((const float *)p.u + ((size_t)(tile.row0 + 8 * b + g) * chunks + c) * 32 + 8 * t4);
                                mma32_f32(part[b], lo, hi, mine ? v[0] : none, mine ? v[1] : none);
                            }
                            if (BF && p.parts == 2) mma32<BF>(part[b], lo, hi, mine ? *(const uint4 *)(u + 64) : zero);
                        }
                    }
                    // this lane's sums 4 b + i: output g or g + 8 (i / 2), token 8 b + 2 t4 or the one behind it
                    bool odd = false;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            odd |= (who >> (8 * b + 2 * t4 + (i & 1)) & 1) && !(fabsf(part[b][i]) <= FLT_MAX);
                    if (odd)  // an infinity of b times u's parts, one of them 0 or of the other sign: NaN, where b u is an infinity
                        for (int o = 0; o < 4 * NB; ++o) {
                            const int t = 8 * (o >> 2) + 2 * t4 + (o & 1);
                            if (!(who >> t & 1)) continue;
                            const float s = whole_sum<BF>(o & 2 ? w1 : w0, p, tile.row0 + t, 32 * c0);
#pragma unroll
                            for (int b = 0; b < NB; ++b)  // (no index but a constant: the sums stay in registers)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (4 * b + i == o && !(fabsf(part[b][i]) <= FLT_MAX)) part[b][i] = s;
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (who >> (8 * b + 2 * t4 + (i & 1)) & 1) acc[0][b][i] += part[b][i];
                }
            }
        }
        // ---------------- the warps' sums
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum_at(m, b, i) = total(m, b, i);
        __syncthreads();
        for (int i = tid; i < tile.n * 8; i += GF_THREADS) {
            const int c = i >> 3, r = 2 * (i & 7), o = m0 + r;
            float2 v[MATS];
#pragma unroll
            for (int m = 0; m < MATS; ++m) {
                v[m] = *(const float2 *)&red[0][m][c][r];
#pragma unroll
                for (int k = 1; k < GF_WARPS; ++k) {
                    const float2 a = *(const float2 *)&red[k][m][c][r];
                    v[m] = make_float2(v[m].x + a.x, v[m].y + a.y);
                }
            }
            float2 z = v[0];
            if (MODE == GP_SWIGLU) z = make_float2(mx4_swiglu<true>(v[0].x, v[MATS - 1].x), mx4_swiglu<true>(v[0].y, v[MATS - 1].y));
            z = make_float2(s_scale[c] * z.x, s_scale[c] * z.y);
            if (o < p.M && s_y[c]) {
                if (p.ytype == MOE_F32) *(float2 *)(s_y[c] + 4 * (size_t)o) = z;
                else if (p.ytype == MOE_BF16) *(uint32_t *)(s_y[c] + 2 * (size_t)o) = grouped_pack<MOE_BF16>(z.x, z.y);
                else *(uint32_t *)(s_y[c] + 2 * (size_t)o) = grouped_pack<MOE_F16>(z.x, z.y);
            }
        }
        __syncthreads();
    }
    if (MODE == GP_LORA && !waited) pdl_wait();
}

template <int MODE, bool BF, int NB>
int launch(const GroupedFewParams &p, cudaStream_t s) {
    const long long tiles = (long long)p.R / (8 * NB) + std::min(p.G, p.R), items = tiles * ((p.M + GF_ROWS - 1) / GF_ROWS);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    moe_pdl_config(&cfg, attr, dim3((unsigned)std::min<long long>(items, 2LL * std::max(1, grouped_sms()))), dim3(GF_THREADS), 0, s);
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, grouped_few_kernel<MODE, BF, NB>, p));
    return MOE_OK;
}

}  // namespace

int grouped_few_launch(const GroupedFewParams &p, int mode, bool bf, cudaStream_t s) {
    if (mode == GP_NK) return bf ? launch<GP_NK, true, 1>(p, s) : launch<GP_NK, false, 1>(p, s);
    if (mode == GP_SWIGLU) return bf ? launch<GP_SWIGLU, true, 1>(p, s) : launch<GP_SWIGLU, false, 1>(p, s);
    if (p.R <= 8) return bf ? launch<GP_LORA, true, 1>(p, s) : launch<GP_LORA, false, 1>(p, s);
    return bf ? launch<GP_LORA, true, 4>(p, s) : launch<GP_LORA, false, 4>(p, s);
}
