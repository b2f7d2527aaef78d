// The tensor-core kernel of the 16-bit products whose rows choose their matrix: moe_grouped_matmul,
// moe_grouped_weight_grad (moe_grouped.cu) and moe_lora_matmul (moe_lora.cu).
//
//   D[m][c] = sum_k A[m][k] B[c][k],  tcgen05.mma kind::f16, fp32 sums in tensor memory.
// The matrix is always the M side (128 rows a CTA) and the rows of the group the N side, up to NT of them: an MMA is
// only as wide as the group's rows are, so ragged groups waste at most GP_GRAN - 1 columns.
//
//              A (M side)                       B (N side)                     reduction
//   GP_NK      W_g[n][k], K-major               rows x[i][k]                   K
//   GP_KN      W_g[k][n], MN-major              rows x[i][k]                   K
//   GP_SWIGLU  16 gate and 16 up rows of W_g    rows x[i][k]                   K
//              in each 32 lanes
//   GP_GRAD    columns of x, MN-major           columns of dy, MN-major        the group's rows
//   GP_LORA    W[n][k], then the adapters'      rows x[t][k], then the rows    K, then 32 ranks of each
//              B_a[n][r]                        u[t] of the adapter's tokens   adapter in the tile
//
// Persistent; a work item is (group, NT-row tile, 128-row tile of the matrix).  Warp roles over rings of mbarriers that
// run on across items:
//   warp 0       the stage's expected bytes and its A tile (TMA boxes);
//   warp 1       its B tile (TMA boxes of 64 and 16 rows);
//   warp 2       the MMAs, by an elected thread;
//   warps 4-11   the epilogue of the previous item from the other accumulator: two warps to a lane quarter;
//   warps 12-19  rows that are no box: picked by an index, u's rows of one adapter, a group's last rows (GP_GRAD).
//                16-byte asynchronous copies, zeros where there is no row;
//   warp 3       hands their stages over once they have landed.  (TMA gathers, four rows an instruction,
//                take about 40 ns each however many are in flight: 32768 rows of 2048 gathered for 1536
//                outputs took 510 us.)
// CG = 2: two CTAs share each MMA (M = 256), every CTA loads half of A and half of B.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_mx4.cuh"
#include "moe_tc.cuh"

enum { GP_NK = 0, GP_KN = 1, GP_SWIGLU = 2, GP_GRAD = 3, GP_LORA = 4 };

#define GP_THREADS 640
#define GP_ABYTES 16384   // 128 rows of 64 reduction steps
#define GP_UBYTES 8192    // GP_LORA: 128 rows of 32 ranks

struct GroupedParams {
    CUtensorMap a, b, b64;    // GP_GRAD: x and dy
    CUtensorMap ab;           // GP_LORA: the adapters' B
    const uint16_t *rows;     // x; GP_LORA: u
    const uint16_t *dy;       // GP_GRAD
    size_t ld, lddy;
    const int32_t *offsets;   // [G + 1], or NULL: one group of R rows
    int G, R;
    const int32_t *x_index;   // B's rows (GP_GRAD: A's): row i is x_index[i] / x_share, NULL: i
    int x_share, x_rows;
    const int32_t *y_index;   // output rows (GP_GRAD: B's rows), NULL: i
    int y_rows;
    const float *scale;       // [y_rows] or NULL
    void *y;
    size_t ldy;               // GP_GRAD: M
    int ytype;
    int M, K, N;              // columns of an output row; reduction (not GP_GRAD); GP_GRAD: output rows of a group
    int accumulate;           // GP_GRAD
    const int32_t *adapter;   // GP_LORA, [R]
    int n_adapters, rank;
    int fmt;                  // 0 fp16, 1 bf16
    int *status;
};

template <int CG, int NT>
struct GroupedGeom {
    static constexpr int GRAN = 16 * CG;                     // rows an MMA's width is rounded up to
    static constexpr int BBYTES = NT / CG * 128;
    static constexpr int STAGE = GP_ABYTES + BBYTES;
    static constexpr int TCOLS = 2 * NT < 32 ? 32 : 2 * NT;  // two accumulators
    static constexpr int O_OFF = 1024, O_FIRST = O_OFF + (MOE_MAX_GROUPS + 4) * 4;
    static constexpr int O_ROWS = O_FIRST + (MOE_MAX_GROUPS + 4) * 4;
    static constexpr int O_XCH = O_ROWS + 2 * NT * 16;
    static constexpr int XCH = 2 * 16 * 80;                  // bytes of an epilogue warp: two chunks
    static constexpr int O_RING = (O_XCH + 8 * XCH + 1023) / 1024 * 1024;
    static constexpr int S = (227 * 1024 - 1024 - O_RING) / STAGE / 2 * 2;  // (even: see the loaders)
    static constexpr size_t SMEM = 1024 + O_RING + (size_t)S * STAGE;
    static_assert(STAGE % 1024 == 0 && TCOLS <= 512 && (3 * S + 5) * 8 + 16 + 80 <= 1024 && S >= 3, "");
};

struct alignas(16) GroupedRow {
    uint8_t *y;  // the output row (NULL: none)
    float scale;
    int pad;
};
struct GroupedItem {
    int g, m, row0, n, npad;  // group, M tile, first row (GP_GRAD: first output row), rows, rows rounded up
    int r0, cnt, steps;       // GP_GRAD: the group's first row and rows; stages of the reduction
};

// Two results to the two 16-bit halves of a word and back.
__device__ __forceinline__ uint32_t grouped_pack(float lo, float hi, bool bf) {
    if (bf) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *(const uint32_t *)&v;
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&v;
}
__device__ __forceinline__ float2 grouped_unpack(uint32_t w, bool bf) {
    if (bf) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*(const __half2 *)&w);
}

// 16 bytes global -> shared (bytes = 16), or zeros (0).
__device__ __forceinline__ void cp_async_16_or_0(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// An arrival (one of the barrier's count) once every copy this thread has issued has landed.
__device__ __forceinline__ void cp_async_mbar_arrive_noinc(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The smallest of a tile's adapters above `last` (-1 to begin with); INT_MAX: none.  ids: this lane's share of the
// tile's tokens; every lane gets the same answer.
__device__ __forceinline__ int grouped_next_adapter(const int (&ids)[8], int last) {
    unsigned best = 0x7FFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (ids[i] > last) best = min(best, (unsigned)ids[i]);
    return (int)__reduce_min_sync(0xffffffffu, best);
}

template <int CG, int NT, int MODE>
__global__ void __launch_bounds__(GP_THREADS, 1) grouped_kernel(const __grid_constant__ GroupedParams p) {
    using G_ = GroupedGeom<CG, NT>;
    constexpr int S = G_::S;
    constexpr bool GRAD = MODE == GP_GRAD, A_MN = GRAD || MODE == GP_KN, B_MN = GRAD;
    constexpr int MROWS = MODE == GP_SWIGLU ? 64 : 128;  // output columns of a CTA's tile
    static_assert(!GRAD || NT / CG == 128, "sixteen pieces of eight columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint64_t *full = (uint64_t *)smem;
    uint64_t *empty = full + S;
    uint64_t *landed = empty + S;
    uint64_t *acc_full = landed + S;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_slot = (uint32_t *)(mma_done + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    int *sums = (int *)(tmem_slot + 4);                       // [20]
    int *off = (int *)(smem + G_::O_OFF);                     // [G + 1]
    int *first = (int *)(smem + G_::O_FIRST);                 // [G + 1] items before a group's
    GroupedRow *e_rows = (GroupedRow *)(smem + G_::O_ROWS);   // [2][NT]
    uint8_t *ring = smem + G_::O_RING;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = CG == 1 ? 0 : (int)cluster_ctarank();
    const bool loaders = GRAD || MODE == GP_LORA || p.x_index;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1 + (loaders ? CG : 0));
            mbar_init(&landed[s], 128);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8 * CG);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc_group<CG>(tmem_slot, G_::TCOLS);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (GP_LORA: the kernel in front computes u and nothing else; it starts this one when everything before it is
    // complete, and only u is waited for, by the warp that loads it)
    if (MODE != GP_LORA) pdl_wait();
    pdl_trigger();

    // ---------------- items: tiles of the M side, inner, by tiles of each group's rows
    const int mt = (p.M + MROWS * CG - 1) / (MROWS * CG);
    const int gran = GRAD ? 64 * CG : G_::GRAN;
    const int gt = GRAD ? (p.N + NT - 1) / NT : 0;  // GP_GRAD: tiles of N
    for (int i = tid; i <= p.G; i += GP_THREADS) off[i] = p.offsets ? p.offsets[i] : i * p.R;
    __syncthreads();
    auto rows_of = [&](int g) -> int {  // rows of a group; none where the offsets are no range of rows
        const int a = off[g], b = off[g + 1];
        return a >= 0 && b >= a && b <= p.R ? b - a : 0;
    };
    constexpr int PER = (MOE_MAX_GROUPS + GP_THREADS - 1) / GP_THREADS;
    {
        int c[PER], t = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int g = tid * PER + i;
            c[i] = t;
            if (g < p.G) {
                const int n = rows_of(g);
                if (!n && off[g + 1] != off[g]) moe_set_status(p.status, MOE_ERR_INVALID);
                t += mt * (GRAD ? gt : (n + NT - 1) / NT);
            }
        }
        int inc = t;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int before = inc - t;
        for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (tid * PER + i < p.G) first[tid * PER + i] = before + c[i];
        if (tid == GP_THREADS - 1) first[p.G] = before + t;
    }
    __syncthreads();
    const int n_items = first[p.G], stride = (int)gridDim.x / CG, item0 = (int)blockIdx.x / CG;
    auto item_at = [&](int j) -> GroupedItem {
        GroupedItem it;
        int lo = 0, hi = p.G;  // the last group whose first item is not after j
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= j) lo = mid;
            else hi = mid;
        }
        it.g = lo;
        const int r = j - first[lo], t = r / mt;
        it.m = r - t * mt;
        it.r0 = off[lo];
        it.cnt = rows_of(lo);
        // near-equal tiles: none is empty, as size <= NT
        const int all = GRAD ? p.N : it.cnt, nt = (all + NT - 1) / NT;
        const int size = ((all + nt - 1) / nt + gran - 1) / gran * gran;
        it.n = min(size, all - t * size);
        it.npad = (it.n + gran - 1) / gran * gran;
        it.row0 = (GRAD ? 0 : it.r0) + t * size;
        it.steps = ((GRAD ? it.cnt : p.K) + 63) / 64;
        return it;
    };
    // GP_LORA: this lane's share of the tile's adapters (-1: none)
    auto tile_adapters = [&](const GroupedItem &it, int (&ids)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = lane + 32 * i;
            const int a = c < it.n ? p.adapter[it.row0 + c] : -1;
            if (a >= p.n_adapters || a < -1) moe_set_status(p.status, MOE_ERR_INVALID);
            ids[i] = a < p.n_adapters ? a : -1;
        }
    };
    const int chunks = MODE == GP_LORA ? (p.rank + 31) / 32 : 0;
    auto extra_stages = [&](const GroupedItem &it) -> int {
        int n = 0;
        if (MODE == GP_LORA) {
            int ids[8];
            tile_adapters(it, ids);
            for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF; a = grouped_next_adapter(ids, a)) n += chunks;
        }
        return n;
    };
    auto source = [&](int i) -> int {  // x's row of position i, -1: none
        if (!p.x_index) return i < p.x_rows ? i : -1;
        const int v = p.x_index[i], r = v / p.x_share;
        return v >= 0 && r < p.x_rows ? r : -1;
    };
    auto target = [&](int i) -> int {
        const int v = p.y_index ? p.y_index[i] : i;
        return v >= 0 && v < p.y_rows ? v : -1;
    };
    if (warp == 0) {
        // ---------------- A, and what a stage's copies bring
        int gs = 0, st = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int j = item0; j < n_items && ok; j += stride) {
            const GroupedItem it = item_at(j);
            const int nb = it.npad / CG, m0 = (it.m * CG + rank) * MROWS;
            for (int kb = 0; kb < it.steps; ++kb, ++gs) {
                if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                uint8_t *dst = ring + (size_t)st * G_::STAGE;
                const uint32_t bar = CG == 1 ? smem_u32(&full[st]) : cluster_map(&full[st], 0);
                const bool whole = !GRAD || 64 * kb + 64 <= it.cnt;  // (else by the loaders)
                const bool box_a = GRAD ? whole && !p.x_index : true, box_b = GRAD ? whole && !p.y_index : !p.x_index;
                if (rank == 0)
                    mbar_arrive_expect_tx_elect(&full[st], CG * ((box_a ? GP_ABYTES : 0u) + (box_b ? nb * 128u : 0u)));
                if (MODE == GP_NK || MODE == GP_LORA) {
                    if (lane == 0) tma_tile_3d<CG>(dst, &p.a, kb * 64, m0, MODE == GP_LORA ? 0 : it.g, bar);
                } else if (MODE == GP_KN) {
                    if (lane < 2) tma_tile_3d<CG>(dst + lane * 8192, &p.a, m0 + 64 * lane, kb * 64, it.g, bar);
                } else if (MODE == GP_SWIGLU) {
                    if (lane < 4) tma_tile_4d<CG>(dst + lane * 4096, &p.a, kb * 64, m0 + 16 * lane, 0, it.g, bar);
                } else if (box_a) {
                    if (lane < 2) tma_tile_2d<CG>(dst + lane * 8192, &p.a, m0 + 64 * lane, it.r0 + 64 * kb, bar);
                }
                __syncwarp();
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (MODE == GP_LORA && ok) {
                int ids[8];
                tile_adapters(it, ids);
                for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF && ok; a = grouped_next_adapter(ids, a))
                    for (int c = 0; c < chunks; ++c, ++gs) {
                        if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                        uint8_t *dst = ring + (size_t)st * G_::STAGE;
                        const uint32_t bar = CG == 1 ? smem_u32(&full[st]) : cluster_map(&full[st], 0);
                        if (rank == 0) mbar_arrive_expect_tx_elect(&full[st], CG * GP_UBYTES);
                        if (lane == 0) tma_tile_3d<CG>(dst, &p.ab, c * 32, m0, a, bar);
                        __syncwarp();
                        if (++st == S) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
            }
        }
        // never leave with copies in flight (a pair: the leader's barriers count both CTAs' copies)
        if (lane == 0 && rank == 0)
            for (int s = 0; s < S && s < gs; ++s) {
                const int last = s + ((gs - 1 - s) / S) * S;
                mbar_wait_bounded(&full[s], (last / S) & 1, p.status);
            }
        if (!ok) settle_after_abort();
    } else if (warp == 1 && (GRAD ? !p.y_index : !p.x_index)) {
        // ---------------- B
        int gs = 0, st = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int j = item0; j < n_items && ok; j += stride) {
            const GroupedItem it = item_at(j);
            const int nb = it.npad / CG, c0 = it.row0 + rank * nb;
            const int extra = extra_stages(it);
            for (int kb = 0; kb < it.steps + extra; ++kb, ++gs) {
                if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                uint8_t *dst = ring + (size_t)st * G_::STAGE + GP_ABYTES;
                const uint32_t bar = CG == 1 ? smem_u32(&full[st]) : cluster_map(&full[st], 0);
                if (GRAD) {
                    if (64 * lane < nb && 64 * kb + 64 <= it.cnt)
                        tma_tile_2d<CG>(dst + lane * 8192, &p.b, c0 + 64 * lane, it.r0 + 64 * kb, bar);
                } else if (kb < it.steps) {
                    // 64 rows a box, the rest by 16
                    const int big = nb / 64, r = lane < big ? 64 * lane : 64 * big + 16 * (lane - big);
                    if (r < nb) tma_tile_2d<CG>(dst + r * 128, lane < big ? &p.b64 : &p.b, kb * 64, c0 + r, bar);
                }
                __syncwarp();
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) settle_after_abort();
    } else if (warp >= 12 && loaders) {
        // ---------------- rows that are no box
        // Two teams of four warps take alternate stages (the ring is an even number of stages: a team sees every phase of the
        // barriers that it waits for).  A copy costs its warp a few instructions one after another, which is what bounds
        // this: 8192^3, every row by index: one team of four warps 921 us, two of two 1442.
        const int team = (warp - 12) >> 2, lt = (tid - 384) & 127;
        int gs = 0, st = 0;
        uint32_t ph = 1;
        bool ok = true;
        auto begin = [&]() -> bool { return gs < S || (ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag)); };
        auto next = [&]() {
            ++gs;
            if (++st == S) {
                st = 0;
                ph ^= 1u;
            }
        };
        // GP_GRAD: a warp's sixteen rows of a stage, looked up by its lanes 0-15 for the team's next stage (of this item or the
        // next) while this one is copied
        int xr = -1, yr = -1;
        auto look_up = [&](const GroupedItem &it, int kb) {
            const int q = kb * 64 + (lt >> 5) * 2 + (lane & 1) + 8 * ((lane >> 1) & 7);
            xr = yr = -1;
            if (kb < it.steps && q < it.cnt) {
                xr = source(it.r0 + q);
                yr = target(it.r0 + q);
                if (xr < 0 || yr < 0) {
                    moe_set_status(p.status, MOE_ERR_INVALID);
                    xr = yr = -1;
                }
            }
        };
        GroupedItem it = {}, after = {};
        if (GRAD && item0 < n_items) {
            after = item_at(item0);
            look_up(after, team);
        }
        for (int j = item0; j < n_items && ok; j += stride) {
            if (GRAD) {
                it = after;
                if (j + stride < n_items) after = item_at(j + stride);
            } else {
                it = item_at(j);
            }
            const int nb = it.npad / CG;
            if (!GRAD) {
                // eight threads a row: piece lt % 8 of rows lt / 8 + 16 i
                constexpr int RI = NT / CG / 16;
                const int piece = lt & 7, r0 = lt >> 3, rows = min(nb, it.n - rank * nb);
                const uint32_t at = smem_u32(ring) + GP_ABYTES + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
                const uint16_t *src[RI];
                int who[RI];  // bytes to copy; GP_LORA: the token's adapter
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const int c = r0 + 16 * i;
                    const int r = c >= rows ? -1 : MODE == GP_LORA ? it.row0 + rank * nb + c : source(it.row0 + rank * nb + c);
                    who[i] = MODE != GP_LORA ? (r >= 0 ? 16 : 0) : r >= 0 ? p.adapter[r] : -1;
                    src[i] = p.rows + (size_t)max(r, 0) * p.ld + 8 * piece + (team == (gs & 1) ? 0 : 64);
                }
                for (int kb = 0; kb < it.steps; ++kb, next()) {
                    if ((gs & 1) != team) continue;
                    if (!begin()) break;
                    if (MODE != GP_LORA) {
                        const uint32_t d = at + (uint32_t)st * G_::STAGE;
                        const int most = kb * 64 + 8 * piece < p.K ? 16 : 0;
#pragma unroll
                        for (int i = 0; i < RI; ++i) {
                            if (16 * i < rows) cp_async_16_or_0(d + i * 2048, src[i], min(most, who[i]));
                            src[i] += kb + 3 > it.steps ? 0 : 128;
                        }
                    }
                    cp_async_mbar_arrive_noinc(&landed[st]);
                }
                if (MODE == GP_LORA && ok) {
                    if (j == item0) pdl_wait();  // u
                    int ids[8];
                    tile_adapters(it, ids);
                    const uint16_t *u = p.rows + (size_t)(it.row0 + rank * nb + r0) * p.ld + 8 * piece;
                    for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF && ok; a = grouped_next_adapter(ids, a))
                        for (int c = 0; c < chunks; ++c, next()) {
                            if ((gs & 1) != team) continue;
                            if (!begin()) break;
                            const uint32_t d = at + (uint32_t)st * G_::STAGE;
#pragma unroll
                            for (int i = 0; i < RI; ++i)
                                if (16 * i < nb) {
                                    const bool some = who[i] == a;
                                    cp_async_16_or_0(d + i * 2048, some ? u + (size_t)16 * i * p.ld + c * 64 : p.rows,
                                                     some ? 16 : 0);
                                }
                            cp_async_mbar_arrive_noinc(&landed[st]);
                        }
                }
            } else {
                // sixteen threads a row (128 columns): piece lt % 16 of rows lt / 16 + 8 i
                const int end = gs + it.steps;  // the next item's first stage
                const bool more = j + stride < n_items, any = it.steps > ((gs & 1) != team);
                if (!any && more) look_up(after, (end & 1) != team);
                const int piece = lt & 15, r0 = lt >> 4;
                const int ca = (it.m * CG + rank) * 128 + 8 * piece, cb = rank * nb + 8 * piece;
                const int in_a = ca < p.M ? 16 : 0, in_b = it.row0 + cb < p.N ? 16 : 0;
                const uint16_t *a = p.rows + (in_a ? ca : 0), *b = p.dy + (in_b ? it.row0 + cb : 0);
                const uint32_t at = smem_u32(ring) + (piece >> 3) * 8192 + r0 * 128 + (((piece ^ r0) & 7) << 4);
                for (int kb = 0; kb < it.steps; ++kb, next()) {
                    if ((gs & 1) != team) continue;
                    if (!begin()) break;
                    const bool whole = 64 * kb + 64 <= it.cnt;
                    const uint32_t d = at + (uint32_t)st * G_::STAGE;
                    if (p.x_index || !whole)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = __shfl_sync(0xffffffffu, xr, 2 * i + (lane >> 4));
                            cp_async_16_or_0(d + i * 1024, a + (size_t)max(r, 0) * p.ld, r >= 0 ? in_a : 0);
                        }
                    if (p.y_index || !whole)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = __shfl_sync(0xffffffffu, yr, 2 * i + (lane >> 4));
                            if (cb < (rank + 1) * nb)
                                cp_async_16_or_0(d + GP_ABYTES + i * 1024, b + (size_t)max(r, 0) * p.lddy, r >= 0 ? in_b : 0);
                        }
                    if (kb + 2 < it.steps) look_up(it, kb + 2);
                    else if (more) look_up(after, (end & 1) != team);
                    cp_async_mbar_arrive_noinc(&landed[st]);
                }
            }
        }
        cp_async_wait_all();
        if (MODE == GP_LORA) pdl_wait();
    } else if (warp == 3 && loaders) {
        // ---------------- the loaders' stages: their copies have landed; the tensor cores may read them
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int j = item0; j < n_items && ok; j += stride) {
            const GroupedItem it = item_at(j);
            const int n = it.steps + extra_stages(it);
            for (int kb = 0; kb < n; ++kb) {
                if (!(ok = mbar_wait_warp(&landed[st], ph, p.status, abort_flag))) break;
                fence_proxy_async_smem();
                if (lane == 0) {
                    if (CG == 1) mbar_arrive1(&full[st]);
                    else mbar_arrive_cluster(cluster_map(&full[st], 0));
                }
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 2 && rank == 0) {
        // ---------------- MMA issuer
        int jl = 0, st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int j = item0; j < n_items && ok; j += stride, ++jl) {
            const GroupedItem it = item_at(j);
            // (a value that a shuffle hands out is known to be the same in every lane: it stays in a uniform register, where
            // the MMA wants its operands)
            const uint32_t idesc = umma_idesc_16(p.fmt, A_MN, B_MN, 128 * CG, __shfl_sync(0xffffffffu, it.npad, 0));
            const int buf = jl & 1;
            const int extra = extra_stages(it);
            if (jl >= 2 && !(ok = mbar_wait_warp(&acc_empty[buf], ((jl / 2) - 1) & 1, p.status, abort_flag))) break;
            tc_fence_after();
            const uint32_t d = __shfl_sync(0xffffffffu, tmem, 0) + buf * NT;
            const int len = GRAD ? __shfl_sync(0xffffffffu, it.cnt, 0) : p.K, n_steps = __shfl_sync(0xffffffffu, it.steps, 0);
            for (int kb = 0; kb < n_steps; ++kb) {
                if (!(ok = mbar_wait_warp(&full[st], ph, p.status, abort_flag))) break;
                tc_fence_after();
                const uint32_t sa = smem_u32(ring) + (uint32_t)st * G_::STAGE;
                const uint64_t a = A_MN ? umma_desc_mn_sw128(sa, 8192) : umma_desc_sw128(sa);
                const uint64_t b = B_MN ? umma_desc_mn_sw128(sa + GP_ABYTES, 8192) : umma_desc_sw128(sa + GP_ABYTES);
                const int left = len - 64 * kb;
                auto step = [&](int q) {
                    umma_f16_elect<CG>(d, a + (uint64_t)(q * (A_MN ? 128 : 2)), b + (uint64_t)(q * (B_MN ? 128 : 2)), idesc,
                                       q > 0 || kb > 0);
                };
                step(0);
                if (left > 48) {  // (no branch between the MMAs)
                    step(1);
                    step(2);
                    step(3);
                } else {
                    if (left > 16) step(1);
                    if (left > 32) step(2);
                }
                umma_commit_group_elect<CG>(&empty[st]);
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            for (int e = 0, c = 0; e < extra && ok; ++e) {
                if (!(ok = mbar_wait_warp(&full[st], ph, p.status, abort_flag))) break;
                tc_fence_after();
                // 32 ranks: u's upper halves in the first 64 bytes of a row, the rest of u in the second, both by the same B_a
                const uint32_t sa = smem_u32(ring) + (uint32_t)st * G_::STAGE;
                const uint64_t a = umma_desc_sw64(sa), b = umma_desc_sw128(sa + GP_ABYTES);
                const bool two = p.rank - 32 * c > 16;
                umma_f16_elect<CG>(d, a, b, idesc, 1);
                umma_f16_elect<CG>(d, a, b + 4, idesc, 1);
                if (two) {
                    umma_f16_elect<CG>(d, a + 2, b + 2, idesc, 1);
                    umma_f16_elect<CG>(d, a + 2, b + 6, idesc, 1);
                }
                umma_commit_group_elect<CG>(&empty[st]);
                if (++c == chunks) c = 0;
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (ok) umma_commit_group_elect<CG>(&acc_full[buf]);
        }
        umma_commit_group_elect<CG>(mma_done);  // every MMA has completed before tensor memory is released
        mbar_wait_bounded(mma_done, 0, p.status);
    } else if (warp >= 4 && warp < 12) {
        // ---------------- epilogue: an accumulator column is an output row.  16-bit results: fragments of 16 lanes x 8 columns,
        // each pair of columns packed, transposed by way of shared memory (stmatrix), so that a lane stores eight
        // consecutive elements of an output row; fp32 results transposed a word at a time, four consecutive elements a store.
        // (Stored straight from the registers, 128 bytes of one output row an instruction: 4864 x 4096 x 512 31.4 us,
        // this way 24.8.)
        const int q = warp & 3, ew = warp - 4, half = ew >> 2, et = ew * 32 + lane;
        const bool bf = p.ytype == MOE_BF16, f32 = p.ytype == MOE_F32;
        const uint32_t xb = smem_u32(smem + G_::O_XCH) + ew * G_::XCH;
        const int size = f32 ? 4 : 2;
        // stmatrix: the address of row lane % 8 of 8 x 8 matrix lane / 8.  Matrices 0, 1: output rows 0-7, elements 0-7 and 8-15;
        // 2, 3: output rows 8-15
        constexpr int PITCH = MODE == GP_SWIGLU ? 48 : 80;  // (no bank conflicts)
        const uint32_t xm = xb + ((lane & 7) + 8 * (lane >> 4)) * PITCH + ((lane >> 3) & 1) * 16;
        int jl = 0;
        for (int j = item0; j < n_items; j += stride, ++jl) {
            const GroupedItem it = item_at(j);
            const int buf = jl & 1;
            if (et < NT && et < it.n) {
                GroupedRow r;
                r.y = nullptr;
                r.scale = 1.f;
                if (GRAD) {
                    r.y = (uint8_t *)p.y + ((size_t)it.g * p.N + it.row0 + et) * p.M * size;
                } else {
                    const int dst = source(it.row0 + et) < 0 ? -1 : target(it.row0 + et);
                    if (dst < 0) {
                        moe_set_status(p.status, MOE_ERR_INVALID);
                    } else {
                        r.y = (uint8_t *)p.y + (size_t)dst * p.ldy * size;
                        if (p.scale) r.scale = p.scale[dst];
                    }
                }
                e_rows[buf * NT + et] = r;
            }
            const bool w = mbar_wait_role(&acc_full[buf], (jl / 2) & 1, p.status, abort_flag);
            if (!bar_and_n(1, 256, w)) break;
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + buf * NT;
            const GroupedRow *rows = e_rows + buf * NT;
            const bool none = GRAD && !it.steps;
            const int m0 = (it.m * CG + rank) * MROWS + MROWS / 4 * q;  // the warp's first element
            // 16 columns: 32x32b, or in fragments the first 16 lanes' registers, then the others'
            auto load = [&](uint32_t (&v)[16], int c0) {
                if (MODE != GP_SWIGLU && f32) {
                    tmem_ld16(tb + c0, v);
                } else {
                    tmem_ld_16x256b_x2(tb + c0, reinterpret_cast<uint32_t(&)[8]>(v[0]));
                    tmem_ld_16x256b_x2(tb + (16u << 16) + c0, reinterpret_cast<uint32_t(&)[8]>(v[8]));
                }
            };
            auto process = [&](uint32_t (&v)[16], int c0, int odd) {
                if (none)
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = 0u;
                if (MODE != GP_SWIGLU && f32) {
                    float *x = (float *)(smem + G_::O_XCH + ew * G_::XCH);  // padded to 36: no bank conflicts
                    const int m = m0 + 4 * (lane & 7);
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[36 * k + lane] = __uint_as_float(v[k]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 4 * k + (lane >> 3);
                        float4 a = *(const float4 *)(x + 36 * c + 4 * (lane & 7));
                        if (c0 + c < it.n && m < p.M) {
                            const GroupedRow r = rows[c0 + c];
                            float4 *o = (float4 *)((float *)r.y + m);
                            if (!GRAD) a = make_float4(r.scale * a.x, r.scale * a.y, r.scale * a.z, r.scale * a.w);
                            if (GRAD && p.accumulate) {
                                const float4 b = *o;
                                a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
                            }
                            if (GRAD || r.y) *o = a;
                        }
                    }
                    __syncwarp();
                    return;
                }
                // registers 4 b + {0, 1}: row lane / 4, columns 8 b + 2 (lane % 4) + {0, 1}; + {2, 3}: row lane / 4 + 8
                uint32_t(&lo)[8] = reinterpret_cast<uint32_t(&)[8]>(v[0]);
                uint32_t(&hi)[8] = reinterpret_cast<uint32_t(&)[8]>(v[8]);
                const int cq = c0 + 2 * (lane & 3);
                const uint32_t to = xm + odd * (G_::XCH / 2), from = xb + odd * (G_::XCH / 2);
                if (MODE == GP_SWIGLU) {
                    float h[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k] = mx4_swiglu<true>(__uint_as_float(lo[k]), __uint_as_float(hi[k]));
                    if (p.scale || f32) {
                        // (e_rows past the last row may hold anything: not stored)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int c = cq + 8 * (k >> 2) + (k & 1), m = m0 + (lane >> 2) + 4 * (k & 2);
                            if (c < it.n) {
                                const GroupedRow r = rows[c];
                                h[k] *= r.scale;
                                if (f32 && r.y && m < p.M) ((float *)r.y)[m] = h[k];
                            }
                        }
                        if (f32) return;
                    }
                    stmatrix_x4_trans(to, grouped_pack(h[0], h[1], bf), grouped_pack(h[2], h[3], bf),
                                      grouped_pack(h[4], h[5], bf), grouped_pack(h[6], h[7], bf));
                    __syncwarp();
                    const int c = lane >> 1, m = m0 + 8 * (lane & 1);
                    const uint4 a = ld_shared_16(from + c * PITCH + 16 * (lane & 1));
                    if (c0 + c < it.n && m < p.M && rows[c0 + c].y) *(uint4 *)(rows[c0 + c].y + 2 * m) = a;
                } else {
                    uint32_t old[8] = {};
                    if (GRAD && p.accumulate) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int c = 8 * k + (lane >> 2), m = m0 + 8 * (lane & 3);
                            if (c0 + c < it.n && m < p.M)
                                st_shared_16(from + c * PITCH + 16 * (lane & 3), *(const uint4 *)(rows[c0 + c].y + 2 * m));
                        }
                        __syncwarp();
                        ldmatrix_x4_trans(to, old[0], old[1], old[2], old[3]);
                        ldmatrix_x4_trans(to + 32, old[4], old[5], old[6], old[7]);
                        __syncwarp();
                    }
                    float s[4] = {1.f, 1.f, 1.f, 1.f};
                    if (!GRAD && p.scale)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (cq + 8 * (k >> 1) + (k & 1) < it.n) s[k] = rows[cq + 8 * (k >> 1) + (k & 1)].scale;
                    auto pack = [&](const uint32_t (&v)[8], int k, uint32_t before) -> uint32_t {
                        float2 o = make_float2(0.f, 0.f);
                        if (GRAD && p.accumulate) o = grouped_unpack(before, bf);
                        return grouped_pack(fmaf(s[k >> 2 << 1], __uint_as_float(v[k]), o.x),
                                            fmaf(s[(k >> 2 << 1) + 1], __uint_as_float(v[k + 1]), o.y), bf);
                    };
                    stmatrix_x4_trans(to, pack(lo, 0, old[0]), pack(lo, 2, old[1]), pack(lo, 4, old[2]), pack(lo, 6, old[3]));
                    stmatrix_x4_trans(to + 32, pack(hi, 0, old[4]), pack(hi, 2, old[5]), pack(hi, 4, old[6]), pack(hi, 6, old[7]));
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = 8 * k + (lane >> 2), m = m0 + 8 * (lane & 3);
                        const uint4 a = ld_shared_16(from + c * PITCH + 16 * (lane & 3));
                        if (c0 + c < it.n && m < p.M && rows[c0 + c].y) *(uint4 *)(rows[c0 + c].y + 2 * m) = a;
                    }
                }
            };
            // a chunk of 16 columns is read from tensor memory while the one before it is worked on (two buffers each: a
            // warp barrier lies between two uses of one)
            uint32_t v0[16], v1[16];
            int c0 = 16 * half;
            if (c0 < it.n) load(v0, c0);
            for (; c0 < it.n; c0 += 64) {
                tmem_ld_wait();
                if (c0 + 32 < it.n) load(v1, c0 + 32);
                process(v0, c0, 0);
                if (c0 + 32 < it.n) {
                    tmem_ld_wait();
                    if (c0 + 64 < it.n) load(v0, c0 + 64);
                    process(v1, c0 + 32, 1);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1) mbar_arrive1(&acc_empty[buf]);
                else mbar_arrive_cluster(cluster_map(&acc_empty[buf], 0));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_group<CG>(tmem, G_::TCOLS);
    }
}

// ------------------------------------------------------------------ host

// Launches the kernel on the current device with one CTA (or pair) an SM (or two), at most `items` of them.
int grouped_launch(const GroupedParams &p, int mode, bool wide, long long items, cudaStream_t s);
// Tensor map of 16-bit elements: `rank` dimensions and box extents innermost first, strides in bytes from the second on.
int grouped_map(CUtensorMap *map, int type, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box, int swizzle_bytes);
