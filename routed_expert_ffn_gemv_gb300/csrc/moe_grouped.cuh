// The tensor-core kernel of the 16-bit products whose rows choose their matrix: moe_grouped_matmul,
// moe_grouped_weight_grad (moe_grouped.cu) and moe_lora_matmul (moe_lora.cu).
//
//   D[m][c] = sum_k A[m][k] B[c][k],  tcgen05.mma kind::f16, fp32 sums in tensor memory.
// The matrix is always the M side (128 rows a CTA) and the rows of the group the N side, up to NT of them: an MMA is
// only as wide as the group's rows are, so ragged groups waste at most GRAN - 1 columns.
//
//              A (M side)                       B (N side)                     reduction
//   GP_NK      W_g[n][k], K-major               rows x[i][k]                   K
//   GP_KN      W_g[k][n], MN-major              rows x[i][k]                   K
//   GP_SWIGLU  16 gate and 16 up rows of W_g    rows x[i][k]                   K
//              in each 32 lanes
//   GP_GRAD    columns of x, MN-major           columns of dy, MN-major        the group's rows
//   GP_LORA    W[n][k], then the adapters'      rows x[t][k], then the rows    K, then 32 ranks of each
//   (bf16),    B_a[n][r]                        u[t] of the adapter's tokens   adapter in the tile
//   GP_LORA_F16
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
// Two shapes (see moe_grouped_matmul for the rule): NT = 32, one CTA an item, for few rows, when reading the matrix is
// the work (77 tokens over 64 experts of 2 x 1408 x 2048: 86 us, HBM's rate); NT = 256 (fp32 results 128, but for the gradient
// of short groups) by pairs of CTAs, when it
// is the MMAs (8192^3: 631 us, 1743 TFLOP/s; by single CTAs, which load twice as much, a prompt's gate/up product took
// 1.7 times as long).
// CG = 1: where items are few, the CTAs of a cluster share an item's reduction and add their sums up over distributed shared
// memory, in the order of their ranks.
// CG = 2: two CTAs share each MMA (M = 256), every CTA loads half of A and half of B.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_mx4.cuh"
#include "moe_tc.cuh"

enum { GP_NK = 0, GP_KN = 1, GP_SWIGLU = 2, GP_GRAD = 3, GP_LORA = 4, GP_LORA_F16 = 5 };

#define GP_THREADS 640
#define GP_ABYTES 16384   // 128 rows of 64 reduction steps
#define GP_UBYTES 8192    // GP_LORA: 128 rows of 32 ranks

struct GroupedParams {
    CUtensorMap a, b, b64;    // GP_GRAD: x and dy
    CUtensorMap ab;           // GP_LORA: the adapters' B
    CUtensorMap yt;           // GP_GRAD: dw by boxes of 32 x 32 (16 x 32 of fp32)
    const uint16_t *rows;     // x; GP_LORA: u
    const uint16_t *dy;       // GP_GRAD
    const uint16_t *lora_b;   // GP_LORA: the adapters' B
    const float *factor;      // GP_LORA, fp16: what each 32 ranks of a token's u are to be multiplied by
    int factors;              // of a token, that may differ: 1 or all
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
    int M, K, N;              // columns of an output row; reduction (not GP_GRAD); GP_GRAD: output rows of a group
    int accumulate;           // GP_GRAD
    const int32_t *adapter;   // GP_LORA, [R]
    int n_adapters, rank, parts;  // parts: 128-byte pieces of u for 32 ranks
    int fmt;                  // 0 fp16, 1 bf16
    int *status;
};

#define GP_ITEMS 96       // items of a CTA that are worked out ahead, in shared memory
#define GP_MAX_SPLIT 8    // CTAs that share an item's reduction

// A sum on the tensor cores drops, at each of its steps of 16, what lies below the last bit of the larger term: 128 steps
// (K = 2048) leave it 1.6e-6 off, relative to the result's norm, which bf16 and fp16 results do not show and fp32 results do
// (fp32 sums rounded to nearest: 1.5e-7).  An accumulator therefore takes ACC_STAGES stages at most, and the epilogue adds an
// item's accumulators up in order: for fp32 results 16 or 32 steps each (2.3e-7, 4.7e-7), for 16-bit ones 512 (6e-6, where
// fp16's half step is 4.9e-4).  Of more accumulators than tensor memory holds, the epilogue adds the first to the second and
// hands it back while the others are filled, and so on: the error does not grow with the reduction (K = 65536, pairs:
// 1.9e-5 off with four accumulators, 5.1e-7 this way).

template <int CG, int NT, int OT>
struct GroupedGeom {
    static constexpr int GRAN = 16 * CG;                     // rows an MMA's width is rounded up to
    static constexpr int BBYTES = NT / CG * 128;
    static constexpr int STAGE = GP_ABYTES + BBYTES;
    static constexpr unsigned SLOTS = OT == MOE_F32 ? 512 / NT : 2;  // accumulators in tensor memory
    static constexpr int TCOLS = (int)SLOTS * NT;                 // (a power of two from 32 on)
    static constexpr int CH = NT >= 64 && OT != MOE_F32 ? 32 : 16;  // columns of an epilogue warp's chunk
    static constexpr int XCH = CH * 80 < 2304 ? 2304 : CH * 80;  // bytes of an epilogue warp
    // CG = 1: partial sums of up to GP_MAX_SPLIT CTAs, for this CTA's share of the rows
    static constexpr int RED = CG == 1 ? (NT + GP_MAX_SPLIT - 1) * 512 : 0;
    static constexpr int O_ITEMS = 1024, O_OFF = O_ITEMS + GP_ITEMS * 16;
    static constexpr int O_FIRST = O_OFF + (MOE_MAX_GROUPS + 4) * 4;
    static constexpr int O_ORDER = O_FIRST + (MOE_MAX_GROUPS + 4) * 4;
    static constexpr int O_ROWS = O_ORDER + MOE_MAX_GROUPS * 2;
    static constexpr int O_XCH = (O_ROWS + 2 * NT * 12 + 511) / 512 * 512;  // (GP_GRAD's boxes: 64-byte swizzle)
    static constexpr int O_RED = O_XCH + 8 * XCH;
    static constexpr int O_RING = (O_RED + RED + 1023) / 1024 * 1024;
    static constexpr int S = (227 * 1024 - 1024 - O_RING) / STAGE / 2 * 2;  // (even: see the loaders)
    static constexpr size_t SMEM = 1024 + O_RING + (size_t)S * STAGE;
    static_assert(STAGE % 1024 == 0 && TCOLS <= 512 && (3 * S + 2 * SLOTS + 4) * 8 + 16 + 80 + 64 <= 1024 && S >= 6, "");
};

struct GroupedItem {
    int g, m, row0, n, npad;  // group, M tile, first row (GP_GRAD: first output row), rows, rows rounded up
    int r0, cnt, steps;       // GP_GRAD: the group's first row and rows; stages of the reduction
};

// Two results to the two halves of a word and back.
template <int OT>
__device__ __forceinline__ uint32_t grouped_pack(float lo, float hi) {
    if (OT == MOE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *(const uint32_t *)&v;
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&v;
}
template <int OT>
__device__ __forceinline__ float2 grouped_unpack(uint32_t w) {
    if (OT == MOE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*(const __half2 *)&w);
}
// Four results to consecutive elements of a row.
template <int OT>
__device__ __forceinline__ void grouped_store4(uint8_t *row, int i, float4 a) {
    if (OT == MOE_F32) *(float4 *)(row + 4 * (size_t)i) = a;
    else *(uint2 *)(row + 2 * (size_t)i) = make_uint2(grouped_pack<OT>(a.x, a.y), grouped_pack<OT>(a.z, a.w));
}

// Shared memory to shared memory of the cluster, counted by a barrier there (shared::cluster addresses).
__device__ __forceinline__ void bulk_s2cluster(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(smem_u32(src)), "r"(bytes), "r"(bar)
                 : "memory");
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

// OT: y's type
template <int CG, int NT, int MODE, int OT>
__global__ void __launch_bounds__(GP_THREADS, 1) grouped_kernel(const __grid_constant__ GroupedParams p) {
    using G_ = GroupedGeom<CG, NT, OT>;
    constexpr int S = G_::S;
    constexpr bool LORA = MODE == GP_LORA || MODE == GP_LORA_F16, BY_POWERS = MODE == GP_LORA_F16;  // u by powers of two
    constexpr bool GRAD = MODE == GP_GRAD, A_MN = GRAD || MODE == GP_KN, B_MN = GRAD;
    constexpr int MROWS = MODE == GP_SWIGLU ? 64 : 128;  // output columns of a CTA's tile
    constexpr int ACC_STAGES = OT != MOE_F32 ? 128 : NT <= 64 || MODE == GP_SWIGLU ? 4 : 8;
    static_assert(!GRAD || NT / CG <= 128, "sixteen pieces of eight columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint64_t *full = (uint64_t *)smem;
    uint64_t *empty = full + S;
    uint64_t *landed = empty + S;
    uint64_t *acc_full = landed + S;
    uint64_t *acc_empty = acc_full + G_::SLOTS;
    uint64_t *mma_done = acc_empty + G_::SLOTS;
    uint64_t *red_full = mma_done + 1;
    uint64_t *flagged = red_full + 1;  // GP_LORA_F16, 16-bit results: an item's has_adapters is there
    uint32_t *tmem_slot = (uint32_t *)(flagged + 2);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    volatile int *bad_item = (volatile int *)(tmem_slot + 2);  // GP_LORA: 1 + the last item with a b that is not finite
    int *sums = (int *)(tmem_slot + 4);                       // [20]
    int *has_adapters = sums + 20;                            // GP_LORA: [2][8] for each epilogue warp's columns of an item: some have an adapter (16-bit results: by a power of two)
    int *off = (int *)(smem + G_::O_OFF);                     // [G] where a group's rows begin, -1: it has none
    int *first = (int *)(smem + G_::O_FIRST);                 // [G + 1] items before those of the i-th group ..
    uint16_t *order = (uint16_t *)(smem + G_::O_ORDER);       // [G] .. and which group that is (pairs)
    uint8_t **e_y = (uint8_t **)(smem + G_::O_ROWS);          // [2][NT] the output rows of an accumulator's columns (NULL: none)
    float *e_s = (float *)(e_y + 2 * NT);                     // [2][NT] and their scale
    int4 *items = (int4 *)(smem + G_::O_ITEMS);
    uint8_t *ring = smem + G_::O_RING;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = CG == 1 ? 0 : (int)cluster_ctarank();
    // CG = 1: the CTAs of a cluster share their item's reduction
    const int ks = CG == 1 ? (int)cluster_nctarank() : 1, kr = CG == 1 ? (int)cluster_ctarank() : 0;
    const bool loaders = GRAD || LORA || p.x_index;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1 + (loaders ? CG : 0));
            mbar_init(&landed[s], 128 + (LORA));
            mbar_init(&empty[s], 1);
        }
        for (unsigned b = 0; b < G_::SLOTS; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8 * CG);
        }
        mbar_init(mma_done, 1);
        mbar_init(red_full, 1);
        mbar_init(flagged, 8);
        *abort_flag = 0;
        *bad_item = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc_group<CG>(tmem_slot, G_::TCOLS);
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || ks > 1) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Accumulators are taken one after another, round tensor memory's slots: an item's (as many as its n stages have use for,
    // then `apart` for GP_LORA's extra stages; none: those go to the last one), the next item's behind them.
    // apart: fp32 results, one for the first 128 ranks of every adapter and one for the others (a token has zeros in the stages
    // of all adapters but one, which lose nothing); fp16, items with a token whose u comes by a power of two, one
    const int all_apart = LORA && OT == MOE_F32 ? (p.rank > 128 ? 2 : 1) : 0;
    auto flags = [&](int buf) -> bool {
        const int4 *h = (const int4 *)(has_adapters + buf * 8);
        const int4 a = h[0], b = h[1];
        return (a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) != 0;
    };
    auto acc_count = [&](int n) -> int { return max(1, (n + ACC_STAGES - 1) / ACC_STAGES); };
    // (GP_LORA: the kernel in front computes u and nothing else; it starts this one when everything before it is
    // complete, and only u is waited for, by the warp that loads it)
    if (!LORA) pdl_wait();
    pdl_trigger();

    // ---------------- items: tiles of the M side, inner, by tiles of each group's rows
    const int mt = (p.M + MROWS * CG - 1) / (MROWS * CG);
    const int gran = GRAD ? 64 * CG : G_::GRAN;
    const int gt = GRAD ? (p.N + NT - 1) / NT : 0;  // GP_GRAD: tiles of N
    // this CTA's items: unit, unit + units, ..
    const int units = (int)gridDim.x / (CG * ks), unit = (int)blockIdx.x / (CG * ks);
    // item `r` of group g: group and M tile, first row, rows, the group's rows
    auto make_item = [&](int g, int r, int begin, int cnt) -> int4 {
        const int t = r / mt;
        // near-equal tiles: none is empty, as size <= NT
        const int all = GRAD ? p.N : cnt, nt = (all + NT - 1) / NT;
        const int size = nt == 1 ? NT : ((all + nt - 1) / nt + gran - 1) / gran * gran;
        return make_int4(g | (r - t * mt) << 10, (GRAD ? 0 : begin) + t * size, min(size, all - t * size), cnt);
    };
    static_assert(MOE_MAX_GROUPS <= 1024 && MOE_MAX_GROUPS < GP_THREADS, "ten bits of a group, a thread each");
    {
        // A thread per group: its items behind those of the groups before it, and of them this CTA's to the table.  Pairs:
        // the groups with the most rows first, so that the last round's items are narrow ones (32768 routes over 128
        // experts of uneven popularity, gate/up 198 -> 192 us).  Not GP_GRAD, whose long and short items, bound by the MMAs
        // and by the stores, had better be mixed.
        int g = tid, begin = tid < p.G && p.offsets ? p.offsets[tid] : 0;
        const int next = tid >= p.G ? 0 : p.offsets ? p.offsets[tid + 1] : p.R;
        const bool bad = begin < 0 || next < begin || next > p.R;  // no range of rows
        int cnt = bad ? 0 : next - begin;
        if (bad) moe_set_status(p.status, MOE_ERR_INVALID);
        if (__syncthreads_or(bad)) {
            // Offsets that descend somewhere: ranges may overlap.  A group's rows begin behind all that earlier groups have,
            // so that there are R rows at most, and no more items than the host counted on.
            int taken = cnt ? next : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, taken, d);
                if (lane >= d) taken = max(taken, v);
            }
            if (lane == 31) sums[warp] = taken;
            const int mine = __shfl_up_sync(0xffffffffu, taken, 1);
            __syncthreads();
            const int in_front = (int)__reduce_max_sync(0xffffffffu, (unsigned)(lane < warp ? sums[lane] : 0));
            if (cnt) begin = min(max(begin, max(in_front, lane ? mine : 0)), next);
            cnt = cnt ? next - begin : 0;
            __syncthreads();
        }
        if (tid < p.G) off[tid] = cnt ? begin : -1;
        if (CG == 2 && !GRAD && p.G > 1) {
            int *rows = first;
            if (tid < (p.G + 3) / 4 * 4) rows[tid] = cnt;
            __syncthreads();
            if (tid < p.G) {
                int before = 0;
#pragma unroll 4
                for (int i = 0; i < p.G; i += 4) {  // (past the last group: no rows, and behind this one)
                    const int4 v = *(const int4 *)&rows[i];
                    before += (v.x > cnt || (v.x == cnt && i < tid)) + (v.y > cnt || (v.y == cnt && i + 1 < tid)) +
                              (v.z > cnt || (v.z == cnt && i + 2 < tid)) + (v.w > cnt || (v.w == cnt && i + 3 < tid));
                }
                order[before] = (uint16_t)tid;
            }
            __syncthreads();
            if (tid < p.G) {
                g = order[tid];
                cnt = rows[g];
                begin = off[g];
            }
            __syncthreads();
        }
        const int mine = tid < p.G ? mt * (GRAD ? gt : (cnt + NT - 1) / NT) : 0;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        const int begins = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) + inc - mine;
        if (tid <= p.G) first[tid] = begins;
        if (mine) {
            int i = begins <= unit ? 0 : (begins - unit + units - 1) / units;
            for (int at = unit + i * units; at < begins + mine && i < GP_ITEMS; ++i, at += units)
                items[i] = make_item(g, at - begins, begin, cnt);
        }
    }
    __syncthreads();
    const int n_items = first[p.G], n_mine = unit < n_items ? (n_items - unit - 1) / units + 1 : 0;
    auto look_up_item = [&](int i) -> int4 {  // (past the table)
        const int at = unit + i * units;
        int lo = 0, hi = p.G;  // the last one whose first item is not after this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= at) lo = mid;
            else hi = mid;
        }
        const int g = CG == 2 && !GRAD && p.G > 1 ? order[lo] : lo;
        const int begin = off[g];
        return make_item(g, at - first[lo], begin, begin < 0 ? 0 : (p.offsets ? p.offsets[g + 1] : p.R) - begin);
    };
    auto item_at = [&](int i) -> GroupedItem {
        const int4 v = i < GP_ITEMS ? items[i] : look_up_item(i);
        GroupedItem it;
        it.g = v.x & 1023;
        it.m = v.x >> 10;
        it.row0 = v.y;
        it.n = v.z;
        it.npad = (v.z + gran - 1) / gran * gran;
        it.r0 = GRAD ? off[it.g] : 0;
        it.cnt = v.w;
        it.steps = ((GRAD ? v.w : p.K) + 63) / 64;
        return it;
    };
    // GP_LORA: this lane's share of the tile's adapters (-1: none).  Read before an item's stages, looked at behind them.
    auto read_adapters = [&](const GroupedItem &it, int (&ids)[8]) {
        if (LORA)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = lane + 32 * i;
                ids[i] = c < it.n ? p.adapter[it.row0 + c] : -1;
            }
    };
    auto check_adapters = [&](int (&ids)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (ids[i] >= p.n_adapters || ids[i] < -1) moe_set_status(p.status, MOE_ERR_INVALID);
            if (ids[i] >= p.n_adapters) ids[i] = -1;
        }
    };
    const int chunks = LORA ? (p.rank + 31) / 32 * p.parts : 1;  // pieces of u: p.parts for 32 ranks of B
    const int shift = LORA && p.parts == 2;
    auto token_factor = [&](int t) -> float {  // fp16: of the token's 32 ranks the largest factor, a power of two
        float f = p.factor[(size_t)t * chunks];
        for (int c = 1; c < p.factors; ++c) f = fmaxf(f, p.factor[(size_t)t * chunks + c]);
        return f;
    };
    auto extra_stages = [&](const int (&ids)[8]) -> int {
        int n = 0;
        for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF; a = grouped_next_adapter(ids, a)) n += chunks;
        return n;
    };
    // of n stages (those of the matrix, then GP_LORA's extra ones) this CTA's [lo, hi)
    auto share = [&](int n, int &lo, int &hi) {
        lo = CG == 1 ? n * kr / ks : 0;
        hi = CG == 1 ? n * (kr + 1) / ks : n;
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
        for (int j = 0; j < n_mine && ok; ++j) {
            const GroupedItem it = item_at(j);
            const int nb = it.npad / CG, m0 = (it.m * CG + rank) * MROWS;
            int lo, hi, ids[8];
            read_adapters(it, ids);
            share(it.steps, lo, hi);
            for (int kb = lo; kb < hi; ++kb, ++gs) {
                if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                uint8_t *dst = ring + (size_t)st * G_::STAGE;
                const uint32_t bar = CG == 1 ? smem_u32(&full[st]) : cluster_map(&full[st], 0);
                const bool whole = !GRAD || 64 * kb + 64 <= it.cnt;  // (else by the loaders)
                const bool box_a = GRAD ? whole && !p.x_index : true, box_b = GRAD ? whole && !p.y_index : !p.x_index;
                if (rank == 0)
                    mbar_arrive_expect_tx_elect(&full[st], CG * ((box_a ? GP_ABYTES : 0u) + (box_b ? nb * 128u : 0u)));
                if (LORA && lane == 0) mbar_arrive1(&landed[st]);
                if (MODE == GP_NK || LORA) {
                    if (lane == 0) tma_tile_3d<CG>(dst, &p.a, kb * 64, m0, LORA ? 0 : it.g, bar);
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
            if (LORA && ok) {
                int e = 0;
                check_adapters(ids);
                share(extra_stages(ids), lo, hi);
                for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF && ok; a = grouped_next_adapter(ids, a))
                    for (int c = 0; c < chunks; ++c, ++e) {
                        if (e < lo || e >= hi) continue;
                        if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                        // (the adapter's B goes through the hands of warp 3, as u does: the leader's barrier counts no bytes)
                        if (rank == 0 && lane == 0) mbar_arrive1(&full[st]);
                        mbar_arrive_expect_tx_elect(&landed[st], GP_UBYTES);
                        if (lane == 0)
                            tma_tile_3d<CG>(ring + (size_t)st * G_::STAGE, &p.ab, (c >> shift) * 32, m0, a, smem_u32(&landed[st]));
                        __syncwarp();
                        ++gs;
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
        for (int j = 0; j < n_mine && ok; ++j) {
            const GroupedItem it = item_at(j);
            const int nb = it.npad / CG, c0 = it.row0 + rank * nb;
            int lo, hi, elo, ehi, ids[8];
            read_adapters(it, ids);
            share(it.steps, lo, hi);
            for (int kb = lo; kb < hi; ++kb, ++gs) {
                if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                uint8_t *dst = ring + (size_t)st * G_::STAGE + GP_ABYTES;
                const uint32_t bar = CG == 1 ? smem_u32(&full[st]) : cluster_map(&full[st], 0);
                if (GRAD) {
                    if (64 * lane < nb && 64 * kb + 64 <= it.cnt)
                        tma_tile_2d<CG>(dst + lane * 8192, &p.b, c0 + 64 * lane, it.r0 + 64 * kb, bar);
                } else {
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
            if (LORA) {  // (the loaders' stages)
                check_adapters(ids);
                share(extra_stages(ids), elo, ehi);
                for (int e = elo; e < ehi; ++e, ++gs) {
                    if (gs >= S && !(ok = mbar_wait_warp(&empty[st], ph, p.status, abort_flag))) break;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
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
        if (GRAD && n_mine) {
            after = item_at(0);
            look_up(after, team);
        }
        for (int j = 0; j < n_mine && ok; ++j) {
            if (GRAD) {
                it = after;
                if (j + 1 < n_mine) after = item_at(j + 1);
            } else {
                it = item_at(j);
            }
            const int nb = it.npad / CG;
            int lo, hi, ids[8];
            read_adapters(it, ids);
            share(it.steps, lo, hi);
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
                    const int r = c >= rows || LORA ? -1 : source(it.row0 + rank * nb + c);
                    who[i] = LORA ? (c < rows ? p.adapter[it.row0 + rank * nb + c] : -1) : r >= 0 ? 16 : 0;
                    src[i] = p.rows + (size_t)max(r, 0) * p.ld + 8 * piece + 64 * (lo + (team != (gs & 1)));
                }
                for (int kb = lo; kb < hi; ++kb, next()) {
                    if ((gs & 1) != team) continue;
                    if (!begin()) break;
                    if (!LORA) {
                        const uint32_t d = at + (uint32_t)st * G_::STAGE;
                        const int most = kb * 64 + 8 * piece < p.K ? 16 : 0;
#pragma unroll
                        for (int i = 0; i < RI; ++i) {
                            if (16 * i < rows) cp_async_16_or_0(d + i * 2048, src[i], min(most, who[i]));
                            src[i] += kb + 3 > hi ? 0 : 128;
                        }
                    }
                    cp_async_mbar_arrive_noinc(&landed[st]);
                }
                if (LORA && ok) {
                    if (j == 0) pdl_wait();  // u
                    int e = 0;
                    check_adapters(ids);
                    share(extra_stages(ids), lo, hi);
                    const uint16_t *u = p.rows + (size_t)(it.row0 + rank * nb + r0) * p.ld + 8 * piece;
                    for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF && ok; a = grouped_next_adapter(ids, a))
                        for (int c = 0; c < chunks; ++c, ++e) {
                            if (e < lo || e >= hi) continue;
                            if ((gs & 1) != team) {
                                next();
                                continue;
                            }
                            if (!begin()) break;
                            const uint32_t d = at + (uint32_t)st * G_::STAGE;
                            if (BY_POWERS && p.factors > 1) {  // one power of two for the token's whole row: the smaller ones' pieces brought to it
#pragma unroll
                                for (int i = 0; i < RI; ++i)
                                    if (16 * i < nb) {
                                        uint4 v = make_uint4(0, 0, 0, 0);
                                        if (who[i] == a) {
                                            const int t = it.row0 + rank * nb + r0 + 16 * i;
                                            const float f = p.factor[(size_t)t * chunks + c] / token_factor(t);
                                            v = *(const uint4 *)(u + (size_t)16 * i * p.ld + c * 64);
                                            uint32_t *w = (uint32_t *)&v;
                                            if (f != 1.f)
#pragma unroll
                                                for (int k = 0; k < 4; ++k) {
                                                    const float2 q = grouped_unpack<MOE_F16>(w[k]);
                                                    w[k] = grouped_pack<MOE_F16>(f * q.x, f * q.y);
                                                }
                                        }
                                        st_shared_16(d + i * 2048, v);
                                    }
                                mbar_arrive1(&landed[st]);
                                next();
                                continue;
                            }
#pragma unroll
                            for (int i = 0; i < RI; ++i)
                                if (16 * i < nb) {
                                    const bool some = who[i] == a;
                                    cp_async_16_or_0(d + i * 2048, some ? u + (size_t)16 * i * p.ld + c * 64 : p.rows,
                                                     some ? 16 : 0);
                                }
                            cp_async_mbar_arrive_noinc(&landed[st]);
                            next();
                        }
                }
            } else {
                // sixteen threads a row (128 columns): piece lt % 16 of rows lt / 16 + 8 i
                const int end = gs + it.steps;  // the next item's first stage
                const bool more = j + 1 < n_mine, any = it.steps > ((gs & 1) != team);
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
        if (LORA) pdl_wait();
    } else if (warp == 3 && loaders) {
        // ---------------- the loaders' stages: their copies have landed; the tensor cores may read them
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int j = 0; j < n_mine && ok; ++j) {
            const GroupedItem it = item_at(j);
            int lo, hi, ids[8];
            read_adapters(it, ids);
            share(it.steps, lo, hi);
            bool extra = !LORA;
            for (int kb = lo;; ++kb) {
                if (kb >= hi) {
                    if (extra) break;
                    extra = true;
                    check_adapters(ids);
                    share(extra_stages(ids), lo, hi);
                    kb = lo;
                    if (kb >= hi) break;
                }
                if (!(ok = mbar_wait_warp(&landed[st], ph, p.status, abort_flag))) break;
                if (LORA && extra) {
                    // The tile's other tokens have zeros for u here, which an infinity or a NaN in b would turn to NaN: rows of
                    // 32 ranks with one of them become zeros, and the epilogue adds them to this adapter's tokens
                    const uint32_t most = p.fmt ? 0x7F807F80u : 0x7C007C00u, at = smem_u32(ring) + (uint32_t)st * G_::STAGE;
                    uint32_t top = 0;  // the largest exponents
#pragma unroll
                    for (int i = 0; i < GP_UBYTES / 512; ++i) {
                        const uint4 v = ld_shared_16(at + i * 512 + lane * 16);
                        top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & most, v.y & most)), __vmaxu2(v.z & most, v.w & most));
                    }
                    const bool any = __any_sync(0xffffffffu, __vcmpeq2(top, most) != 0);
                    if (any)
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t row = at + (lane + 32 * i) * 64;
                            uint32_t bad = 0;
                            for (int k = 0; k < 4; ++k) {
                                const uint4 v = ld_shared_16(row + 16 * k);
                                bad |= __vcmpeq2(v.x & most, most) | __vcmpeq2(v.y & most, most) | __vcmpeq2(v.z & most, most) |
                                       __vcmpeq2(v.w & most, most);
                            }
                            if (bad)
                                for (int k = 0; k < 4; ++k) st_shared_16(row + 16 * k, make_uint4(0, 0, 0, 0));
                        }
                    if (any && lane == 0) *bad_item = j + 1;
                    __syncwarp();
                }
                fence_proxy_async_smem();
                __syncwarp();
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
        int st = 0;
        unsigned seq = 0;  // accumulators taken so far
        uint32_t ph = 0;
        bool ok = true;
        for (int j = 0; j < n_mine && ok; ++j) {
            const GroupedItem it = item_at(j);
            // (a value that a shuffle hands out is known to be the same in every lane: it stays in a uniform register, where
            // the MMA wants its operands)
            const uint32_t idesc = umma_idesc_16(p.fmt, A_MN, B_MN, 128 * CG, __shfl_sync(0xffffffffu, it.npad, 0));
            int lo, hi, ids[8];
            read_adapters(it, ids);
            share(__shfl_sync(0xffffffffu, it.steps, 0), lo, hi);
            bool fresh = true;  // nothing summed yet
            uint32_t d = 0;
            auto take = [&]() -> bool {  // the next accumulator
                const unsigned slot = seq % G_::SLOTS, round = seq / G_::SLOTS;
                if (round >= 1 && !(ok = mbar_wait_warp(&acc_empty[slot], (round - 1) & 1, p.status, abort_flag))) return false;
                tc_fence_after();
                d = __shfl_sync(0xffffffffu, tmem, 0) + slot * NT;
                ++seq;
                fresh = true;
                return true;
            };
            if (!take()) break;
            const int len = GRAD ? __shfl_sync(0xffffffffu, it.cnt, 0) : p.K;
            for (int kb = lo; ok;) {  // (an accumulator's stages by themselves: its address stays in a uniform register)
                const uint32_t acc = d;
                for (const int end = min(hi, kb + ACC_STAGES); kb < end; ++kb) {
                    if (!(ok = mbar_wait_warp(&full[st], ph, p.status, abort_flag))) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring) + (uint32_t)st * G_::STAGE;
                    const uint64_t a = A_MN ? umma_desc_mn_sw128(sa, 8192) : umma_desc_sw128(sa);
                    const uint64_t b = B_MN ? umma_desc_mn_sw128(sa + GP_ABYTES, 8192) : umma_desc_sw128(sa + GP_ABYTES);
                    const int left = len - 64 * kb;
                    auto step = [&](int q) {
                        umma_f16_elect<CG>(acc, a + (uint64_t)(q * (A_MN ? 128 : 2)), b + (uint64_t)(q * (B_MN ? 128 : 2)), idesc,
                                           q > 0 || !fresh);
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
                    fresh = false;
                    umma_commit_group_elect<CG>(&empty[st]);
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok || kb >= hi) break;
                umma_commit_group_elect<CG>(&acc_full[(seq - 1) % G_::SLOTS]);
                if (!take()) break;
            }
            uint32_t dx[2] = {d, d};
            bool fresh_x[2] = {fresh, fresh};
            int apart = all_apart;
            if (LORA) {
                check_adapters(ids);
                if (OT != MOE_F32 && BY_POWERS && ok && (ok = mbar_wait_warp(flagged, j & 1, p.status, abort_flag))) apart = flags(j & 1);
                share(__shfl_sync(0xffffffffu, extra_stages(ids), 0), lo, hi);
                if (apart && ok) umma_commit_group_elect<CG>(&acc_full[(seq - 1) % G_::SLOTS]);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (x < apart && ok && take()) {
                        dx[x] = d;
                        fresh_x[x] = true;
                    }
            }
            for (int e = lo, c = LORA ? lo % chunks : 0; LORA && e < hi && ok; ++e) {
                if (!(ok = mbar_wait_warp(&full[st], ph, p.status, abort_flag))) break;
                const bool other = OT == MOE_F32 && apart == 2 && c >= 4 * p.parts;  // (pieces of 32 ranks)
                const uint32_t d = other ? dx[1] : dx[0];
                const bool fresh = other ? fresh_x[1] : fresh_x[0];
                tc_fence_after();
                // 32 ranks: u's upper halves in the first 64 bytes of a row, the rest of u in the second, both by the same B_a
                const uint32_t sa = smem_u32(ring) + (uint32_t)st * G_::STAGE;
                const uint64_t a = umma_desc_sw64(sa), b = umma_desc_sw128(sa + GP_ABYTES);
                umma_f16_elect<CG>(d, a, b, idesc, !fresh);
                umma_f16_elect<CG>(d, a, b + 4, idesc, 1);
                if (p.rank - 32 * (c >> shift) > 16) {
                    umma_f16_elect<CG>(d, a + 2, b + 2, idesc, 1);
                    umma_f16_elect<CG>(d, a + 2, b + 6, idesc, 1);
                }
                fresh_x[0] &= other;
                fresh_x[1] &= !other;
                if (++c == chunks) c = 0;
                umma_commit_group_elect<CG>(&empty[st]);
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (ok)
                for (unsigned a = seq - max(apart, 1); a < seq; ++a) umma_commit_group_elect<CG>(&acc_full[a % G_::SLOTS]);
        }
        umma_commit_group_elect<CG>(mma_done);  // every MMA has completed before tensor memory is released
        mbar_wait_bounded(mma_done, 0, p.status);
    } else if (warp >= 4 && warp < 12) {
        // ---------------- epilogue: an accumulator column is an output row.  16-bit results: fragments of 16 lanes x 8 columns,
        // each pair of columns packed, transposed by way of shared memory (stmatrix), so that a lane stores eight
        // consecutive elements of an output row; fp32 results transposed a word at a time, four consecutive elements a store.
        // (Stored straight from the registers, 128 bytes of one output row an instruction: 4864 x 4096 x 512 31.4 us,
        // this way 24.8.)
        constexpr bool F32 = OT == MOE_F32;
        constexpr int CH = G_::CH, NB = CH / 8, SIZE = F32 ? 4 : 2;
        const int q = warp & 3, ew = warp - 4, half = ew >> 2, et = ew * 32 + lane;
        const uint32_t xb = smem_u32(smem + G_::O_XCH) + ew * G_::XCH;
        // stmatrix: the address of row lane % 8 of 8 x 8 matrix lane / 8.  Matrices 0, 1: output rows 0-7, elements 0-7 and 8-15;
        // 2, 3: output rows 8-15
        constexpr int PITCH = MODE == GP_SWIGLU ? 48 : 80;  // (no bank conflicts)
        const uint32_t xm = xb + ((lane & 7) + 8 * (lane >> 4)) * PITCH + ((lane >> 3) & 1) * 16;
        // this thread's row of an item, read an item ahead: its indexes, then (once they are there) its output row and scale
        int ix = 0, iy = 0;
        uint8_t *row = nullptr;
        float scale = 1.f;
        int ia = -1;  // GP_LORA: its adapter
        auto fetch = [&](const GroupedItem &it) {
            if (LORA) ia = et < it.n ? p.adapter[it.row0 + et] : -1;
            if (GRAD || et >= it.n) return;
            ix = p.x_index ? p.x_index[it.row0 + et] : it.row0 + et;
            iy = p.y_index ? p.y_index[it.row0 + et] : it.row0 + et;
        };
        auto resolve = [&](const GroupedItem &it) {
            row = nullptr;
            scale = 1.f;
            if (et >= it.n) return;
            if (GRAD) {
                row = (uint8_t *)p.y + ((size_t)it.g * p.N + it.row0 + et) * p.M * SIZE;
            } else if (ix >= 0 && ix / (p.x_index ? p.x_share : 1) < p.x_rows && iy >= 0 && iy < p.y_rows) {
                row = (uint8_t *)p.y + (size_t)iy * p.ldy * SIZE;
                if (LORA) {  // (the adapter's part alone is multiplied)
                    if (BY_POWERS && ia >= 0 && ia < p.n_adapters) scale = token_factor(iy);
                } else if (p.scale) {
                    scale = p.scale[iy];
                }
            } else {
                moe_set_status(p.status, MOE_ERR_INVALID);
            }
        };
        auto add16 = [&](uint32_t (&v)[16], uint32_t at) {  // another accumulator
            uint32_t u[16];
            tmem_ld16(at, u);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(u[k]));
        };
        auto add16_by = [&](uint32_t (&v)[16], uint32_t at, const float *by) {  // one that is apart, its columns multiplied
            uint32_t u[16];
            tmem_ld16(at, u);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(fmaf(by[k], __uint_as_float(u[k]), __uint_as_float(v[k])));
        };
        // GP_LORA: 32 ranks (those of piece c of u, with their first piece) of adapter a for output o of token t, where b is not
        // finite among them, else 0.  By the whole u: an infinity times its parts may be infinities of both signs, or of a part
        // that is 0, NaN.
        auto not_finite = [&](int a, int c, int o, int t) -> float {
            if (shift && (c & 1)) return 0.f;
            const uint16_t *b = p.lora_b + ((size_t)a * p.M + o) * p.rank, *u = p.rows + (size_t)t * p.ld + c * 64;
            auto value = [&](uint16_t h) -> float {
                return p.fmt ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
            };
            float s = 0.f;
            bool bad = false;
            const int c0 = 32 * (c >> shift);
            for (int k = 0; k < 32 && c0 + k < p.rank; ++k) {
                const float v = value(b[c0 + k]);
                bad |= !(fabsf(v) <= 3.4028235e38f);
                s = fmaf(v, value(u[k]) + value(u[32 + k]) + (shift ? value(u[64 + k]) : 0.f), s);
            }
            return bad ? (!BY_POWERS ? s : s * p.factor[(size_t)t * chunks + c]) : 0.f;
        };
        unsigned seq = 0;  // accumulators handed back so far
        auto hand_back = [&](unsigned a) {
            if (lane == 0) {
                if (CG == 1) mbar_arrive1(&acc_empty[a % G_::SLOTS]);
                else mbar_arrive_cluster(cluster_map(&acc_empty[a % G_::SLOTS], 0));
            }
        };
        GroupedItem it = {};
        if (n_mine) {
            it = item_at(0);
            fetch(it);
            if (BY_POWERS) pdl_wait();  // the factors
            resolve(it);
        }
        for (int j = 0; j < n_mine; ++j) {
            const int buf = j & 1;
            if (et < NT) {
                e_y[buf * NT + et] = row;
                e_s[buf * NT + et] = scale;
            }
            int apart = all_apart;
            bool w = true;
            if (LORA && (F32 || BY_POWERS)) {
                const bool any = __any_sync(0xffffffffu, ia >= 0 && ia < p.n_adapters && (F32 || scale != 1.f));
                if (lane == 0) has_adapters[buf * 8 + ew] = any;
                if (!F32) {
                    if (lane == 0) mbar_arrive1(flagged);
                    w = mbar_wait_warp(flagged, buf, p.status, abort_flag);
                    apart = flags(buf);
                }
            }
            GroupedItem nx = {};
            if (j + 1 < n_mine) {
                nx = item_at(j + 1);
                fetch(nx);
            }
            unsigned used;  // accumulators
            {
                int lo, hi;
                share(it.steps, lo, hi);
                used = acc_count(hi - lo);
            }
            const uint32_t quarter = tmem + ((uint32_t)(32 * q) << 16);
            // as many as the last pass adds up: those that tensor memory holds, one for 16-bit results
            const unsigned held = F32 ? G_::SLOTS - apart : 1;
            for (; used > held && w; --used, ++seq) {  // the first added to the second (the columns that are this warp's below, too)
                for (unsigned a = seq; a < seq + 2 && w; ++a)
                    w = mbar_wait_warp(&acc_full[a % G_::SLOTS], (a / G_::SLOTS) & 1, p.status, abort_flag);
                if (!w) break;
                tc_fence_after();
                const uint32_t from = quarter + seq % G_::SLOTS * NT, to = quarter + (seq + 1) % G_::SLOTS * NT;
                for (int c0 = CH * half; c0 < it.n; c0 += 2 * CH)
#pragma unroll
                    for (int h = 0; h < CH; h += 16) {
                        uint32_t v[16];
                        tmem_ld16(from + c0 + h, v);
                        add16(v, to + c0 + h);
                        tmem_st16(to + c0 + h, v);
                    }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                hand_back(seq);
            }
            for (unsigned a = seq; a < seq + used + apart && w; ++a)
                w = mbar_wait_role(&acc_full[a % G_::SLOTS], (a / G_::SLOTS) & 1, p.status, abort_flag);
            if (!bar_and_n(1, 256, w)) break;
            if (j + 1 < n_mine) resolve(nx);
            tc_fence_after();
            const uint32_t tb = quarter + seq % G_::SLOTS * NT;
            auto other = [&](unsigned a) -> uint32_t { return quarter + (seq + a) % G_::SLOTS * NT; };  // the item's a-th accumulator
            // GP_LORA: of this CTA's extra stages the range; of the accumulators that are apart, those that some of them went to (1 the
            // first, 2 the second)
            int elo = 0, ehi = 0, added = 0;
            if (LORA && ks > 1) {
                int ids[8];
                read_adapters(it, ids);
                check_adapters(ids);
                share(extra_stages(ids), elo, ehi);
                for (int e = elo; e < min(ehi, elo + chunks); ++e) added |= apart == 2 && e % chunks >= 4 * p.parts ? 2 : 1;
            } else if (LORA && apart && (!F32 || flags(buf))) {
                added = 3;
            }
            uint8_t *const *ys = e_y + buf * NT;
            const float *ss = e_s + buf * NT;
            const bool none = GRAD && !it.steps, keep = none && p.accumulate;  // (keep: an empty group's matrix is left as it was)
            const int m0 = (it.m * CG + rank) * MROWS + MROWS / 4 * q;  // the warp's first element
            if (CG == 1 && ks > 1) {
                // the cluster's only item: each CTA adds up its share of the rows, `per` of them (the last ones fewer)
                const int per = (it.n + ks - 1) / ks, own = max(0, min(per, it.n - kr * per));
                int lo, hi;
                share(it.steps, lo, hi);
                const bool some = hi > lo || (!apart && ehi > elo);  // (else nothing was summed)
                float *x = (float *)(smem + G_::O_XCH);  // [NT][128]
                static_assert(CG == 2 || NT * 512 <= 8 * G_::XCH, "sums of an item");
                if (16 * half < it.n) {
                    uint32_t v[16];
                    tmem_ld16(tb + 16 * half, v);
                    tmem_ld_wait();
                    for (unsigned a = 1; a < used; ++a) add16(v, other(a) + 16 * half);
                    if (!some)
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = 0u;
                    for (int a = 0; a < apart; ++a)
                        if (added >> a & 1) add16_by(v, other(used + a) + 16 * half, ss + 16 * half);
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[(16 * half + k) * 128 + 32 * q + lane] = __uint_as_float(v[k]);
                }
                if (LORA && *bad_item > j) {
                    int e = 0, ids[8];
                    read_adapters(it, ids);
                    check_adapters(ids);
                    for (int a = grouped_next_adapter(ids, -1); a != 0x7FFFFFFF; a = grouped_next_adapter(ids, a))
                        for (int c = 0; c < chunks; ++c, ++e)
                            if (e >= elo && e < ehi && m0 + lane < p.M)
                                for (int k = 16 * half; k < min(it.n, 16 * half + 16); ++k)
                                    if (p.adapter[it.row0 + k] == a)
                                        x[k * 128 + 32 * q + lane] += not_finite(a, c, m0 + lane, it.row0 + k);
                }
                fence_proxy_async_smem();
                if (et == 0 && own) mbar_arrive_expect_tx(red_full, (uint32_t)(own * ks) * 512u);
                bar_sync_n(2, 256);
                // to each CTA its rows, in one copy
                const int rows = max(0, min(per, it.n - et * per));
                if (et < ks && rows)
                    bulk_s2cluster(cluster_map(smem + G_::O_RED + kr * per * 512, et), x + et * per * 128, rows * 512u,
                                   cluster_map(red_full, et));
                if (own) {
                    const bool there = mbar_wait_role(red_full, 0, p.status, abort_flag);
                    if (!bar_and_n(3, 256, there)) break;
                    const float *sum = (const float *)(smem + G_::O_RED);
                    auto total = [&](int r, int m) -> float4 {  // in the order of the CTAs
                        float4 a = *(const float4 *)(sum + r * 128 + m);
                        for (int k = 1; k < ks; ++k) {
                            const float4 b = *(const float4 *)(sum + (k * per + r) * 128 + m);
                            a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
                        }
                        return a;
                    };
                    constexpr int QUADS = MROWS / 4;
                    for (int i = et; i < own * QUADS; i += 256) {
                        const int r = i / QUADS, c = kr * per + r, m = 4 * (i % QUADS), mg = it.m * MROWS + m;
                        float4 a;
                        if (MODE == GP_SWIGLU) {
                            const int at = 2 * (m & ~15) + (m & 15);
                            const float4 g = total(r, at), u = total(r, at + 16);
                            a = make_float4(mx4_swiglu<F32>(g.x, u.x), mx4_swiglu<F32>(g.y, u.y), mx4_swiglu<F32>(g.z, u.z),
                                            mx4_swiglu<F32>(g.w, u.w));
                        } else {
                            a = total(r, m);
                        }
                        const float s = LORA ? 1.f : ss[c];
                        if (mg < p.M && ys[c]) grouped_store4<OT>(ys[c], mg, make_float4(s * a.x, s * a.y, s * a.z, s * a.w));
                    }
                }
            } else {
                for (int c0 = CH * half; c0 < it.n && !keep; c0 += 2 * CH) {
                    if (F32 && MODE != GP_SWIGLU) {
                        uint32_t v[CH / 16][16];
#pragma unroll
                        for (int h = 0; h < CH / 16; ++h) tmem_ld16(tb + c0 + 16 * h, v[h]);
                        tmem_ld_wait();
                        for (unsigned a = 1; a < used; ++a)
#pragma unroll
                            for (int h = 0; h < CH / 16; ++h) add16(v[h], other(a) + c0 + 16 * h);
                        for (int a = 0; a < apart; ++a)
                            if (added >> a & 1)
#pragma unroll
                                for (int h = 0; h < CH / 16; ++h) add16_by(v[h], other(used + a) + c0 + 16 * h, ss + c0 + 16 * h);
                        float *x = (float *)(smem + G_::O_XCH + ew * G_::XCH);
                        if (GRAD) {  // whole boxes by TMA: see below
                            if (lane == 0) tma_store_wait_read();
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 16; ++k) x[32 * k + lane] = none ? 0.f : __uint_as_float(v[0][k]);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0 && m0 < p.M) {
                                if (p.accumulate) tma_add_3d(&p.yt, m0, it.row0 + c0, it.g, xb);
                                else tma_store_3d(&p.yt, m0, it.row0 + c0, it.g, xb);
                            }
                            continue;
                        }
                        // padded to 36: no bank conflicts
                        const int m = m0 + 4 * (lane & 7);
#pragma unroll
                        for (int h = 0; h < CH / 16; ++h) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) x[36 * k + lane] = none ? 0.f : __uint_as_float(v[h][k]);
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int r = 4 * k + (lane >> 3), c = c0 + 16 * h + r;
                                float4 a = *(const float4 *)(x + 36 * r + 4 * (lane & 7));
                                if (c < it.n && m < p.M && ys[c]) {
                                    const float s = LORA ? 1.f : ss[c];
                                    a = make_float4(s * a.x, s * a.y, s * a.z, s * a.w);
                                    grouped_store4<OT>(ys[c], m, a);
                                }
                            }
                            __syncwarp();
                        }
                        continue;
                    }
                    // registers 4 b + {0, 1}: row lane / 4, columns 8 b + 2 (lane % 4) + {0, 1}; + {2, 3}: row lane / 4 + 8
                    uint32_t lo[4 * NB], hi[4 * NB];  // (GP_SWIGLU: gate and up)
                    tmem_ld_16x256b(tb + c0, lo);
                    tmem_ld_16x256b(tb + (16u << 16) + c0, hi);
                    tmem_ld_wait();
                    for (unsigned a = 1; F32 && a < used; ++a) {
                        uint32_t u[4 * NB];
                        tmem_ld_16x256b(other(a) + c0, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4 * NB; ++k) lo[k] = __float_as_uint(__uint_as_float(lo[k]) + __uint_as_float(u[k]));
                        tmem_ld_16x256b(other(a) + (16u << 16) + c0, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4 * NB; ++k) hi[k] = __float_as_uint(__uint_as_float(hi[k]) + __uint_as_float(u[k]));
                    }
                    const int cq = c0 + 2 * (lane & 3);
                    if (LORA && (added & 1))  // (fp16)
#pragma unroll
                        for (int side = 0; side < 2; ++side) {
                            uint32_t u[4 * NB];
                            tmem_ld_16x256b(other(used) + ((uint32_t)(16 * side) << 16) + c0, u);
                            tmem_ld_wait();
                            uint32_t *v = side ? hi : lo;
#pragma unroll
                            for (int k = 0; k < 4 * NB; ++k)
                                v[k] = __float_as_uint(fmaf(ss[cq + 8 * (k >> 2) + (k & 1)], __uint_as_float(u[k]), __uint_as_float(v[k])));
                        }
                    if (none)
#pragma unroll
                        for (int k = 0; k < 4 * NB; ++k) lo[k] = hi[k] = 0u;
                    if (MODE == GP_SWIGLU)
#pragma unroll
                        for (int k = 0; k < 4 * NB; ++k)
                            lo[k] = __float_as_uint(mx4_swiglu<F32>(__uint_as_float(lo[k]), __uint_as_float(hi[k])));
                    if (!GRAD && p.scale)
#pragma unroll
                        for (int k = 0; k < 2 * NB; ++k) {  // (rows past the last one are not stored)
                            const int c = cq + 8 * (k >> 1) + (k & 1), r = 4 * (k >> 1) + (k & 1);
                            const float s = c < it.n ? ss[c] : 0.f;
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                lo[r + h] = __float_as_uint(s * __uint_as_float(lo[r + h]));
                                if (MODE != GP_SWIGLU) hi[r + h] = __float_as_uint(s * __uint_as_float(hi[r + h]));
                            }
                        }
                    if (F32) {  // GP_SWIGLU: 32 bytes of four output rows an instruction
#pragma unroll
                        for (int k = 0; k < 4 * NB; ++k) {
                            const int c = cq + 8 * (k >> 2) + (k & 1), m = m0 + (lane >> 2) + 4 * (k & 2);
                            if (c < it.n && m < p.M && ys[c]) ((float *)ys[c])[m] = __uint_as_float(lo[k]);
                        }
                        continue;
                    }
                    constexpr int PARTS = MODE == GP_SWIGLU ? 2 : 4, LINES = 32 / PARTS;  // 16-byte pieces of an output row
                    const int part = lane % PARTS, m = m0 + 8 * part;
                    if (GRAD && p.accumulate) {
#pragma unroll
                        for (int k = 0; k < CH / LINES; ++k) {
                            const int c = LINES * k + lane / PARTS;
                            if (c0 + c < it.n && m < p.M)
                                st_shared_16(xb + c * PITCH + 16 * part, *(const uint4 *)(ys[c0 + c] + 2 * (size_t)m));
                        }
                        __syncwarp();
#pragma unroll
                        for (int b = 0; b < NB / 2; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t old[4];
                                ldmatrix_x4_trans(xm + 16 * b * PITCH + 32 * h, old[0], old[1], old[2], old[3]);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    uint32_t *v = (h ? hi : lo) + 8 * b + 2 * k;
                                    const float2 o = grouped_unpack<OT>(old[k]);
                                    v[0] = __float_as_uint(__uint_as_float(v[0]) + o.x);
                                    v[1] = __float_as_uint(__uint_as_float(v[1]) + o.y);
                                }
                            }
                        __syncwarp();
                    }
                    auto pack = [&](const uint32_t *v) -> uint32_t {
                        return grouped_pack<OT>(__uint_as_float(v[0]), __uint_as_float(v[1]));
                    };
                    if (GRAD && CH == 32 && !p.accumulate) {
                        // whole boxes: stored by TMA (rows past N, and columns past M, are not); 128 groups of 256 rows, 1536 x
                        // 2048: 215 us by the lanes' own stores, 188 this way
                        if (lane == 0) tma_store_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int b = 0; b < NB / 2; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t *v = (h ? hi : lo) + 8 * b;
                                const int r = (lane & 7) + 8 * (lane >> 4) + 16 * b, piece = ((lane >> 3) & 1) + 2 * h;
                                stmatrix_x4_trans(xb + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4), pack(v), pack(v + 2), pack(v + 4), pack(v + 6));
                            }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && m0 < p.M) tma_store_3d(&p.yt, m0, it.row0 + c0, it.g, xb);
                        continue;
                    }
#pragma unroll
                    for (int b = 0; b < NB / 2; ++b) {
                        const uint32_t *l = lo + 8 * b, *h = hi + 8 * b;
                        stmatrix_x4_trans(xm + 16 * b * PITCH, pack(l), pack(l + 2), pack(l + 4), pack(l + 6));
                        if (MODE != GP_SWIGLU) stmatrix_x4_trans(xm + 16 * b * PITCH + 32, pack(h), pack(h + 2), pack(h + 4), pack(h + 6));
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < CH / LINES; ++k) {
                        const int c = LINES * k + lane / PARTS;
                        const uint4 a = ld_shared_16(xb + c * PITCH + 16 * part);
                        if (c0 + c < it.n && m < p.M && ys[c0 + c]) *(uint4 *)(ys[c0 + c] + 2 * (size_t)m) = a;
                    }
                    __syncwarp();
                }
                if (LORA && *bad_item > j) {
                    __syncwarp();
                    for (int c0 = CH * half; c0 < it.n; c0 += 2 * CH)
                        for (int c = c0; c < min(it.n, c0 + CH); ++c) {
                            const int a = p.adapter[it.row0 + c];
                            if (a < 0 || a >= p.n_adapters || m0 + lane >= p.M || !ys[c]) continue;
                            float s = 0.f;
                            for (int k = 0; k < chunks; ++k) s += not_finite(a, k, m0 + lane, it.row0 + c);
                            if (s != 0.f) {  // (or NaN)
                                uint8_t *o = ys[c] + (size_t)SIZE * (m0 + lane);
                                if (F32) *(float *)o += s;
                                else *(uint16_t *)o = (uint16_t)grouped_pack<OT>(grouped_unpack<OT>(*(uint16_t *)o).x + s, 0.f);
                            }
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            for (used += apart; used; --used, ++seq) hand_back(seq);
            it = nx;
        }
        if (GRAD && lane == 0) tma_store_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || ks > 1) cluster_sync_all();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_group<CG>(tmem, G_::TCOLS);
    }
}

// ------------------------------------------------------------------ host

// Launches the kernel on the current device: one CTA (or pair) an SM (or two), at most as many as `items`; where there are few
// of them (not wide), clusters share one item's reduction of `stages` stages.  One translation unit for each y type.
int grouped_launch_f32(const GroupedParams &p, int mode, bool wide, long long items, int stages, cudaStream_t s);
int grouped_launch_bf16(const GroupedParams &p, int mode, bool wide, long long items, int stages, cudaStream_t s);
int grouped_launch_f16(const GroupedParams &p, int mode, bool wide, long long items, int stages, cudaStream_t s);
static inline int grouped_launch(const GroupedParams &p, int ytype, int mode, bool wide, long long items, int stages,
                                 cudaStream_t s) {
    return ytype == MOE_F32    ? grouped_launch_f32(p, mode, wide, items, stages, s)
           : ytype == MOE_BF16 ? grouped_launch_bf16(p, mode, wide, items, stages, s)
                               : grouped_launch_f16(p, mode, wide, items, stages, s);
}
// GP_GRAD: reductions of at most 512 rows on average.
static inline bool grouped_grad_short(int R, int G) { return R <= 512LL * G; }
// SMs of the current device (0: none).
int grouped_sms();
// Tensor map of elements of `type`: `rank` dimensions and box extents innermost first, strides in bytes from the second on.
int grouped_map(CUtensorMap *map, int type, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box, int swizzle_bytes);

// ------------------------------------------------------------------ few rows (moe_grouped_few.cu)

#define GF_MAX_R 32                      // rows of a call
#define GF_MAX_TILES GF_MAX_R

struct GroupedFewParams {
    const uint16_t *x, *w;
    size_t ldx;
    const int32_t *offsets;  // as in GroupedParams
    int G, R;
    const int32_t *x_index;
    int x_share, x_rows;
    const int32_t *y_index;
    int y_rows;
    const float *scale;
    void *y;
    size_t ldy;
    int ytype, M, K;
    const int32_t *adapter;  // GP_LORA
    const uint16_t *b, *u;   // (fp16: u in fp32, 32 ranks to a piece)
    int n_adapters, rank, parts;
    int *status;
};
// GP_NK, GP_SWIGLU, GP_LORA with R <= GF_MAX_R.
int grouped_few_launch(const GroupedFewParams &p, int mode, bool bf, cudaStream_t s);
