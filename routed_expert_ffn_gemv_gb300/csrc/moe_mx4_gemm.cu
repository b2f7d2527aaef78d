// The routed experts' products over MXFP4 weights and MXFP4 activations
// (moe_mx4_expert_gateup, moe_mx4_expert_down) on the block-scaled tensor cores.
//
//   D[128 weight rows][N routes] += (A . SFA)[rows][64] * (B . SFB)[routes][64]^T,
//   tcgen05.mma kind::mxf4: E2M1 operands read from shared memory, one E8M0 scale per 32 columns
//   read from tensor memory, exact products, fp32 sums in tensor memory.
// The weights are the M side, so that an expert's few routes cost only as wide an MMA as they are.
//
//  * few routes (MX4_LOCAL_R): each CTA groups them by expert itself; otherwise mx4_count_kernel and
//    mx4_place_kernel sort them, experts with the most routes first, and lay their rows out.  Chunks are at
//    most NT routes of one expert.  The order of the routes inside an expert is not fixed; a route's result
//    does not depend on it.
//  * mx4_gemm_kernel: persistent, one CTA per SM; a work item is (chunk, 128-row weight tile).
//    Warp roles, mbarrier rings that run on across items:
//      warps 0, 1  a stage of 256 columns: the tile's two 8704-byte blocks (codes and scales, one
//                  bulk copy: the slot image is in operand order) and the chunk's code rows, as runs
//                  of mx4_place_kernel's output, or, for few routes, four rows to a TMA gather
//                  straight into the 128-byte-swizzled operand layout;
//      warp 2      the four MMAs of a stage and one commit, by an elected thread;
//      warps 4-7   the stage's scales into tensor memory.  Each warp writes its own
//                  lane quarter (the tensor core reads a copy in each);
//      warps 8-15  the epilogue of the previous item from the other accumulator.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "moe_mx4_gemm.cuh"
#include "moe_tc.cuh"

#define MXG_THREADS 512
#define MXG_WBYTES (2 * MX4_TB)  // weights of a stage: two tile blocks
#define MXG_ITEMS 64              // items of a CTA that are looked up ahead, in shared memory

#define MXG_ROUTE_BLOCKS 256

namespace {

// ------------------------------------------------------------------ workspace

// Routes that every CTA groups for itself (LOCAL): as many as its tables leave the ring room for.  Measured,
// gate/up: 2000 routes over 128 experts 41.0 us against 49.0 with two kernels in front, 2000 over 16
// 11.7 against 14.2, over 8 (four rows to a TMA copy, 128 rows a chunk) 19.9 against 20.3.
#define MX4_LOCAL_R 2048

// Most routes of a chunk: a few where experts have few (more stages in the ring), else as wide as tensor
// and shared memory allow, which is less beside the tables of LOCAL.  The larger saves passes over the
// weights: 32768 routes over 128 experts of uneven popularity (one draw) are 241 chunks of at most 176, 227
// of at most 192.
#define MXG_NT_SMALL 32
#define MXG_NT_LOCAL 176
#define MXG_NT_LARGE 192
int chunk_routes(int T, int E, int k) {
    const long R = (long)T * k;
    return R <= 16L * E ? MXG_NT_SMALL : R <= MX4_LOCAL_R ? MXG_NT_LOCAL : MXG_NT_LARGE;
}

struct GemmWs {
    size_t o_rows, o_slot, o_pos, o_n, o_hist, ints;  // in ints; [0] is the number of chunks
    size_t Rp;                                // positions: every expert's start at a multiple of 8
    size_t codes, scales, total;              // in bytes
};

// Chunks of at most NT routes that R routes can make.
int most_chunks(long R, int E, int NT) { return (int)(R / NT + std::min<long>(E, R)); }

// (the tables hold the chunks of the smallest kind, so that the size grows with T whatever kind a call takes)
GemmWs gemm_ws(int T, int H, int F, int E, int k) {
    GemmWs L;
    const long R = (long)T * k;
    const int max_chunks = most_chunks(R, E, MXG_NT_SMALL);
    L.Rp = (size_t)(R + 7 * std::min<long>(E, R) + 7) / 8 * 8;
    size_t o = 16;
    L.o_rows = o; o += L.Rp;
    L.o_slot = o; o += max_chunks;
    L.o_pos = o;  o += max_chunks;
    L.o_n = o;    o += max_chunks;
    L.o_hist = o; o += (size_t)MXG_ROUTE_BLOCKS * E;
    L.ints = o;
    L.codes = (o * 4 + 1023) / 1024 * 1024;
    const size_t stages = (std::max(H, F) + 255) / 256, rows = R > MX4_LOCAL_R ? stages * L.Rp : 0;
    L.scales = L.codes + rows * 128;
    L.total = L.scales + rows * 8;
    return L;
}

// ------------------------------------------------------------------ routes by expert

// The eight scale bytes of a row from block 8q on (fewer at the row's end: zeros).
__device__ __forceinline__ uint2 scale8(const uint8_t *row, int q, int KS) {
    if ((KS & 7) == 0 && ((uintptr_t)row & 7) == 0) return *(const uint2 *)(row + 8 * q);
    uint32_t v[2] = {0u, 0u};
    const int n = min(8, KS - 8 * q);
    for (int i = 0; i < n; ++i) v[i >> 2] |= (uint32_t)row[8 * q + i] << (8 * (i & 3));
    return make_uint2(v[0], v[1]);
}

// Two kernels of the same blocks of consecutive routes.  The first counts each block's routes per expert.
// In the second every block adds the counts up (all blocks: the experts' starts, at multiples of 8; the
// blocks before: its own cursors), gives its routes their positions and takes their rows there, in
// operand order by stages of 256 columns: codes [stage][position][128 bytes], 16-byte piece j at
// j ^ (position % 8) (the 128-byte swizzle; chunks start at multiples of 8), scales [stage][position][8
// bytes], zeros past K.  So a stage of a chunk is two runs of bytes.  One more block writes the chunk
// table.  Bound by the latency of its row copies, hence 1024 threads a block.  Measured, 32768 routes:
// one cluster of 8 CTAs for the positions and a gather kernel took 17 + 8 us, this kernel with 256
// threads a block 27 us; gathering by TMA inside the product kernel (four rows a copy, 48 copies a stage) kept two
// warps busy all the time, about 80 clocks a copy, and bound it.
#define MXG_ROUTE_THREADS 256  // routes of a block at a time
#define MXG_PLACE_THREADS 1024

__global__ void __launch_bounds__(MXG_ROUTE_THREADS)
mx4_count_kernel(const int32_t *__restrict__ ids, int R, int E, int32_t *__restrict__ hist, int *status) {
    __shared__ int h[MOE_MAX_E];
    const int tid = threadIdx.x, seg = (R + gridDim.x - 1) / gridDim.x, r0 = blockIdx.x * seg, r1 = min(R, r0 + seg);
    for (int e = tid; e < E; e += MXG_ROUTE_THREADS) h[e] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    for (int r = r0 + tid; r < r1; r += MXG_ROUTE_THREADS) {
        const int e = ids[r];
        if (e >= 0 && e < E) atomicAdd(&h[e], 1);
        else if (e != -1) moe_set_status(status, MOE_ERR_INVALID);
    }
    __syncthreads();
    for (int e = tid; e < E; e += MXG_ROUTE_THREADS) hist[blockIdx.x * E + e] = h[e];
}

// Exclusive sums of v over the block's threads.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += warp_sums[w];
    return x - v;
}

__global__ void __launch_bounds__(MXG_PLACE_THREADS)
mx4_place_kernel(const int32_t *__restrict__ ids, int R, int E, const int32_t *__restrict__ table, int n_slots, int NT,
                 const int32_t *__restrict__ hist, const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                 int K, int div, size_t Rp, int32_t *__restrict__ ints, int32_t *__restrict__ rows,
                 int32_t *__restrict__ c_slot, int32_t *__restrict__ c_pos, int32_t *__restrict__ c_n,
                 uint8_t *__restrict__ xg, uint8_t *__restrict__ sg, int *status) {
    constexpr int PARTS = MXG_PLACE_THREADS / MOE_MAX_E;
    __shared__ __align__(16) int cnt[MOE_MAX_E];
    __shared__ int cur[MOE_MAX_E], order[MOE_MAX_E], sums[MXG_PLACE_THREADS / 32], part[2][PARTS][MOE_MAX_E];
    __shared__ int s_pos[MXG_ROUTE_THREADS], s_src[MXG_ROUTE_THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, blocks = gridDim.x - 1;
    const int seg = (R + blocks - 1) / blocks, r0 = blockIdx.x * seg, r1 = min(R, r0 + seg);
    const int KS = K / 32, NKS = (K + 255) / 256;
    // (the count kernel lets this one start after everything before it is complete: ids may be read)
    const int first_id = tid < MXG_ROUTE_THREADS && r0 + tid < r1 ? ids[r0 + tid] : -1;
    pdl_wait();
    pdl_trigger();
    {
        const int e = tid % MOE_MAX_E, q = tid / MOE_MAX_E;
        int t = 0, before = 0;
        if (e < E)
#pragma unroll 16
            for (int b = q; b < blocks; b += PARTS) {
                const int v = hist[b * E + e];
                before += b < (int)blockIdx.x ? v : 0;
                t += v;
            }
        part[0][q][e] = t;
        part[1][q][e] = before;
    }
    __syncthreads();
    int total = 0, before = 0;
    if (tid < MOE_MAX_E)
        for (int q = 0; q < PARTS; ++q) {
            total += part[0][q][tid];
            before += part[1][q][tid];
        }
    const int off = block_exclusive((total + 7) & ~7, sums);
    if (tid < MOE_MAX_E) {
        cnt[tid] = total;
        cur[tid] = off + before;
    }
    __syncthreads();
    if ((int)blockIdx.x == blocks) {
        // chunks, the experts with the most routes first
        if (tid < MOE_MAX_E) {
            int o = 0;
#pragma unroll 4
            for (int j = 0; j < MOE_MAX_E; j += 4) {
                const int4 v = *(const int4 *)&cnt[j];
                o += (v.x > total || (v.x == total && j < tid)) + (v.y > total || (v.y == total && j + 1 < tid)) +
                     (v.z > total || (v.z == total && j + 2 < tid)) + (v.w > total || (v.w == total && j + 3 < tid));
            }
            order[o] = tid;
            cur[tid] = off;
        }
        __syncthreads();
        const int e = tid < MOE_MAX_E ? order[tid] : 0, n = tid < MOE_MAX_E ? cnt[e] : 0, nc = (n + NT - 1) / NT;
        const int first = block_exclusive(nc, sums);
        if (tid == MXG_PLACE_THREADS - 1) ints[0] = first;
        if (n > 0) {
            int slot = table ? table[e] : e;
            if (slot < 0 || slot >= n_slots) {
                moe_set_status(status, MOE_ERR_INVALID);
                slot = -1;
            }
            // near-equal chunks that start at multiples of 8 (NT is one: no chunk is empty)
            const int size = ((n + nc - 1) / nc + 7) & ~7;
            for (int c = 0; c < nc; ++c) {
                c_slot[first + c] = slot;
                c_pos[first + c] = cur[e] + c * size;
                c_n[first + c] = min(size, n - c * size);
            }
        }
        return;
    }
    for (int rb = r0; rb < r1; rb += MXG_ROUTE_THREADS) {
        if (tid < MXG_ROUTE_THREADS) {
            // the lanes of one expert reserve their positions together
            const int r = rb + tid, id = rb == r0 ? first_id : r < r1 ? ids[r] : -1, e = id >= 0 && id < E ? id : -1;
            const unsigned peers = __match_any_sync(0xffffffffu, e);
            int pos = -1;
            if (e >= 0) {
                const int lead = __ffs(peers) - 1;
                int at = 0;
                if (lane == lead) at = atomicAdd(&cur[e], __popc(peers));
                at = __shfl_sync(peers, at, lead);
                pos = at + __popc(peers & ((1u << lane) - 1));
                rows[pos] = r;
            }
            s_pos[tid] = pos;
            s_src[tid] = r / div;
        }
        __syncthreads();
        // a warp takes eight rows.  Codes: lane l piece l % 8 of a stage of rows l / 8 and l / 8 + 4, four
        // stages at a time, every load before the first store (the copies are all latency)
        const int j = lane & 7, ka = 8 * warp + (lane >> 3), at[2] = {s_pos[ka], s_pos[ka + 4]};
        const uint8_t *src[2] = {codes + (size_t)s_src[ka] * (K / 2) + 16 * j, codes + (size_t)s_src[ka + 4] * (K / 2) + 16 * j};
        const int ks = 8 * warp + (lane >> 2), ats = s_pos[ks];
        const uint8_t *srcs = scales + (size_t)s_src[ks] * KS;
#pragma unroll 1
        for (int q0 = 0; q0 < NKS; q0 += 4) {
            uint4 v[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[i][q] = make_uint4(0, 0, 0, 0);
                    if (at[i] >= 0 && 128 * (q0 + q) + 16 * j < K / 2) v[i][q] = *(const uint4 *)(src[i] + 128 * (q0 + q));
                }
            // scales: lane l stage l % 4 of row l / 4
            const int qs = q0 + (lane & 3);
            const bool has = ats >= 0 && qs < NKS;
            const uint2 sc = has ? scale8(srcs, qs, KS) : make_uint2(0, 0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (at[i] >= 0 && q0 + q < NKS)
                        *(uint4 *)(xg + ((size_t)(q0 + q) * Rp + at[i]) * 128 + ((j ^ (at[i] & 7)) << 4)) = v[i][q];
            if (has) *(uint2 *)(sg + ((size_t)qs * Rp + ats) * 8) = sc;
        }
        __syncthreads();
    }
}
static_assert(MXG_PLACE_THREADS == 4 * MXG_ROUTE_THREADS, "eight rows a warp");
static_assert(MXG_ROUTE_THREADS == MOE_MAX_E, "a thread per expert");

// ------------------------------------------------------------------ the products

struct GemmParams {
    CUtensorMap map;         // LOCAL: the code rows, boxes of 128 bytes of one row
    const uint8_t *scales;   // LOCAL: [rows][K / 32]
    const uint8_t *xg, *sg;  // otherwise mx4_place_kernel's rows
    size_t Rp;
    const uint8_t *pool;
    size_t slot_bytes;
    const int32_t *ints, *rows, *c_slot, *c_pos, *c_n;  // mx4_place_kernel's tables
    const int32_t *ids, *table;                         // LOCAL
    int R, E, n_slots;
    const float *weights;    // down
    void *out;
    int K, R_out, div;       // columns, output row length, routes per code row
    int MT;                  // weight tiles of an item list
    size_t mat;              // byte offset of the matrix in an image
    int *status;
};

// (at most R / NT + E chunks)
typedef Mx4Chunks<MX4_LOCAL_R, MX4_LOCAL_R / MXG_NT_SMALL + MOE_MAX_E> GemmChunks;

// A ring stage and its scales in tensor memory share their index: a landed stage means that the MMAs
// that read the scales' previous contents are done, so the scale slots need no wait of their own.
// A stage lives about 3000 clocks (its copies, its scales, its MMAs): as many stages as fit.  Gate/up
// exchanges eight routes at a time, down (three stages an item, its epilogue the longer part) 16.
template <int NT, bool DOWN, bool LOCAL>
struct GemmGeom {
    static constexpr int NI = (NT + 31) / 32;                // 32-route groups
    static constexpr int STAGE = MXG_WBYTES + NT * 128;      // weights, code rows
    static constexpr int SSTAGE = NI * 256;                  // scales of the rows
    static constexpr int S = NT > MXG_NT_SMALL ? (DOWN ? 4 : 5) : (DOWN ? 8 : 9);  // ring stages
    static constexpr int SFCOL = 2 * NT;                     // scales after the two accumulators, 24 columns a stage
    static constexpr int XCH = DOWN ? 8 * 16 * 36 * 4 : 4 * 2 * 2 * 4 * 32 * 4;
    static constexpr int O_XCH = 1024 + MXG_ITEMS * 16, O_ROWS = O_XCH + XCH, O_LOC = O_ROWS + 2 * NT * 8;
    static constexpr int O_SC = (O_LOC + (LOCAL ? (int)sizeof(GemmChunks) : 0) + 15) / 16 * 16;
    static constexpr int O_RING = (O_SC + S * SSTAGE + 1023) / 1024 * 1024;
    static constexpr size_t SMEM = 1024 + O_RING + (size_t)S * STAGE;
    static_assert(SFCOL + S * 24 <= 512 && STAGE % 1024 == 0 && O_LOC % 16 == 0 && SMEM <= 227 * 1024, "tensor and shared memory");
};

// A work item: slot (-1: none), first position and number of its routes, weight tile.
typedef int4 Item;

// Four rows of the map's box width to 4 x 128 bytes of shared memory.  x is a multiple of 128.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int x, const int (&r)[4], uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_u32(bar))
        : "memory");
}

// LOCAL: few routes, grouped by the CTA itself; otherwise mx4_place_kernel's tables.
template <int NT, bool DOWN, int OT, bool LOCAL>
__global__ void __launch_bounds__(MXG_THREADS, 1) mx4_gemm_kernel(const __grid_constant__ GemmParams p) {
    using G = GemmGeom<NT, DOWN, LOCAL>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint64_t *s_full = (uint64_t *)smem;
    uint64_t *s_empty = s_full + G::S;
    uint64_t *sf_full = s_empty + G::S;
    uint64_t *acc_full = sf_full + G::S;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *mma_done = acc_empty + 2;
    uint32_t *tmem_slot = (uint32_t *)(mma_done + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    static_assert((3 * G::S + 6) * 8 <= 1024, "barriers");
    Item *items = (Item *)(smem + 1024);                  // [MXG_ITEMS]
    float *xch = (float *)(smem + G::O_XCH);              // gate/up [4 pairs][2][2 ways][4 routes][32], down [8][16][36]
    int2 *e_rows = (int2 *)(smem + G::O_ROWS);            // [2 accumulators][NT]: route, its weight's bits
    GemmChunks &loc = *(GemmChunks *)(smem + G::O_LOC);   // LOCAL
    uint8_t *ring = smem + G::O_RING, *sring = smem + G::O_SC;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::S; ++s) {
            mbar_init(&s_full[s], LOCAL ? 1 : 2);
            mbar_init(&s_empty[s], 1);
            mbar_init(&sf_full[s], 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (LOCAL)
        mx4_local_chunks<MXG_THREADS>(loc, (uint16_t *)ring, p.ids, p.R, p.E, p.table, p.n_slots, NT, nullptr, p.status);
    auto route_at = [&](int pos) -> int { return LOCAL ? (int)loc.rows[pos] : p.rows[pos]; };
    const int MT = p.MT, n_items = (LOCAL ? loc.nch : p.ints[0]) * MT;
    // this CTA's items are blockIdx.x, + gridDim.x, ..; every role looks them up, and from global memory
    // each look costs an L2 round trip
    const int n_mine = (int)blockIdx.x < n_items ? (n_items - (int)blockIdx.x - 1) / (int)gridDim.x + 1 : 0;
    auto look_up = [&](int i) -> Item {
        const int j = blockIdx.x + i * gridDim.x, c = j / MT;
        return LOCAL ? make_int4(loc.slot[c], loc.pos[c], loc.n[c], j - c * MT)
                     : make_int4(p.c_slot[c], p.c_pos[c], p.c_n[c], j - c * MT);
    };
    for (int i = threadIdx.x; i < min(n_mine, MXG_ITEMS); i += MXG_THREADS) items[i] = look_up(i);
    __syncthreads();
    auto item_at = [&](int i) -> Item { return i < MXG_ITEMS ? items[i] : look_up(i); };
    const int K = p.K, KB = (K + 127) / 128, NKS = (KB + 1) / 2, KS = K / 32;

    if (warp < 2) {
        // ---------------- producers.  LOCAL: warp 0 the stage's expected bytes, its weights and the even
        // groups of four code rows, warp 1 the odd groups.  Otherwise warp 0 the weights, warp 1
        // the chunk's rows and scales, runs of bytes.
        const uint64_t once = l2_evict_first();
        int g = 0, st_i = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int i = 0; i < n_mine && ok; ++i) {
            const Item it = item_at(i);
            const int slot = __shfl_sync(0xffffffffu, it.x, 0), m = __shfl_sync(0xffffffffu, it.w, 0);
            if (slot < 0) continue;
            const int pos0 = __shfl_sync(0xffffffffu, it.y, 0), n = __shfl_sync(0xffffffffu, it.z, 0);
            const int npad = (n + 7) & ~7, q = 2 * lane + warp;  // this lane's group of four rows
            int r4[4];
            if (LOCAL)
                for (int k = 0; k < 4; ++k) {
                    const int at = 4 * q + k;
                    r4[k] = route_at(pos0 + (at < n ? at : 0)) / p.div;  // rows past the chunk: unused columns
                }
            const uint8_t *w = p.pool + (size_t)slot * p.slot_bytes + p.mat + (size_t)m * KB * MX4_TB;
            const uint8_t *xrow = p.xg + (size_t)pos0 * 128, *srow = p.sg + (size_t)pos0 * 8;
            for (int kc = 0; kc < NKS; ++kc, ++g) {
                if (g >= G::S && !(ok = mbar_wait_warp(&s_empty[st_i], ph, p.status, abort_flag))) break;
                uint8_t *st = ring + (size_t)st_i * G::STAGE;
                uint64_t *full = &s_full[st_i];
                if (warp == 0) {
                    const uint32_t wb = 2 * kc + 1 < KB ? MXG_WBYTES : MX4_TB;
                    mbar_arrive_expect_tx_elect(full, LOCAL ? wb + (uint32_t)npad * 128u : wb);
                    // few routes read an expert's weights about once, many in several chunks
                    if (LOCAL) bulk_g2s_elect_hint(st, w, wb, full, once);
                    else bulk_g2s_elect(st, w, wb, full);
                    w += MXG_WBYTES;
                } else if (!LOCAL) {
                    // (an arrival of its own: a copy takes its thread about 100 clocks)
                    const uint32_t sb = (uint32_t)((n + 1) & ~1) * 8u;
                    mbar_arrive_expect_tx_elect(full, (uint32_t)n * 128u + sb);
                    bulk_g2s_elect(st + MXG_WBYTES, xrow, (uint32_t)n * 128u, full);
                    bulk_g2s_elect(sring + st_i * G::SSTAGE, srow, sb, full);
                    xrow += p.Rp * 128;
                    srow += p.Rp * 8;
                }
                if (LOCAL) {
                    if (4 * q < npad) tma_gather4(st + MXG_WBYTES + q * 512, &p.map, kc * 128, r4, full);
                    __syncwarp();
                }
                if (++st_i == G::S) {
                    st_i = 0;
                    ph ^= 1u;
                }
            }
        }
        // never leave with copies in flight
        if (threadIdx.x == 0)
            for (int s = 0; s < G::S && s < g; ++s) {
                const int last = s + ((g - 1 - s) / G::S) * G::S;
                mbar_wait_bounded(&s_full[s], (last / G::S) & 1, p.status);
            }
        if (!ok) settle_after_abort();
    } else if (warp == 2) {
        // ---------------- MMA issuer: the whole warp, one elected thread inside each instruction
        int jl = 0, st_i = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int i = 0; i < n_mine && ok; ++i) {
            const Item it = item_at(i);
            if (it.x < 0) continue;
            const int npad = __shfl_sync(0xffffffffu, (it.z + 7) & ~7, 0);
            const uint32_t id0 = umma_idesc_mxf4(128, npad, 0), id2 = umma_idesc_mxf4(128, npad, 2);
            const int buf = jl & 1;
            if (jl >= 2 && !(ok = mbar_wait_warp(&acc_empty[buf], ((jl / 2) - 1) & 1, p.status, abort_flag))) break;
            tc_fence_after();
            const uint32_t d = tmem + buf * NT;
            for (int kc = 0; kc < NKS; ++kc) {
                // (the scale warps saw the stage land before they arrived)
                if (!(ok = mbar_wait_warp(&sf_full[st_i], ph, p.status, abort_flag))) break;
                tc_fence_after();
                const uint32_t st = smem_u32(ring) + (uint32_t)st_i * G::STAGE;
                const uint64_t a = umma_desc_sw64(st), b = umma_desc_sw128(st + MXG_WBYTES);
                const uint32_t sf = tmem + G::SFCOL + 24 * st_i;
                const int steps = (K - 256 * kc + 63) / 64;
                umma_mxf4(d, a, b, id0, sf, sf + 8, kc > 0);
                if (steps > 1) umma_mxf4(d, a + 2, b + 2, id2, sf, sf + 8, 1);
                if (steps > 2) umma_mxf4(d, a + (MX4_TB >> 4), b + 4, id0, sf + 4, sf + 16, 1);
                if (steps > 3) umma_mxf4(d, a + (MX4_TB >> 4) + 2, b + 6, id2, sf + 4, sf + 16, 1);
                umma_commit_elect(&s_empty[st_i]);
                if (++st_i == G::S) {
                    st_i = 0;
                    ph ^= 1u;
                }
            }
            if (ok) umma_commit_elect(&acc_full[buf]);
            ++jl;
        }
        umma_commit_elect(mma_done);  // every MMA has completed before tensor memory is released
        mbar_wait_bounded(mma_done, 0, p.status);
    } else if (warp >= 4 && warp < 8) {
        // ---------------- scales
        const uint32_t t0 = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + G::SFCOL;
        constexpr int NI = G::NI;
        int st_i = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int j = 0; j < n_mine && ok; ++j) {
            const Item it = item_at(j);
            if (it.x < 0) continue;
            const int pos0 = it.y, n = it.z;
            // LOCAL: the routes' scales from their rows, loaded two stages ahead (a load takes about as long
            // as a stage); otherwise they landed with the stage
            const uint8_t *row[NI];
            uint2 n0[NI], n1[NI];
            if (LOCAL)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int at = 32 * i + lane;
                    row[i] = at < n ? p.scales + (size_t)(route_at(pos0 + at) / p.div) * KS : nullptr;
                    n0[i] = row[i] ? scale8(row[i], 0, KS) : make_uint2(0, 0);
                    n1[i] = row[i] && NKS > 1 ? scale8(row[i], 1, KS) : make_uint2(0, 0);
                }
            for (int kc = 0; kc < NKS; ++kc) {
                uint32_t v[24];
                if (!(ok = mbar_wait_warp(&s_full[st_i], ph, p.status, abort_flag))) break;
                tc_fence_after();
                const uint8_t *st = ring + (size_t)st_i * G::STAGE;
                if (!LOCAL)
#pragma unroll
                    for (int i = 0; i < NI; ++i) n0[i] = *(const uint2 *)(sring + st_i * G::SSTAGE + 8 * (32 * i + lane));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[8 + i] = i < NI ? n0[i < NI ? i : 0].x : 0u;
                    v[16 + i] = i < NI ? n0[i < NI ? i : 0].y : 0u;
                }
                if (LOCAL)
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        n0[i] = n1[i];
                        if (row[i] && kc + 2 < NKS) n1[i] = scale8(row[i], kc + 2, KS);
                    }
                const uint4 a = *(const uint4 *)(st + 8192 + 16 * lane);
                uint4 b = make_uint4(0, 0, 0, 0);
                if (2 * kc + 1 < KB) b = *(const uint4 *)(st + MX4_TB + 8192 + 16 * lane);
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
#pragma unroll
                for (int i = 0; i < 3; ++i) tmem_st8(t0 + 24 * st_i + 8 * i, *reinterpret_cast<uint32_t(*)[8]>(&v[8 * i]));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sf_full[st_i]);
                if (++st_i == G::S) {
                    st_i = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp >= 8) {
        // ---------------- epilogue: lane quarter q, lane = weight row 32 q + lane of the tile; the two
        // warps of a quarter take alternate groups of routes.  The next item's routes and weights are
        // read while this one is worked on.  Gate/up: lanes 0-63 hold gate rows, 64-127 the same up
        // rows; a gate warp and its up warp trade halves of the group, so that both work on SwiGLU.
        // (Measured, 32768 routes, gate/up 82.5 us and down 78.7: the warps as two groups on alternate items
        // 86.6 and 79.3, tensor memory read a group ahead 85.3 and 79.9, the accumulator released after its
        // last load instead of its last store 83.6 and 78.3.)
        const int q = warp & 3, ew = warp - 8, half = ew >> 2, et = ew * 32 + lane;
        int jl = 0, xs = 0;
        auto next_item = [&](int i, Item &it) {  // the first item from i on that has a slot
            for (; i < n_mine; ++i)
                if ((it = item_at(i)).x >= 0) break;
            return i;
        };
        Item it = make_int4(-1, 0, 0, 0);
        int i = next_item(0, it);
        int route = i < n_mine && et < it.z ? route_at(it.y + et) : 0;
        float weight = DOWN && i < n_mine && et < it.z ? p.weights[route] : 0.f;
        while (i < n_mine) {
            const int n = it.z, m = it.w, buf = jl & 1;
            if (et < n) e_rows[buf * NT + et] = make_int2(route, __float_as_int(weight));
            Item nx = it;
            i = next_item(i + 1, nx);
            const bool more = i < n_mine && et < nx.z;
            if (more) route = route_at(nx.y + et);
            const bool w = mbar_wait_role(&acc_full[buf], (jl / 2) & 1, p.status, abort_flag);
            if (!bar_and_n(1, 256, w)) break;
            if (DOWN && more) weight = p.weights[route];
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + buf * NT;
            if (!DOWN) {
                constexpr int ES = OT == MOE_BF16 ? 2 : 4;
                const int pair = (q & 1) + 2 * half, up = q >> 1, f = 64 * m + 32 * (q & 1) + lane;
                uint8_t *out = (uint8_t *)p.out + (size_t)f * ES;
                for (int c0 = 8 * half; c0 < n; c0 += 16, ++xs) {
                    uint32_t v[8];
                    tmem_ld8(tb + c0, v);
                    // the gate warp keeps routes 0-3 of the group and hands over 4-7, the up warp the other
                    // way round
                    float *xb = xch + (size_t)(pair * 2 + (xs & 1)) * 256 + lane;
                    const int2 *row = e_rows + buf * NT + c0 + 4 * up;
                    uint8_t *o[4];
                    const int nn = f < p.R_out ? min(4, n - c0 - 4 * up) : 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = out + (size_t)row[k].x * (p.R_out * ES);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 4; ++k) xb[128 * up + 32 * k] = __uint_as_float(up ? v[k] : v[4 + k]);
                    bar_sync_n(2 + pair, 64);
                    float h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float other = xb[128 * (1 - up) + 32 * k];
                        const float gv = up ? other : __uint_as_float(v[k]);
                        const float uv = up ? __uint_as_float(v[4 + k]) : other;
                        h[k] = mx4_swiglu<OT == MOE_F32>(gv, uv);
                    }
                    auto put = [&](int k) {
                        if (OT == MOE_BF16) *(__nv_bfloat16 *)o[k] = __float2bfloat16(h[k]);
                        else *(float *)o[k] = h[k];
                    };
                    if (nn == 4) {  // no branch between the stores
#pragma unroll
                        for (int k = 0; k < 4; ++k) put(k);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < nn) put(k);
                    }
                }
            } else {
                // 32 rows x 16 routes by way of shared memory (padded: no bank conflicts), so that a store
                // covers four rows of four routes: a quarter of the store instructions
                float *xb = xch + ew * 576;
                const int o = 128 * m + 32 * q + 4 * (lane & 7);
                float *out = (float *)p.out + o;
                for (int c0 = 16 * half; c0 < n; c0 += 32) {
                    uint32_t v[16];
                    tmem_ld16(tb + c0, v);
                    const int nn = o < p.R_out ? n - c0 : 0;
                    int2 d[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) d[k] = e_rows[buf * NT + c0 + 4 * k + (lane >> 3)];
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) xb[36 * k + lane] = __uint_as_float(v[k]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 4 * k + (lane >> 3);
                        const float4 a = *(const float4 *)(xb + 36 * r + 4 * (lane & 7));
                        const float wt = __int_as_float(d[k].y);
                        if (r < nn)
                            *(float4 *)(out + (size_t)d[k].x * p.R_out) = make_float4(wt * a.x, wt * a.y, wt * a.z, wt * a.w);
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(&acc_empty[buf]);
            ++jl;
            it = nx;
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

// Code rows [rows][K/2] as boxes of 128 bytes of one row (TMA gathers), 128-byte swizzle; columns
// past the row's end read 0.
int encode_codes_map(const uint8_t *codes, long rows, int K, CUtensorMap *map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return MOE_ERR_UNSUPPORTED;
    const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {128, 1};
    const cuuint32_t es[2] = {1, 1};
    if (enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)codes, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <int NT, bool DOWN, int OT, bool LOCAL>
int launch_gemm_t(const GemmParams &p, int max_chunks, cudaStream_t s) {
    using G = GemmGeom<NT, DOWN, LOCAL>;
    static std::mutex mu;
    static int sms[64] = {0};
    int dev = -1;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    int n = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!sms[dev]) {
            MOE_TRY_CUDA(cudaFuncSetAttribute(mx4_gemm_kernel<NT, DOWN, OT, LOCAL>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM));
            MOE_TRY_CUDA(cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev));
        }
        n = sms[dev];
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const long items = (long)max_chunks * p.MT;
    moe_pdl_config(&cfg, attr, dim3((unsigned)std::min<long>(items, n)), dim3(MXG_THREADS), G::SMEM, s);
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<NT, DOWN, OT, LOCAL>, p));
    return MOE_OK;
}

template <bool DOWN, int OT>
int launch_gemm(const GemmParams &p, int NT, int max_chunks, cudaStream_t s) {
    if (p.R <= MX4_LOCAL_R)
        return NT == MXG_NT_SMALL ? launch_gemm_t<MXG_NT_SMALL, DOWN, OT, true>(p, max_chunks, s)
                                  : launch_gemm_t<MXG_NT_LOCAL, DOWN, OT, true>(p, max_chunks, s);
    return NT == MXG_NT_SMALL ? launch_gemm_t<MXG_NT_SMALL, DOWN, OT, false>(p, max_chunks, s)
                              : launch_gemm_t<MXG_NT_LARGE, DOWN, OT, false>(p, max_chunks, s);
}

int run_product(bool down, const uint8_t *codes, const uint8_t *scales, int T, int H, int F, int E, int k,
                const int32_t *ids, const float *weights, const int32_t *table, int n_slots, const void *pool,
                size_t slot_bytes, void *out, int otype, void *workspace, cudaStream_t s) {
    const int NT = chunk_routes(T, E, k);
    const GemmWs L = gemm_ws(T, H, F, E, k);
    int32_t *w = (int32_t *)workspace;
    GemmParams p;
    p.K = down ? F : H;
    p.R_out = down ? H : F;
    p.div = down ? 1 : k;
    p.R = T * k;
    if (p.R <= MX4_LOCAL_R) {
        const int rc = encode_codes_map(codes, down ? (long)T * k : T, p.K, &p.map);
        if (rc != MOE_OK) return rc;
    }
    p.scales = scales;
    uint8_t *xg = (uint8_t *)workspace + L.codes, *sg = (uint8_t *)workspace + L.scales;
    p.xg = xg;
    p.sg = sg;
    p.Rp = L.Rp;
    p.pool = (const uint8_t *)pool;
    p.slot_bytes = slot_bytes;
    p.ints = w;
    p.rows = w + L.o_rows;
    p.c_slot = w + L.o_slot;
    p.c_pos = w + L.o_pos;
    p.c_n = w + L.o_n;
    p.ids = ids;
    p.table = table;
    p.E = E;
    p.n_slots = n_slots;
    p.weights = weights;
    p.out = out;
    p.MT = down ? (H + 127) / 128 : (F + 63) / 64;
    p.mat = down ? mx4_gu_bytes(H, F) : 0;
    p.status = moe_status_word_device_ptr();
    const int max_chunks = most_chunks(p.R, E, NT);

    if (p.R > MX4_LOCAL_R) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        const int blocks = std::min(MXG_ROUTE_BLOCKS, (p.R + MXG_ROUTE_THREADS - 1) / MXG_ROUTE_THREADS);
        moe_pdl_config(&cfg, attr, dim3(blocks), dim3(MXG_ROUTE_THREADS), 0, s);
        MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, mx4_count_kernel, ids, p.R, E, w + L.o_hist, p.status));
        moe_pdl_config(&cfg, attr, dim3(blocks + 1), dim3(MXG_PLACE_THREADS), 0, s);
        MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, mx4_place_kernel, ids, p.R, E, table, n_slots, NT,
                                        (const int32_t *)(w + L.o_hist), codes, scales, p.K, p.div, L.Rp, w,
                                        w + L.o_rows, w + L.o_slot, w + L.o_pos, w + L.o_n, xg, sg, p.status));
    }
    if (down) return launch_gemm<true, MOE_F32>(p, NT, max_chunks, s);
    return otype == MOE_BF16 ? launch_gemm<false, MOE_BF16>(p, NT, max_chunks, s)
                             : launch_gemm<false, MOE_F32>(p, NT, max_chunks, s);
}

}  // namespace

int mx4_ffn_check(int T, int H, int F, int E, int k) {
    MOE_CHECK(T >= 0 && H > 0 && F > 0 && H % 32 == 0 && F % 32 == 0);
    MOE_CHECK(E >= 1 && E <= MOE_MAX_E && k >= 1 && k <= MOE_MAX_K && k <= E);
    MOE_CHECK((long long)T * k <= 1 << 24);
    // a row of h in bytes, a tile's columns and the number of work items are ints in the kernels
    if (H > 1 << 28 || F > 1 << 28) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int mx4_pool_check(int H, int F, int n_slots, const void *pool, size_t slot_bytes) {
    MOE_CHECK(pool && n_slots >= 1 && ((uintptr_t)pool & 255) == 0 && slot_bytes % 256 == 0);
    MOE_CHECK(slot_bytes >= moe_expert_image_bytes(MOE_MXFP4, H, F));
    return MOE_OK;
}

extern "C" int moe_mx4_expert_workspace(int T, int H, int F, int E, int k, size_t *bytes) {
    MOE_CHECK(bytes);
    const int rc = mx4_ffn_check(T, H, F, E, k);
    if (rc != MOE_OK) return rc;
    *bytes = (gemm_ws(T, H, F, E, k).total + 255) / 256 * 256;
    return MOE_OK;
}

extern "C" int moe_mx4_expert_gateup(const uint8_t *x_codes, const uint8_t *x_scales, int T, int H, int F, int E,
                                     int k, const int32_t *ids, const int32_t *d_slot_table, int n_slots,
                                     const void *pool, size_t slot_bytes, void *h, int htype, void *workspace,
                                     size_t ws_bytes, moe_stream_t s) {
    size_t need = 0;
    int rc = moe_mx4_expert_workspace(T, H, F, E, k, &need);
    if (rc != MOE_OK) return rc;
    MOE_CHECK(htype == MOE_F32 || htype == MOE_BF16);
    if (T == 0) return MOE_OK;
    MOE_CHECK(x_codes && x_scales && ids && h && workspace && ws_bytes >= need);
    MOE_CHECK(((uintptr_t)x_codes & 15) == 0 && ((uintptr_t)workspace & 255) == 0);
    MOE_CHECK(((uintptr_t)h & (htype == MOE_BF16 ? 1 : 3)) == 0);
    if ((rc = mx4_pool_check(H, F, n_slots, pool, slot_bytes)) != MOE_OK) return rc;
    return run_product(false, x_codes, x_scales, T, H, F, E, k, ids, nullptr, d_slot_table, n_slots, pool, slot_bytes,
                       h, htype, workspace, moe_cuda_stream(s));
}

extern "C" int moe_mx4_expert_down(const uint8_t *h_codes, const uint8_t *h_scales, int T, int H, int F, int E, int k,
                                   const int32_t *ids, const float *weights, const int32_t *d_slot_table, int n_slots,
                                   const void *pool, size_t slot_bytes, float *partial, void *workspace,
                                   size_t ws_bytes, moe_stream_t s) {
    size_t need = 0;
    int rc = moe_mx4_expert_workspace(T, H, F, E, k, &need);
    if (rc != MOE_OK) return rc;
    if (T == 0) return MOE_OK;
    MOE_CHECK(h_codes && h_scales && ids && weights && partial && workspace && ws_bytes >= need);
    MOE_CHECK(((uintptr_t)h_codes & 15) == 0 && ((uintptr_t)workspace & 255) == 0 && ((uintptr_t)partial & 15) == 0);
    if ((rc = mx4_pool_check(H, F, n_slots, pool, slot_bytes)) != MOE_OK) return rc;
    return run_product(true, h_codes, h_scales, T, H, F, E, k, ids, weights, d_slot_table, n_slots, pool, slot_bytes,
                       partial, MOE_F32, workspace, moe_cuda_stream(s));
}
