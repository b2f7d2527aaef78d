// Internals shared by the MXFP4 product and layer translation units.
#pragma once

#include "moe_mx4.cuh"

// Argument checks of the product and layer calls (sizes; pool).
int mx4_ffn_check(int T, int H, int F, int E, int k);
int mx4_pool_check(int H, int F, int n_slots, const void *pool, size_t slot_bytes);

// ------------------------------------------------------------------ few routes: chunks by every CTA
//
// Up to MAXR routes are grouped by expert by each CTA for itself in shared memory: a warp match ranks the
// routes of each 32 among those of their expert, a thread per expert adds the 32s up, a block-wide sum
// gives the experts' positions.  No atomics: every CTA arrives at the same tables (they share chunks), and
// no kernel has to run in front.
template <int MAXR, int MAXC>
struct alignas(16) Mx4Chunks {
    uint16_t rows[MAXR];                                      // position -> route
    int slot[MAXC], pos[MAXC], n[MAXC];                       // per chunk
    int eslot[MOE_MAX_E], off[MOE_MAX_E];                     // per expert: slot (or -1), first position
    int sums[32];
    int nch;                                                  // chunks
};

// Called by every thread of a block of NTHR (a multiple of 32, at least MOE_MAX_E and MAXR / 4); syncs the
// block.  Routes of -1 are not served; ids outside [0, E) and slots outside [0, n_slots) are recorded and
// not served either.  Chunks of at most NR routes.  `table`: global or shared memory, or NULL.  `scratch`:
// shared, 2 * E bytes for every 32 of MAXR.  `served`: shared [MAXR], 1 for the routes that are, or NULL.
template <int NTHR, int MAXR, int MAXC>
__device__ __forceinline__ void mx4_local_chunks(Mx4Chunks<MAXR, MAXC> &c, uint16_t *scratch, const int32_t *ids, int R,
                                                 int E, const int32_t *table, int n_slots, int NR, int *served,
                                                 int *status) {
    constexpr int PASSES = (MAXR + NTHR - 1) / NTHR;
    static_assert(PASSES <= 4 && NTHR >= MOE_MAX_E && NTHR % 32 == 0, "threads");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = (R + 31) / 32;
    int id[PASSES], rank[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = tid + i * NTHR;
        id[i] = r < R ? ids[r] : -1;
    }
    if (tid < E) {
        const int s = table ? table[tid] : tid;
        c.eslot[tid] = s >= 0 && s < n_slots ? s : -1;
    }
    if (groups > 1)
        for (int i = tid; i < (groups * E + 1) / 2; i += NTHR) ((uint32_t *)scratch)[i] = 0;
    __syncthreads();
    if (groups <= 1) {
        // a warp's worth of routes: its first warp does it all, experts in the order of their first routes
        if (warp == 0) {
            if (id[0] != -1 && (id[0] < 0 || id[0] >= E || c.eslot[id[0]] < 0)) {
                moe_set_status(status, MOE_ERR_INVALID);
                id[0] = -1;
            }
            const unsigned peers = __match_any_sync(0xffffffffu, id[0]);
            const int cnt = __popc(peers), head = __ffs(peers) - 1, nc = (cnt + NR - 1) / NR;
            const bool lead = id[0] >= 0 && head == lane;
            int incl = lead ? cnt | nc << 16 : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const int b = incl - (lead ? cnt | nc << 16 : 0), pos = b & 0xFFFF;
            if (lead)
                for (int i = 0; i < nc; ++i) {  // near-equal chunks
                    const int lo = cnt * i / nc, hi = cnt * (i + 1) / nc;
                    c.slot[(b >> 16) + i] = c.eslot[id[0]];
                    c.pos[(b >> 16) + i] = pos + lo;
                    c.n[(b >> 16) + i] = hi - lo;
                }
            const int start = __shfl_sync(0xffffffffu, pos, head);
            if (id[0] >= 0) c.rows[start + __popc(peers & ((1u << lane) - 1))] = (uint16_t)lane;
            if (served && lane < R) served[lane] = id[0] >= 0;
            if (lane == 31) c.nch = incl >> 16;
        }
        __syncthreads();
        return;
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = tid + i * NTHR;
        if (id[i] != -1 && (id[i] < 0 || id[i] >= E || c.eslot[id[i]] < 0)) {
            moe_set_status(status, MOE_ERR_INVALID);
            id[i] = -1;
        }
        const unsigned peers = __match_any_sync(0xffffffffu, id[i]);
        rank[i] = __popc(peers & ((1u << lane) - 1));
        if (id[i] >= 0 && rank[i] == 0) scratch[(r >> 5) * E + id[i]] = (uint16_t)__popc(peers);
        if (served && r < R) served[r] = id[i] >= 0;
    }
    __syncthreads();
    int total = 0;
    if (tid < E)
#pragma unroll 4
        for (int g = 0; g < groups; ++g) {
            const int v = scratch[g * E + tid];
            scratch[g * E + tid] = (uint16_t)total;
            total += v;
        }
    const int nc = (total + NR - 1) / NR, pk = total | nc << 16;
    int incl = pk;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) c.sums[warp] = incl;
    __syncthreads();
    int b = incl - pk;
    for (int w = 0; w < warp; ++w) b += c.sums[w];
    if (tid == NTHR - 1) c.nch = (b + pk) >> 16;
    if (tid < E) {
        c.off[tid] = b & 0xFFFF;
        for (int i = 0; i < nc; ++i) {  // near-equal chunks
            const int lo = total * i / nc, hi = total * (i + 1) / nc;
            c.slot[(b >> 16) + i] = c.eslot[tid];
            c.pos[(b >> 16) + i] = (b & 0xFFFF) + lo;
            c.n[(b >> 16) + i] = hi - lo;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = tid + i * NTHR;
        if (id[i] >= 0) c.rows[c.off[id[i]] + scratch[(r >> 5) * E + id[i]] + rank[i]] = (uint16_t)r;
    }
    fence_proxy_async_smem();  // the scratch becomes part of a copy ring
    __syncthreads();
}
