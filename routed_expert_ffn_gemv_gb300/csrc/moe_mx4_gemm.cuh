// Internals shared by the MXFP4 product and layer translation units.
#pragma once

#include "moe_mx4.cuh"

// Argument checks of the product and layer calls (sizes; pool).
int mx4_ffn_check(int T, int H, int F, int E, int k);
int mx4_pool_check(int H, int F, int n_slots, const void *pool, size_t slot_bytes);

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// ------------------------------------------------------------------ few routes: chunks by every CTA
//
// Up to MX4_LOCAL_R routes are grouped by expert by each CTA for itself in shared memory: thread r
// compares route r with every other one (its rank among the routes of its expert, their number, the
// first of them), a block-wide sum gives the experts' positions in the order of their first routes.
// Everyone arrives at the same tables, without a kernel in front.
#define MX4_LOCAL_R 256

struct Mx4Chunks {
    alignas(16) int id[MX4_LOCAL_R];                          // served expert of a route, or -1
    int slot[MX4_LOCAL_R], pos[MX4_LOCAL_R], n[MX4_LOCAL_R];  // per chunk
    int rows[MX4_LOCAL_R];                                    // position -> route
    int base[MX4_LOCAL_R];                                    // of an expert, at its first route
    int scan[MX4_LOCAL_R / 32];
    int nch;                                                  // chunks
};

// Called by every thread of a block of at least MX4_LOCAL_R; syncs the block.  Routes of -1 are not
// served; ids outside [0, E) and slots outside [0, n_slots) are recorded and not served either.
// Chunks of at most NR routes.  `table`: global or shared memory, or NULL.
__device__ __forceinline__ void mx4_local_chunks(Mx4Chunks &c, const int32_t *ids, int R, int E, const int32_t *table,
                                                 int n_slots, int NR, int *status) {
    const int r = threadIdx.x, lane = r & 31, warp = r >> 5;
    int id = -1, slot = -1;
    if (r < MX4_LOCAL_R) {
        if (r < R) {
            id = ids[r];
            bool bad = id != -1 && (id < 0 || id >= E);
            if (!bad && id >= 0) {
                slot = table ? table[id] : id;
                bad = slot < 0 || slot >= n_slots;
            }
            if (bad) {
                moe_set_status(status, MOE_ERR_INVALID);
                id = -1;
            }
        }
        c.id[r] = id;
    }
    __syncthreads();
    int cnt = 0, rank = 0, first = MX4_LOCAL_R, pk = 0, incl = 0;
    if (r < MX4_LOCAL_R) {
        if (id >= 0)
#pragma unroll 4
            for (int q = 0; q < R; q += 4) {
                const int4 v = *(const int4 *)&c.id[q];
                const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool eq = w[i] == id;
                    cnt += eq;
                    rank += eq && q + i < r;
                    first = min(first, eq ? q + i : MX4_LOCAL_R);
                }
            }
        if (id >= 0 && rank == 0) pk = cnt | ((cnt + NR - 1) / NR) << 16;
        incl = pk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) c.scan[warp] = incl;
    }
    __syncthreads();
    if (r < MX4_LOCAL_R) {
        int b = incl - pk;
        for (int w = 0; w < warp; ++w) b += c.scan[w];
        if (r == MX4_LOCAL_R - 1) c.nch = (b + pk) >> 16;
        if (pk) {
            c.base[r] = b & 0xFFFF;
            const int c0 = b >> 16, nc = pk >> 16;
            for (int i = 0; i < nc; ++i) {  // near-equal chunks
                const int lo = cnt * i / nc, hi = cnt * (i + 1) / nc;
                c.slot[c0 + i] = slot;
                c.pos[c0 + i] = (b & 0xFFFF) + lo;
                c.n[c0 + i] = hi - lo;
            }
        }
    }
    __syncthreads();
    if (id >= 0) c.rows[c.base[first] + rank] = r;
    __syncthreads();
}
