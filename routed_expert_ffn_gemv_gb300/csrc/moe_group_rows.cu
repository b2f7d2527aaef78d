// moe_group_rows: a stable sort of row numbers by small group ids.
//
// A warp ranks 32 consecutive ids among themselves by a warp match and counts them in a table of its own, so that no
// atomic decides an order.  Latency bounds it (32768 ids over 128 groups 6.7 us a call among others, 262 KB of traffic; 9.8 us when
// each id was ranked twice, by clusters of eight CTAs).  Few ids: one cluster, each CTA a run of the ids, the CTAs' counts exchanged through
// distributed shared memory.  Many: a kernel that counts and a kernel that places, the counts of every block between
// them in the workspace.
#include <algorithm>
#include <mutex>

#include "moe_ptx.cuh"

#define GR_WARPS 32
#define GR_THREADS (32 * GR_WARPS)
#define GR_CTA_IDS 2048                    // ids of a CTA of the cluster, while there are few
#define GR_MAX_CTAS 16
#define GR_LANE_IDS 8                      // most ids of a thread
#define GR_CLUSTER_IDS (GR_MAX_CTAS * GR_THREADS * GR_LANE_IDS)  // most ids that one cluster takes
#define GR_BLOCKS 148

namespace {

// Exclusive sums of v over the block's threads in order; sums: [GR_WARPS + 1] shared, the last one the total.
__device__ __forceinline__ int block_sums(int v, int *sums) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int t = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += t;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = lane < GR_WARPS ? sums[lane] : 0, all = w;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int t = __shfl_up_sync(0xffffffffu, all, d);
            if (lane >= d) all += t;
        }
        sums[lane] = all - w;
        if (lane == 31) sums[GR_WARPS] = all;
    }
    __syncthreads();
    const int r = sums[warp] + inc - v;
    return r;
}

// A warp's ids [i0, i1): the count of each group in `table` [G] (zeroed), by rank when `rows` is given: table then holds the
// group's next position.
__device__ __forceinline__ void warp_pass(const int32_t *ids, int i0, int i1, int G, int *table, int32_t *rows, int *status) {
    const int lane = threadIdx.x % 32;
    for (int b = i0; b < i1; b += 32) {
        const int i = b + lane, id = i < i1 ? ids[i] : -1;
        const bool in = id >= 0 && id < G;
        if (!rows && !in && id != -1) moe_set_status(status, MOE_ERR_INVALID);
        const unsigned peers = __match_any_sync(0xffffffffu, in ? id : -1);
        const int before = __popc(peers & ((1u << lane) - 1u));
        int at = 0;
        if (in) at = table[id];
        __syncwarp();
        if (in && before == 0) table[id] = at + __popc(peers);
        __syncwarp();
        if (rows && in) rows[at + before] = i;
    }
}

// Where the groups begin: total [G] counts -> first [G] (shared), and offsets from the block that writes them.  Returns the
// number of grouped ids.
__device__ __forceinline__ int group_starts(const int *total, int *first, int G, int32_t *offsets, int *sums) {
    int base = 0;
    for (int g0 = 0; g0 < G; g0 += GR_THREADS) {
        const int g = g0 + threadIdx.x, v = g < G ? total[g] : 0;
        const int at = base + block_sums(v, sums);
        if (g < G) {
            first[g] = at;
            if (offsets) offsets[g] = at;
        }
        base += sums[GR_WARPS];
        __syncthreads();
    }
    if (offsets && threadIdx.x == 0) offsets[G] = base;
    return base;
}

size_t table_bytes(int G) { return (size_t)(GR_WARPS + 2) * G * 4; }
size_t cluster_bytes(int G) { return (size_t)(GR_WARPS + 1 + 3) * G * 4; }

// A thread keeps its ids and their ranks among the warp's ids of the same group between the count and the placement.
__global__ void __launch_bounds__(GR_THREADS, 1)
    group_cluster_kernel(const int32_t *ids, int n, int G, int32_t *offsets, int32_t *rows, int *status) {
    extern __shared__ int sm[];
    __shared__ int sums[GR_WARPS + 1];
    constexpr int P = GR_WARPS + 1;  // (padded: no bank conflicts)
    int *count = sm, *total = sm + P * G, *first = total + G, *start = first + G;  // [G][warps], this CTA's, all, and where it begins
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int ctas = (int)cluster_nctarank(), me = (int)cluster_ctarank();
    for (int i = tid; i < P * G; i += GR_THREADS) count[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int turns = (n + ctas * GR_THREADS - 1) / (ctas * GR_THREADS);  // of 32 ids a warp
    const int i0 = (me * GR_WARPS + warp) * turns * 32 + lane;
    int id[GR_LANE_IDS], rank[GR_LANE_IDS];
#pragma unroll
    for (int t = 0; t < GR_LANE_IDS; ++t) id[t] = t < turns && i0 + 32 * t < n ? ids[i0 + 32 * t] : -1;
#pragma unroll
    for (int t = 0; t < GR_LANE_IDS; ++t) {
        if (t >= turns) break;
        if (id[t] < -1 || id[t] >= G) {
            moe_set_status(status, MOE_ERR_INVALID);
            id[t] = -1;
        }
        const unsigned peers = __match_any_sync(0xffffffffu, id[t]);
        const int before = __popc(peers & ((1u << lane) - 1u));
        int *c = &count[max(id[t], 0) * P + warp];
        rank[t] = id[t] >= 0 ? *c + before : 0;
        __syncwarp();
        if (id[t] >= 0 && before == 0) *c = rank[t] + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int g = warp; g < G; g += GR_WARPS) {  // counts -> the warps' places among the CTA's ids of the group
        const int c = count[g * P + lane];
        int inc = c;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        count[g * P + lane] = inc - c;
        if (lane == 31) total[g] = inc;
    }
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
    // the cluster's counts, and those of the CTAs in front
    for (int g = tid; g < G; g += GR_THREADS) {
        int t = 0, before = 0;
        for (int c = 0; c < ctas; ++c) {
            const int v = ctas > 1 ? __float_as_int(ld_cluster_f32(cluster_map(&total[g], c))) : total[g];
            if (c < me) before += v;
            t += v;
        }
        first[g] = t;
        start[g] = before;
    }
    __syncthreads();
    const int all = group_starts(first, first, G, me == 0 ? offsets : nullptr, sums);
    for (int g = tid; g < G; g += GR_THREADS) start[g] += first[g];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < GR_LANE_IDS; ++t)
        if (id[t] >= 0 && t < turns) rows[start[id[t]] + count[id[t] * P + warp] + rank[t]] = i0 + 32 * t;
    for (int i = all + me * GR_THREADS + tid; i < n; i += ctas * GR_THREADS) rows[i] = -1;
    if (ctas > 1) cluster_sync_all();  // (no CTA leaves while its counts are read)
}

__global__ void __launch_bounds__(GR_THREADS, 1)
    group_count_kernel(const int32_t *ids, int n, int G, int32_t *hist, int *status) {
    extern __shared__ int sm[];
    const int tid = threadIdx.x, warp = tid / 32;
    for (int i = tid; i < GR_WARPS * G; i += GR_THREADS) sm[i] = 0;
    __syncthreads();
    pdl_wait();
    const int seg = (n + (int)gridDim.x * GR_WARPS - 1) / ((int)gridDim.x * GR_WARPS);
    const int i0 = (int)min((long long)n, ((long long)blockIdx.x * GR_WARPS + warp) * seg), i1 = min(n, i0 + seg);
    warp_pass(ids, i0, i1, G, sm + warp * G, nullptr, status);
    __syncthreads();
    for (int g = tid; g < G; g += GR_THREADS) {
        int t = 0;
        for (int w = 0; w < GR_WARPS; ++w) t += sm[w * G + g];
        hist[(size_t)blockIdx.x * G + g] = t;
    }
}

__global__ void __launch_bounds__(GR_THREADS, 1)
    group_place_kernel(const int32_t *ids, int n, int G, const int32_t *hist, int32_t *offsets, int32_t *rows, int *status) {
    extern __shared__ int sm[];
    __shared__ int sums[GR_WARPS + 1];
    int *count = sm, *total = sm + GR_WARPS * G, *first = total + G;
    const int tid = threadIdx.x, warp = tid / 32;
    for (int i = tid; i < GR_WARPS * G; i += GR_THREADS) count[i] = 0;
    __syncthreads();
    pdl_wait();
    const int seg = (n + (int)gridDim.x * GR_WARPS - 1) / ((int)gridDim.x * GR_WARPS);
    const int i0 = (int)min((long long)n, ((long long)blockIdx.x * GR_WARPS + warp) * seg), i1 = min(n, i0 + seg);
    warp_pass(ids, i0, i1, G, count + warp * G, nullptr, nullptr);
    for (int g = tid; g < G; g += GR_THREADS) {
        int t = 0, before = 0;
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int v = hist[(size_t)b * G + g];
            before += b < (int)blockIdx.x ? v : 0;
            t += v;
        }
        total[g] = before;
        first[g] = t;
    }
    __syncthreads();
    const int all = group_starts(first, first, G, blockIdx.x == 0 ? offsets : nullptr, sums);
    __syncthreads();
    for (int g = tid; g < G; g += GR_THREADS) {
        int t = first[g] + total[g];
        for (int w = 0; w < GR_WARPS; ++w) {
            const int c = count[w * G + g];
            count[w * G + g] = t;
            t += c;
        }
    }
    __syncthreads();
    warp_pass(ids, i0, i1, G, count + warp * G, rows, status);
    for (long long i = (long long)all + blockIdx.x * GR_THREADS + tid; i < n; i += (long long)gridDim.x * GR_THREADS)
        rows[i] = -1;
}

int prepare_device() {
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = -1;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
        const int most = (int)table_bytes(MOE_MAX_GROUPS);
        MOE_TRY_CUDA(cudaFuncSetAttribute(group_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)cluster_bytes(MOE_MAX_GROUPS)));
        MOE_TRY_CUDA(cudaFuncSetAttribute(group_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
        MOE_TRY_CUDA(cudaFuncSetAttribute(group_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        MOE_TRY_CUDA(cudaFuncSetAttribute(group_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        done[dev] = true;
    }
    return MOE_OK;
}

int check(int n, int G) {
    MOE_CHECK(n >= 0 && n <= 1 << 24 && G >= 1 && G <= MOE_MAX_GROUPS);
    return MOE_OK;
}

}  // namespace

extern "C" int moe_group_rows_workspace(int n, int G, size_t *bytes) {
    MOE_CHECK(bytes);
    const int rc = check(n, G);
    if (rc != MOE_OK) return rc;
    *bytes = n > GR_CLUSTER_IDS ? (size_t)GR_BLOCKS * G * 4 : 0;
    return MOE_OK;
}

extern "C" int moe_group_rows(const int32_t *ids, int n, int G, int32_t *offsets, int32_t *rows, void *workspace,
                              size_t ws_bytes, moe_stream_t s) {
    size_t need = 0;
    int rc = moe_group_rows_workspace(n, G, &need);
    if (rc != MOE_OK) return rc;
    MOE_CHECK(offsets && (n == 0 || (ids && rows)));
    MOE_CHECK(!need || (workspace && ((uintptr_t)workspace & 3) == 0 && ws_bytes >= need));
    if ((rc = prepare_device()) != MOE_OK) return rc;
    int *status = moe_status_word_device_ptr();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (!need) {
        int ctas = 1;
        while (ctas < GR_MAX_CTAS && (long long)ctas * GR_CTA_IDS < n) ctas *= 2;
        moe_pdl_config(&cfg, attr, dim3(ctas), dim3(GR_THREADS), cluster_bytes(G), moe_cuda_stream(s));
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, group_cluster_kernel, ids, n, G, offsets, rows, status));
        return MOE_OK;
    }
    moe_pdl_config(&cfg, attr, dim3(GR_BLOCKS), dim3(GR_THREADS), (size_t)GR_WARPS * G * 4, moe_cuda_stream(s));
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, group_count_kernel, ids, n, G, (int32_t *)workspace, status));
    moe_pdl_config(&cfg, attr, dim3(GR_BLOCKS), dim3(GR_THREADS), table_bytes(G), moe_cuda_stream(s));
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, group_place_kernel, ids, n, G, (const int32_t *)workspace, offsets, rows, status));
    return MOE_OK;
}
