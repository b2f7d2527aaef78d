// Launches of the kernel in moe_grouped.cuh, for the translation units of its three y types.
#pragma once

#include <algorithm>
#include <mutex>

#include "moe_grouped.cuh"

template <int CG, int NT, int MODE, int OT>
static int grouped_launch_t(const GroupedParams &p, long long items, int stages, cudaStream_t s) {
    using G = GroupedGeom<CG, NT, OT>;
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = -1;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            MOE_TRY_CUDA(cudaFuncSetAttribute(grouped_kernel<CG, NT, MODE, OT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)G::SMEM));
            ready[dev] = true;
        }
    }
    const int n = std::max(CG, grouped_sms());
    items = std::max(1LL, items);
    int cluster = CG;
    // CG = 1: as many CTAs to an item as there are SMs for, each with four stages of the reduction at least
    if (CG == 1)
        while (cluster < GP_MAX_SPLIT && items * (cluster + 1) <= n && (cluster + 1) * 4 <= stages) ++cluster;
    const long long units = std::min<long long>(items, n / cluster);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    moe_pdl_config(&cfg, attr, dim3((unsigned)(units * cluster)), dim3(GP_THREADS), G::SMEM, s);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, grouped_kernel<CG, NT, MODE, OT>, p));
    return MOE_OK;
}

// Pairs: tiles of 256 rows; of 128 with fp32 results, so that tensor memory holds four accumulators.
template <int OT>
static int grouped_launch_modes(const GroupedParams &p, int mode, bool wide, long long items, int stages, cudaStream_t s) {
    constexpr int WIDE = OT == MOE_F32 ? 128 : 256;
    switch (mode) {
        case GP_NK:
            return wide ? grouped_launch_t<2, WIDE, GP_NK, OT>(p, items, stages, s)
                        : grouped_launch_t<1, 32, GP_NK, OT>(p, items, stages, s);
        case GP_KN:
            return wide ? grouped_launch_t<2, WIDE, GP_KN, OT>(p, items, stages, s)
                        : grouped_launch_t<1, 32, GP_KN, OT>(p, items, stages, s);
        case GP_SWIGLU:
            return wide ? grouped_launch_t<2, WIDE, GP_SWIGLU, OT>(p, items, stages, s)
                        : grouped_launch_t<1, 32, GP_SWIGLU, OT>(p, items, stages, s);
        case GP_LORA:
            return wide ? grouped_launch_t<2, WIDE, GP_LORA, OT>(p, items, stages, s)
                        : grouped_launch_t<1, 32, GP_LORA, OT>(p, items, stages, s);
        case GP_LORA_F16:
            return wide ? grouped_launch_t<2, WIDE, GP_LORA_F16, OT>(p, items, stages, s)
                        : grouped_launch_t<1, 32, GP_LORA_F16, OT>(p, items, stages, s);
        default:
            // fp32: tiles of 128, for four accumulators instead of two, with long reductions only (128 groups of 256 rows, 1536 x 2048: 403 us
            // against 331)
            if (OT == MOE_F32 && !grouped_grad_short(p.R, p.G)) return grouped_launch_t<2, WIDE, GP_GRAD, OT>(p, items, stages, s);
            return grouped_launch_t<2, 256, GP_GRAD, OT>(p, items, stages, s);
    }
}
