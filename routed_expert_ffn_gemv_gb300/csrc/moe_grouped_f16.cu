// The kernels of moe_grouped.cuh with fp16 results.
#include "moe_grouped_launch.cuh"

int grouped_launch_f16(const GroupedParams &p, int mode, bool wide, long long items, int stages, cudaStream_t s) {
    return grouped_launch_modes<MOE_F16>(p, mode, wide, items, stages, s);
}
