// Launch of the adapter kernels (host side): clusters that take tasks.
#pragma once

#include <cuda_runtime.h>

#include "moe_adapter.cuh"
#include "moe_launch.h"

namespace moe {

struct AdLaunch {
    cudaLaunchConfig_t c;
    cudaLaunchAttribute at[1];
};

// Fills in l (grid, clusters, shared memory) and g->max_tasks for a kernel that
// takes the tasks of `list`.
void ad_launch(AdLaunch* l, AdArgs* g, const void* fn, int list, int threads, size_t smem, cudaStream_t s);

cudaError_t launch_adapter_few(const AdArgs& g, moe_dtype dtype, cudaStream_t s);

}  // namespace moe
