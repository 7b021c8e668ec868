// Launches of the adapter kernel for few rows, and what the launches of both
// adapter kernels share.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "moe_adapter_few.cuh"
#include "moe_adapter_launch.h"

namespace moe {

// Clusters of cs CTAs that the device holds at once (cached per kernel).
static int resident_clusters(const void* fn, const cudaLaunchConfig_t& c, int cs) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int>, int> known;
    int dev = 0;
    cudaGetDevice(&dev);
    const auto key = std::make_tuple(dev, fn, cs);
    std::lock_guard<std::mutex> lk(mu);
    auto it = known.find(key);
    if (it != known.end()) return it->second;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &c) != cudaSuccess || n < 1) return 1;
    known[key] = n;
    return n;
}

// The tasks of a batch.  Adapters without a row have none, and the host does not
// know them: their number is estimated as if every row had drawn its adapter,
// with a last task half full.  (A batch that uses few adapters of a large table
// is taken for more tasks than it has, and gets smaller clusters: 2048 bf16 rows
// in runs of 16 adapters take k_adapter 64 us with a table of 64, 110 with 256.)
static double tasks_of(const AdArgs& g, int list) {
    const double classes = g.n + 1, used = classes * (1.0 - std::exp(-g.T / classes));
    return used * std::max(1.0, g.T / used / ad_rows(list) + 0.5);
}

void ad_launch(AdLaunch* l, AdArgs* g, const void* fn, int list, int threads, size_t smem, cudaStream_t s) {
    g->max_tasks = ad_max_tasks(g->n, g->T, list);
    l->c = cudaLaunchConfig_t{};
    l->c.blockDim = dim3((unsigned)threads);
    l->c.dynamicSmemBytes = smem;
    l->c.stream = s;
    l->at[0].id = cudaLaunchAttributeClusterDimension;
    l->at[0].val.clusterDim.y = 1;
    l->at[0].val.clusterDim.z = 1;
    l->c.attrs = l->at;
    l->c.numAttrs = 1;
    // CTAs of a cluster: the batch takes its rounds of tasks over the clusters
    // that the device holds at once, a round a task's time by the cluster's size
    // and some that does not shrink with it (start, meeting: 0.15 of a task on
    // one CTA).  No cluster leaves a CTA without a few shares of the products.
    // Measured at d = 6144 with clusters of 1, 2, 4 and 8 (k_adapter_few, rank 16,
    // us): 128 rows of 5 adapters 32, 19, 13, 10.7; 768 rows 33, 23, 19, 25; 4096
    // rows 76, 66, 79, 100.
    const int units = std::max(g->d_in / 64, g->d_out / 64);
    const double tasks = tasks_of(*g, list);
    double best = 0.0;
    int cs = 1, held = 1;
    for (int c = 1; c <= 8 && (c == 1 || c * 4 <= units); c *= 2) {
        l->c.gridDim = dim3((unsigned)c);
        l->at[0].val.clusterDim.x = (unsigned)c;
        const int n = resident_clusters(fn, l->c, c);
        const double cost = std::ceil(tasks / n) * (1.0 / c + 0.15);
        if (c == 1 || cost < best) {
            best = cost;
            cs = c;
            held = n;
        }
    }
    l->at[0].val.clusterDim.x = (unsigned)cs;
    l->c.gridDim = dim3((unsigned)(cs * std::min(g->max_tasks, held)));
}

template <typename XT, int RT>
static cudaError_t launch_t(AdArgs g, cudaStream_t s) {
    using Tile = AfTile<XT, RT>;
    auto fn = k_adapter_few<XT, RT>;
    const cudaError_t e = allow_smem((const void*)fn, Tile::SMEM);
    if (e != cudaSuccess) return e;
    AdLaunch l;
    ad_launch(&l, &g, (const void*)fn, Tile::LIST, (Tile::NW + Tile::NP) * 32, Tile::SMEM, s);
    return cudaLaunchKernelEx(&l.c, fn, g);
}

template <typename XT>
static cudaError_t launch_few(const AdArgs& g, cudaStream_t s) {
    if (g.r_max <= 16) return launch_t<XT, 16>(g, s);
    if (g.r_max <= 32) return launch_t<XT, 32>(g, s);
    if (g.r_max <= 64) return launch_t<XT, 64>(g, s);
    return launch_t<XT, 128>(g, s);
}

cudaError_t launch_adapter_few(const AdArgs& g, moe_dtype dtype, cudaStream_t s) {
    return dtype == MOE_F32 ? launch_few<float>(g, s)
           : dtype == MOE_BF16 ? launch_few<__nv_bfloat16>(g, s)
                               : launch_few<int8_t>(g, s);
}

}  // namespace moe
