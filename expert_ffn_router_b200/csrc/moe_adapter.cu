// moe_adapter, moe_adapter_plan: argument checks and launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <string>
#include <tuple>

#include "moe.h"
#include "moe_adapter.cuh"
#include "moe_launch.h"

namespace moe {

static moe_status check_plan_args(int n_adapters, int T, const void* plan, size_t plan_bytes) {
    if (n_adapters < 1 || n_adapters > kAdMaxN) return fail(MOE_EINVAL, "n_adapters must be in [1, 1024]");
    if (T < 0) return fail(MOE_EINVAL, "T < 0");
    moe_status st = check_ptr(plan, "plan");
    if (st != MOE_OK) return st;
    const size_t need = ad_plan_carve(nullptr, n_adapters, T).bytes;
    if (plan_bytes < need)
        return fail(MOE_ENOSPACE, "plan has " + std::to_string(plan_bytes) + " bytes, needs " + std::to_string(need));
    return MOE_OK;
}

// Bytes a [T][d] array with rows ld elements apart spans.
static size_t span(int T, int d, long long ld, size_t size) { return ((size_t)(T - 1) * (size_t)ld + d) * size; }

static bool overlap(const void* p, size_t np, const void* q, size_t nq) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && a < b + nq && b < a + np;
}

// CTAs of a task's cluster.
static int cluster_size(const AdArgs& g) {
    const int units = std::max(g.d_in / 32, g.d_out / 16);
    return units >= 64 ? 8 : units >= 32 ? 4 : units >= 16 ? 2 : 1;
}

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

template <typename XT, int RT, int MR>
static cudaError_t launch_adapter_t(const AdArgs& g, cudaStream_t s) {
    auto fn = k_adapter<XT, RT, MR>;
    const size_t smem = AdTile<XT, RT, MR>::SMEM;
    cudaError_t e = allow_smem((const void*)fn, smem);
    if (e != cudaSuccess) return e;
    const int cs = cluster_size(g);
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)cs);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    const int tasks = ad_max_tasks(g.n, g.T, AdTile<XT, RT, MR>::LIST);
    c.gridDim.x = (unsigned)(cs * std::min(tasks, resident_clusters((const void*)fn, c, cs)));
    return cudaLaunchKernelEx(&c, fn, g);
}

template <typename XT, int RT>
static cudaError_t launch_adapter_rt(const AdArgs& g, cudaStream_t s) {
    if (g.T < 1024) return launch_adapter_t<XT, RT, 16>(g, s);
    return launch_adapter_t<XT, RT, 64>(g, s);
}

template <typename XT>
static cudaError_t launch_adapter(const AdArgs& g, cudaStream_t s) {
    if (g.r_max <= 16) return launch_adapter_rt<XT, 16>(g, s);
    if (g.r_max <= 32) return launch_adapter_rt<XT, 32>(g, s);
    if (g.r_max <= 64) return launch_adapter_rt<XT, 64>(g, s);
    return launch_adapter_rt<XT, 128>(g, s);
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_plan_bytes(int32_t n_adapters, int32_t max_tokens) {
    if (n_adapters < 1 || n_adapters > kAdMaxN || max_tokens < 0) {
        fail(MOE_EINVAL, "n_adapters must be in [1, 1024] and max_tokens >= 0");
        return 0;
    }
    return ad_plan_carve(nullptr, n_adapters, max_tokens).bytes;
}

moe_status moe_adapter_plan(int32_t n_adapters, const int32_t* adapter_of, int32_t T, void* plan, size_t plan_bytes,
                            moe_stream_t stream) {
    moe_status st = check_plan_args(n_adapters, T, plan, plan_bytes);
    if (st != MOE_OK) return st;
    if (T > 0 && (st = check_ptr(adapter_of, "adapter_of")) != MOE_OK) return st;
    const size_t smem = ad_plan_smem(n_adapters);
    cudaError_t e = allow_smem((const void*)k_adapter_plan, smem);
    if (e == cudaSuccess) {
        k_adapter_plan<<<1, kAdPlanThreads, smem, (cudaStream_t)stream>>>(adapter_of, T, n_adapters,
                                                                          ad_plan_carve(plan, n_adapters, T));
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, std::string("moe_adapter_plan: ") + cudaGetErrorString(e));
}

moe_status moe_adapter(const moe_adapters* ad, void* plan, size_t plan_bytes, const void* x, moe_dtype dtype,
                       const float* sx, int64_t ldx, int32_t T, const float* base, int64_t ldbase, float* y,
                       int64_t ldy, moe_stream_t stream) {
    moe_status st;
    if (!ad) return fail(MOE_EINVAL, "ad is NULL");
    if (ad->r_max < 8 || ad->r_max > kAdMaxRank || ad->r_max % 8)
        return fail(MOE_EINVAL, "r_max must be a multiple of 8 in [8, 128]");
    if (ad->d_in < 16 || ad->d_in > 32768 || ad->d_in % 16 || ad->d_out < 16 || ad->d_out > 32768 || ad->d_out % 16)
        return fail(MOE_EINVAL, "d_in and d_out must be multiples of 16 in [16, 32768]");
    if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_I8)
        return fail(MOE_EINVAL, "dtype must be MOE_F32, MOE_BF16 or MOE_I8");
    if ((dtype == MOE_I8) != (sx != nullptr)) return fail(MOE_EINVAL, "sx goes with MOE_I8 rows, and only with them");
    if ((st = check_plan_args(ad->n_adapters, T, plan, plan_bytes)) != MOE_OK) return st;
    const size_t size = dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 1;
    if (ldx < ad->d_in || (ldx * size) % 16)
        return fail(MOE_EINVAL, "ldx must be >= d_in and keep rows on 16 bytes");
    if (ldy < ad->d_out || ldy % 4 || (base && (ldbase < ad->d_out || ldbase % 4)))
        return fail(MOE_EINVAL, "ldy and ldbase must be >= d_out and multiples of 4");
    if (T == 0) return MOE_OK;
    if ((st = check_ptr(ad->a, "ad->a")) != MOE_OK) return st;
    if ((st = check_ptr(ad->b, "ad->b")) != MOE_OK) return st;
    if ((st = check_ptr(ad->rank, "ad->rank", true)) != MOE_OK) return st;
    if ((st = check_ptr(ad->scale, "ad->scale", true)) != MOE_OK) return st;
    if ((st = check_ptr(x, "x")) != MOE_OK) return st;
    if ((st = check_ptr(sx, "sx", true)) != MOE_OK) return st;
    if ((st = check_ptr(base, "base", true)) != MOE_OK) return st;
    if ((st = check_ptr(y, "y")) != MOE_OK) return st;
    const size_t ny = span(T, ad->d_out, ldy, 4), nab = (size_t)ad->n_adapters * ad->r_max * 2;
    const bool in_place = base == y;
    if (in_place && ldbase != ldy) return fail(MOE_EINVAL, "base is y, but ldbase is not ldy");
    if ((!in_place && overlap(y, ny, base, span(T, ad->d_out, ldbase, 4))) ||
        overlap(y, ny, x, span(T, ad->d_in, ldx, size)) || overlap(y, ny, sx, (size_t)T * 4) ||
        overlap(y, ny, ad->a, nab * ad->d_in) || overlap(y, ny, ad->b, nab * ad->d_out) ||
        overlap(y, ny, ad->rank, (size_t)ad->n_adapters * 4) || overlap(y, ny, ad->scale, (size_t)ad->n_adapters * 4) ||
        overlap(y, ny, plan, plan_bytes))
        return fail(MOE_EINVAL, "y overlaps an input");
    AdArgs g{};
    g.a = static_cast<const __nv_bfloat16*>(ad->a);
    g.b = static_cast<const __nv_bfloat16*>(ad->b);
    g.rank = ad->rank;
    g.scale = ad->scale;
    g.n = ad->n_adapters;
    g.r_max = ad->r_max;
    g.d_in = ad->d_in;
    g.d_out = ad->d_out;
    g.T = T;
    g.plan = ad_plan_carve(plan, g.n, T);
    g.x = x;
    g.sx = sx;
    g.ldx = ldx;
    g.base = base;
    g.ldbase = ldbase;
    g.y = y;
    g.ldy = ldy;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == MOE_F32    ? launch_adapter<float>(g, s)
                          : dtype == MOE_BF16 ? launch_adapter<__nv_bfloat16>(g, s)
                                              : launch_adapter<int8_t>(g, s);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, std::string("moe_adapter: ") + cudaGetErrorString(e));
}

}  // extern "C"
