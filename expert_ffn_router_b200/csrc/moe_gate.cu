// moe_gate: argument checks and launch of the expert selection.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "moe.h"
#include "moe_gate.cuh"
#include "moe_launch.h"

namespace moe {

moe_status check_rule(const moe_config* c, const moe_gate_rule* r) {
    if (!r) return fail(MOE_EINVAL, "rule is NULL");
    if (r->score != MOE_SCORE_SIGMOID && r->score != MOE_SCORE_SOFTMAX)
        return fail(MOE_EINVAL, "rule->score must be MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX");
    if (r->raw_weights != 0 && r->raw_weights != 1) return fail(MOE_EINVAL, "rule->raw_weights must be 0 or 1");
    if (r->n_groups < 0 || r->n_groups > 32) return fail(MOE_EINVAL, "rule->n_groups must be in [0, 32]");
    if (r->n_groups <= 1) return MOE_OK;
    if (c->n_experts % r->n_groups) return fail(MOE_EINVAL, "rule->n_groups must divide n_experts");
    if (r->topk_groups < 1 || r->topk_groups > r->n_groups)
        return fail(MOE_EINVAL, "rule->topk_groups must be in [1, n_groups]");
    if (r->group_value != MOE_GROUP_TOP2 && r->group_value != MOE_GROUP_MAX)
        return fail(MOE_EINVAL, "rule->group_value must be MOE_GROUP_TOP2 or MOE_GROUP_MAX");
    if (c->top_k > r->topk_groups * (c->n_experts / r->n_groups))
        return fail(MOE_EINVAL, "top_k exceeds the experts of topk_groups groups");
    return MOE_OK;
}

template <typename LT, int NPL, bool VEC>
static cudaError_t launch_gate_t(const GateArgs& a, cudaStream_t s) {
    const void* fn = (const void*)k_gate<LT, NPL, VEC>;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // a warp a row: CTAs of 8 warps, smaller ones while that leaves SMs without any
    const int warps = std::max(1, std::min(kWarps, a.T / sms));
    const size_t smem = (size_t)warps * gate_smem(a.E, NPL);
    const cudaError_t e = allow_smem(fn, (size_t)kWarps * gate_smem(a.E, NPL));
    if (e != cudaSuccess) return e;
    const int grid = std::min((a.T + warps - 1) / warps, persistent_grid(fn, smem, warps * 32));
    k_gate<LT, NPL, VEC><<<grid, warps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename LT, bool VEC>
static cudaError_t launch_gate_v(const GateArgs& a, cudaStream_t s) {
    if constexpr (!VEC) {
        if (a.E <= 32) return launch_gate_t<LT, 1, false>(a, s);
        if (a.E <= 64) return launch_gate_t<LT, 2, false>(a, s);
    }
    if (a.E <= 128) return launch_gate_t<LT, 4, VEC>(a, s);
    if (a.E <= 256) return launch_gate_t<LT, 8, VEC>(a, s);
    if (a.E <= 512) return launch_gate_t<LT, 16, VEC>(a, s);
    return launch_gate_t<LT, 32, VEC>(a, s);
}

template <typename LT>
static cudaError_t launch_gate_l(const GateArgs& a, cudaStream_t s) {
    // four neighbours at a time where every row (and plane) starts on them
    const bool vec = a.E > 64 && a.E % 4 == 0 && a.ld % 4 == 0 && a.plane % 4 == 0 &&
                     (uintptr_t)a.logits % (4 * sizeof(LT)) == 0;
    return vec ? launch_gate_v<LT, true>(a, s) : launch_gate_v<LT, false>(a, s);
}

cudaError_t launch_gate(const moe_config* c, const moe_gate_rule* r, const void* logits, moe_dtype dt, long long ld,
                        int nplanes, long long plane, int T, const float* bias, int32_t* idx, float* w,
                        cudaStream_t s) {
    GateArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.plane = plane;
    a.nplanes = nplanes;
    a.bias = bias;
    a.T = T;
    a.E = c->n_experts;
    a.k = c->top_k;
    a.softmax = r->score == MOE_SCORE_SOFTMAX;
    a.G = std::max(1, (int)r->n_groups);
    a.gs = a.E / a.G;
    a.keep = a.G > 1 ? r->topk_groups : 1;
    a.gmax = r->group_value == MOE_GROUP_MAX;
    a.raw = r->raw_weights;
    a.scale = c->routed_scale;
    a.topp = c->topp;
    a.idx = idx;
    a.w = w;
    return dt == MOE_BF16 ? launch_gate_l<__nv_bfloat16>(a, s) : launch_gate_l<float>(a, s);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_gate(const moe_config* cfg, const moe_gate_rule* rule, const void* logits, moe_dtype dtype,
                               int64_t ld, int32_t T, const float* bias, int32_t* topk_idx, float* topk_w,
                               moe_stream_t stream) try {
    moe_status st = check_selection(cfg);
    if (st != MOE_OK) return st;
    if ((st = check_rule(cfg, rule)) != MOE_OK) return st;
    if ((st = check_dtype(dtype)) != MOE_OK) return st;
    if (T < 0) return fail(MOE_EINVAL, "T < 0");
    if (ld < cfg->n_experts) return fail(MOE_EINVAL, "ld is smaller than n_experts");
    if (T == 0) return MOE_OK;
    if (!logits) return fail(MOE_EINVAL, "logits is NULL");
    if ((uintptr_t)logits % (dtype == MOE_BF16 ? 2 : 4)) return fail(MOE_EALIGN, "logits is not aligned to its elements");
    if ((st = check_ptr(bias, "bias", true)) != MOE_OK) return st;
    if ((st = check_ptr(topk_idx, "topk_idx")) != MOE_OK) return st;
    if ((st = check_ptr(topk_w, "topk_w")) != MOE_OK) return st;
    const cudaError_t e = launch_gate(cfg, rule, logits, dtype, ld, 1, 0, T, bias, topk_idx, topk_w,
                                      (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, std::string("moe_gate: ") + cudaGetErrorString(e));
} catch (...) {  // (out of host memory)
    return MOE_ECUDA;
}
