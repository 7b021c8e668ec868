// Expert selection from router logits (moe_gate): scores by sigmoid or
// softmax, a bias, group-limited top-k, optional truncation, weights.
#pragma once

#include <float.h>

#include "moe_common.cuh"

namespace moe {

struct GateArgs {
    const void* logits;  // [nplanes][T][E], rows ld apart; a row's logits are the planes' sum, added in order
    long long ld, plane;
    int nplanes;
    const float* bias;  // nullptr: none
    int T, E, k;
    int softmax;        // score rule
    int G, gs, keep;    // groups (1: none), experts per group, groups that stay
    int gmax;           // a group counts as its largest value (else the sum of its two largest)
    int raw;            // weights are not renormalised
    float scale, topp;
    int32_t* idx;
    float* w;
};

__device__ __forceinline__ float gate_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float gate_load(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

template <typename LT>
__device__ __forceinline__ float gate_logit(const GateArgs& a, int t, int e) {
    const LT* p = static_cast<const LT*>(a.logits) + (size_t)t * a.ld + e;
    float v = gate_load(p);
    for (int i = 1; i < a.nplanes; ++i) v += gate_load(p + (size_t)i * a.plane);
    return v;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The whole rule for one row by one warp, in double precision: every
// comparison is decided as the definition has it.  sel: E doubles of this
// warp's shared memory.
template <typename LT>
static __device__ void gate_row_f64(const GateArgs& a, int t, double* sel) {
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k;
    float m = -INFINITY;
    double z = 1.0;
    auto fits = [&](int e, float l) { return l > -INFINITY && (!a.bias || __ldg(a.bias + e) > -INFINITY); };  // false for NaN
    if (a.softmax) {
        for (int e = lane; e < E; e += 32) {
            const float l = gate_logit<LT>(a, t, e);
            if (fits(e, l)) m = fmaxf(m, l);
        }
        m = warp_max(m);
        z = 0.0;
        for (int e = lane; e < E; e += 32) {
            const float l = gate_logit<LT>(a, t, e);
            if (fits(e, l)) z += l == m ? 1.0 : exp((double)l - (double)m);  // +inf logits share the mass
        }
        z = warp_sum_f64(z);
    }
    auto score = [&](float l) {
        if (!a.softmax) return 1.0 / (1.0 + exp(-(double)l));
        return (l == m ? 1.0 : exp((double)l - (double)m)) / z;
    };
    for (int e = lane; e < E; e += 32) {
        const float l = gate_logit<LT>(a, t, e);
        double v = -INFINITY;
        if (fits(e, l)) v = a.bias ? score(l) + (double)__ldg(a.bias + e) : (double)l;
        sel[e] = v;
    }
    __syncwarp();
    unsigned stay = kFull;
    if (a.G > 1) {
        double v1 = -INFINITY, v2 = -INFINITY;  // lane g: the two largest of group g
        if (lane < a.G)
            for (int e = lane * a.gs; e < (lane + 1) * a.gs; ++e) {
                double v = sel[e];
                if (!a.bias && v > -INFINITY) v = score((float)v);
                if (v > v1) {
                    v2 = v1;
                    v1 = v;
                } else if (v > v2) {
                    v2 = v;
                }
            }
        const double gv = !a.gmax && v2 > -INFINITY ? v1 + v2 : v1;
        int better = 0;
        for (int g = 0; g < a.G; ++g) {
            const double o = __shfl_sync(kFull, gv, g);
            if (o > gv || (o == gv && g < lane)) ++better;
        }
        stay = __ballot_sync(kFull, lane < a.G && gv > -INFINITY && better < a.keep);
    }
    int my_e = -1;
    for (int j = 0; j < k; ++j) {
        double bv = -INFINITY;
        int be = 0x7fffffff;
        for (int e = lane; e < E; e += 32) {
            const double v = sel[e];
            if (v > bv && (a.G == 1 || (stay >> (e / a.gs)) & 1u)) {
                bv = v;
                be = e;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double ov = __shfl_xor_sync(kFull, bv, o);
            const int oe = __shfl_xor_sync(kFull, be, o);
            if (ov > bv || (ov == bv && oe < be)) {
                bv = ov;
                be = oe;
            }
        }
        if (be == 0x7fffffff) break;  // no expert is left (the same for every lane)
        if (lane == j) my_e = be;
        __syncwarp();
        if (lane == 0) sel[be] = -INFINITY;
        __syncwarp();
    }
    double s = my_e >= 0 ? score(gate_logit<LT>(a, t, my_e)) : 0.0;
    if (a.topp > 0.0f && a.topp < 1.0f) {
        const double whole = (double)a.topp * warp_sum_f64(s);
        double before = 0.0;
        for (int j = 0; j < k - 1; ++j) {
            const double o = __shfl_sync(kFull, s, j);
            if (lane > j) before += o;
        }
        if (lane > 0 && !(before < whole)) {
            my_e = -1;
            s = 0.0;
        }
    }
    const double sum = warp_sum_f64(s);
    if (lane < k) {
        a.idx[(size_t)t * k + lane] = my_e;
        a.w[(size_t)t * k + lane] = (float)((a.raw ? s : sum > 0.0 ? s / sum : 0.0) * (double)a.scale);
    }
}

// One warp per row.  Dynamic shared memory: kWarps * E doubles.
template <typename LT>
__global__ void __launch_bounds__(kThreads) k_gate(const GateArgs a) {
    extern __shared__ double gate_sm[];
    const int warp = threadIdx.x >> 5;
    for (long long t = (long long)blockIdx.x * kWarps + warp; t < a.T; t += (long long)gridDim.x * kWarps) {
        gate_row_f64<LT>(a, (int)t, gate_sm + (size_t)warp * a.E);
        __syncwarp();
    }
}

}  // namespace moe
