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

// The largest of a warp's floats (none of them NaN).
__device__ __forceinline__ float gate_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + exp(-l)) within 3e-7 of it: 2^x within 2^-22, by s (1 - s) <= 1/4;
// the sum 2^-24; the reciprocal 2^-23.
__device__ __forceinline__ float gate_sigmoid(float l) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
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
static __device__ __noinline__ void gate_row_f64(const GateArgs& a, int t, double* sel) {
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
        a.w[(size_t)t * k + lane] = my_e < 0 ? 0.0f : (float)((a.raw ? s : sum > 0.0 ? s / sum : 0.0) * (double)a.scale);
    }
}

// ---------------------------------------------------------------------------
// The same in float32 where that decides, one warp per row.
//
// Scores and selection values are computed with fast float32 functions, whose
// error is bounded by `eps`; the values of a row are mapped onto a fixed-point
// scale of its own range, and value and index (complemented: the lower index
// is the larger key) share a 32-bit key, so a round of the top-k is one
// warp-wide integer maximum over the lanes' heads.  A lane sorts its values
// once (a network) and gives them up one by one.  Where two neighbours of the
// k largest and those that may belong to them, or the last group that stays and
// the first that does not, are nearer than their errors allow to tell -- and the
// experts' logits and biases are not the same, in which case the index decides --
// these alone are compared in double precision (with 256 sigmoids in one row of
// 300).  Rows with infinite values or scores near underflow are done again by
// gate_row_f64: that takes some 20 us, a warp to itself.
//
// Lane l holds the experts (i / V) * 32 V + l V + i % V, V = min(NPL, 4), so
// that it reads 16 (bf16: 8) bytes at a time where rows allow it (VEC).
//
// Bound by the instructions a row takes, not by its bytes: 1090 for 256 experts
// in 8 groups, 8 selected (ncu, 66% of the issue slots): 65536 such rows in
// 99 us, 0.72 TB/s against 6.55 of a copy, where every row in double precision
// took 426.  1024 experts, 32 selected: 4096 rows in 35 us (double 107).  One
// row: 4.0 us, the launch and a chain of some thirty dependent steps.
//
// Without a bias the scale is that of the logits, so a finite mask value far below
// them takes all of it: the others share few keys and go to double precision.
// 65536 rows of 256, a quarter masked: 71 us with -inf or -30, 98 with -1e4, 420
// to 500 with -1e9 or the type's lowest value.
// ---------------------------------------------------------------------------
// Descending: odd-even merge sort, the places known to the compiler.
template <int N, int P, int K>
__device__ __forceinline__ void gate_merge(unsigned (&v)[N]) {
#pragma unroll
    for (int x = 0; x < N - K; ++x)
        if (x >= K % P && ((x - K % P) / K) % 2 == 0 && x / (2 * P) == (x + K) / (2 * P)) {
            const unsigned a = v[x], b = v[x + K];
            v[x] = max(a, b);
            v[x + K] = min(a, b);
        }
    if constexpr (K > 1) gate_merge<N, P, K / 2>(v);
}
template <int N, int P = 1>
__device__ __forceinline__ void gate_sort(unsigned (&v)[N]) {
    if constexpr (P < N) {
        gate_merge<N, P, P>(v);
        gate_sort<N, P * 2>(v);
    }
}

template <typename LT, int NPL, bool VEC>
__device__ __forceinline__ void gate_load_row(const GateArgs& a, int t, float (&l)[NPL]) {
    constexpr int V = NPL < 4 ? NPL : 4;
    const int lane = threadIdx.x & 31;
    const LT* row = static_cast<const LT*>(a.logits) + (size_t)t * a.ld;
    for (int p = 0; p < a.nplanes; ++p, row += a.plane) {
#pragma unroll
        for (int i = 0; i < NPL; i += V) {
            const int e = i * 32 + lane * V;
            float v[V];
            if (VEC) {
                if (e < a.E) {
                    if constexpr (sizeof(LT) == 4) {
                        const float4 x = ld_stream_f4(row + e);
                        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                    } else {
                        const uint2 x = __ldg(reinterpret_cast<const uint2*>(row + e));
                        v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
                        v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = -INFINITY;
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = e + j < a.E ? gate_load(row + e + j) : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) l[i + j] = p ? l[i + j] + v[j] : v[j];
        }
    }
}

// Shared memory of a warp: E doubles and 32 for the groups' distance (before and
// after that float32 values and sorted keys in the same place).
__host__ __device__ constexpr int gate_smem(int E, int npl) {
    return ((E + 32) * 8 > npl * 128 + 128 ? (E + 32) * 8 : npl * 128 + 128) / 16 * 16 + 16;
}

// Which groups stay: bit g L of the result for group g, whose values lie at
// v[g (gs + L)] on.  lo, hi (float only): the smallest value of those that stay,
// the largest of the others.
template <typename T>
__device__ __forceinline__ unsigned gate_groups(const GateArgs& a, int L, const T* v, T& lo, T& hi) {
    const int lane = threadIdx.x & 31, g = lane / L, sub = lane % L;
    const T none = -INFINITY;
    T v1 = none, v2 = none;
    if (g < a.G)
#pragma unroll 4
        for (int i = sub; i < a.gs; i += L) {
            const T x = v[g * (a.gs + L) + i];
            if constexpr (sizeof(T) == 4) {
                v2 = fmaxf(v2, fminf(v1, x));
                v1 = fmaxf(v1, x);
            } else if (x > v1) {
                v2 = v1;
                v1 = x;
            } else if (x > v2) {
                v2 = x;
            }
        }
    for (int o = 1; o < L; o *= 2) {
        const T x1 = __shfl_xor_sync(kFull, v1, o), x2 = __shfl_xor_sync(kFull, v2, o);
        const T small = x1 < v1 ? x1 : v1, big = x1 < v1 ? v1 : x1, rest = x2 < v2 ? v2 : x2;
        v1 = big;
        v2 = small < rest ? rest : small;
    }
    const T gv = !a.gmax && v2 > none ? v1 + v2 : v1;
    int better = 0;
#pragma unroll 4
    for (int j = 0; j < a.G; ++j) {
        const T x = __shfl_sync(kFull, gv, j * L);
        better += x > gv || (x == gv && j < g);
    }
    const bool in = g < a.G && gv > none && better < a.keep;
    if constexpr (sizeof(T) == 4) {
        lo = -gate_max(in ? -gv : none);
        hi = gate_max(g < a.G && !in ? gv : none);
    }
    return __ballot_sync(kFull, in);
}

__device__ __forceinline__ double gate_score_f64(float l, float m, double z, int softmax) {
    return softmax ? exp((double)l - (double)m) / z : 1.0 / (1.0 + exp(-(double)l));
}
// Sum of the exponentials of a row (softmax; 1 otherwise), in double.
template <typename LT>
static __device__ __noinline__ double gate_sum_f64(const GateArgs& a, int t, float m) {
    if (!a.softmax) return 1.0;
    double z = 0.0;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float l = gate_logit<LT>(a, t, e);
        if (l > -INFINITY && (!a.bias || __ldg(a.bias + e) > -INFINITY)) z += exp((double)l - (double)m);
    }
    return warp_sum_f64(z);
}
// The groups of a row in double precision.
template <typename LT>
static __device__ __noinline__ unsigned gate_groups_f64(const GateArgs& a, int t, float m, int L, double* v) {
    const double z = gate_sum_f64<LT>(a, t, m);
#pragma unroll 4
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float l = gate_logit<LT>(a, t, e), b = a.bias ? __ldg(a.bias + e) : 0.0f;
        v[e + e / a.gs * L] = l > -INFINITY && b > -INFINITY ? gate_score_f64(l, m, z, a.softmax) + (double)b : -INFINITY;
    }
    __syncwarp();
    double lo, hi;
    const unsigned stay = gate_groups<double>(a, L, v, lo, hi);
    __syncwarp();
    return stay;
}
// c <= 64 experts (e0 of lane i the i-th, e1 the 32 + i-th) in the rule's order, by
// their values in double precision: the first 32 of them, one a lane.
template <typename LT>
static __device__ __noinline__ int gate_order_f64(const GateArgs& a, int t, float m, int c, int e0, int e1) {
    const int lane = threadIdx.x & 31;
    const double z = a.bias ? gate_sum_f64<LT>(a, t, m) : 1.0;
    auto value = [&](int e) {
        const float l = gate_logit<LT>(a, t, e);
        return a.bias ? gate_score_f64(l, m, z, a.softmax) + (double)__ldg(a.bias + e) : (double)l;
    };
    const double v0 = lane < c ? value(e0) : -INFINITY, v1 = lane + 32 < c ? value(e1) : -INFINITY;
    int r0 = 0, r1 = 0;
    for (int j = 0; j < c; ++j) {
        const double x = __shfl_sync(kFull, j < 32 ? v0 : v1, j & 31);
        const int o = __shfl_sync(kFull, j < 32 ? e0 : e1, j & 31);
        r0 += x > v0 || (x == v0 && o < e0);
        r1 += x > v1 || (x == v1 && o < e1);
    }
    int out = -1;
    for (int j = 0; j < c; ++j) {  // lane rank takes the j-th
        const int to = __shfl_sync(kFull, j < 32 ? r0 : r1, j & 31), o = __shfl_sync(kFull, j < 32 ? e0 : e1, j & 31);
        if (lane == to) out = o;
    }
    return out;
}

template <typename LT, int NPL, bool VEC>
__global__ void __launch_bounds__(kThreads, NPL <= 4 ? 4 : NPL == 8 ? 3 : 2) k_gate(const __grid_constant__ GateArgs a) {
    constexpr int V = NPL < 4 ? NPL : 4;
    constexpr int IB = NPL == 1 ? 5 : NPL == 2 ? 6 : NPL == 4 ? 7 : NPL == 8 ? 8 : NPL == 16 ? 9 : 10;  // index bits
    constexpr int VB = 31 - IB < 23 ? 31 - IB : 23;                                                    // value bits
    constexpr unsigned IM = (1u << IB) - 1;
    extern __shared__ double gate_sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    double* sel = reinterpret_cast<double*>(reinterpret_cast<uint8_t*>(gate_sm) + (size_t)warp * gate_smem(a.E, NPL));
    float* fs = reinterpret_cast<float*>(sel);
    unsigned* us = reinterpret_cast<unsigned*>(sel);
    const int k = a.k, G = a.G;
    // groups: L lanes share one; a group's values lie L words apart from the next one's, other banks
    int L = 1;
    while (L * 2 * G <= 32) L *= 2;
    float b[NPL];
    int pos[NPL];      // place among the groups' values in shared memory
    unsigned gbit[NPL];  // its group's bit, 0 behind the last expert
    bool b_out = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i / V * 32 * V + lane * V + i % V;
        b[i] = a.bias && e < a.E ? fmaxf(__ldg(a.bias + e), -INFINITY) : 0.0f;  // NaN: -inf
        const int g = G > 1 && e < a.E ? e / a.gs : 0;
        pos[i] = e < a.E ? e + g * L : a.E + 32;  // (a place that nobody reads)
        gbit[i] = e < a.E ? 1u << (g * L) : 0u;
        b_out |= b[i] == -INFINITY;
    }
    b_out = __any_sync(kFull, b_out);
    for (long long t0 = (long long)blockIdx.x * warps + warp; t0 < a.T; t0 += (long long)gridDim.x * warps) {
        const int t = (int)t0;
        float l[NPL], v[NPL];
        gate_load_row<LT, NPL, VEC>(a, t, l);
        float m = -INFINITY, z = 1.0f, eps = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            l[i] = fmaxf(l[i], -INFINITY);  // NaN: -inf
            if (b_out && b[i] == -INFINITY) l[i] = -INFINITY;
        }
        bool redo = false;
        if (a.softmax) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) m = fmaxf(m, l[i]);
            m = gate_max(m);
            redo = m == INFINITY;
        }
        if (a.softmax && (a.bias || a.raw || G > 1)) {
            float e_sum = 0.0f;
            if (a.raw) {
#pragma unroll
                for (int i = 0; i < NPL; ++i) e_sum += v[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
            } else {
#pragma unroll
                for (int i = 0; i < NPL; ++i) e_sum += v[i] = l[i] > -INFINITY ? __expf(l[i] - m) : 0.0f;
            }
            z = warp_sum(e_sum);
            const float rz = __frcp_rn(z);
#pragma unroll
            for (int i = 0; i < NPL; ++i) v[i] = __fmul_rn(v[i], rz);  // (not fused: the border's search has it again)
            eps = 4e-6f * rz;  // of the largest score: exponential and sum, 32 roundings of 2^-23
        } else if (!a.softmax && (a.bias || G > 1)) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) v[i] = gate_sigmoid(l[i]);
            eps = 4e-7f;
        }
        // selection values (and the scores plus bias that groups count by)
        float top = -INFINITY, bot = INFINITY, widest = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (a.bias) v[i] = __fadd_rn(v[i], b[i]);
            if (G > 1) widest = fmaxf(widest, l[i] > -INFINITY ? fabsf(v[i]) : 0.0f);
            if (G > 1) {
                fs[pos[i]] = l[i] > -INFINITY ? v[i] : -INFINITY;
            }
        }
        unsigned stay = kFull;
        if (G > 1) {
            __syncwarp();
            float lo, hi;
            stay = gate_groups<float>(a, L, fs, lo, hi);
            __syncwarp();
            widest = gate_max(widest);
            redo |= !(widest < 1e37f);  // a sum of two might leave float32
            // two sums of two values each, six roundings of at most 2^-24 of twice the widest value
            if (hi > -INFINITY && !(lo - hi > 4.0f * eps + 1e-6f * widest) && !redo)
                stay = gate_groups_f64<LT>(a, t, m, L, sel);
        }
        if (!a.bias) {  // by the logits themselves, which are exact
            eps = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) v[i] = l[i];
        }
        unsigned key[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const bool in = l[i] > -INFINITY && (stay & gbit[i]);
            key[i] = in;
            top = fmaxf(top, in ? v[i] : -INFINITY);
            bot = fminf(bot, in ? v[i] : INFINITY);
        }
        top = gate_max(top);
        bot = -gate_max(-bot);
        const float range = top - bot;
        redo |= top > bot && !(range < 1e37f);  // infinite, or nearly
        const float inv = range > 0.0f && range < 1e37f ? 0.9999990f / range : 0.0f;
        const float off = fmaxf(fabsf(top), fabsf(bot));
        // the distance that tells two values apart: both errors, the value's own rounding, and the scale's
        const float tol_f = (2.0f * eps + (a.bias ? 2.5e-7f * off : 0.0f)) * inv * (float)(1 << VB) + 4.0f;
        const unsigned tol = tol_f < 1e9f ? (unsigned)tol_f : 1000000000u;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i / V * 32 * V + lane * V + i % V;
            const unsigned f = __float_as_uint(fmaf(v[i] - bot, inv, 1.0f)) & 0x7fffffu;  // [1, 2): the mantissa
            key[i] = key[i] ? 0x80000000u | (f >> (23 - VB)) << IB | (IM - (unsigned)e) : 0u;
        }
        if (NPL > 1) gate_sort<NPL>(key);
        // the lane's keys one by one: head, then next, read ahead; zeros behind the last
        unsigned head = key[0], mine = 0u, mine2 = 0u;
        if (NPL > 1) {
#pragma unroll
            for (int i = 1; i < NPL; ++i) us[i * 32 + lane] = key[i];
        }
        us[NPL * 32 + lane] = 0u;
        const unsigned* next_at = us + 32 + lane;
        unsigned next = NPL > 1 ? key[NPL > 1 ? 1 : 0] : 0u;
        __syncwarp();
        auto give = [&](unsigned mx) {
            const bool own = head == mx;
            head = own ? next : head;
            next_at += own && next ? 32 : 0;
            next = *next_at;
        };
        unsigned mx = __reduce_max_sync(kFull, head);
#pragma unroll 2
        for (int j = 0; j < k; ++j) {  // (zeros, once no expert is left)
            mine = lane == j ? mx : mine;
            give(mx);
            mx = __reduce_max_sync(kFull, head);
        }
        // candidates: the i-th in lane i's `mine`, the 32 + i-th in its `mine2`
        int c = __popc(__ballot_sync(kFull, mine != 0u));
        const unsigned kth = __shfl_sync(kFull, mine, k - 1);
        int e_mine = mine ? (int)(IM - (mine & IM)) : -1;
        float l_mine = e_mine >= 0 ? gate_logit<LT>(a, t, e_mine) : 0.0f;
        const float b_mine = a.bias && e_mine >= 0 ? __ldg(a.bias + e_mine) : 0.0f;
        const unsigned near = __shfl_down_sync(kFull, mine, 1);
        const float l_nx = __shfl_down_sync(kFull, l_mine, 1), b_nx = __shfl_down_sync(kFull, b_mine, 1);
        // neighbours that the keys do not tell apart
        bool unsure = __any_sync(kFull, lane < c - 1 && (mine >> IB) - (near >> IB) <= tol &&
                                            !(l_mine == l_nx && b_mine == b_nx));
        if (c == k && mx && (kth >> IB) - (mx >> IB) <= tol) {
            // others may belong to the k: those not clearly below the last of them that are not its equals (or that
            // are, if the order of the k is not sure).  All experts above that line are counted, their values computed
            // again, operation by operation; more than stand among the k, and the others are to be compared.
            const float l_k = __shfl_sync(kFull, l_mine, k - 1), b_k = __shfl_sync(kFull, b_mine, k - 1);
            const unsigned last = kth;
            int above = 0;
#pragma unroll 1
            for (int e = lane; e < a.E && !unsure; e += 32) {
                const float le = fmaxf(gate_logit<LT>(a, t, e), -INFINITY), be = a.bias ? __ldg(a.bias + e) : 0.0f;
                if (!(le > -INFINITY && be > -INFINITY) || (le == l_k && be == b_k)) continue;
                if (G > 1 && !((stay >> (e / a.gs * L)) & 1u)) continue;
                float ve = le;
                if (a.bias)
                    ve = __fadd_rn(a.softmax ? __fmul_rn(a.raw ? expf(le - m) : __expf(le - m), __frcp_rn(z))
                                             : gate_sigmoid(le), be);
                const unsigned f = (__float_as_uint(fmaf(ve - bot, inv, 1.0f)) & 0x7fffffu) >> (23 - VB);
                above += (0x80000000u >> IB | f) + tol + 2u >= last >> IB;
            }
            const int among = __popc(__ballot_sync(kFull, lane < k && !(l_mine == l_k && b_mine == b_k)));
            if (unsure || __reduce_add_sync(kFull, above) > among) {
                unsure = true;
                while (mx && (last >> IB) - (mx >> IB) <= tol) {
                    if (c == 64) {
                        redo = true;  // more candidates than two a lane
                        break;
                    }
                    if (lane == c) mine = mx;
                    if (lane + 32 == c) mine2 = mx;
                    give(mx);
                    ++c;
                    mx = __reduce_max_sync(kFull, head);
                }
                e_mine = mine ? (int)(IM - (mine & IM)) : -1;
            }
        }
        redo = __any_sync(kFull, redo);
        if (unsure && !redo) {
            e_mine = gate_order_f64<LT>(a, t, m, c, e_mine, (int)(IM - (mine2 & IM)));
            l_mine = e_mine >= 0 ? gate_logit<LT>(a, t, e_mine) : 0.0f;
        }
        if (lane >= k) e_mine = -1;
        // weights of the selected, in full float32 (the truncation's sums in double): off by 4e-8 to 6e-8 of the
        // exact ones, where double precision and one rounding gave 2.5e-8.  (In double, as for the truncation: 0.4
        // us more for 512 rows of 256, on the chain of every row.)
        float w = 0.0f;
        int e_out = e_mine;
        const bool cut = a.topp > 0.0f && a.topp < 1.0f;
        if (!cut) {
            const float s = e_mine < 0 ? 0.0f : a.softmax ? expf(l_mine - m) : __fdiv_rn(1.0f, 1.0f + expf(-l_mine));
            const float sum = warp_sum(s);
            redo |= e_mine >= 0 && !(s > 1e-30f);  // near underflow
            w = a.raw ? (a.softmax ? __fdiv_rn(s, z) : s) : __fdiv_rn(s, sum);
        } else {
            double s = 0.0;
            if (e_mine >= 0)
                s = a.softmax ? exp((double)l_mine - (double)m) : 1.0 / (1.0 + exp(-(double)l_mine));
            const double whole = (double)a.topp * warp_sum_f64(s);
            double before = s;  // the sum of the slots up to this one, then without it
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const double x = __shfl_up_sync(kFull, before, o);
                if (lane >= o) before += x;
            }
            before = __shfl_up_sync(kFull, before, 1);
            redo |= lane > 0 && e_mine >= 0 && fabs(before - whole) < 1e-12 * whole;  // the order of the sum might tell
            if (lane > 0 && !(before < whole)) {
                e_out = -1;
                s = 0.0;
            }
            const double sum = warp_sum_f64(s);
            redo |= e_mine >= 0 && !(sum > 1e-30);
            w = (float)(a.raw ? (a.softmax ? s / (double)z : s) : s / sum);
        }
        if (__any_sync(kFull, redo)) {
            __syncwarp();
            gate_row_f64<LT>(a, t, sel);
        } else if (lane < k) {
            a.idx[(size_t)t * k + lane] = e_out;
            a.w[(size_t)t * k + lane] = e_out >= 0 ? w * a.scale : 0.0f;
        }
        __syncwarp();
    }
}

}  // namespace moe
