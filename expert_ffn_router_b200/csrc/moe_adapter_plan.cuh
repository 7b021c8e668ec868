// The plan of a batch's adapters (moe_adapter_plan).
#pragma once

#include "moe_adapter.cuh"

namespace moe {

// Exclusive scan of n ints in shared memory by a kAdPlanThreads CTA (n at
// most twice the threads); returns the total.
static __device__ int ad_exscan(int* a, int n, int* red) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i0 = 2 * tid, i1 = 2 * tid + 1;
    const int v0 = i0 < n ? a[i0] : 0, v1 = i1 < n ? a[i1] : 0;
    int v = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int base = 0, total = 0;
    for (int i = 0; i < kAdPlanThreads / 32; ++i) {
        if (i < warp) base += red[i];
        total += red[i];
    }
    const int ex = base + v - v0 - v1;
    if (i0 < n) a[i0] = ex;
    if (i1 < n) a[i1] = ex + v0;
    __syncthreads();
    return total;
}

// One CTA: counts the rows of each class (adapter, or none), then places them
// in their order in the batch, kAdPlanThreads rows at a time; a row's place is
// its class's start + the rows of its class in earlier warps + in its own.
// Dynamic shared memory: ad_plan_smem(n).
constexpr size_t ad_plan_smem(int n) { return (size_t)(n + 1) * (2 + kAdPlanThreads / 32) * 4; }

__global__ void __launch_bounds__(kAdPlanThreads) k_adapter_plan(const int32_t* __restrict__ adapter_of, int T,
                                                                  int n, AdPlan p) {
    extern __shared__ int ad_sm[];
    __shared__ int red[kAdPlanThreads / 32];
    constexpr int W = kAdPlanThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int C = n + 1;
    int* start = ad_sm;     // [C]
    int* tfirst = start + C;  // [C] first task of the class
    int* hist = tfirst + C;   // [W][C]
    auto klass = [&](int t) {
        const int a = __ldg(adapter_of + t);
        return a < 0 || a >= n ? n : a;
    };
    if (tid == 0) {
        p.hdr->status = 0;
        p.hdr->status_info = 0;
        p.hdr->magic = kAdMagic;
        p.hdr->T = T;
        p.hdr->n_adapters = n;
    }
    for (int c = tid; c < C; c += kAdPlanThreads) start[c] = 0;
    __syncthreads();
    for (int t = tid; t < T; t += kAdPlanThreads) {
        const int a = __ldg(adapter_of + t);
        if (a < -1 || a >= n) set_status(reinterpret_cast<WsHeader*>(p.hdr), MOE_EDEVICE, t);
        atomicAdd(&start[klass(t)], 1);
    }
    __syncthreads();
    for (int c = tid; c < C; c += kAdPlanThreads) hist[c] = start[c];  // the counts, until the placing below
    __syncthreads();
    ad_exscan(start, C, red);
    for (int l = 0; l < kAdLists; ++l) {
        const int R = ad_rows(l);
        for (int c = tid; c < C; c += kAdPlanThreads) tfirst[c] = (hist[c] + R - 1) / R;
        __syncthreads();
        const int n_tasks = ad_exscan(tfirst, C, red);
        if (tid == 0) p.hdr->n_tasks[l] = n_tasks;
        for (int c = tid; c < C; c += kAdPlanThreads) {
            const int b = start[c], cnt = hist[c];
            for (int i = 0; i * R < cnt; ++i)
                p.tasks[l][tfirst[c] + i] = make_int4(c < n ? c : -1, b + i * R, min(R, cnt - i * R), 0);
        }
        __syncthreads();
    }
    for (int t0 = 0; t0 < T; t0 += kAdPlanThreads) {
        for (int i = tid; i < W * C; i += kAdPlanThreads) hist[i] = 0;
        __syncthreads();
        const int t = t0 + tid;
        const int c = t < T ? klass(t) : C;
        const unsigned peers = __match_any_sync(kFull, c);
        const int rank = __popc(peers & lanemask_lt());
        if (c < C && rank == 0) hist[warp * C + c] = __popc(peers);
        __syncthreads();
        for (int i = tid; i < C; i += kAdPlanThreads) {
            int run = start[i];
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                const int h = hist[w * C + i];
                hist[w * C + i] = run;
                run += h;
            }
            start[i] = run;
        }
        __syncthreads();
        if (c < C) p.order[hist[warp * C + c] + rank] = t;
        __syncthreads();
    }
    for (int l = 0; l < kAdLists; ++l)  // an adapter's rows ascend
        for (int i = tid; i < p.hdr->n_tasks[l]; i += kAdPlanThreads) {
            const int4 k = p.tasks[l][i];
            p.tasks[l][i].w = p.order[k.y + k.z - 1] - p.order[k.y] == k.z - 1;
        }
}

}  // namespace moe
