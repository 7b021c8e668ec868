// Low-rank adapters of many requests beside a shared projection (moe_adapter):
// y[t] = base[t] + scale_a * B_a (A_a x[t]), a the adapter of row t.
#pragma once

#include "moe_common.cuh"

namespace moe {

// The batch's plan in device memory: the rows grouped by adapter (those
// without one last), cut into tasks of at most kAdTask rows.
constexpr int kAdTask = 64;
constexpr int kAdMaxN = 1024;
constexpr int kAdMaxRank = 128;
constexpr int32_t kAdMagic = 0x41445031;
constexpr int kAdPlanThreads = 1024;

struct AdPlanHeader {
    int32_t status, status_info;  // as in WsHeader: moe_poll_status reads them
    int32_t magic, T, n_adapters;
    int32_t n_tasks;
    int32_t pad[10];
};
static_assert(sizeof(AdPlanHeader) == 64, "plan header must stay 64 bytes");

struct AdPlan {
    AdPlanHeader* hdr;
    int32_t* order;  // [T] rows, grouped
    int4* tasks;     // [n_tasks] (adapter or -1, first place in order, rows, 0)
    size_t bytes;
};

// Rows in tasks of kAdTask: every adapter of the batch, and the rows without
// one, may end with a task that is not full.
inline int ad_max_tasks(int n_adapters, int T) { return std::min(T, n_adapters + 1) + T / kAdTask; }

inline AdPlan ad_plan_carve(void* base, int n_adapters, int T) {
    AdPlan p{};
    char* b = static_cast<char*>(base);
    p.hdr = reinterpret_cast<AdPlanHeader*>(b);
    size_t off = sizeof(AdPlanHeader);
    p.order = reinterpret_cast<int32_t*>(b + off);
    off = align_up(off + (size_t)T * 4, 16);
    p.tasks = reinterpret_cast<int4*>(b + off);
    p.bytes = off + (size_t)ad_max_tasks(n_adapters, T) * 16;
    return p;
}

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

static __global__ void __launch_bounds__(kAdPlanThreads) k_adapter_plan(const int32_t* __restrict__ adapter_of, int T,
                                                                  int n, AdPlan p) {
    extern __shared__ int ad_sm[];
    __shared__ int red[kAdPlanThreads / 32];
    constexpr int W = kAdPlanThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    for (int c = tid; c < C; c += kAdPlanThreads) tfirst[c] = (start[c] + kAdTask - 1) / kAdTask;
    __syncthreads();
    ad_exscan(start, C, red);
    const int n_tasks = ad_exscan(tfirst, C, red);
    if (tid == 0) p.hdr->n_tasks = n_tasks;
    for (int c = tid; c < C; c += kAdPlanThreads) {
        const int b = start[c], e = c + 1 < C ? start[c + 1] : T;
        for (int i = 0; b + i * kAdTask < e; ++i)
            p.tasks[tfirst[c] + i] = make_int4(c < n ? c : -1, b + i * kAdTask, min(kAdTask, e - b - i * kAdTask), 0);
    }
    __syncthreads();
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
}

struct AdArgs {
    const __nv_bfloat16* a;
    const __nv_bfloat16* b;
    const int32_t* rank;
    const float* scale;
    int n, r_max, d_in, d_out, T;
    AdPlan plan;
    const void* x;
    const float* sx;
    long long ldx;
    const float* base;
    long long ldbase;
    float* y;
    long long ldy;
};

// The plan is this call's (same rows, same adapters); recorded if not.
__device__ __forceinline__ bool ad_plan_fits(const AdArgs& g) {
    const AdPlanHeader* h = g.plan.hdr;
    if (h->magic == kAdMagic && h->T == g.T && h->n_adapters == g.n) return true;
    if (threadIdx.x == 0) set_status(reinterpret_cast<WsHeader*>(g.plan.hdr), MOE_EDEVICE, -1);
    return false;
}

__device__ __forceinline__ float ad_x(const float* x, size_t i) { return __ldg(x + i); }
__device__ __forceinline__ float ad_x(const __nv_bfloat16* x, size_t i) { return __bfloat162float(__ldg(x + i)); }
__device__ __forceinline__ float ad_x(const int8_t* x, size_t i) { return (float)__ldg(x + i); }

// One CTA per task, row after row: h = A x by one warp per component, then a
// thread per output.
template <typename XT>
__global__ void __launch_bounds__(kThreads) k_adapter(const AdArgs g) {
    __shared__ float h[kAdMaxRank];
    if (!ad_plan_fits(g)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    WsHeader* hdr = reinterpret_cast<WsHeader*>(g.plan.hdr);
    if ((int)blockIdx.x >= g.plan.hdr->n_tasks) return;
    const int4 task = g.plan.tasks[blockIdx.x];
    const int ad = idx_in(hdr, task.x, -1, g.n, 701);
    const int n = idx_in(hdr, task.z, 0, kAdTask + 1, 702);
    const int r = ad < 0 ? 0 : g.rank ? min(max(__ldg(g.rank + ad), 0), g.r_max) : g.r_max;
    const float scale = ad < 0 ? 0.0f : g.scale ? __ldg(g.scale + ad) : 1.0f;
    const __nv_bfloat16* A = g.a + (size_t)max(ad, 0) * g.r_max * g.d_in;
    const __nv_bfloat16* B = g.b + (size_t)max(ad, 0) * g.d_out * g.r_max;
    const XT* x = static_cast<const XT*>(g.x);
    for (int i = 0; i < n; ++i) {
        const int t = idx_in(hdr, g.plan.order[idx_in(hdr, task.y + i, 0, g.T, 703)], 0, g.T, 704);
        const float sx = g.sx ? __ldg(g.sx + t) : 1.0f;
        __syncthreads();
        for (int j = warp; j < r; j += kWarps) {
            float s = 0.0f;
            for (int c = lane; c < g.d_in; c += 32)
                s = fmaf(ad_x(x, (size_t)t * g.ldx + c), __bfloat162float(__ldg(A + (size_t)j * g.d_in + c)), s);
            s = warp_sum(s);
            if (lane == 0) h[j] = s * sx;
        }
        __syncthreads();
        for (int o = tid; o < g.d_out; o += kThreads) {
            float s = 0.0f;
            for (int j = 0; j < r; ++j) s = fmaf(h[j], __bfloat162float(__ldg(B + (size_t)o * g.r_max + j)), s);
            s *= scale;
            g.y[(size_t)t * g.ldy + o] = g.base ? g.base[(size_t)t * g.ldbase + o] + s : s;
        }
    }
}

}  // namespace moe
