// Low-rank adapters of many requests beside a shared projection (moe_adapter):
// y[t] = base[t] + scale_a * B_a (A_a x[t]), a the adapter of row t.
#pragma once

#include <cooperative_groups.h>

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

// ---------------------------------------------------------------------------
// Operands.  Every product is bf16 x bf16 on the tensor cores with float32
// sums: codes and bf16 rows are exact as they are, a float32 value v is the
// exact sum of three bf16 parts (its leading 8 bits, the next 8, the last 8,
// each cut off by truncation), so three products give all its 24 bits.
// ---------------------------------------------------------------------------
// Two floats' leading halves as a bf16 pair (truncated).
__device__ __forceinline__ uint32_t ad_hi2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float ad_rest(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
struct AdSplit {
    uint32_t p[3];
};
__device__ __forceinline__ AdSplit ad_split2(float a, float b) {
    AdSplit s;
    s.p[0] = ad_hi2(a, b);
    a = ad_rest(a);
    b = ad_rest(b);
    s.p[1] = ad_hi2(a, b);
    s.p[2] = ad_hi2(ad_rest(a), ad_rest(b));
    return s;
}

template <typename XT>
struct AdX;  // 8 neighbouring values of a row: as loaded, and as PARTS x 4 bf16 pairs
template <>
struct AdX<__nv_bfloat16> {
    static constexpr int PARTS = 1;
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = ld_stream(p); }
    __device__ __forceinline__ void parts(uint32_t (&o)[PARTS][4]) const {
        o[0][0] = v.x;
        o[0][1] = v.y;
        o[0][2] = v.z;
        o[0][3] = v.w;
    }
};
template <>
struct AdX<float> {
    static constexpr int PARTS = 3;
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream_f4(p);
        b = ld_stream_f4(p + 4);
    }
    __device__ __forceinline__ void parts(uint32_t (&o)[PARTS][4]) const {
        const AdSplit s[4] = {ad_split2(a.x, a.y), ad_split2(a.z, a.w), ad_split2(b.x, b.y), ad_split2(b.z, b.w)};
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[q][i] = s[i].p[q];
    }
};
template <>
struct AdX<int8_t> {
    static constexpr int PARTS = 1;
    uint2 v;
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
    __device__ __forceinline__ void load(const int8_t* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    // a code c as the float 2^23 + (c + 128), less 2^23 + 128: exact, and so is its bf16 half
    static __device__ __forceinline__ uint32_t two(uint32_t u, uint32_t sel0, uint32_t sel1) {
        const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, sel0)) - 8388736.0f;
        const float b = __uint_as_float(__byte_perm(u, 0x4b000000u, sel1)) - 8388736.0f;
        return ad_hi2(a, b);
    }
    __device__ __forceinline__ void parts(uint32_t (&o)[PARTS][4]) const {
        const uint32_t x = v.x ^ 0x80808080u, y = v.y ^ 0x80808080u;
        o[0][0] = two(x, 0x7540, 0x7541);
        o[0][1] = two(x, 0x7542, 0x7543);
        o[0][2] = two(y, 0x7540, 0x7541);
        o[0][3] = two(y, 0x7542, 0x7543);
    }
};

// D (16 x 8, float32) += A (16 x 16 bf16) B (16 x 8 bf16)
__device__ __forceinline__ void ad_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ad_ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
// The first n of 8 bf16 values, the others 0.
__device__ __forceinline__ uint4 ad_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = n >= 2 * i + 2 ? w[i] : n == 2 * i + 1 ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// One cluster of CTAs per task (the rows of one adapter, at most kAdTask):
//  1. each CTA multiplies its share of d_in: a warp holds 16 rows and a slice
//     of the columns, all RT components, operands straight from global memory
//     in the order the MMA wants them (a lane's 16 bytes are 8 neighbouring
//     columns; the same columns stand in the same places of both operands, so
//     their order within the k index is free);
//  2. the partial A x meet in the cluster's shared memory: each CTA sums its
//     share of the components over all CTAs in rank order and hands the sums
//     (scaled) to every CTA;
//  3. each CTA multiplies its share of d_out: a warp keeps A x of its 16 rows
//     in registers and walks over B, 16 outputs at a time; lane (g, i) of the
//     two 8-column MMAs gets 4 neighbouring outputs of rows g and g + 8, one
//     16-byte access each to base and y.
// RT: components held, a multiple of 16, at least r_max.
// ---------------------------------------------------------------------------
template <int RT>
struct AdSmem {
    static constexpr int LD = RT + 4;
    float part[kWarps][16][LD];  // per warp; then the summed components [kAdTask][LD]
    float sum[kAdTask][LD];      // this CTA's share
};

template <typename XT, int RT>
__global__ void __launch_bounds__(kThreads) k_adapter(const AdArgs g) {
    namespace cg = cooperative_groups;
    constexpr int NT = RT / 8;             // 8-component tiles
    constexpr int NQ = (RT + 31) / 32;     // 32-component steps of the expansion
    constexpr int PARTS = AdX<XT>::PARTS;
    constexpr int LD = AdSmem<RT>::LD;
    extern __shared__ __align__(16) uint8_t ad_raw[];
    AdSmem<RT>& sm = *reinterpret_cast<AdSmem<RT>*>(ad_raw);
    float(*fin)[LD] = reinterpret_cast<float(*)[LD]>(&sm.part[0][0][0]);
    __shared__ int s_row[kAdTask];
    cg::cluster_group cl = cg::this_cluster();
    const int cs = (int)cl.num_blocks(), cr = (int)cl.block_rank();
    if (!ad_plan_fits(g)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    WsHeader* hdr = reinterpret_cast<WsHeader*>(g.plan.hdr);
    const int ti = blockIdx.x / cs;
    if (ti >= g.plan.hdr->n_tasks) return;
    const int4 task = g.plan.tasks[ti];
    const int ad = idx_in(hdr, task.x, -1, g.n, 701);
    const int n = idx_in(hdr, task.z, 0, kAdTask + 1, 702);
    const int r = ad < 0 ? 0 : g.rank ? min(max(__ldg(g.rank + ad), 0), g.r_max) : g.r_max;
    if (tid < n) s_row[tid] = idx_in(hdr, g.plan.order[idx_in(hdr, task.y + tid, 0, g.T, 703)], 0, g.T, 704);
    __syncthreads();
    // this CTA's outputs, 16 at a time
    const int groups = g.d_out / 16;
    const int o_lo = (int)((long long)groups * cr / cs), o_hi = (int)((long long)groups * (cr + 1) / cs);
    if (r == 0) {  // no update: base, or 0
        if (g.base == g.y) return;
        const int w4 = (o_hi - o_lo) * 4;
        for (int i = tid; i < n * w4; i += kThreads) {
            const int t = s_row[i / w4], o = o_lo * 16 + (i % w4) * 4;
            const float4 v = g.base ? *reinterpret_cast<const float4*>(g.base + (size_t)t * g.ldbase + o)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(g.y + (size_t)t * g.ldy + o) = v;
        }
        return;
    }
    const int mt = n <= 16 ? 1 : n <= 32 ? 2 : 4;  // 16-row tiles; the other warps split the columns
    const int m = warp % mt, sl = warp / mt, nsl = kWarps / mt;
    const int gr = lane >> 2, gi = lane & 3;
    const int j0 = m * 16 + gr, j1 = j0 + 8;  // the lane's two rows of the task

    // ---- 1. A x over this CTA's columns
    {
        const int steps = (g.d_in + 31) / 32;
        const int lo = (int)((long long)steps * cr / cs), hi = (int)((long long)steps * (cr + 1) / cs);
        const __nv_bfloat16* A = g.a + (size_t)ad * g.r_max * g.d_in + (size_t)gr * g.d_in + gi * 8;
        const XT* x0 = static_cast<const XT*>(g.x) + (j0 < n ? (size_t)s_row[j0] * g.ldx : 0) + gi * 8;
        const XT* x1 = static_cast<const XT*>(g.x) + (j1 < n ? (size_t)s_row[j1] * g.ldx : 0) + gi * 8;
        float acc[NT][4] = {}, low[PARTS > 1 ? NT : 1][4] = {};
        for (int st = lo + sl; st < hi; st += nsl) {
            const bool in = st * 32 + gi * 8 < g.d_in;
            AdX<XT> u0, u1;
            u0.zero();
            u1.zero();
            if (in && j0 < n) u0.load(x0 + st * 32);
            if (in && j1 < n) u1.load(x1 + st * 32);
            uint4 w[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                w[i] = in && i * 8 + gr < r ? ad_ldg16(A + (size_t)i * 8 * g.d_in + st * 32) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t p0[PARTS][4], p1[PARTS][4];
            u0.parts(p0);
            u1.parts(p1);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (i * 8 >= r) break;
                ad_mma(acc[i], p0[0][0], p1[0][0], p0[0][1], p1[0][1], w[i].x, w[i].y);
                ad_mma(acc[i], p0[0][2], p1[0][2], p0[0][3], p1[0][3], w[i].z, w[i].w);
#pragma unroll
                for (int q = 1; q < PARTS; ++q) {
                    ad_mma(low[i], p0[q][0], p1[q][0], p0[q][1], p1[q][1], w[i].x, w[i].y);
                    ad_mma(low[i], p0[q][2], p1[q][2], p0[q][3], p1[q][3], w[i].z, w[i].w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (PARTS > 1)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] += low[i][c];
            *reinterpret_cast<float2*>(&sm.part[warp][gr][i * 8 + gi * 2]) = make_float2(acc[i][0], acc[i][1]);
            *reinterpret_cast<float2*>(&sm.part[warp][gr + 8][i * 8 + gi * 2]) = make_float2(acc[i][2], acc[i][3]);
        }
    }
    __syncthreads();

    // ---- 2. the cluster's sum
    const int r4 = (r + 3) / 4;
    for (int i = tid; i < n * r4; i += kThreads) {
        const int j = i / r4, c = (i % r4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < nsl; ++k) {
            const float4 o = *reinterpret_cast<const float4*>(&sm.part[k * mt + j / 16][j % 16][c]);
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        }
        *reinterpret_cast<float4*>(&sm.sum[j][c]) = v;
    }
    cl.sync();  // every CTA's share is in place, and none of them needs `part` any more
    {
        const float scale = g.scale ? __ldg(g.scale + ad) : 1.0f;
        for (int i = cr + cs * tid; i < n * r4; i += cs * kThreads) {
            const int j = i / r4, c = (i % r4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cs; ++k) {
                const float4 o = *reinterpret_cast<const float4*>(cl.map_shared_rank(&sm.sum[j][c], k));
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            const float f = g.sx ? scale * __ldg(g.sx + s_row[j]) : scale;
            v.x *= f;
            v.y *= f;
            v.z *= f;
            v.w *= f;
            for (int k = 0; k < cs; ++k) *reinterpret_cast<float4*>(cl.map_shared_rank(&fin[j][c], k)) = v;
        }
    }
    cl.sync();  // the sums are everywhere; no CTA reads another's memory after this

    // ---- 3. B (A x) over this CTA's outputs
    uint32_t h[NQ][3][2][4];  // [step][part][half][a0 a1 a2 a3]
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        float v0[8], v1[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int k = q * 32 + gi * 8 + c;
            v0[c] = j0 < n && k < r ? fin[j0][k] : 0.0f;
            v1[c] = j1 < n && k < r ? fin[j1][k] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const AdSplit a0 = ad_split2(v0[4 * u], v0[4 * u + 1]), a1 = ad_split2(v1[4 * u], v1[4 * u + 1]);
            const AdSplit a2 = ad_split2(v0[4 * u + 2], v0[4 * u + 3]), a3 = ad_split2(v1[4 * u + 2], v1[4 * u + 3]);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                h[q][p][u][0] = a0.p[p];
                h[q][p][u][1] = a1.p[p];
                h[q][p][u][2] = a2.p[p];
                h[q][p][u][3] = a3.p[p];
            }
        }
    }
    if (m * 16 >= n) return;  // a tile without rows (the warp's slice of the outputs is other warps' too)
    const __nv_bfloat16* B =
        g.b + (size_t)ad * g.d_out * g.r_max + (size_t)(4 * (gr >> 1) + (gr & 1)) * g.r_max + gi * 8;
    const size_t y0 = (size_t)(j0 < n ? s_row[j0] : 0) * g.ldy + gi * 4, y1 = (size_t)(j1 < n ? s_row[j1] : 0) * g.ldy + gi * 4;
    const size_t b0 = (size_t)(j0 < n ? s_row[j0] : 0) * g.ldbase + gi * 4,
                 b1 = (size_t)(j1 < n ? s_row[j1] : 0) * g.ldbase + gi * 4;
    for (int o = o_lo + sl; o < o_hi; o += nsl) {
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
        if (g.base) {
            if (j0 < n) v0 = *reinterpret_cast<const float4*>(g.base + b0 + o * 16);
            if (j1 < n) v1 = *reinterpret_cast<const float4*>(g.base + b1 + o * 16);
        }
        uint4 w[2][NQ];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int left = r - q * 32 - gi * 8;  // components this lane still has
                w[u][q] = left > 0 ? ad_first(ad_ldg16(B + (size_t)(o * 16 + 2 * u) * g.r_max + q * 32), left)
                                   : make_uint4(0u, 0u, 0u, 0u);
            }
        float acc[2][4] = {}, low[2][4] = {};
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            if (q * 32 >= r) break;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    float(&d)[4] = p ? low[u] : acc[u];
                    ad_mma(d, h[q][p][0][0], h[q][p][0][1], h[q][p][0][2], h[q][p][0][3], w[u][q].x, w[u][q].y);
                    ad_mma(d, h[q][p][1][0], h[q][p][1][1], h[q][p][1][2], h[q][p][1][3], w[u][q].z, w[u][q].w);
                }
            }
        }
        v0.x += acc[0][0] + low[0][0];
        v0.y += acc[0][1] + low[0][1];
        v0.z += acc[1][0] + low[1][0];
        v0.w += acc[1][1] + low[1][1];
        v1.x += acc[0][2] + low[0][2];
        v1.y += acc[0][3] + low[0][3];
        v1.z += acc[1][2] + low[1][2];
        v1.w += acc[1][3] + low[1][3];
        if (j0 < n) *reinterpret_cast<float4*>(g.y + y0 + o * 16) = v0;
        if (j1 < n) *reinterpret_cast<float4*>(g.y + y1 + o * 16) = v1;
    }
}

}  // namespace moe
