// Low-rank adapters of many requests beside a shared projection (moe_adapter):
// y[t] = base[t] + scale_a * B_a (A_a x[t]), a the adapter of row t.
#pragma once

#include <cooperative_groups.h>

#include "moe_common.cuh"

namespace moe {

// The batch's plan in device memory: the rows grouped by adapter (those
// without one last), cut into tasks -- twice: of at most 16 rows (small
// batches) and of at most 64.
constexpr int kAdLists = 2;
__host__ __device__ constexpr int ad_rows(int list) { return list == 0 ? 16 : 64; }
constexpr int kAdMaxN = 1024;
constexpr int kAdMaxRank = 128;
constexpr int32_t kAdMagic = 0x41445031;
constexpr int kAdPlanThreads = 1024;

struct AdPlanHeader {
    int32_t status, status_info;  // as in WsHeader: moe_poll_status reads them
    int32_t magic, T, n_adapters;
    int32_t n_tasks[kAdLists];
    int32_t pad[9];
};
static_assert(sizeof(AdPlanHeader) == 64, "plan header must stay 64 bytes");

struct AdPlan {
    AdPlanHeader* hdr;
    int32_t* order;  // [T] rows, grouped
    int4* tasks[kAdLists];  // (adapter or -1, first place in order, rows, 0)
    size_t bytes;
};

// Every adapter of the batch, and the rows without one, may end with a task
// that is not full.
inline int ad_max_tasks(int n_adapters, int T, int list) {
    return std::min(T, n_adapters + 1) + T / ad_rows(list);
}

inline AdPlan ad_plan_carve(void* base, int n_adapters, int T) {
    AdPlan p{};
    char* b = static_cast<char*>(base);
    p.hdr = reinterpret_cast<AdPlanHeader*>(b);
    size_t off = sizeof(AdPlanHeader);
    p.order = reinterpret_cast<int32_t*>(b + off);
    off = align_up(off + (size_t)T * 4, 16);
    for (int l = 0; l < kAdLists; ++l) {
        p.tasks[l] = reinterpret_cast<int4*>(b + off);
        off += (size_t)ad_max_tasks(n_adapters, T, l) * 16;
    }
    p.bytes = off;
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

// 8 neighbouring values of a row of a stage (ld bytes apart), as PARTS x 4 bf16
// pairs.  at(): byte offset of the 16-byte chunk c of row j; its place is
// moved by the row so that a warp's reads meet no bank twice.
template <typename XT>
struct AdX;
template <>
struct AdX<__nv_bfloat16> {
    static constexpr int PARTS = 1;
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ ((j & 1) << 2)) << 4); }
    static __device__ __forceinline__ void get(const uint8_t* sx, int j, int c8, int ld, uint32_t (&o)[PARTS][4]) {
        const uint4 v = *reinterpret_cast<const uint4*>(sx + at(j, c8, ld));
        o[0][0] = v.x;
        o[0][1] = v.y;
        o[0][2] = v.z;
        o[0][3] = v.w;
    }
};
template <>
struct AdX<float> {
    static constexpr int PARTS = 3;
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ (j & 1)) << 4); }
    static __device__ __forceinline__ void get(const uint8_t* sx, int j, int c8, int ld, uint32_t (&o)[PARTS][4]) {
        const float4 a = *reinterpret_cast<const float4*>(sx + at(j, 2 * c8, ld));
        const float4 b = *reinterpret_cast<const float4*>(sx + at(j, 2 * c8 + 1, ld));
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
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ (ld == 64 ? j & 2 : (j & 3) << 1)) << 4); }
    // a code c as the float 2^23 + (c + 128), less 2^23 + 128: exact, and so is its bf16 half
    static __device__ __forceinline__ uint32_t two(uint32_t u, uint32_t sel0, uint32_t sel1) {
        const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, sel0)) - 8388736.0f;
        const float b = __uint_as_float(__byte_perm(u, 0x4b000000u, sel1)) - 8388736.0f;
        return ad_hi2(a, b);
    }
    static __device__ __forceinline__ void get(const uint8_t* sx, int j, int c8, int ld, uint32_t (&o)[PARTS][4]) {
        const uint2 v = *reinterpret_cast<const uint2*>(sx + at(j, c8 >> 1, ld) + (c8 & 1) * 8);
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

// 16 bytes global -> shared, asynchronous; the second form writes zeros if !in.
__device__ __forceinline__ void ad_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ad_cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ad_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ad_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The first n of 8 bf16 values, the others 0.
__device__ __forceinline__ uint4 ad_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = n >= 2 * i + 2 ? w[i] : n == 2 * i + 1 ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// A cluster of CTAs takes one task (up to MR rows of one adapter) after the
// other.  Each CTA
//  1. multiplies its share of d_in, KC columns a stage;
//  2. meets the others: the partial A x are summed over the cluster's shared
//     memory (each CTA sums its share of the components in rank order and
//     hands the scaled sums to all);
//  3. multiplies its share of d_out, 16 outputs a warp and stage.
// One queue of asynchronous copies runs ahead through both products, so B and
// base are on their way while the cluster meets.
// MMA operands: a lane's 16 bytes are 8 neighbouring columns (components); the
// same ones stand in the same places of both operands, so their order within
// the k index is free.  Of the two 8-output tiles of a group lane (gr, gi)
// gets 4 neighbouring outputs of rows gr and gr + 8: one 16-byte access each.
// RT: components held, a multiple of 16, at least r_max.
// ---------------------------------------------------------------------------
template <typename XT, int RT, int MR>
struct AdTile {
    static constexpr int LIST = MR == 16 ? 0 : 1;  // the plan's list
    static constexpr int LD = RT + 4;
    static constexpr int KC = MR == 16 ? 128 : 64;
    static constexpr int X_LD = KC * (int)sizeof(XT), A_LD = KC * 2;
    static constexpr int X_BYTES = MR * X_LD, A_BYTES = RT * A_LD;                    // product 1
    static constexpr int BASE_BYTES = kWarps * 1024, B_BYTES = kWarps * 16 * RT * 2;  // product 2
    static constexpr int STAGE = X_BYTES + A_BYTES > BASE_BYTES + B_BYTES ? X_BYTES + A_BYTES : BASE_BYTES + B_BYTES;
    static constexpr int SUM_ROWS = MR == 16 ? (RT >= 64 ? 16 : RT == 32 ? 32 : 64) : 64;
    static constexpr int SUM_BYTES = (SUM_ROWS + MR) * LD * 4;
    // stages: what two CTAs of an SM can hold, up to 8
    static constexpr int NS0 = (111 * 1024 - SUM_BYTES) / STAGE;
    static constexpr int NS = NS0 > 8 ? 8 : NS0 < 3 ? 3 : NS0;
    static constexpr int SMEM = NS * STAGE + SUM_BYTES;
    static_assert(SMEM <= 227 * 1024 - 1024, "shared memory");
    // chunk c of a row of A, of B
    static __device__ __forceinline__ int a_at(int j, int c) { return j * A_LD + ((c ^ ((j & 1) << 2)) << 4); }
    static __device__ __forceinline__ int b_at(int j, int c) {
        return j * RT * 2 + ((RT >= 64 ? c ^ ((j & 1) << 2) : c) << 4);
    }
};

template <typename XT, int RT, int MR>
__global__ void __launch_bounds__(kThreads) k_adapter(const AdArgs g) {
    namespace cg = cooperative_groups;
    using Tile = AdTile<XT, RT, MR>;
    constexpr int NT = RT / 8;                                            // 8-component tiles
    constexpr int NTW = MR == 16 ? (NT > 8 ? NT / 8 : 1) : (NT > 2 ? NT / 2 : 1);  // of them, a warp's at most
    constexpr int NQ = (RT + 31) / 32;                                    // 32-component steps of product 2
    constexpr int PARTS = AdX<XT>::PARTS, LD = Tile::LD, NS = Tile::NS, KC = Tile::KC;
    constexpr int CHX = Tile::X_LD / 16, XRP = kThreads / CHX, XP = (MR + XRP - 1) / XRP;  // x: chunks a row, rows a pass
    constexpr int CHA = Tile::A_LD / 16, ARP = kThreads / CHA, AP = (RT + ARP - 1) / ARP;  // A
    constexpr int BRP = kThreads / NT;                                                     // B: rows a pass
    extern __shared__ __align__(16) uint8_t ad_raw[];
    float(*sum)[LD] = reinterpret_cast<float(*)[LD]>(ad_raw + NS * Tile::STAGE);  // this CTA's share
    float(*fin)[LD] = sum + Tile::SUM_ROWS;                                        // the cluster's sums, scaled
    __shared__ int s_row[MR];
    cg::cluster_group cl = cg::this_cluster();
    const int cs = (int)cl.num_blocks(), cr = (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gr = lane >> 2, gi = lane & 3;
    WsHeader* hdr = reinterpret_cast<WsHeader*>(g.plan.hdr);
    const int n_tasks = g.plan.hdr->n_tasks[Tile::LIST];
    {  // the plan is this call's (same rows, same adapters)?
        const AdPlanHeader* h = g.plan.hdr;
        if (h->magic != kAdMagic || h->T != g.T || h->n_adapters != g.n) {
            if (tid == 0) set_status(hdr, MOE_EDEVICE, -1);
            return;
        }
    }
    // this CTA's outputs, 16 at a time, and its columns, KC at a time
    const int groups = g.d_out / 16;
    const int o_lo = (int)((long long)groups * cr / cs), o_hi = (int)((long long)groups * (cr + 1) / cs);
    const int steps = (g.d_in + KC - 1) / KC;
    const int k_lo = (int)((long long)steps * cr / cs), ns1 = (int)((long long)steps * (cr + 1) / cs) - k_lo;
    const uint32_t smem = smem_u32(ad_raw);

    for (int ti = blockIdx.x / cs; ti < n_tasks; ti += gridDim.x / cs) {
        const int4 task = __ldg(g.plan.tasks[Tile::LIST] + ti);
        const int ad = idx_in(hdr, task.x, -1, g.n, 701);
        const int n = idx_in(hdr, task.z, 0, MR + 1, 702);
        const int r = ad < 0 ? 0 : g.rank ? min(max(__ldg(g.rank + ad), 0), g.r_max) : g.r_max;
        __syncthreads();  // the task before has left the shared memory
        if (tid < n)
            s_row[tid] = idx_in(hdr, __ldg(g.plan.order + idx_in(hdr, task.y + tid, 0, g.T, 703)), 0, g.T, 704);
        __syncthreads();
        if (r == 0) {  // no update: base, or 0
            if (g.base == g.y) continue;
            const int w4 = (o_hi - o_lo) * 4;
            for (int i = tid; i < n * w4; i += kThreads) {
                const int t = s_row[i / w4], o = o_lo * 16 + (i % w4) * 4;
                const float4 v = g.base ? *reinterpret_cast<const float4*>(g.base + (size_t)t * g.ldbase + o)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(g.y + (size_t)t * g.ldy + o) = v;
            }
            continue;
        }
        const int mt = MR == 16 || n <= 16 ? 1 : n <= 32 ? 2 : 4;  // 16-row tiles
        const int m = MR == 16 ? 0 : warp % mt, sl = MR == 16 ? warp : warp / mt, nsl = MR == 16 ? kWarps : kWarps / mt;
        const int j0 = m * 16 + gr, j1 = j0 + 8;  // the lane's two rows of the task
        const bool on0 = j0 < n, on1 = j1 < n;

        // ---- the queue of copies: stages [0, ns1) of product 1, [ns1, ns) of product 2
        const int ns = ns1 + (o_hi - o_lo + nsl - 1) / nsl;
        const int xj = tid / CHX, xc = tid % CHX, aj = tid / CHA, ac = tid % CHA, bj = tid / NT, bc = tid % NT;
        const XT* xp[XP];
#pragma unroll
        for (int p = 0; p < XP; ++p)
            xp[p] = static_cast<const XT*>(g.x) + (size_t)(xj + p * XRP < n ? s_row[xj + p * XRP] : 0) * g.ldx +
                    k_lo * KC + xc * (16 / (int)sizeof(XT));
        const __nv_bfloat16* ap = g.a + ((size_t)ad * g.r_max + aj) * g.d_in + k_lo * KC + ac * 8;
        const __nv_bfloat16* bp = g.b + ((size_t)ad * g.d_out + o_lo * 16 + bj) * g.r_max + bc * 8;
        const float* p0 = g.base + (size_t)(on0 ? s_row[j0] : 0) * g.ldbase + (o_lo + sl) * 16 + gi * 4;
        const float* p1 = g.base + (size_t)(on1 ? s_row[j1] : 0) * g.ldbase + (o_lo + sl) * 16 + gi * 4;
        const uint32_t xd = AdX<XT>::at(xj, xc, Tile::X_LD), adst = Tile::X_BYTES + Tile::a_at(aj, ac);
        const uint32_t bdst = Tile::BASE_BYTES + Tile::b_at(bj, bc), based = warp * 1024 + lane * 16;
        int issued = 0, ibuf = 0;
        auto issue = [&]() {
            const uint32_t st = smem + ibuf * Tile::STAGE;
            if (issued < ns1) {
                const int left = g.d_in - (k_lo + issued) * KC;  // columns from this stage on
                if (left >= KC) {
#pragma unroll
                    for (int p = 0; p < XP; ++p)
                        if (xj + p * XRP < n) ad_cp16(st + xd + p * XRP * Tile::X_LD, xp[p]);
#pragma unroll
                    for (int p = 0; p < AP; ++p)
                        if (aj + p * ARP < r) ad_cp16(st + adst + p * ARP * Tile::A_LD, ap + (size_t)p * ARP * g.d_in);
                } else {  // the last columns, zeros behind them
                    const bool xin = xc * (16 / (int)sizeof(XT)) < left, ain = ac * 8 < left;
#pragma unroll
                    for (int p = 0; p < XP; ++p)
                        if (xj + p * XRP < n) ad_cp16(st + xd + p * XRP * Tile::X_LD, xin ? xp[p] : g.x, xin);
#pragma unroll
                    for (int p = 0; p < AP; ++p)
                        if (aj + p * ARP < r)
                            ad_cp16(st + adst + p * ARP * Tile::A_LD, ain ? ap + (size_t)p * ARP * g.d_in : g.a, ain);
                }
#pragma unroll
                for (int p = 0; p < XP; ++p) xp[p] += KC;
                ap += KC;
            } else if (issued < ns) {
                const int o0 = o_lo + (issued - ns1) * nsl;
                if (g.base && o0 + sl < o_hi) {  // each lane its own: read back by the lane alone
                    if (on0) ad_cp16(st + based, p0);
                    if (on1) ad_cp16(st + based + 512, p1);
                }
                p0 += nsl * 16;
                p1 += nsl * 16;
                const int no = min(nsl, o_hi - o0) * 16;
                if (bc * 8 < r)
                    for (int j = bj, p = 0; j < no; j += BRP, ++p)
                        ad_cp16(st + bdst + p * BRP * RT * 2, bp + (size_t)p * BRP * g.r_max);
                bp += (size_t)nsl * 16 * g.r_max;
            }
            ad_cp_commit();
            ++issued;
            ibuf = ibuf + 1 == NS ? 0 : ibuf + 1;
        };
#pragma unroll 1
        for (int s = 0; s < NS - 1; ++s) issue();
        int buf = 0;
        auto next_stage = [&]() {  // stage there for all, the one before it free
            ad_cp_wait<NS - 2>();
            __syncthreads();
            issue();
            const uint8_t* st = ad_raw + buf * Tile::STAGE;
            buf = buf + 1 == NS ? 0 : buf + 1;
            return st;
        };

        // ---- 1. A x over this CTA's columns: warps split the rows, then the
        // components, then (few of both) the 32-column steps of a stage
        const int nn = min(nsl, NT);  // warps over the components
        const int kw = min(nsl / nn, KC / 32);
        const int ni = sl % nn, ki = sl / nn;
        {
            float acc[NTW][4] = {}, low[PARTS > 1 ? NTW : 1][4] = {};
            for (int s = 0; s < ns1; ++s) {
                const uint8_t* st = next_stage();
                if (m * 16 >= n) continue;
#pragma unroll
                for (int hf = 0; hf < KC / 32; ++hf) {
                    if (kw > 1 && hf % kw != ki) continue;
                    uint32_t u0[PARTS][4], u1[PARTS][4];
                    AdX<XT>::get(st, j0, hf * 4 + gi, Tile::X_LD, u0);
                    AdX<XT>::get(st, j1, hf * 4 + gi, Tile::X_LD, u1);
#pragma unroll
                    for (int i = 0; i < NTW; ++i) {
                        const int tile = ni + i * nn;
                        if (tile * 8 >= r) break;
                        const uint4 w =
                            *reinterpret_cast<const uint4*>(st + Tile::X_BYTES + Tile::a_at(tile * 8 + gr, hf * 4 + gi));
                        ad_mma(acc[i], u0[0][0], u1[0][0], u0[0][1], u1[0][1], w.x, w.y);
                        ad_mma(acc[i], u0[0][2], u1[0][2], u0[0][3], u1[0][3], w.z, w.w);
#pragma unroll
                        for (int q = 1; q < PARTS; ++q) {
                            ad_mma(low[i], u0[q][0], u1[q][0], u0[q][1], u1[q][1], w.x, w.y);
                            ad_mma(low[i], u0[q][2], u1[q][2], u0[q][3], u1[q][3], w.z, w.w);
                        }
                    }
                }
            }
            if (ki < kw) {
                const int jb = ki * 16 * mt;  // the steps' sums one after the other
#pragma unroll
                for (int i = 0; i < NTW; ++i) {
                    const int tile = ni + i * nn;
                    if (tile * 8 >= r) break;
                    if (PARTS > 1)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[i][c] += low[i][c];
                    *reinterpret_cast<float2*>(&sum[jb + j0][tile * 8 + gi * 2]) = make_float2(acc[i][0], acc[i][1]);
                    *reinterpret_cast<float2*>(&sum[jb + j1][tile * 8 + gi * 2]) = make_float2(acc[i][2], acc[i][3]);
                }
            }
        }

        // ---- 2. the cluster's sum
        cl.sync();
        {
            const int r4 = (r + 3) / 4;
            const float scale = g.scale ? __ldg(g.scale + ad) : 1.0f;
            for (int i = cr + cs * tid; i < n * r4; i += cs * kThreads) {
                const int j = i / r4, c = (i % r4) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < cs; ++k)
                    for (int q = 0; q < kw; ++q) {
                        const float4 o = *reinterpret_cast<const float4*>(cl.map_shared_rank(&sum[q * 16 * mt + j][c], k));
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
        cl.sync();  // the sums are everywhere; no CTA reads another's memory until the next task's sum

        // ---- 3. B (A x) over this CTA's outputs: A x of the warp's rows in registers
        uint32_t h[NQ][3][2][4];  // [step][part][half][a0 a1 a2 a3]
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            float v0[8], v1[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int k = q * 32 + gi * 8 + c;
                v0[c] = on0 && k < r ? fin[j0][k] : 0.0f;
                v1[c] = on1 && k < r ? fin[j1][k] : 0.0f;
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
        float* y0 = g.y + (size_t)(on0 ? s_row[j0] : 0) * g.ldy + (o_lo + sl) * 16 + gi * 4;
        float* y1 = g.y + (size_t)(on1 ? s_row[j1] : 0) * g.ldy + (o_lo + sl) * 16 + gi * 4;
        const int jw = sl * 16 + 4 * (gr >> 1) + (gr & 1);  // the lane's first output row of a stage
        for (int o = o_lo + sl; o - sl < o_hi; o += nsl, y0 += nsl * 16, y1 += nsl * 16) {
            const uint8_t* st = next_stage();
            if (o >= o_hi || m * 16 >= n) continue;
            float acc[2][4] = {}, low[2][4] = {};
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int left = r - q * 32;  // components from this step on
                if (left <= 0) break;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 w = *reinterpret_cast<const uint4*>(st + Tile::BASE_BYTES + Tile::b_at(jw + 2 * u, (q * 4 + gi) % NT));
                    if (left < 32) w = ad_first(w, left - gi * 8);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        float(&d)[4] = p ? low[u] : acc[u];
                        ad_mma(d, h[q][p][0][0], h[q][p][0][1], h[q][p][0][2], h[q][p][0][3], w.x, w.y);
                        ad_mma(d, h[q][p][1][0], h[q][p][1][1], h[q][p][1][2], h[q][p][1][3], w.z, w.w);
                    }
                }
            }
            float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
            if (g.base) {
                v0 = *reinterpret_cast<const float4*>(st + based);
                v1 = *reinterpret_cast<const float4*>(st + based + 512);
            }
            v0.x += acc[0][0] + low[0][0];
            v0.y += acc[0][1] + low[0][1];
            v0.z += acc[1][0] + low[1][0];
            v0.w += acc[1][1] + low[1][1];
            v1.x += acc[0][2] + low[0][2];
            v1.y += acc[0][3] + low[0][3];
            v1.z += acc[1][2] + low[1][2];
            v1.w += acc[1][3] + low[1][3];
            if (on0) *reinterpret_cast<float4*>(y0) = v0;
            if (on1) *reinterpret_cast<float4*>(y1) = v1;
        }
        ad_cp_wait<0>();  // (only empty groups are left)
    }
}

}  // namespace moe
