// Low-rank adapters of many requests beside a shared projection (moe_adapter):
// y[t] = base[t] + scale_a * B_a (A_a x[t]), a the adapter of row t.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "moe_common.cuh"

namespace moe {

// The batch's plan in device memory: the rows grouped by adapter (those
// without one last), cut into tasks -- twice: of at most 8 rows (small
// batches) and of at most 64.
constexpr int kAdLists = 2;
__host__ __device__ constexpr int ad_rows(int list) { return list == 0 ? 8 : 64; }
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
    int4* tasks[kAdLists];  // (adapter or -1, first place in order, rows, 1 if they are neighbours in the batch)
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

struct AdArgs {
    const __nv_bfloat16* a;
    const __nv_bfloat16* b;
    const int32_t* rank;
    const float* scale;
    int n, r_max, d_in, d_out, T;
    AdPlan plan;
    int max_tasks;  // the tasks the plan's list can hold
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
__device__ __forceinline__ void ad_split2(float a, float b, uint32_t (&p)[3]) {
    p[0] = ad_hi2(a, b);
    a = ad_rest(a);
    b = ad_rest(b);
    p[1] = ad_hi2(a, b);
    p[2] = ad_hi2(ad_rest(a), ad_rest(b));
}

// 8 neighbouring values of a row that are not bf16: as loaded, and as PARTS
// chunks of 8 bf16 values.  (bf16 rows are copied as they are.)
template <typename XT>
struct AdX;
template <>
struct AdX<__nv_bfloat16> {
    static constexpr int PARTS = 1;
    int none;
    __device__ __forceinline__ void load(const __nv_bfloat16*) {}
    __device__ __forceinline__ void parts(uint4 (&)[PARTS]) const {}
};
template <>
struct AdX<float> {
    static constexpr int PARTS = 3;
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream_f4(p);
        b = ld_stream_f4(p + 4);
    }
    __device__ __forceinline__ void parts(uint4 (&o)[PARTS]) const {
        uint32_t s[4][3];
        ad_split2(a.x, a.y, s[0]);
        ad_split2(a.z, a.w, s[1]);
        ad_split2(b.x, b.y, s[2]);
        ad_split2(b.z, b.w, s[3]);
#pragma unroll
        for (int q = 0; q < 3; ++q) o[q] = make_uint4(s[0][q], s[1][q], s[2][q], s[3][q]);
    }
};
template <>
struct AdX<int8_t> {
    static constexpr int PARTS = 1;
    uint2 v;
    __device__ __forceinline__ void load(const int8_t* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    // a code c as the float 2^23 + (c + 128), less 2^23 + 128: exact, and so is its bf16 half
    static __device__ __forceinline__ uint32_t two(uint32_t u, uint32_t sel0, uint32_t sel1) {
        const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, sel0)) - 8388736.0f;
        const float b = __uint_as_float(__byte_perm(u, 0x4b000000u, sel1)) - 8388736.0f;
        return ad_hi2(a, b);
    }
    __device__ __forceinline__ void parts(uint4 (&o)[PARTS]) const {
        const uint32_t x = v.x ^ 0x80808080u, y = v.y ^ 0x80808080u;
        o[0] = make_uint4(two(x, 0x7540, 0x7541), two(x, 0x7542, 0x7543), two(y, 0x7540, 0x7541), two(y, 0x7542, 0x7543));
    }
};

// Shared-memory descriptor of a K-major operand whose rows are 128 bytes (64
// bf16 values) in the 128-byte swizzle: the 16-byte chunk c of row j lies at
// j * 128 + ((c ^ (j & 7)) << 4), 8 rows per 1024 bytes (1024-byte aligned).
__device__ __forceinline__ uint64_t ad_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ int ad_place(int j, int c) { return j * 128 + ((c ^ (j & 7)) << 4); }
// The same for rows of 32 bytes (16 values) in the 32-byte swizzle: chunk c of
// row j at j * 32 + ((c ^ ((j >> 2) & 1)) << 4), 8 rows per 256 bytes.
__device__ __forceinline__ uint64_t ad_desc32(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (16ull << 32) | (1ull << 46) | (6ull << 61);
}
// True for one lane of a converged warp.  The MMA and the tiled copies take
// their operands from uniform registers: the warps that issue them run
// converged on values that are uniform by construction (votes, shuffles, loop
// counters), and only the instructions themselves are one lane's.  In a branch
// on the lane's number each of them cost about 200 cycles.
__device__ __forceinline__ bool ad_elect() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p)::"memory");
    return p != 0;
}
__device__ __forceinline__ int ad_uniform(int v) { return __shfl_sync(kFull, v, 0); }
// D[tmem] (128 x n, float32) (+)= A (128 x 16) B (n x 16)^T, bf16, one CTA.
__device__ __forceinline__ void ad_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D float32, A and B bf16, both K-major, M = 128, N = n (a multiple of 16).
__host__ __device__ constexpr uint32_t ad_idesc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// ---------------------------------------------------------------------------
// The cluster's meeting points: an mbarrier in every CTA that one thread of
// each CTA of the cluster arrives on, so that the copying warp need not take
// part.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t ad_peer(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ad_peer_ld(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void ad_peer_st8(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void ad_peer_arrive(uint64_t* bar, int rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(ad_peer(smem_u32(bar), rank))
                 : "memory");
}
// Waits for a stage's barrier, bounded (the clock is read once in 1024 tries).
__device__ __forceinline__ bool ad_wait(uint64_t* bar, uint32_t parity, WsHeader* hdr, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 1023u) == 1023u) {
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) {
                set_status(hdr, MOE_ETIMEOUT, site);
                return false;
            }
        }
    }
}
// Waits for a phase of such a meeting point, what the peers wrote before it included.
__device__ __forceinline__ bool ad_meet(uint64_t* bar, uint32_t parity, WsHeader* hdr, int site) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 1023u) == 1023u) {
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) {
                set_status(hdr, MOE_ETIMEOUT, site);
                return false;
            }
        }
    }
}
// Orders shared-memory writes (this thread's, and those it has acquired)
// before the tensor core's reads, in the whole cluster.
__device__ __forceinline__ void ad_fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void ad_cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void ad_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ int ad_cluster_size() {
    int v;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(v));
    return v;
}
__device__ __forceinline__ int ad_cluster_rank() {
    int v;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
    return v;
}

// Tiled copies: box at (x, y) of a 2-D map, at (x, y, z) of a 3-D one; rows
// y0..y3 of a 2-D map whose box is one row.
__device__ __forceinline__ void ad_tma_2d(uint32_t dst, const void* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void ad_tma_3d(uint32_t dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void ad_tma_rows4(uint32_t dst, const void* map, int x, int y0, int y1, int y2, int y3,
                                             uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(smem_u32(bar))
        : "memory");
}
// The first n of 8 bf16 values, the others 0.
__device__ __forceinline__ uint4 ad_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = n >= 2 * i + 2 ? w[i] : n == 2 * i + 1 ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void ad_st16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A warp: w (a multiple of 16) values of a row of base, or zeros, into y.
__device__ __forceinline__ void ad_copy_row(const float* base, float* y, int w) {
    const int lane = threadIdx.x & 31;
    for (int i0 = lane * 4; i0 < w; i0 += 8 * 128) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = base && i0 + u * 128 < w ? *reinterpret_cast<const float4*>(base + i0 + u * 128)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u * 128 < w) *reinterpret_cast<float4*>(y + i0 + u * 128) = v[u];
    }
}

// ---------------------------------------------------------------------------
// Many rows: a cluster of CTAs takes one task (up to 64 rows of one adapter)
// after the other.  Each CTA
//  1. multiplies its share of d_in: D1 [component][row] = A x^T;
//  2. meets the others: the partial D1 are summed over the cluster's shared
//     memory in rank order, scaled, and split into three bf16 parts H;
//  3. multiplies its share of d_out, OC outputs a stage: D2 [output][row] =
//     B H^T, and adds base.
// The weights are the MMA's 128-row operand (components or outputs; rows past
// them give lanes that nobody reads), the batch's rows its columns, so that a
// lane of the accumulator is an output and a warp's accesses to a row of base
// and y are contiguous: of two accumulators one holds the even outputs, one
// the odd ones, and a lane has 8 bytes.
// Warps: NE read tensor memory, add and store; one issues the MMAs, one the
// tiled copies, which keep a ring of stages full through both products and on
// into the next task; NP put rows that are not bf16 into their parts, and clear
// what lies in B behind a rank that is no multiple of 16.
// Measured (B200, 8192 bf16 rows of 6144 in runs, 16 adapters, ranks 4 to 64): 117
// us, 4.4 TB/s of the rows, base and outputs, 0.67 of a copy.  The adding warps
// drain product 1, meet and drain product 2 in turn, so base and y do not move
// meanwhile.  Rows that do not lie together are gathered four at a time: rank 64
// throughout, 126 us in runs, 211 mixed; float32 rows, which pass the parting
// warps either way, 204 and 205.
// RT: components held, a multiple of 16, at least r_max.
// ---------------------------------------------------------------------------
template <typename XT, int RT>
struct AdTile {
    static constexpr int NR = 64, LIST = 1;  // the plan's list
    static constexpr int PARTS = AdX<XT>::PARTS;
    static constexpr int NE = 16, NP = PARTS > 1 ? 8 : 4;
    static constexpr int WARPS = NE + 2 + NP;
    static constexpr int OC = 256;
    static constexpr int KS = RT / 16;                        // 16-component slices of B, each two tiles of 128 outputs
    static constexpr int KBK = (RT + 63) / 64;                // 64-component blocks of H
    static constexpr int A_BLK = RT * 128, X_BLK = NR * 128;  // 64 columns of A, of a part of x
    static constexpr int P1_BLK = A_BLK + PARTS * X_BLK, FLOOR = 32768;
    static constexpr int STAGE0 = KS * 8192 > P1_BLK ? KS * 8192 : P1_BLK;
    static constexpr int STAGE = STAGE0 > FLOOR ? STAGE0 : FLOOR;
    static constexpr int KB = STAGE / P1_BLK > 4 ? 4 : STAGE / P1_BLK;  // 64-column blocks a stage
    static constexpr int LD = RT + 4;
    static constexpr int SUM_BYTES = NR * LD * 4, H_BYTES = 3 * KBK * X_BLK;
    static constexpr int OVER = (KB - 1) * A_BLK + 16384 - STAGE;  // A's 128 rows read this far behind a stage
    static constexpr int REST = SUM_BYTES + H_BYTES > OVER ? SUM_BYTES + H_BYTES : OVER;
    static constexpr int NS0 = (225 * 1024 - REST - 1024) / STAGE;
    static constexpr int NS = NS0 > 6 ? 6 : NS0;
    static constexpr int SMEM = NS * STAGE + REST + 1024;
    // D1 is read out and begun anew every FLUSH stages (32 to 48 steps of the
    // MMA), the parts added in registers: a sum over all 6144 columns within
    // tensor memory was off by 2.8e-6 of the result (its adder truncates); so y is
    // off by 5e-7 for bf16 rows and 1.1e-6 for float32 ones, whose three parts are 48
    // steps (rank 64, no base; plain float32 products: 3e-7 and 6e-7).
    static constexpr int FLUSH = KB >= 4 ? 2 : KB == 3 ? 3 : 4;
    // tensor memory: D2 2 x 2 x NR columns, D1 2 x NR.  No CTA of a kernel that
    // uses tensor memory fits beside this one, so its columns are free.
    static constexpr int D1 = 4 * NR, TCOLS = 512;
    static_assert(KB >= 1 && NS >= 2 && SMEM > 152 * 1024, "tile");
};

struct AdRow {  // a row of base and of y, from the CTA's first output on
    const float* base;
    float* y;
};

template <typename XT, int RT>
__global__ void __launch_bounds__(AdTile<XT, RT>::WARPS * 32, 1)
    k_adapter(const AdArgs g, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g) {
    using Tile = AdTile<XT, RT>;
    constexpr int NR = Tile::NR;
    constexpr int PARTS = Tile::PARTS, KB = Tile::KB, KBK = Tile::KBK, KS = Tile::KS, OC = Tile::OC, NS = Tile::NS;
    constexpr int LD = Tile::LD, NE = Tile::NE, NP = Tile::NP;
    constexpr bool CONV = !std::is_same<XT, __nv_bfloat16>::value;
    extern __shared__ uint8_t ad_raw[];
    uint8_t* sbase = ad_raw + ((1024 - (smem_u32(ad_raw) & 1023u)) & 1023u);
    uint8_t* hbuf = sbase + NS * Tile::STAGE;                                    // H [part][block][row] swizzled
    float(*sum)[LD] = reinterpret_cast<float(*)[LD]>(hbuf + Tile::H_BYTES);       // this CTA's share of A x
    __shared__ uint64_t full[NS], fixed[NS], empty[NS], d1full[2], d1empty[2], hfull, d2full[2], d2empty[2], drain, meet_a, meet_b;
    __shared__ uint32_t s_tmem;
    __shared__ int x_row[NR], e_row[NR];  // a task's rows, for the parting and the adding warps
    __shared__ __align__(16) AdRow e_ptr[NR];
    const int cs = ad_cluster_size(), cr = ad_cluster_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t_first = blockIdx.x / cs, t_step = gridDim.x / cs;
    WsHeader* hdr = reinterpret_cast<WsHeader*>(g.plan.hdr);
    int4 task = t_first < g.max_tasks ? __ldg(g.plan.tasks[Tile::LIST] + t_first) : make_int4(-1, 0, 0, 0);
    const int n_tasks = g.plan.hdr->n_tasks[Tile::LIST];
    {  // the plan is this call's (same rows, same adapters)?
        const AdPlanHeader* h = g.plan.hdr;
        if (h->magic != kAdMagic || h->T != g.T || h->n_adapters != g.n) {
            if (tid == 0) set_status(hdr, MOE_EDEVICE, -1);
            return;
        }
    }
    if (t_first >= n_tasks) return;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&fixed[i], NP);
            mbar_init(&empty[i], 1 + NP);  // the MMAs that read it, the parting warps
        }
        mbar_init(&hfull, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&d1full[i], 1);
            mbar_init(&d1empty[i], NE);
            mbar_init(&d2full[i], 1);
            mbar_init(&d2empty[i], NE);
        }
        mbar_init(&drain, 1);
        mbar_init(&meet_a, cs);
        mbar_init(&meet_b, cs);
        fence_mbar_init();
    }
    if (warp == NE) tmem_alloc(&s_tmem, Tile::TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    ad_cluster_arrive();  // barriers ready; waited for before the first access to a peer
    const uint32_t tbase = s_tmem;
    // this CTA's outputs, 16 at a time, and its columns, 64 at a time
    const int groups = g.d_out / 16, blocks = (g.d_in + 63) / 64;
    const int o_lo = (int)((long long)groups * cr / cs), o_hi = (int)((long long)groups * (cr + 1) / cs);
    const int k_lo = (int)((long long)blocks * cr / cs), k_hi = (int)((long long)blocks * (cr + 1) / cs);
    auto rank_of = [&](int ad) { return ad < 0 ? 0 : g.rank ? min(max(__ldg(g.rank + ad), 0), g.r_max) : g.r_max; };
    auto row_of = [&](int j) {
        return idx_in(hdr, __ldg(g.plan.order + idx_in(hdr, task.y + j, 0, g.T, 703)), 0, g.T, 704);
    };
    // B's last slice of 16 components holds some behind the rank (behind r_max the copy fills in zeros)
    auto cut = [&](int r) { return r % 16 != 0 && r != g.r_max; };

    if (warp == NE + 1) {
        // ------------------------------------------------------------ tiled copies
        int slot = 0;
        uint32_t ph = 0, issued = 0;
        bool ok = true;
        const uint32_t ring = smem_u32(sbase);
        for (int ti = t_first; ti < n_tasks && ok; ti += t_step) {
            if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
            const int ad = ad_uniform(idx_in(hdr, task.x, -1, g.n, 701));
            const int n = ad_uniform(idx_in(hdr, task.z, 0, NR + 1, 702));
            const int r = ad_uniform(rank_of(ad));
            if (r == 0) continue;
            int row[(NR + 31) / 32];  // a lane's rows, those behind the last the last again
#pragma unroll
            for (int i = 0; i < (NR + 31) / 32; ++i) row[i] = CONV ? 0 : row_of(min(lane + 32 * i, n - 1));
            const int rs = (r + 15) / 16, n4 = (n + 3) / 4;
            const bool run = ad_uniform(task.w) != 0;  // neighbours: one box (a row behind them is nobody's)
            const int row0 = ad_uniform(row[0]);
            auto take = [&]() -> uint32_t {  // the next stage, free
                ok = __all_sync(kFull, ad_wait(&empty[slot], ph ^ 1u, hdr, 0x7201));
                return ring + slot * Tile::STAGE;
            };
            auto next = [&]() {
                ++issued;
                if (++slot == NS) {
                    slot = 0;
                    ph ^= 1u;
                }
            };
            for (int k = k_lo; k < k_hi && ok; k += KB) {
                const int nb = min(KB, k_hi - k);
                const uint32_t st = take();
                if (!ok) break;
                if (ad_elect()) {
                    mbar_arrive_expect_tx(&full[slot], (uint32_t)nb * (rs * 2048 + (CONV ? 0 : run ? NR * 128 : n4 * 512)));
                    for (int b = 0; b < nb; ++b) {
                        for (int i = 0; i < rs; ++i)
                            ad_tma_2d(st + b * Tile::A_BLK + i * 2048, &map_a, (k + b) * 64, ad * g.r_max + i * 16, &full[slot]);
                        if (!CONV && run)
                            ad_tma_2d(st + KB * Tile::A_BLK + b * Tile::X_BLK, &map_x, (k + b) * 64, row0, &full[slot]);
                    }
                }
                __syncwarp();
                if (!CONV && !run) {
#pragma unroll
                    for (int h = 0; h < (NR + 31) / 32; ++h)
                        for (int i = 0; i < 8 && 8 * h + i < n4; ++i) {
                            const int y0 = __shfl_sync(kFull, row[h], 4 * i), y1 = __shfl_sync(kFull, row[h], 4 * i + 1);
                            const int y2 = __shfl_sync(kFull, row[h], 4 * i + 2), y3 = __shfl_sync(kFull, row[h], 4 * i + 3);
                            if (ad_elect())
                                for (int b = 0; b < nb; ++b)
                                    ad_tma_rows4(st + KB * Tile::A_BLK + b * Tile::X_BLK + (8 * h + i) * 512, &map_g,
                                                 (k + b) * 64, y0, y1, y2, y3, &full[slot]);
                            __syncwarp();
                        }
                }
                next();
            }
            for (int o = o_lo; o < o_hi && ok; o += OC / 16) {
                const uint32_t st = take();
                if (!ok) break;
                const int z = (int)(((long long)ad * g.d_out + o * 16) / 2);
                if (ad_elect()) {
                    mbar_arrive_expect_tx(&full[slot], (uint32_t)rs * 8192);
                    for (int i = 0; i < rs; ++i)
                        for (int u = 0; u < 2; ++u) ad_tma_3d(st + (u * KS + i) * 4096, &map_b, i * 16, u, z, &full[slot]);
                }
                __syncwarp();
                next();
            }
        }
        // every copy has landed before the CTA exits
        for (int s = 0; s < NS; ++s) {
            const uint32_t n_s = issued / NS + ((uint32_t)s < issued % NS ? 1u : 0u);
            if (n_s) ad_wait(&full[s], (n_s - 1) & 1u, hdr, 0x7202);
        }
    } else if (warp > NE + 1) {
        // ------------------------------------------------------------ parts of x, ends of B
        constexpr int NPT = NP * 32, RPP = NPT / 8;  // rows a pass, 8 chunks of 8 values each
        constexpr int XB = NR / RPP;                 // chunks of a block of x a thread has
        constexpr int XD = 2;                        // stages of x loaded ahead
        static_assert(RPP % 8 == 0 && NR % RPP == 0, "parts");
        const int pt = tid - (NE + 2) * 32, c = pt & 7, jr = pt >> 3;
        const int place = ad_place(jr, c);  // (a row RPP further: RPP * 128 further)
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
        // these warps take part in every stage, if only to stay in its phase
        auto next = [&]() {
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == NS) {
                slot = 0;
                ph ^= 1u;
            }
        };
        auto wait = [&]() {  // (the slot's last stage done first: else `ph` could name the phase before it)
            if (ok) ok = ad_wait(&empty[slot], ph ^ 1u, hdr, 0x7203) && ad_wait(&full[slot], ph, hdr, 0x7204);
            __syncwarp();
        };
        auto done = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fixed[slot]);
        };
        for (int ti = t_first; ti < n_tasks; ti += t_step) {
            if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
            const int n = idx_in(hdr, task.z, 0, NR + 1, 706);
            const int r = rank_of(idx_in(hdr, task.x, -1, g.n, 705));
            if (r == 0) continue;
            if constexpr (CONV) {
                named_sync(2, NPT);  // the rows before are no longer read
                if (pt < n) x_row[pt] = row_of(pt);
                named_sync(2, NPT);
                const XT* X = static_cast<const XT*>(g.x) + c * 8;
                AdX<XT> xv[XD][KB * XB];
                auto load_x = [&](int k, AdX<XT>(&v)[KB * XB]) {  // of the stage that starts at block k
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int i = 0; i < XB; ++i) {
                            const int j = jr + i * RPP, col = (k + b) * 64;
                            if (k + b < k_hi && col + c * 8 < g.d_in && j < n)
                                v[b * XB + i].load(X + (size_t)x_row[j] * g.ldx + col);
                        }
                };
#pragma unroll
                for (int d = 0; d < XD; ++d) load_x(k_lo + d * KB, xv[d]);
                for (int k = k_lo; k < k_hi; k += KB) {
                    if (ok) ok = ad_wait(&empty[slot], ph ^ 1u, hdr, 0x7203);
                    const uint32_t st = smem_u32(sbase + slot * Tile::STAGE) + KB * Tile::A_BLK + place;
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int i = 0; i < XB; ++i)
                            if (k + b < k_hi && (k + b) * 64 + c * 8 < g.d_in && jr + i * RPP < n) {
                                uint4 q[PARTS];
                                xv[0][b * XB + i].parts(q);
#pragma unroll
                                for (int p = 0; p < PARTS; ++p)
                                    ad_st16(st + (b * PARTS + p) * Tile::X_BLK + i * RPP * 128, q[p]);
                            }
                    done();
                    next();
#pragma unroll
                    for (int d = 0; d + 1 < XD; ++d)
#pragma unroll
                        for (int i = 0; i < KB * XB; ++i) xv[d][i] = xv[d + 1][i];
                    load_x(k + XD * KB, xv[XD - 1]);
                }
            } else {
                for (int k = k_lo; k < k_hi; k += KB) {
                    wait();
                    next();
                }
            }
            for (int o = o_lo; o < o_hi; o += OC / 16) {
                wait();
                if (cut(r)) {
                    const int e = r % 16;  // components of the last slice
#pragma unroll
                    for (int i = 0; i < 2 * 128 / NPT; ++i) {
                        const int u = (pt + i * NPT) / 128, j = (pt + i * NPT) % 128;
                        uint8_t* row = sbase + slot * Tile::STAGE + (u * KS + r / 16) * 4096 + j * 32;
                        uint4* lo = reinterpret_cast<uint4*>(row + (((j >> 2) & 1) << 4));
                        uint4* hi = reinterpret_cast<uint4*>(row + ((((j >> 2) & 1) ^ 1) << 4));
                        if (e < 8) *lo = ad_first(*lo, e);
                        *hi = ad_first(*hi, max(e - 8, 0));
                    }
                    done();
                }
                next();
            }
        }
    } else if (warp == NE) {
        // ------------------------------------------------------------ MMA issuer
        int slot = 0;
        uint32_t ph = 0, fph = 0, round = 0, parts1 = 0, tiles = 0;  // fph: bit s, the phase of fixed[s]
        bool ok = true, issued = false;
        const uint32_t ring = smem_u32(sbase), tm = ad_uniform(tbase);
        const uint64_t dh = ad_desc(smem_u32(hbuf));
        auto take = [&](bool fix) -> uint32_t {
            ok = __all_sync(kFull, ad_wait(&full[slot], ph, hdr, 0x7211));
            if (fix) {
                ok = __all_sync(kFull, ok && ad_wait(&fixed[slot], (fph >> slot) & 1u, hdr, 0x7212));
                fph ^= 1u << slot;
            }
            tc_fence_after();
            return ring + slot * Tile::STAGE;
        };
        auto next = [&]() {
            issued = true;
            if (++slot == NS) {
                slot = 0;
                ph ^= 1u;
            }
        };
        for (int ti = t_first; ti < n_tasks && ok; ti += t_step) {
            if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
            const int r = ad_uniform(rank_of(idx_in(hdr, task.x, -1, g.n, 711)));
            if (r == 0) continue;
            const uint32_t idesc = ad_idesc((ad_uniform(idx_in(hdr, task.z, 1, NR + 1, 712)) + 15) / 16 * 16);
            for (int k = k_lo, s = 0; k < k_hi && ok; k += KB, ++s) {
                const uint32_t st = take(CONV);
                const int buf = parts1 & 1;
                if (s % Tile::FLUSH == 0) {
                    ok = __all_sync(kFull, ok && ad_wait(&d1empty[buf], ((parts1 >> 1) & 1u) ^ 1u, hdr, 0x7213));
                    tc_fence_after();
                }
                if (!ok) break;
                const int nb = min(KB, k_hi - k);
                const bool last = s % Tile::FLUSH == Tile::FLUSH - 1 || k + KB >= k_hi;
                if (ad_elect()) {
                    for (int b = 0; b < nb; ++b) {
                        const int ks = min(4, (g.d_in - (k + b) * 64) / 16);  // of 16 columns
                        const uint64_t da = ad_desc(st + b * Tile::A_BLK);
                        const uint64_t dx = ad_desc(st + KB * Tile::A_BLK + b * PARTS * Tile::X_BLK);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i >= ks) break;
#pragma unroll
                            for (int p = 0; p < PARTS; ++p)
                                ad_mma(tm + Tile::D1 + buf * NR, da + i * 2, dx + p * (Tile::X_BLK >> 4) + i * 2, idesc,
                                       (s % Tile::FLUSH) | b | i | p);
                        }
                    }
                    tc_commit(&empty[slot]);
                    if (last) tc_commit(&d1full[buf]);
                }
                __syncwarp();
                parts1 += last;
                next();
            }
            if (!ok) break;
            ok = __all_sync(kFull, ad_wait(&hfull, round & 1u, hdr, 0x7214));
            ++round;
            const int rs = (r + 15) / 16;
            const bool fix = cut(r);
            for (int o = o_lo; o < o_hi && ok; o += OC / 16, ++tiles) {
                const uint32_t st = take(fix);
                const int buf = tiles & 1;
                ok = __all_sync(kFull, ok && ad_wait(&d2empty[buf], ((tiles >> 1) & 1u) ^ 1u, hdr, 0x7215));
                if (!ok) break;
                tc_fence_after();
                if (ad_elect()) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint64_t db = ad_desc32(st + u * KS * 4096);
#pragma unroll
                        for (int p = 2; p >= 0; --p)  // the small parts first
#pragma unroll
                            for (int i = 0; i < KS; ++i) {
                                if (i >= rs) break;
                                ad_mma(tm + (buf * 2 + u) * NR, db + i * 256,
                                       dh + ((p * KBK + (i >> 2)) * (Tile::X_BLK >> 4) + (i & 3) * 2), idesc, (2 - p) | i);
                            }
                    }
                    tc_commit(&empty[slot]);
                    tc_commit(&d2full[buf]);
                }
                __syncwarp();
                next();
            }
        }
        // every MMA issued has completed before tensor memory is released
        if (issued) {
            if (ad_elect()) tc_commit(&drain);
            __syncwarp();
            ad_wait(&drain, 0, hdr, 0x7216);
        }
    } else {
        // ------------------------------------------------------------ sums and outputs
        constexpr int NT = NE * 32;
        constexpr int NB = NR * 4 / NE / 16;  // blocks of 16 rows a warp has
        constexpr int PF = 1;                 // blocks of 8 rows loaded ahead
        const int q = warp & 3, rb0 = (warp >> 2) * 16 * NB;  // tensor-memory lanes, first row
        const uint32_t tl = tbase + ((uint32_t)(32 * q) << 16);
        uint32_t round = 0, parts1 = 0, tiles = 0;
        bool ok = true, met = false;
        for (int ti = t_first; ti < n_tasks; ti += t_step) {
            if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
            const int ad = idx_in(hdr, task.x, -1, g.n, 721);
            const int n = idx_in(hdr, task.z, 0, NR + 1, 722);
            const int r = rank_of(ad);
            named_sync(1, NT);  // the rows before are no longer read
            if (tid < n) {
                const size_t t = (size_t)row_of(tid);
                e_row[tid] = (int)t;
                e_ptr[tid] = AdRow{g.base + t * g.ldbase + o_lo * 16, g.y + t * g.ldy + o_lo * 16};
            }
            named_sync(1, NT);
            if (r == 0) {  // no update: base, or 0
                if (g.base == g.y) continue;
                for (int j = warp; j < n; j += NE)
                    ad_copy_row(g.base ? e_ptr[j].base : nullptr, e_ptr[j].y, (o_hi - o_lo) * 16);
                continue;
            }
            // base of 8 rows of a stage of outputs, the lane's two of each row,
            // PF blocks ahead of the sums
            const int nb = min(max((n - rb0 + 7) / 8, 0), 2 * NB);
            const int width = (o_hi - o_lo) * 16;
            int po = 2 * (32 * q + lane), pb = 0;  // the lane's output, from o_lo on
            auto fetch = [&](float2(&v)[8]) {
                if (g.base && po < width) {
                    const AdRow* rows = e_ptr + rb0 + pb * 8;
                    if (rb0 + pb * 8 + 8 <= n) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const float2*>(rows[k].base + po);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (rb0 + pb * 8 + k < n) v[k] = *reinterpret_cast<const float2*>(rows[k].base + po);
                    }
                }
                if (++pb >= nb) {
                    pb = 0;
                    po += OC;
                }
            };
            float2 bv[PF + 1][8];
#pragma unroll
            for (int d = 0; d <= PF; ++d)
#pragma unroll
                for (int k = 0; k < 8; ++k) bv[d][k] = make_float2(0.f, 0.f);

            // ---- 1. the parts of D1 -> this CTA's share
            static_assert(NB == 1, "16 rows a warp");
            float share[16] = {};
            for (int k = k_lo; k < k_hi; k += KB * Tile::FLUSH, ++parts1) {
                const int buf = parts1 & 1;
                if (ok) ok = ad_wait(&d1full[buf], (parts1 >> 1) & 1u, hdr, 0x7221);
                tc_fence_after();
                if (32 * q < r && rb0 < n) {
                    int v[16];
                    tmem_ld16(tl + Tile::D1 + buf * NR + rb0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) share[i] += __int_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d1empty[buf]);
            }
            if (nb > 0)
#pragma unroll
                for (int d = 0; d < PF; ++d) fetch(bv[d]);
            if (round > 0) ad_meet(&meet_b, (round - 1) & 1u, hdr, 0x7222);  // no peer reads `sum` any more
            if (32 * q + lane < r && rb0 < n)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[rb0 + i][32 * q + lane] = share[i];
            named_sync(1, NT);

            // ---- 2. the cluster's sum
            if (!met) ad_cluster_wait();
            met = true;
            if (tid < cs) ad_peer_arrive(&meet_a, tid);
            ad_meet(&meet_a, round & 1u, hdr, 0x7223);
            {
                const int r4 = (r + 15) / 16 * 4;  // fours of components, those behind the rank 0
                const float scale = g.scale ? __ldg(g.scale + ad) : 1.0f;
                // few values: every CTA sums them all; many: each its share, handed to all
                const bool all = n * r4 <= 2 * NT;
                for (int i = all ? tid : cr + cs * tid; i < n * r4; i += all ? NT : cs * NT) {
                    const int j = i / r4, c = (i % r4) * 4;
                    float v[4] = {};
                    if (c < r) {
                        const uint32_t at = smem_u32(&sum[j][c]);
#pragma unroll 4
                        for (int k = 0; k < cs; ++k) {
                            const float4 o = ad_peer_ld(ad_peer(at, k));
                            v[0] += o.x;
                            v[1] += o.y;
                            v[2] += o.z;
                            v[3] += o.w;
                        }
                        const float f = g.sx ? scale * __ldg(g.sx + e_row[j]) : scale;
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = c + k < r ? v[k] * f : 0.0f;
                    }
                    uint32_t p0[3], p1[3];
                    ad_split2(v[0], v[1], p0);
                    ad_split2(v[2], v[3], p1);
                    const uint32_t to = smem_u32(hbuf) + (c >> 6) * Tile::X_BLK + ad_place(j, (c & 63) >> 3) + (c & 4) * 2;
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        if (all) ad_peer_st8(ad_peer(to + p * KBK * Tile::X_BLK, cr), p0[p], p1[p]);
                        else
                            for (int k = 0; k < cs; ++k) ad_peer_st8(ad_peer(to + p * KBK * Tile::X_BLK, k), p0[p], p1[p]);
                    }
                }
                ad_fence_async();  // H is read by the MMAs
                named_sync(1, NT);
                if (tid < cs) ad_peer_arrive(&meet_b, tid);
                if (!all) ad_meet(&meet_b, round & 1u, hdr, 0x7224);
                if (tid == 0) {
                    ad_fence_async();
                    mbar_arrive(&hfull);
                }
                ++round;
            }

            // ---- 3. D2 + base -> y
            for (int o = o_lo; o < o_hi; o += OC / 16, ++tiles) {
                const int buf = tiles & 1;
                const int oo = (o - o_lo) * 16 + 2 * (32 * q + lane);
                const bool in = oo < width;
                if (ok) ok = ad_wait(&d2full[buf], (tiles >> 1) & 1u, hdr, 0x7225);
                tc_fence_after();
                for (int b = 0; b < nb; ++b) {
                    const int rb = rb0 + 8 * b;
                    int v0[8], v1[8];
                    const uint32_t td = tl + buf * 2 * NR + rb;
                    tmem_ld8(td, v0);
                    tmem_ld8(td + NR, v1);
                    fetch(bv[PF]);
                    tmem_ld_wait();
                    if (in) {
                        const AdRow* rows = e_ptr + rb;
                        float2 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = make_float2(bv[0][k].x + __int_as_float(v0[k]), bv[0][k].y + __int_as_float(v1[k]));
                        if (rb + 8 <= n) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) *reinterpret_cast<float2*>(rows[k].y + oo) = v[k];
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (rb + k < n) *reinterpret_cast<float2*>(rows[k].y + oo) = v[k];
                        }
                    }
#pragma unroll
                    for (int d = 0; d < PF; ++d)
#pragma unroll
                        for (int k = 0; k < 8; ++k) bv[d][k] = bv[d + 1][k];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d2empty[buf]);
            }
        }
        __syncwarp();
        if (!met) ad_cluster_wait();
        if (round > 0) ad_meet(&meet_b, (round - 1) & 1u, hdr, 0x7226);  // no peer reads `sum` any more
    }
    __syncwarp();
    if (warp >= NE) ad_cluster_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == NE) tmem_dealloc(tbase, Tile::TCOLS);
}

}  // namespace moe
