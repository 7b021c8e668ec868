// Low-rank adapters for few rows (moe_adapter on small batches).
#pragma once

#include "moe_adapter.cuh"

namespace moe {

// 8 neighbouring values of a row of a stage as PARTS x 4 bf16 pairs.  at():
// byte offset of the 16-byte chunk c of row j, rows ld bytes apart; its place
// is moved by the row so that a warp's reads meet no bank twice.
template <typename XT>
struct AfX;
template <>
struct AfX<__nv_bfloat16> {
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ ((j & 1) << 2)) << 4); }
    static __device__ __forceinline__ void get(const uint8_t* row, int sw, int c8, uint32_t (&o)[1][4]) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + ((c8 ^ (sw << 2)) << 4));
        o[0][0] = v.x;
        o[0][1] = v.y;
        o[0][2] = v.z;
        o[0][3] = v.w;
    }
    static __device__ __forceinline__ int swap(int j) { return j & 1; }
};
template <>
struct AfX<float> {
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ (j & 1)) << 4); }
    static __device__ __forceinline__ void get(const uint8_t* row, int sw, int c8, uint32_t (&o)[3][4]) {
        const float4 a = *reinterpret_cast<const float4*>(row + (((2 * c8) ^ sw) << 4));
        const float4 b = *reinterpret_cast<const float4*>(row + (((2 * c8 + 1) ^ sw) << 4));
        uint32_t s[4][3];
        ad_split2(a.x, a.y, s[0]);
        ad_split2(a.z, a.w, s[1]);
        ad_split2(b.x, b.y, s[2]);
        ad_split2(b.z, b.w, s[3]);
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[q][i] = s[i][q];
    }
    static __device__ __forceinline__ int swap(int j) { return j & 1; }
};
template <>
struct AfX<int8_t> {
    static __device__ __forceinline__ int at(int j, int c, int ld) { return j * ld + ((c ^ ((j & 3) << 1)) << 4); }
    static __device__ __forceinline__ void get(const uint8_t* row, int sw, int c8, uint32_t (&o)[1][4]) {
        AdX<int8_t> v;
        v.v = *reinterpret_cast<const uint2*>(row + (((c8 >> 1) ^ (sw << 1)) << 4) + (c8 & 1) * 8);
        uint4 q[1];
        v.parts(q);
        o[0][0] = q[0].x;
        o[0][1] = q[0].y;
        o[0][2] = q[0].z;
        o[0][3] = q[0].w;
    }
    static __device__ __forceinline__ int swap(int j) { return j & 3; }
};

// D (16 x 8, float32) += A (16 x 16 bf16) B (16 x 8 bf16)
__device__ __forceinline__ void af_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared, asynchronous.
__device__ __forceinline__ void af_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival on `bar`, once all its copies so far have landed.
__device__ __forceinline__ void af_cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void af_cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Few rows: as k_adapter, a cluster of CTAs takes one task (up to 8 rows of one
// adapter) after the other: its share of A x, the cluster's sum, its share of
// the outputs.  The weights, read once, bound it; the steps between the loads
// are what it is built for: mma.sync with the weights as the 16-row operand and
// the rows as the 8 columns, straight from a stage in shared memory (no
// tensor memory to allocate, drain and read, no descriptors, no parts of x to
// write back), and rows gathered by 16-byte copies of NP warps that run ahead
// through both products.
// MMA operands: a lane's 16 bytes are 8 neighbouring columns (components); the
// same ones stand in the same places of both operands, so their order within
// the k index is free.  The 16 weight rows of an MMA of product 2 are the
// outputs 0 2 4 .. 14 1 3 .. 15, so that a lane has 2 neighbouring outputs.
// Three CTAs on an SM (64 registers, 75 KB) so that the starts, meetings and ends
// of some hide behind the copies of others.  Measured (B200, d = 6144): one row,
// rank 16, 8.6 us -- the chain plan -> task -> row -> x -> A x -> meeting -> y of
// one task; 64 rows of 64 adapters, ranks 4 to 64, fp32: 21.7 us, 1.8 TB/s of the
// weights and rows; 8192 rows of rank 16: 119 us, 4.3 TB/s.  What holds the larger
// ranks back is mma.sync itself (11 cycles for 16 x 8 x 16 on a scheduler, and three
// parts of A x): 210 us for 8192 rows of rank 64.
// RT: components held, a multiple of 16, at least r_max.
// ---------------------------------------------------------------------------
template <typename XT, int RT>
struct AfTile {
    static constexpr int NR = 8, LIST = 0;  // the plan's list
    static constexpr int PARTS = AdX<XT>::PARTS;
    static constexpr int NW = 8, NP = 2;           // multiplying and copying warps
    static constexpr int CTAS = RT <= 64 ? 3 : 1;  // on an SM
    static constexpr int KC = RT == 16 ? 256 : 128, OC = 128;
    static constexpr int KW = KC / 32, NN = NW / KW, NTW = RT / 16 / NN;  // product 1: warps on the steps, on the components
    static constexpr int X_LD = KC * (int)sizeof(XT), A_LD = KC * 2, BASE_LD = OC * 4 + 16;
    static constexpr int X_BYTES = NR * X_LD, BASE_BYTES = NR * BASE_LD;
    static constexpr int S1 = X_BYTES + RT * A_LD, S2 = BASE_BYTES + OC * RT * 2;
    static constexpr int STAGE = ((S1 > S2 ? S1 : S2) + 127) / 128 * 128;
    static constexpr int LD = RT + 4;
    static constexpr int SUM_BYTES = NR * LD * 4, PART_BYTES = KW * SUM_BYTES;
    static constexpr int NS0 = ((CTAS == 3 ? 74 : 200) * 1024 - 2 * SUM_BYTES - PART_BYTES) / STAGE;
    static constexpr int NS = NS0 > 8 ? 8 : NS0 < 3 ? 3 : NS0;
    static constexpr int SMEM = NS * STAGE + 2 * SUM_BYTES + PART_BYTES;
    static_assert(NTW >= 1 && SMEM <= 226 * 1024, "tile");
    static __device__ __forceinline__ int a_at(int j, int c) { return X_BYTES + j * A_LD + ((c ^ ((j & 1) << 2)) << 4); }
    // chunk c of a row of B: of outputs j and j + 2, one of the lanes' pairs, in different banks
    static __device__ __forceinline__ int b_at(int j, int c) {
        if (RT >= 64) return BASE_BYTES + j * RT * 2 + ((c ^ ((j & 2) << 1)) << 4);
        if (RT == 32) return BASE_BYTES + (j ^ ((j >> 1) & 1)) * 64 + (c << 4);
        return BASE_BYTES + j * 32 + (c << 4);
    }
};

template <typename XT, int RT>
__global__ void __launch_bounds__((AfTile<XT, RT>::NW + AfTile<XT, RT>::NP) * 32, AfTile<XT, RT>::CTAS)
    k_adapter_few(const AdArgs g) {
    using Tile = AfTile<XT, RT>;
    constexpr int NR = Tile::NR, NTW = Tile::NTW, NN = Tile::NN, KW = Tile::KW, KC = Tile::KC, OC = Tile::OC;
    constexpr int NQ = (RT + 31) / 32, NCH = RT / 8;  // 32-component steps of product 2, chunks of a row of B
    constexpr int PARTS = Tile::PARTS, LD = Tile::LD, NS = Tile::NS, NW = Tile::NW, SZ = (int)sizeof(XT);
    extern __shared__ __align__(128) uint8_t ad_raw[];
    float(*part)[NR][LD] = reinterpret_cast<float(*)[NR][LD]>(ad_raw + NS * Tile::STAGE);  // per step of a stage
    float(*sum)[LD] = part[KW];                                                           // this CTA's share
    float(*fin)[LD] = sum + NR;                                                           // the cluster's sums, scaled
    __shared__ uint64_t full[NS], empty[NS], meet_a, meet_b;
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
            mbar_init(&full[i], Tile::NP * 32);
            mbar_init(&empty[i], NW);
        }
        mbar_init(&meet_a, cs);
        mbar_init(&meet_b, cs);
        fence_mbar_init();
    }
    __syncthreads();
    ad_cluster_arrive();  // barriers ready; waited for before the first access to a peer
    // this CTA's outputs, 16 at a time, and its columns, KC at a time
    const int groups = g.d_out / 16, steps = (g.d_in + KC - 1) / KC;
    const int o_lo = (int)((long long)groups * cr / cs), o_hi = (int)((long long)groups * (cr + 1) / cs);
    const int k_lo = (int)((long long)steps * cr / cs), k_hi = (int)((long long)steps * (cr + 1) / cs);
    auto rank_of = [&](int ad) { return ad < 0 ? 0 : g.rank ? min(max(__ldg(g.rank + ad), 0), g.r_max) : g.r_max; };
    auto row_of = [&](int j) {
        return idx_in(hdr, __ldg(g.plan.order + idx_in(hdr, task.y + j, 0, g.T, 733)), 0, g.T, 734);
    };

    if (warp >= NW) {
        // ------------------------------------------------------------ copies
        constexpr int NPT = Tile::NP * 32;
        constexpr int CHX = KC * SZ / 16, CHA = KC * 2 / 16, CHY = OC / 4;  // 16-byte chunks of a row
        static_assert(NPT % CHX == 0 && NPT % CHA == 0 && NPT % CHY == 0 && NPT % NCH == 0, "copies");
        constexpr int XRP = NPT / CHX, ARP = NPT / CHA, YRP = NPT / CHY, BRP = NPT / NCH;  // rows a pass
        static_assert(ARP % 2 == 0 && BRP % 4 == 0, "a row a pass further has the same swizzle");
        constexpr int XP = (NR + XRP - 1) / XRP, YP = (NR + YRP - 1) / YRP;
        const int pt = tid - NW * 32;
        const int xc = pt % CHX, xr = pt / CHX, ac = pt % CHA, ar = pt / CHA;
        const int yc = pt % CHY, yr = pt / CHY, bc = pt % NCH, br = pt / NCH;
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
        auto take = [&]() -> uint32_t {  // the next stage, free
            if (ok) ok = ad_wait(&empty[slot], ph ^ 1u, hdr, 0x7301);
            return smem_u32(ad_raw + slot * Tile::STAGE);
        };
        auto next = [&]() {
            af_cp_arrive(&full[slot]);
            if (++slot == NS) {
                slot = 0;
                ph ^= 1u;
            }
        };
        for (int ti = t_first; ti < n_tasks; ti += t_step) {
            if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
            const int ad = idx_in(hdr, task.x, -1, g.n, 731);
            const int n = idx_in(hdr, task.z, 0, NR + 1, 732);
            const int r = rank_of(ad);
            if (r == 0) continue;
            const __nv_bfloat16* A = g.a + ((size_t)ad * g.r_max + ar) * g.d_in + k_lo * KC + ac * 8;
            const __nv_bfloat16* B = g.b + ((size_t)ad * g.d_out + o_lo * 16 + br) * g.r_max + bc * 8;
            const size_t a_step = (size_t)ARP * g.d_in, b_step = (size_t)BRP * g.r_max;
            const XT* xp[XP];
            const float* yp[YP];
#pragma unroll
            for (int p = 0; p < XP; ++p)
                xp[p] = static_cast<const XT*>(g.x) + (xr + p * XRP < n ? (size_t)row_of(xr + p * XRP) : 0) * g.ldx +
                        k_lo * KC + xc * (16 / SZ);
#pragma unroll
            for (int p = 0; p < YP; ++p)
                yp[p] = g.base + (yr + p * YRP < n ? (size_t)row_of(yr + p * YRP) : 0) * g.ldbase + o_lo * 16 + yc * 4;
            const uint32_t ap = Tile::a_at(ar, ac), bp = Tile::b_at(br, bc);
            for (int k = k_lo; k < k_hi; ++k) {
                const uint32_t st = take();
                const int cols = g.d_in - k * KC;  // from this stage on
                if (ok) {
                    if (xc * (16 / SZ) < cols)
#pragma unroll
                        for (int p = 0; p < XP; ++p)
                            if (xr + p * XRP < n) af_cp16(st + AfX<XT>::at(xr + p * XRP, xc, Tile::X_LD), xp[p]);
                    if (ac * 8 < cols) {
                        const __nv_bfloat16* src = A;
                        uint32_t dst = st + ap;
#pragma unroll 4
                        for (int j = ar; j < r; j += ARP, src += a_step, dst += ARP * Tile::A_LD) af_cp16(dst, src);
                    }
                }
#pragma unroll
                for (int p = 0; p < XP; ++p) xp[p] += KC;
                A += KC;
                next();
            }
            for (int o = o_lo; o < o_hi; o += OC / 16) {
                const uint32_t st = take();
                const int no = min(OC / 16, o_hi - o) * 16;
                if (ok) {
                    if (g.base && yc * 4 < no)
#pragma unroll
                        for (int p = 0; p < YP; ++p)
                            if (yr + p * YRP < n) af_cp16(st + (yr + p * YRP) * Tile::BASE_LD + yc * 16, yp[p]);
                    if (bc * 8 < r) {
                        const __nv_bfloat16* src = B;
                        uint32_t dst = st + bp;
#pragma unroll 4
                        for (int j = br; j < no; j += BRP, src += b_step, dst += BRP * RT * 2) af_cp16(dst, src);
                    }
                }
#pragma unroll
                for (int p = 0; p < YP; ++p) yp[p] += OC;
                B += (size_t)OC * g.r_max;
                next();
            }
        }
        af_cp_wait_all();  // every copy has landed before the CTA exits
        __syncwarp();
        ad_cluster_wait();
        return;
    }

    // ---------------------------------------------------------------- products
    const int gr = lane >> 2, gi = lane & 3;
    const int ni = warp % NN, ki = warp / NN;
    int slot = 0;
    uint32_t ph = 0, round = 0;
    bool ok = true, met = false;
    const uint8_t* st = ad_raw;  // the slot's stage
    auto wait_stage = [&]() {
        if (ok) ok = ad_wait(&full[slot], ph, hdr, 0x7303);
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        st += Tile::STAGE;
        if (++slot == NS) {
            slot = 0;
            ph ^= 1u;
            st = ad_raw;
        }
    };
    const int x_swap = AfX<XT>::swap(gr);
    for (int ti = t_first; ti < n_tasks; ti += t_step) {
        if (ti != t_first) task = __ldg(g.plan.tasks[Tile::LIST] + ti);
        const int ad = idx_in(hdr, task.x, -1, g.n, 735);
        const int n = idx_in(hdr, task.z, 0, NR + 1, 736);
        const int r = rank_of(ad);
        if (r == 0) {  // no update: base, or 0
            if (g.base != g.y)
                for (int j = warp; j < n; j += NW) {
                    const size_t t = (size_t)row_of(j);
                    ad_copy_row(g.base ? g.base + t * g.ldbase + o_lo * 16 : nullptr, g.y + t * g.ldy + o_lo * 16,
                                (o_hi - o_lo) * 16);
                }
            continue;
        }
        // the lane's two rows of the outputs
        const bool on0 = 2 * gi < n, on1 = 2 * gi + 1 < n;
        float* y0 = g.y + (on0 ? (size_t)row_of(2 * gi) : 0) * g.ldy + (o_lo + warp) * 16 + gr * 2;
        float* y1 = g.y + (on1 ? (size_t)row_of(2 * gi + 1) : 0) * g.ldy + (o_lo + warp) * 16 + gr * 2;

        // ---- 1. A x over this CTA's columns
        {
            float acc[NTW][4] = {}, low[PARTS > 1 ? NTW : 1][4] = {};
            for (int k = k_lo; k < k_hi; ++k) {
                wait_stage();
                const int left = g.d_in - k * KC - ki * 32;  // columns from the warp's step on
                if (left > 0) {
                    uint32_t u[PARTS][4];
                    AfX<XT>::get(st + gr * Tile::X_LD, x_swap, ki * 4 + gi, u);
                    const bool out = gi * 8 >= left;  // behind the last column
                    if (out)
#pragma unroll
                        for (int q = 0; q < PARTS; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) u[q][i] = 0u;
#pragma unroll
                    for (int i = 0; i < NTW; ++i) {
                        const int t = ni + i * NN;
                        if (t * 16 >= r) break;
                        uint4 w0 = *reinterpret_cast<const uint4*>(st + Tile::a_at(t * 16 + gr, ki * 4 + gi));
                        uint4 w1 = *reinterpret_cast<const uint4*>(st + Tile::a_at(t * 16 + gr + 8, ki * 4 + gi));
                        if (out) w0 = w1 = make_uint4(0u, 0u, 0u, 0u);
                        af_mma(acc[i], w0.x, w1.x, w0.y, w1.y, u[0][0], u[0][1]);
                        af_mma(acc[i], w0.z, w1.z, w0.w, w1.w, u[0][2], u[0][3]);
#pragma unroll
                        for (int q = 1; q < PARTS; ++q) {
                            af_mma(low[i], w0.x, w1.x, w0.y, w1.y, u[q][0], u[q][1]);
                            af_mma(low[i], w0.z, w1.z, w0.w, w1.w, u[q][2], u[q][3]);
                        }
                    }
                }
                release();
            }
#pragma unroll
            for (int i = 0; i < NTW; ++i) {
                const int t = ni + i * NN;
                if (t * 16 >= r) break;
                if (PARTS > 1)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][c] += low[i][c];
                float* d = &part[ki][2 * gi][t * 16 + gr];
                d[0] = acc[i][0];
                d[LD] = acc[i][1];
                d[8] = acc[i][2];
                d[LD + 8] = acc[i][3];
            }
        }
        if (round > 0) ad_meet(&meet_b, (round - 1) & 1u, hdr, 0x7304);  // no peer reads `sum` any more
        named_sync(1, NW * 32);
        const int r4 = (r + 3) / 4;
        for (int i = tid; i < n * r4; i += NW * 32) {
            const int j = i / r4, c = (i % r4) * 4;
            float4 v = *reinterpret_cast<const float4*>(&part[0][j][c]);
#pragma unroll
            for (int k = 1; k < KW; ++k) {
                const float4 o = *reinterpret_cast<const float4*>(&part[k][j][c]);
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            *reinterpret_cast<float4*>(&sum[j][c]) = v;
        }
        named_sync(1, NW * 32);

        // ---- 2. the cluster's sum, every CTA for itself
        if (!met) ad_cluster_wait();
        met = true;
        if (tid < cs) ad_peer_arrive(&meet_a, tid);
        ad_meet(&meet_a, round & 1u, hdr, 0x7305);
        {
            const float scale = g.scale ? __ldg(g.scale + ad) : 1.0f;
            for (int i = tid; i < n * r4; i += NW * 32) {
                const int j = i / r4, c = (i % r4) * 4;
                const uint32_t at = smem_u32(&sum[j][c]);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = 0; k < cs; ++k) {
                    const float4 o = ad_peer_ld(ad_peer(at, k));
                    v.x += o.x;
                    v.y += o.y;
                    v.z += o.z;
                    v.w += o.w;
                }
                const float f = g.sx ? scale * __ldg(g.sx + row_of(j)) : scale;
                *reinterpret_cast<float4*>(&fin[j][c]) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            }
            named_sync(1, NW * 32);
            if (tid < cs) ad_peer_arrive(&meet_b, tid);
            ++round;
        }

        // ---- 3. B (A x) over this CTA's outputs: A x in registers
        uint32_t h[NQ][3][4];  // [step][part][pairs]
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            float v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int k = q * 32 + gi * 8 + c;
                v[c] = gr < n && k < r ? fin[gr][k] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t p[3];
                ad_split2(v[2 * u], v[2 * u + 1], p);
                h[q][0][u] = p[0];
                h[q][1][u] = p[1];
                h[q][2][u] = p[2];
            }
        }
        // the lane's places in B: where it has no components left (its part of A x
        // is 0), the first ones, which are finite if the output is
        int at0[NQ], at1[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int c = q * 32 + gi * 8 < r ? q * 4 + gi : 0;
            at0[q] = Tile::b_at(warp * 16 + 2 * gr, c);
            at1[q] = Tile::b_at(warp * 16 + 2 * gr + 1, c);
        }
        const bool ragged = (r & 7) != 0;  // the last 8 components are cut
        for (int o = o_lo; o < o_hi; o += OC / 16, y0 += OC, y1 += OC) {
            wait_stage();
            if (o + warp < o_hi) {
                float a[4] = {}, b[4] = {};
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    if (q * 32 >= r) break;
                    uint4 w0 = *reinterpret_cast<const uint4*>(st + at0[q]);
                    uint4 w1 = *reinterpret_cast<const uint4*>(st + at1[q]);
                    if (ragged) {
                        const int left = max(r - q * 32 - gi * 8, 0);
                        w0 = ad_first(w0, left);
                        w1 = ad_first(w1, left);
                    }
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        float(&d)[4] = p ? b : a;
                        af_mma(d, w0.x, w1.x, w0.y, w1.y, h[q][p][0], h[q][p][1]);
                        af_mma(d, w0.z, w1.z, w0.w, w1.w, h[q][p][2], h[q][p][3]);
                    }
                }
                float2 v0 = make_float2(0.f, 0.f), v1 = v0;
                if (g.base) {
                    v0 = *reinterpret_cast<const float2*>(st + 2 * gi * Tile::BASE_LD + (warp * 16 + gr * 2) * 4);
                    v1 = *reinterpret_cast<const float2*>(st + (2 * gi + 1) * Tile::BASE_LD + (warp * 16 + gr * 2) * 4);
                }
                if (on0) *reinterpret_cast<float2*>(y0) = make_float2(v0.x + (a[0] + b[0]), v0.y + (a[2] + b[2]));
                if (on1) *reinterpret_cast<float2*>(y1) = make_float2(v1.x + (a[1] + b[1]), v1.y + (a[3] + b[3]));
            }
            release();
        }
    }
    __syncwarp();
    if (!met) ad_cluster_wait();
    if (round > 0) ad_meet(&meet_b, (round - 1) & 1u, hdr, 0x7307);  // no peer reads `sum` any more
}

}  // namespace moe
