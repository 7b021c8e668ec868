// moe_adapter, moe_adapter_plan: argument checks and launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <string>
#include <type_traits>

#include "moe.h"
#include "moe_adapter.cuh"
#include "moe_adapter_launch.h"
#include "moe_adapter_plan.cuh"
#include "moe_launch.h"

namespace moe {

// Which of the two kernels takes a call.  k_adapter (tasks of 64 rows on
// tcgen05) needs long tasks and ranks that keep mma.sync busy.  Measured (B200,
// d = 6144, rank 64, base given; us with k_adapter_few and with k_adapter, rows
// in runs | mixed):
//   8192 rows of 16 adapters   bf16 214 126 | 215 211   fp32 265 204 | 265 205   codes 220 153 | 220 152
//   8192 rows of 64 adapters   bf16 240 176 | 240 280   fp32 295 293 | 295 295   codes 247 214 | 248 212
//   2048 rows of 4 adapters    bf16  69  59 |  69 105   fp32  84 100 |  84 100   codes  71  74 |  71  74
//   2048 rows of 16 adapters   bf16  70  63 |  70 106   fp32  84 101 |  84 101   codes  71  80 |  71  78
// rank 128, 8 adapters in runs, 8192 rows: bf16 437 143, fp32 525 213; 2048 rows:
// bf16 129 74, fp32 154 108.  Rank 16, bf16 in runs, 8192 rows: 119 111, fp32 144
// 204.  The host knows the adapters of the table, not those that the batch uses,
// nor whether its rows lie in runs (the plan does, on the device), so the rule
// does not take the faster kernel everywhere: 8192 rows of 16 adapters of a table
// of more than 32 (and of 64 adapters, in runs) run on k_adapter_few, 2048 mixed
// bf16 rows and 2048 fp32 rows of up to 8 adapters on k_adapter.
static bool ad_few(const AdArgs& g) {
    return g.r_max <= 32 || g.T < 2048 || g.T / 256 < g.n;
}

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

// Tensor map of bf16 values, `rank` dimensions (the first one contiguous, the
// others `pitch` bytes apart), zeros outside.
static cudaError_t make_map(CUtensorMap* tm, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* pitch,
                            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    if (!enc) return cudaErrorNotSupported;
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, pitch, box, step,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A: rows of components, 64 columns x 16 rows a box.  B: outputs in pairs, 16
// components x 128 outputs of one parity a box.  x (bf16): 64 columns of `rows`
// neighbouring rows, and of one.
static cudaError_t make_maps(const AdArgs& g, bool x_bf16, int rows, CUtensorMap* a, CUtensorMap* b, CUtensorMap* x,
                             CUtensorMap* x1) {
    const cuuint64_t da[2] = {(cuuint64_t)g.d_in, (cuuint64_t)g.n * g.r_max}, pa[1] = {(cuuint64_t)g.d_in * 2};
    const cuuint32_t ba[2] = {64, 16};
    cudaError_t e = make_map(a, g.a, 2, da, pa, ba, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const cuuint64_t db[3] = {(cuuint64_t)g.r_max, 2, (cuuint64_t)g.n * g.d_out / 2};
    const cuuint64_t pb[2] = {(cuuint64_t)g.r_max * 2, (cuuint64_t)g.r_max * 4};
    const cuuint32_t bb[3] = {16, 1, 128};
    e = make_map(b, g.b, 3, db, pb, bb, CU_TENSOR_MAP_SWIZZLE_32B);
    if (e != cudaSuccess || !x_bf16) {
        *x = *x1 = *a;
        return e;
    }
    const cuuint64_t dx[2] = {(cuuint64_t)g.d_in, (cuuint64_t)g.T}, px[1] = {(cuuint64_t)g.ldx * 2};
    const cuuint32_t bx[2] = {64, (cuuint32_t)rows}, b1[2] = {64, 1};
    e = make_map(x, g.x, 2, dx, px, bx, CU_TENSOR_MAP_SWIZZLE_128B);
    return e == cudaSuccess ? make_map(x1, g.x, 2, dx, px, b1, CU_TENSOR_MAP_SWIZZLE_128B) : e;
}

template <typename XT, int RT>
static cudaError_t launch_adapter_t(AdArgs g, cudaStream_t s) {
    using Tile = AdTile<XT, RT>;
    auto fn = k_adapter<XT, RT>;
    cudaError_t e = allow_smem((const void*)fn, Tile::SMEM);
    if (e != cudaSuccess) return e;
    AdLaunch l;
    ad_launch(&l, &g, (const void*)fn, Tile::LIST, Tile::WARPS * 32, Tile::SMEM, s);
    CUtensorMap ma, mb, mx, m1;
    if ((e = make_maps(g, std::is_same<XT, __nv_bfloat16>::value, Tile::NR, &ma, &mb, &mx, &m1)) != cudaSuccess) return e;
    return cudaLaunchKernelEx(&l.c, fn, g, ma, mb, mx, m1);
}

template <typename XT>
static cudaError_t launch_many(const AdArgs& g, cudaStream_t s) {
    return g.r_max <= 64 ? launch_adapter_t<XT, 64>(g, s) : launch_adapter_t<XT, 128>(g, s);  // r_max > 32: ad_few
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_plan_bytes(int32_t n_adapters, int32_t max_tokens) try {
    if (n_adapters < 1 || n_adapters > kAdMaxN || max_tokens < 0) {
        fail(MOE_EINVAL, "n_adapters must be in [1, 1024] and max_tokens >= 0");
        return 0;
    }
    return ad_plan_carve(nullptr, n_adapters, max_tokens).bytes;
} catch (...) {  // (out of host memory)
    return 0;
}

moe_status moe_adapter_plan(int32_t n_adapters, const int32_t* adapter_of, int32_t T, void* plan, size_t plan_bytes,
                            moe_stream_t stream) try {
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
} catch (...) {
    return MOE_ECUDA;
}

moe_status moe_adapter(const moe_adapters* ad, void* plan, size_t plan_bytes, const void* x, moe_dtype dtype,
                       const float* sx, int64_t ldx, int32_t T, const float* base, int64_t ldbase, float* y,
                       int64_t ldy, moe_stream_t stream) try {
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
    const cudaError_t e = ad_few(g) ? launch_adapter_few(g, dtype, s)
                          : dtype == MOE_F32    ? launch_many<float>(g, s)
                          : dtype == MOE_BF16 ? launch_many<__nv_bfloat16>(g, s)
                                              : launch_many<int8_t>(g, s);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, std::string("moe_adapter: ") + cudaGetErrorString(e));
} catch (...) {
    return MOE_ECUDA;
}

}  // extern "C"
