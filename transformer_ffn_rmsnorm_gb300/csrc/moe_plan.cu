// moe_plan.cu -- the two ends of the routed block: sorting the (token, slot)
// pairs by expert, and adding each token's weighted results.
//
// The plan is one CTA: it counts the pairs of each expert in shared memory,
// scans the counts, cuts every expert's rows into token tiles of equal width
// (rounded to the 32 columns a tile can end on) and deals the sorted
// positions out.  Equal lanes of a warp count once (match_any), so a few
// popular experts cost no serialised atomics.  The order of an expert's rows depends
// on the order of the warps, the results do not: every column of a product
// is computed the same way wherever it stands.  Other CTAs of the same launch
// write the 16-bit activations of the products where those are not x itself.
//
// The combination adds a token's k fp32 rows in slot order with fp32 weights
// and rounds once.  Bound by reading those rows.
#include <algorithm>

#include "moe.cuh"

namespace ffn {
namespace {

using moe::Plan;
using moe::Tile;

constexpr int kPlanThreads = 1024;

struct PlanParams {
    const int32_t *idx;
    int pairs, k, experts, tile;
    Plan plan;
    const void *x;
    void *x16;
    int64_t nvec;   // 8-element vectors of x
    bool perm;
    unsigned *err;
};

// exclusive prefix sums of two values over the block's 1024 threads
__device__ __forceinline__ void scan2(int &a, int &b, int (*s_warp)[32], int &total_a, int &total_b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sa = a, sb = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ta = __shfl_up_sync(0xffffffffu, sa, o), tb = __shfl_up_sync(0xffffffffu, sb, o);
        if (lane >= o) {
            sa += ta;
            sb += tb;
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = sa;
        s_warp[1][warp] = sb;
    }
    __syncthreads();
    if (warp == 0) {
        int wa = s_warp[0][lane], wb = s_warp[1][lane];
        const int oa = wa, ob = wb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ta = __shfl_up_sync(0xffffffffu, wa, o), tb = __shfl_up_sync(0xffffffffu, wb, o);
            if (lane >= o) {
                wa += ta;
                wb += tb;
            }
        }
        s_warp[0][lane] = wa - oa;
        s_warp[1][lane] = wb - ob;
        if (lane == 31) {
            s_warp[2][0] = wa;
            s_warp[2][1] = wb;
        }
    }
    __syncthreads();
    a = s_warp[0][warp] + sa - a;
    b = s_warp[1][warp] + sb - b;
    total_a = s_warp[2][0];
    total_b = s_warp[2][1];
}

template <typename T>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const PlanParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x > 0) {
        // fp16 copy of x
        const uint4 *src = static_cast<const uint4 *>(p.x);
        uint4 *dst = static_cast<uint4 *>(p.x16);
        bool bad = false;
        const int64_t step = static_cast<int64_t>(gridDim.x - 1) * kPlanThreads;
        for (int64_t i = static_cast<int64_t>(blockIdx.x - 1) * kPlanThreads + threadIdx.x; i < p.nvec; i += step) {
            float f[8];
            Vec16<T>::unpack(src[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) bad |= fabsf(f[e]) > 65504.f && fabsf(f[e]) < INFINITY;
            if (p.perm) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float t = f[e + 1];
                    f[e + 1] = f[e + 2];
                    f[e + 2] = t;
                }
            }
            dst[i] = Vec16<__half>::pack(f);
        }
        if (bad) atomicOr(p.err, DEVERR_RANGE);
        return;
    }
    __shared__ int s_count[moe::kMaxExperts], s_first[moe::kMaxExperts], s_row0[moe::kMaxExperts];
    __shared__ int s_warp[3][32];
    __shared__ int s_widest;
    const int lane = threadIdx.x & 31;
    s_count[threadIdx.x] = 0;
    if (threadIdx.x == 0) s_widest = 0;
    __syncthreads();
    const int rounds = (p.pairs + kPlanThreads - 1) / kPlanThreads;
    for (int r = 0; r < rounds; ++r) {
        const int i = r * kPlanThreads + threadIdx.x;
        const int e = i < p.pairs ? p.idx[i] : -1;
        const bool ok = e >= 0 && e < p.experts;
        const unsigned same = __match_any_sync(0xffffffffu, ok ? e : -1);
        if (ok && __ffs(same) - 1 == lane) atomicAdd(&s_count[e], __popc(same));
    }
    __syncthreads();
    const int c = s_count[threadIdx.x];
    const int nt = (c + p.tile - 1) / p.tile;
    int row0 = c, first = nt, total, ntiles;
    scan2(row0, first, s_warp, total, ntiles);
    s_first[threadIdx.x] = first;
    s_row0[threadIdx.x] = row0;
    if (nt) atomicMax(&s_widest, (((c + nt - 1) / nt) + 31) & ~31);
    __syncthreads();
    if (threadIdx.x == 0) {
        p.plan.header[0] = ntiles;
        p.plan.header[1] = s_widest;
    }
    for (int q = threadIdx.x; q < ntiles; q += kPlanThreads) {
        // the last expert whose first tile is at or before q and that has tiles
        int lo = 0, hi = p.experts - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_first[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        const int ce = s_count[lo], n = (ce + p.tile - 1) / p.tile;
        Tile t;
        t.expert = lo;
        t.first = s_first[lo];
        t.count = n;
        t.cols = (((ce + n - 1) / n) + 31) & ~31;
        t.row0 = s_row0[lo];
        t.rows = ce;
        t.pad0 = t.pad1 = 0;
        p.plan.tiles[q] = t;
    }
    __syncthreads();
    s_count[threadIdx.x] = row0;   // next free row of each expert
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
        const int i = r * kPlanThreads + threadIdx.x;
        const int e = i < p.pairs ? p.idx[i] : -1;
        const bool ok = e >= 0 && e < p.experts;
        const unsigned same = __match_any_sync(0xffffffffu, ok ? e : -1);
        const int leader = __ffs(same) - 1;
        int base = 0;
        if (ok && leader == lane) base = atomicAdd(&s_count[e], __popc(same));
        base = __shfl_sync(0xffffffffu, base, leader);
        const int at = base + __popc(same & ((1u << lane) - 1u));
        if (i < p.pairs) p.plan.pos[i] = ok ? at : -1;
        if (ok) p.plan.row_token[at] = i / p.k;
    }
}

struct CombineParams {
    const int *pos;
    const float *w, *part;
    const void *res;
    void *y;
    int64_t rows, nvec;   // nvec: 8-element vectors of a row
    int k;
};

template <typename T>
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t n = p.rows * p.nvec;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / p.nvec, c = i - t * p.nvec;
        float f[8];
        if (p.res) {
            Vec16<T>::unpack(__ldcs(static_cast<const uint4 *>(p.res) + i), f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = 0.f;
        }
        float sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll 4
        for (int j = 0; j < p.k; ++j) {
            const int at = p.pos[t * p.k + j];
            if (at < 0) continue;
            const float w = p.w[t * p.k + j];
            const float4 *src = reinterpret_cast<const float4 *>(p.part) + (static_cast<int64_t>(at) * p.nvec + c) * 2;
            const float4 a = __ldcs(src), b = __ldcs(src + 1);
            const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, v[e], sum[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += sum[e];
        static_cast<uint4 *>(p.y)[i] = Vec16<T>::pack(f);
    }
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t moe_plan_bytes(int64_t pairs, int64_t experts, int tile) {
    return 256 + align256(static_cast<size_t>(moe::max_tiles(pairs, experts, tile)) * sizeof(Tile)) +
           2 * align256(static_cast<size_t>(pairs) * sizeof(int));
}

Plan moe_plan_carve(void *base, int64_t pairs, int64_t experts, int tile) {
    char *b = static_cast<char *>(base);
    Plan p;
    p.header = reinterpret_cast<int *>(b);
    b += 256;
    p.tiles = reinterpret_cast<Tile *>(b);
    b += align256(static_cast<size_t>(moe::max_tiles(pairs, experts, tile)) * sizeof(Tile));
    p.row_token = reinterpret_cast<int *>(b);
    b += align256(static_cast<size_t>(pairs) * sizeof(int));
    p.pos = reinterpret_cast<int *>(b);
    return p;
}

cudaError_t launch_moe_plan(const int32_t *idx, int64_t rows, int k, int experts, int tile, const Plan &plan,
                            const void *x, void *x16, int64_t d, int dt, bool perm, cudaStream_t s) {
    PlanParams p{};
    p.idx = idx;
    p.pairs = static_cast<int>(rows * k);
    p.k = k;
    p.experts = experts;
    p.tile = tile;
    p.plan = plan;
    p.x = x;
    p.x16 = x16;
    p.nvec = rows * d / 8;
    p.perm = perm;
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    // the copy's CTAs: up to four vectors a thread, at most two a multiprocessor
    const int64_t copy = x16 ? std::min<int64_t>((p.nvec + 4 * kPlanThreads - 1) / (4 * kPlanThreads), 2 * sm_count()) : 0;
    const dim3 grid(static_cast<unsigned>(1 + copy));
    LaunchScope scope(K_MOE_PLAN, s);
    const cudaError_t e = dt == DT_BF16
                              ? launch_dependent(moe_plan_kernel<__nv_bfloat16>, grid, dim3(kPlanThreads), 0, s, p)
                              : launch_dependent(moe_plan_kernel<__half>, grid, dim3(kPlanThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_moe_combine(const Plan &plan, const float *w, const float *part, const void *res, void *y,
                               int64_t rows, int k, int64_t d, int dt, cudaStream_t s) {
    CombineParams p{plan.pos, w, part, res, y, rows, d / 8, k};
    const int64_t blocks = std::min<int64_t>((rows * p.nvec + 255) / 256, 32 * static_cast<int64_t>(sm_count()));
    LaunchScope scope(K_MOE_COMBINE, s);
    const cudaError_t e =
        dt == DT_BF16 ? launch_dependent(moe_combine_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(blocks)),
                                         dim3(256), 0, s, p)
                      : launch_dependent(moe_combine_kernel<__half>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                         s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ffn
