// moe_plan.cu -- the two ends of the routed block: sorting the (token, slot)
// pairs by expert, and adding each token's weighted results.
//
// The plan counts the pairs of each expert in shared memory, scans the
// counts, cuts every expert's rows into token tiles of equal width and deals
// the sorted positions out.  Up to 256 pairs (decode) every CTA of one
// launch does that for itself and copies a share of x's rows to their sorted
// places; more pairs are sorted by one CTA and copied by a second kernel (a
// launch is then small beside the products).  In the large form the order of an expert's
// rows depends on the order of the warps; the results do not: every column
// of a product is computed the same way wherever it stands.
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

constexpr int kSmallPairs = 256;   // up to here one launch plans and copies

struct PlanParams {
    const int32_t *idx;
    int pairs, k, experts;
    moe::Cut cut;
    Plan plan;
    const void *x;
    void *xs;
    int nvec;   // 8-element vectors of a row of x
    bool to_f16, perm;
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

// One 8-element vector of x as the products read it.
template <typename T>
__device__ __forceinline__ uint4 convert_vec(const PlanParams &p, const uint4 &v, bool &bad) {
    if (!p.to_f16) return v;
    float f[8];
    Vec16<T>::unpack(v, f);
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
    return Vec16<__half>::pack(f);
}

struct PlanShared {
    int count[moe::kMaxExperts], first[moe::kMaxExperts], row0[moe::kMaxExperts];
    int warp[3][32];
    int widest;
};

// From the experts' counts in sh.count: first tiles, first rows, the tables.
__device__ __forceinline__ void plan_tables(const PlanParams &p, PlanShared &sh) {
    const int c = sh.count[threadIdx.x];
    const int nt = (c + p.cut.tile - 1) / p.cut.tile;
    int row0 = c, first = nt, total, ntiles;
    scan2(row0, first, sh.warp, total, ntiles);
    sh.first[threadIdx.x] = first;
    sh.row0[threadIdx.x] = row0;
    auto width = [&](int rows, int tiles) {
        return ((rows + tiles - 1) / tiles + p.cut.gran - 1) / p.cut.gran * p.cut.gran;
    };
    if (nt) atomicMax(&sh.widest, width(c, nt));
    __syncthreads();
    if (threadIdx.x == 0) {
        p.plan.header[0] = ntiles;
        p.plan.header[1] = sh.widest;
        p.plan.header[2] = total;
    }
    for (int q = threadIdx.x; q < ntiles; q += kPlanThreads) {
        // the last expert whose first tile is at or before q (one without
        // tiles shares its first with the next one)
        int lo = 0, hi = p.experts - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sh.first[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        Tile t;
        t.expert = lo;
        t.first = sh.first[lo];
        t.rows = sh.count[lo];
        t.count = (t.rows + p.cut.tile - 1) / p.cut.tile;
        t.cols = width(t.rows, t.count);
        t.row0 = sh.row0[lo];
        t.pad0 = t.pad1 = 0;
        p.plan.tiles[q] = t;
    }
}

// Few pairs: every CTA sorts them for itself, by counting for each pair the
// pairs before it in sorted order (no scan: two barriers in all), and copies
// its piece of one sorted row; the first CTA writes the tables.
template <typename T>
__global__ void __launch_bounds__(kSmallPairs) moe_plan_small_kernel(const PlanParams p) {
    __shared__ __align__(16) int s_e[kSmallPairs], s_lead[kSmallPairs], s_tiles[kSmallPairs];
    __shared__ int s_token, s_ntiles, s_widest;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int i = threadIdx.x, r = blockIdx.y;
    int e = i < p.pairs ? p.idx[i] : -1;
    if (e < 0 || e >= p.experts) e = -1;
    s_e[i] = e;
    if (i == 0) s_token = -1;
    if (i == 0) s_ntiles = s_widest = 0;
    __syncthreads();
    int at = -1, rank = 0, count = 0;
    if (e >= 0) {
        const int4 *v = reinterpret_cast<const int4 *>(s_e);
        int less = 0;
        for (int j = 0; 4 * j < p.pairs; ++j) {
            const int4 o = v[j];
            const int all[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                less += all[q] >= 0 && all[q] < e;
                count += all[q] == e;
                rank += all[q] == e && 4 * j + q < i;
            }
        }
        at = less + rank;
        if (at == r) s_token = i / p.k;
    }
    if (blockIdx.x == 0 && r == 0) {
        const bool lead = e >= 0 && rank == 0;   // the expert's first pair
        const int nt = lead ? (count + p.cut.tile - 1) / p.cut.tile : 0;
        s_lead[i] = lead ? e : 0x7fffffff;
        s_tiles[i] = nt;
        const int total = __syncthreads_count(e >= 0);
        if (lead) {
            int first = 0;
            for (int j = 0; j < p.pairs; ++j) first += s_lead[j] < e ? s_tiles[j] : 0;
            Tile t;
            t.expert = e;
            t.first = first;
            t.rows = count;
            t.count = nt;
            t.cols = ((count + nt - 1) / nt + p.cut.gran - 1) / p.cut.gran * p.cut.gran;
            t.row0 = at;
            t.pad0 = t.pad1 = 0;
            for (int q = 0; q < nt; ++q) p.plan.tiles[first + q] = t;
            atomicMax(&s_ntiles, first + nt);
            atomicMax(&s_widest, t.cols);
        }
        if (i < p.pairs) p.plan.pos[i] = at;
        __syncthreads();
        if (i == 0) {
            p.plan.header[0] = s_ntiles;
            p.plan.header[1] = s_widest;
            p.plan.header[2] = total;
        }
    } else {
        __syncthreads();
    }
    if (s_token < 0) return;
    const uint4 *src = static_cast<const uint4 *>(p.x) + static_cast<int64_t>(s_token) * p.nvec;
    uint4 *dst = static_cast<uint4 *>(p.xs) + static_cast<int64_t>(r) * p.nvec;
    bool bad = false;
    for (int c = blockIdx.x * kSmallPairs + i; c < p.nvec; c += gridDim.x * kSmallPairs)
        dst[c] = convert_vec<T>(p, src[c], bad);
    if (bad) atomicOr(p.err, DEVERR_RANGE);
}

// Many pairs: one CTA.  A pair's rank among its expert's is the counter's
// value when it came (a few experts: counted by warp ballots, so that the
// counters are not hit 32 times a warp).
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const PlanParams p) {
    __shared__ PlanShared sh;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int kBatch = 8;   // index loads in flight a thread
    const int lane = threadIdx.x & 31;
    sh.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.widest = 0;
    __syncthreads();
    auto load = [&](int i) {
        const int e = i < p.pairs ? p.idx[i] : -1;
        return e < p.experts ? e : -1;
    };
    for (int i0 = threadIdx.x; i0 - static_cast<int>(threadIdx.x) < p.pairs; i0 += kBatch * kPlanThreads) {
        int e[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) e[b] = load(i0 + b * kPlanThreads);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kPlanThreads;
            int rank = 0;
            if (p.experts <= 16) {
                for (int x = 0; x < p.experts; ++x) {
                    const unsigned m = __ballot_sync(0xffffffffu, e[b] == x);
                    int base = 0;
                    if (m && lane == 0) base = atomicAdd(&sh.count[x], __popc(m));
                    base = __shfl_sync(0xffffffffu, base, 0);
                    if (e[b] == x) rank = base + __popc(m & ((1u << lane) - 1u));
                }
            } else if (e[b] >= 0) {
                rank = atomicAdd(&sh.count[e[b]], 1);
            }
            if (i < p.pairs) p.plan.pos[i] = e[b] >= 0 ? rank : -1;
        }
    }
    __syncthreads();
    plan_tables(p, sh);
    for (int i0 = threadIdx.x; i0 < p.pairs; i0 += kBatch * kPlanThreads) {
        int e[kBatch], rank[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kPlanThreads;
            e[b] = load(i);
            rank[b] = i < p.pairs ? p.plan.pos[i] : -1;   // written by this thread above
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kPlanThreads;
            if (i >= p.pairs || e[b] < 0) continue;
            const int at = sh.row0[e[b]] + rank[b];
            p.plan.pos[i] = at;
            p.plan.row_token[at] = i / p.k;
        }
    }
}

// The sorted copy of x's rows, after moe_plan_kernel: a row per CTA.
template <typename T>
__global__ void __launch_bounds__(256) moe_gather_kernel(const PlanParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int r = blockIdx.x;
    if (r >= p.plan.header[2]) return;
    const uint4 *src = static_cast<const uint4 *>(p.x) + static_cast<int64_t>(p.plan.row_token[r]) * p.nvec;
    uint4 *dst = static_cast<uint4 *>(p.xs) + static_cast<int64_t>(r) * p.nvec;
    bool bad = false;
    for (int c0 = threadIdx.x; c0 < p.nvec; c0 += 2 * blockDim.x) {
        const int c1 = c0 + blockDim.x;
        const uint4 a = src[c0], b = c1 < p.nvec ? src[c1] : make_uint4(0, 0, 0, 0);
        dst[c0] = convert_vec<T>(p, a, bad);
        if (c1 < p.nvec) dst[c1] = convert_vec<T>(p, b, bad);
    }
    if (bad) atomicOr(p.err, DEVERR_RANGE);
}

struct CombineParams {
    const int *pos;
    const float *w, *part;
    const void *res;
    void *y;
    int64_t nvec;         // 8-element vectors of a row
    int64_t split_stride; // floats from one split of part to the next
    int k, splits;
};

template <typename T>
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    for (int64_t c = blockIdx.y * blockDim.x + threadIdx.x; c < p.nvec; c += gridDim.y * blockDim.x) {
        const int64_t i = t * p.nvec + c;
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
            const float *src = p.part + (static_cast<int64_t>(at) * p.nvec + c) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            for (int sp = 0; sp < p.splits; ++sp, src += p.split_stride) {
                const float4 a = __ldcs(reinterpret_cast<const float4 *>(src)),
                             b = __ldcs(reinterpret_cast<const float4 *>(src) + 1);
                v[0] += a.x;
                v[1] += a.y;
                v[2] += a.z;
                v[3] += a.w;
                v[4] += b.x;
                v[5] += b.y;
                v[6] += b.z;
                v[7] += b.w;
            }
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

namespace {

template <typename T>
cudaError_t launch_plan(const PlanParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.pairs <= kSmallPairs) {
        // two vectors a thread
        const dim3 grid(static_cast<unsigned>((p.nvec + 2 * kSmallPairs - 1) / (2 * kSmallPairs)),
                        static_cast<unsigned>(p.pairs));
        LaunchScope scope(K_MOE_PLAN, s);
        e = launch_dependent(moe_plan_small_kernel<T>, grid, dim3(kSmallPairs), 0, s, p);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    {
        LaunchScope scope(K_MOE_PLAN, s);
        e = launch_dependent(moe_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    }
    if (e != cudaSuccess) return e;
    const unsigned threads = static_cast<unsigned>(std::min<int64_t>(256, (p.nvec + 31) / 32 * 32));
    LaunchScope scope(K_MOE_PLAN, s);
    e = launch_dependent(moe_gather_kernel<T>, dim3(static_cast<unsigned>(p.pairs)), dim3(threads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_plan(const int32_t *idx, int64_t rows, int k, int experts, moe::Cut cut, const Plan &plan,
                            const void *x, void *xs, int64_t d, int dt, bool to_f16, bool perm, cudaStream_t s) {
    PlanParams p{};
    p.idx = idx;
    p.pairs = static_cast<int>(rows * k);
    p.k = k;
    p.experts = experts;
    p.cut = cut;
    p.plan = plan;
    p.x = x;
    p.xs = xs;
    p.nvec = static_cast<int>(d / 8);
    p.to_f16 = to_f16;
    p.perm = perm;
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    return dt == DT_BF16 ? launch_plan<__nv_bfloat16>(p, s) : launch_plan<__half>(p, s);
}

cudaError_t launch_moe_combine(const Plan &plan, const float *w, const float *part, int splits, const void *res,
                               void *y, int64_t rows, int k, int64_t d, int dt, cudaStream_t s) {
    CombineParams p{plan.pos, w, part, res, y, d / 8, rows * k * d, k, splits};
    const unsigned threads = static_cast<unsigned>(std::min<int64_t>(256, (p.nvec + 31) / 32 * 32));
    const dim3 grid(static_cast<unsigned>(rows),
                    static_cast<unsigned>(std::min<int64_t>((p.nvec + threads - 1) / threads, 65535)));
    LaunchScope scope(K_MOE_COMBINE, s);
    const cudaError_t e =
        dt == DT_BF16 ? launch_dependent(moe_combine_kernel<__nv_bfloat16>, grid, dim3(threads), 0, s, p)
                      : launch_dependent(moe_combine_kernel<__half>, grid, dim3(threads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int moe_down_splits(int64_t pairs, int64_t experts, int64_t d, int64_t ffn) {
    const int64_t units = std::min(pairs, experts) * ((d + 127) / 128), stages = (ffn + 127) / 128;
    constexpr int64_t kSms = 152;   // (not the current device's: the workspace depends on it)
    if (pairs > 1024) return 1;   // tiles enough, and each split writes a row a pair
    int best = 1;
    double least = 0.;
    for (int s = 1; s <= 8 && stages / s >= 4; ++s) {
        const double t = static_cast<double>((units * s + kSms - 1) / kSms) / s;
        if (s == 1 || t < 0.98 * least) {
            best = s;
            least = t;
        }
    }
    return best;
}

}  // namespace ffn
