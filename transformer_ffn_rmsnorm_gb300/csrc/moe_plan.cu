// moe_plan.cu -- the two ends of the routed block: sorting the (token, slot)
// pairs by expert, and adding each token's weighted results.
//
// The plan counts the pairs of each expert, scans the counts, cuts every
// expert's rows into token tiles of equal width and deals the sorted
// positions out.  Up to 256 pairs (decode) every CTA of one launch does that
// for itself and copies a piece of a row of x to its sorted place.  More pairs
// take three kernels: counts of chunks of pairs (shared-memory atomics, whose
// old values are the pairs' ranks), one CTA's scan over chunks and experts, and
// the copy, a warp a row.  (One CTA for the first two took 21 us for 24576
// pairs, the atomics of 32 warps one after the other.)  In the large form the
// order of an expert's rows depends on the order of the warps; the results do
// not: every column of a product is computed the same way wherever it stands.
//
// Where h is fp16, the copy also sets the row's levels to 0 and its scale to 1
// (moe.cuh).
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
constexpr int kChunkThreads = 256, kMaxChunks = 512;

// pairs of a chunk: a multiple of 256, at most kMaxChunks chunks
constexpr int64_t chunk_pairs(int64_t pairs) {
    return ((pairs + kMaxChunks - 1) / kMaxChunks + kChunkThreads - 1) / kChunkThreads * kChunkThreads;
}

struct PlanParams {
    const int32_t *idx;
    int pairs, k, experts;
    moe::Cut cut;
    Plan plan;
    const void *x;
    void *xs;
    int nvec;   // 8-element vectors of a row of x
    int chunk, chunks;
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
    int part[kPlanThreads];
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
        p.plan.header[2] = 0;
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
        t.done = t.odd = 0;
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
        __syncthreads();
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
            t.done = t.odd = 0;
            for (int q = 0; q < nt; ++q) p.plan.tiles[first + q] = t;
            atomicMax(&s_ntiles, first + nt);
            atomicMax(&s_widest, t.cols);
        }
        if (i < p.pairs) p.plan.pos[i] = at;
        __syncthreads();
        if (i == 0) {
            p.plan.header[0] = s_ntiles;
            p.plan.header[1] = s_widest;
            p.plan.header[2] = 0;
        }
    } else {
        __syncthreads();
    }
    if (s_token < 0) return;
    if (p.plan.scale && blockIdx.x == 0) {
        if (i == 0) p.plan.scale[r] = 1.f;
        for (int c = i; c < p.plan.nlevel; c += kSmallPairs)
            p.plan.level[static_cast<int64_t>(r) * p.plan.nlevel + c] = make_uint4(0, 0, 0, 0);
    }
    const uint4 *src = static_cast<const uint4 *>(p.x) + static_cast<int64_t>(s_token) * p.nvec;
    uint4 *dst = static_cast<uint4 *>(p.xs) + static_cast<int64_t>(r) * p.nvec;
    bool bad = false;
    for (int c = blockIdx.x * kSmallPairs + i; c < p.nvec; c += gridDim.x * kSmallPairs)
        dst[c] = convert_vec<T>(p, src[c], bad);
    if (bad) atomicOr(p.err, DEVERR_RANGE);
}

// Many pairs: a CTA counts a chunk's pairs by expert; a pair's rank in the
// chunk is the counter's value when it came.
__global__ void __launch_bounds__(kChunkThreads) moe_count_kernel(const PlanParams p) {
    __shared__ int s_count[moe::kMaxExperts];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int e = threadIdx.x; e < p.experts; e += kChunkThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
    for (int j = threadIdx.x; j < p.chunk; j += kChunkThreads) {
        const int64_t i = i0 + j;
        if (i >= p.pairs) break;
        const int e = p.idx[i];
        p.plan.pos[i] = e >= 0 && e < p.experts ? atomicAdd(&s_count[e], 1) : -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kChunkThreads)
        p.plan.hist[static_cast<int64_t>(blockIdx.x) * p.experts + e] = s_count[e];
}

// One CTA: the tables, and in place of each chunk's count of an expert the
// sorted row of the chunk's first pair there.  Up to 32 threads an expert,
// each a run of chunks.
__global__ void __launch_bounds__(kPlanThreads) moe_scan_kernel(const PlanParams p) {
    __shared__ PlanShared sh;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int per = min(32, kPlanThreads / p.experts);
    const int e = threadIdx.x % p.experts, g = threadIdx.x / p.experts;
    const bool on = g < per;
    const int c0 = on ? p.chunks * g / per : 0, c1 = on ? p.chunks * (g + 1) / per : 0;
    sh.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.widest = 0;
    int sum = 0;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += p.plan.hist[static_cast<int64_t>(c) * p.experts + e];
    sh.part[threadIdx.x] = sum;
    __syncthreads();
    int before = 0;
    if (on) {
        for (int q = 0; q < g; ++q) before += sh.part[q * p.experts + e];
        if (g == per - 1) sh.count[e] = before + sum;
    }
    __syncthreads();
    plan_tables(p, sh);
    int row = sh.row0[e] + before;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        int *h = p.plan.hist + static_cast<int64_t>(c) * p.experts + e;
        const int n = *h;
        *h = row;
        row += n;
    }
}

// A warp per pair: its sorted row, and x's row copied there.
template <typename T>
__global__ void __launch_bounds__(256) moe_gather_kernel(const PlanParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (i >= p.pairs) return;
    const int rank = p.plan.pos[i];
    if (rank < 0) return;
    const int at = p.plan.hist[i / p.chunk * p.experts + p.idx[i]] + rank;
    __syncwarp();   // every lane has read the rank
    if (lane == 0) p.plan.pos[i] = at;
    if (p.plan.scale) {
        if (lane == 0) p.plan.scale[at] = 1.f;
        for (int c = lane; c < p.plan.nlevel; c += 32)
            p.plan.level[static_cast<int64_t>(at) * p.plan.nlevel + c] = make_uint4(0, 0, 0, 0);
    }
    const uint4 *src = static_cast<const uint4 *>(p.x) + i / p.k * p.nvec;
    uint4 *dst = static_cast<uint4 *>(p.xs) + static_cast<int64_t>(at) * p.nvec;
    bool bad = false;
    for (int v0 = lane; v0 < p.nvec; v0 += 8 * 32) {
        uint4 v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b)
            if (v0 + 32 * b < p.nvec) v[b] = src[v0 + 32 * b];
#pragma unroll
        for (int b = 0; b < 8; ++b)
            if (v0 + 32 * b < p.nvec) dst[v0 + 32 * b] = convert_vec<T>(p, v[b], bad);
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

size_t hist_bytes(int64_t pairs, int64_t experts) {
    if (pairs <= kSmallPairs) return 0;
    const int64_t chunk = chunk_pairs(pairs);
    return align256(static_cast<size_t>((pairs + chunk - 1) / chunk) * experts * sizeof(int));
}

}  // namespace

size_t moe_plan_bytes(int64_t pairs, int64_t experts, int tile) {
    return 256 + align256(static_cast<size_t>(moe::max_tiles(pairs, experts, tile)) * sizeof(Tile)) +
           hist_bytes(pairs, experts) + align256(static_cast<size_t>(pairs) * sizeof(int));
}

// (the number of chunks falls by half where they grow by 256 pairs)
size_t moe_plan_bytes_upto(int64_t pairs, int64_t experts, int tile) {
    const int64_t full = static_cast<int64_t>(kMaxChunks) * kChunkThreads;
    return moe_plan_bytes(pairs, experts, tile) - hist_bytes(pairs, experts) +
           std::max(hist_bytes(pairs, experts), hist_bytes(std::min(pairs, full), experts));
}

Plan moe_plan_carve(void *base, int64_t pairs, int64_t experts, int tile) {
    char *b = static_cast<char *>(base);
    Plan p;
    p.header = reinterpret_cast<int *>(b);
    b += 256;
    p.tiles = reinterpret_cast<Tile *>(b);
    b += align256(static_cast<size_t>(moe::max_tiles(pairs, experts, tile)) * sizeof(Tile));
    p.hist = reinterpret_cast<int *>(b);
    b += hist_bytes(pairs, experts);
    p.pos = reinterpret_cast<int *>(b);
    p.scale = nullptr;
    p.level = nullptr;
    p.nlevel = 0;
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
        e = launch_dependent(moe_count_kernel, dim3(static_cast<unsigned>(p.chunks)), dim3(kChunkThreads), 0, s, p);
    }
    if (e == cudaSuccess) {
        LaunchScope scope(K_MOE_PLAN, s);
        e = launch_dependent(moe_scan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    }
    if (e != cudaSuccess) return e;
    LaunchScope scope(K_MOE_PLAN, s);
    e = launch_dependent(moe_gather_kernel<T>, dim3(static_cast<unsigned>((p.pairs + 7) / 8)), dim3(256), 0, s, p);
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
    p.chunk = static_cast<int>(chunk_pairs(p.pairs));
    p.chunks = (p.pairs + p.chunk - 1) / p.chunk;
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

// Where few units leave a last round part empty, splitting fills it, but a unit
// has a fixed cost (its epilogue, the pipeline's fill: about a stage of 128
// values) and every split a row a pair for the combine kernel to add (about
// three stages, and the rows' traffic).
// Down plus combine, each timed by itself between events (in a call they overlap
// a little, and each figure holds some 5 us of launch): 1 token, 4 of 32 Q4
// experts of 5120 x 2176: one split 28.8 us, two 28.1, three 27.9, four 32.3; 16
// tokens, 2 of 8 of 4096 x 14336: one 79.8, two 73.7, four 72.1, seven 78.5.
int moe_down_splits(int64_t pairs, int64_t experts, int64_t d, int64_t ffn) {
    const int64_t units = std::min(pairs, experts) * ((d + 127) / 128), stages = (ffn + 127) / 128;
    constexpr int64_t kSms = 152;   // (not the current device's: the workspace depends on it)
    if (pairs > kMoeSplitPairs) return 1;   // tiles enough, and each split writes a row a pair
    int best = 1;
    double least = 0.;
    for (int s = 1; s <= kMoeMaxSplits && stages / s >= 4; ++s) {
        const double rounds = static_cast<double>((units * s + kSms - 1) / kSms);
        const double t = rounds * (static_cast<double>(stages) / s + 1.) +
                         (s - 1) * (3. + static_cast<double>(pairs * d) / 800000.);
        if (s == 1 || t < least) {
            best = s;
            least = t;
        }
    }
    return best;
}

}  // namespace ffn
