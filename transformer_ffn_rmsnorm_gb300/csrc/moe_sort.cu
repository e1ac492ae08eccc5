// moe_sort.cu -- the tokens of a routed layer in the order of their experts, and
// back, with the gradients:
//
//   sort:     xs[pos_tj] = x_t        pos_tj: place of the pair (t, j) among all pairs with an
//                                     expert, by expert, then token, then slot
//   unsort:   y_t = [res_t +] sum_j w_tj ys[pos_tj]        (w = 1: the gradient of sort)
//   its gradient:  dys[pos_tj] = w_tj dy_t,   dw_tj = <ys[pos_tj], dy_t>
//
// All four are bound by HBM: k rows written (or read) for each one read (or
// written).  A CTA has a token: its row is read once, in 16-byte vectors, and
// goes to k places; or the k rows are read together and added in fp32.
//
// The order is stable, whatever the number of CTAs: a pair's rank among its
// expert's is counted, not dealt out by atomics.  Up to 1024 pairs each CTA counts
// the pairs before its token's k for itself, one launch in all (384 pairs 2.9 us, 7.1
// in three).  Up to 8192 a cluster of eight CTAs counts an eighth of the pairs each
// (ranks inside a warp by comparing lanes, then warp after warp), reads the others'
// counts and writes the places, and the copy follows; more pairs take a CTA a chunk (of
// pieces of 1024 pairs, one after the other), a scan over the chunks' counts and the
// copy.  (1026 pairs 7.1 us by a cluster, 8.8 by chunks; 24576, three pieces a CTA of a
// cluster, 27.6 and 24.6.)
#include <algorithm>

#include "moe.cuh"
#include "moe_sort.cuh"

namespace ffn {
namespace {

constexpr int kSmallPairs = 1024;
constexpr int kCountThreads = 1024, kMaxChunks = 512;
constexpr int kCluster = 8, kClusterPairs = kCluster * kCountThreads;
constexpr int kRowThreads = 128;

int64_t chunk_pairs(int64_t pairs) {
    return ((pairs + kMaxChunks - 1) / kMaxChunks + kCountThreads - 1) / kCountThreads * kCountThreads;
}

struct SortParams {
    const int32_t *idx;
    int pairs, k, experts;
    int32_t *pos, *offsets;
    int *hist;            // [chunks][experts]
    int chunk, chunks;
    const uint4 *x;       // rows of nvec vectors
    uint4 *xs;
    const float *x_scales;
    float *xs_scales;
    int nvec, nscales;
};

// One token's row (vectors first, first + step, ...) and scales to its k places.
__device__ __forceinline__ void copy_row(const SortParams &p, int64_t t, const int *at, int first, int step,
                                         bool scales) {
    const uint4 *src = p.x + t * p.nvec;
    for (int v0 = first; v0 < p.nvec; v0 += 4 * step) {
        uint4 v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (v0 + b * step < p.nvec) v[b] = __ldcs(src + v0 + b * step);
        for (int j = 0; j < p.k; ++j) {
            if (at[j] < 0) continue;
            uint4 *dst = p.xs + static_cast<int64_t>(at[j]) * p.nvec;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (v0 + b * step < p.nvec) __stcs(dst + v0 + b * step, v[b]);
        }
    }
    if (!p.x_scales || !scales) return;
    for (int c = threadIdx.x; c < p.nscales; c += blockDim.x) {
        const float s = p.x_scales[t * p.nscales + c];
        for (int j = 0; j < p.k; ++j)
            if (at[j] >= 0) p.xs_scales[static_cast<int64_t>(at[j]) * p.nscales + c] = s;
    }
}

// Few pairs, a thread each: CTA (piece, t) counts the places of token t's pairs and copies
// a piece of its row; the row of CTAs after the last token's writes offsets.
__global__ void __launch_bounds__(kSmallPairs) moe_sort_small_kernel(const SortParams p) {
    __shared__ int s_count[moe::kMaxExperts];
    __shared__ int s_at[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int i = threadIdx.x, tokens = p.pairs / p.k;
    int e = i < p.pairs ? p.idx[i] : p.experts;
    if (e < 0 || e >= p.experts) e = p.experts;   // after every expert
    const int t = blockIdx.y;
    if (t < tokens) {
        for (int j = 0; j < p.k; ++j) {
            const int own = t * p.k + j;
            int mine = p.idx[own];
            if (mine < 0 || mine >= p.experts) mine = p.experts;
            const int before = __syncthreads_count(e < mine || (e == mine && i < own));
            if (i == 0) s_at[j] = mine < p.experts ? before : -1;
        }
        __syncthreads();
        if (blockIdx.x == 0 && i < p.k) p.pos[t * p.k + i] = s_at[i];
        copy_row(p, t, s_at, blockIdx.x * blockDim.x + i, gridDim.x * blockDim.x, blockIdx.x == 0);
        return;
    }
    if (blockIdx.x) return;
    for (int f = i; f < p.experts; f += blockDim.x) s_count[f] = 0;
    __syncthreads();
    if (e < p.experts) atomicAdd(&s_count[e], 1);
    __syncthreads();
    if (i >= 32) return;
    int before = 0;
    for (int f0 = 0; f0 < p.experts; f0 += 32) {
        const int f = f0 + i;
        int incl = f < p.experts ? s_count[f] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (i >= o) incl += v;
        }
        if (f < p.experts) p.offsets[f + 1] = before + incl;
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (i == 0) p.offsets[0] = 0;
}

// The sum of an expert's counts in the warps before `before`.
__device__ __forceinline__ int count_before(const uint8_t *counts, int before) {
    const uint4 lo = reinterpret_cast<const uint4 *>(counts)[0], hi = reinterpret_cast<const uint4 *>(counts)[1];
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t n = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int left = before - 4 * i;   // bytes of the word that count
        const uint32_t ones = left >= 4 ? 0x01010101u : left <= 0 ? 0u : 0x01010101u & ((1u << (8 * left)) - 1u);
        n = __dp4a(w[i], ones, n);
    }
    return static_cast<int>(n);
}

// Pairs i0 .. i0 + count - 1 by a CTA: counts by expert to s_run, each pair's rank among
// them of its expert to pos (-1: none).  s_count: [experts][32 warps].
__device__ __forceinline__ void count_pairs(const SortParams &p, int64_t i0, int count, uint8_t *s_count, int *s_run) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.experts; e += kCountThreads) s_run[e] = 0;   // (read after a barrier)
    for (int c = 0; c < count && i0 + c < p.pairs; c += kCountThreads) {
        for (int w = threadIdx.x; w < p.experts * 8; w += kCountThreads) reinterpret_cast<uint32_t *>(s_count)[w] = 0u;
        __syncthreads();
        const int64_t i = i0 + c + threadIdx.x;
        const bool in = c + threadIdx.x < count && i < p.pairs;
        int e = in ? p.idx[i] : -1;
        if (e < 0 || e >= p.experts) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int ahead = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && ahead == 0) s_count[e * 32 + warp] = static_cast<uint8_t>(__popc(same));
        __syncthreads();
        if (in) p.pos[i] = e >= 0 ? s_run[e] + ahead + count_before(s_count + e * 32, warp) : -1;
        __syncthreads();
        for (int f = threadIdx.x; f < p.experts; f += kCountThreads) s_run[f] += count_before(s_count + f * 32, 32);
        __syncthreads();
    }
}

// The sum over the threads before this one of a CTA of 1024 and, in total, over all.
__device__ __forceinline__ int scan_threads(int n, int *s_warp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const int w = s_warp[lane];
    return incl - n + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

// A cluster: the places of all pairs and the experts' first rows.
__global__ void __launch_bounds__(kCountThreads) moe_sort_cluster_kernel(const SortParams p) {
    extern __shared__ __align__(16) uint8_t s_count[];
    __shared__ int s_run[moe::kMaxExperts], s_base[moe::kMaxExperts], s_warp[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int rank = static_cast<int>(ptx::cluster_ctarank()), e = threadIdx.x;
    const int64_t i0 = static_cast<int64_t>(rank) * p.chunk;
    count_pairs(p, i0, p.chunk, s_count, s_run);
    ptx::cluster_sync();
    int before = 0, total = 0;
    if (e < p.experts) {
        const uint32_t mine = ptx::smem_u32(&s_run[e]);
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            int n;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(ptx::mapa_shared(mine, r)) : "memory");
            before += r < rank ? n : 0;
            total += n;
        }
    }
    const int first = scan_threads(total, s_warp);
    if (e < p.experts) {
        s_base[e] = first + before;
        if (rank == 0) p.offsets[e + 1] = first + total;
    }
    if (rank == 0 && e == 0) p.offsets[0] = 0;
    ptx::cluster_sync();   // the others have read this CTA's counts; s_base is written
    for (int c = threadIdx.x; c < p.chunk; c += kCountThreads) {
        const int64_t i = i0 + c;
        if (i >= p.pairs) break;
        const int at = p.pos[i];   // (this thread wrote it)
        if (at >= 0) p.pos[i] = at + s_base[p.idx[i]];
    }
}

// A chunk of pairs: counts by expert to hist, ranks to pos.
__global__ void __launch_bounds__(kCountThreads) moe_sort_count_kernel(const SortParams p) {
    extern __shared__ __align__(16) uint8_t s_count[];
    __shared__ int s_run[moe::kMaxExperts];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    count_pairs(p, static_cast<int64_t>(blockIdx.x) * p.chunk, p.chunk, s_count, s_run);
    for (int e = threadIdx.x; e < p.experts; e += kCountThreads)
        p.hist[static_cast<int64_t>(blockIdx.x) * p.experts + e] = s_run[e];
}

// One CTA: the experts' first rows, and in place of each chunk's count of an
// expert the sorted row of its first pair there.  Up to 32 threads an expert,
// each a run of chunks.
__global__ void __launch_bounds__(1024) moe_sort_scan_kernel(const SortParams p) {
    __shared__ int s_part[1024], s_first[1024], s_warp[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int per = min(32, 1024 / p.experts);
    const int e = threadIdx.x % p.experts, g = threadIdx.x / p.experts;
    const bool on = g < per;
    const int c0 = on ? p.chunks * g / per : 0, c1 = on ? p.chunks * (g + 1) / per : 0;
    s_first[threadIdx.x] = 0;
    int sum = 0;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += p.hist[static_cast<int64_t>(c) * p.experts + e];
    s_part[threadIdx.x] = sum;
    __syncthreads();
    int before = 0;
    if (on) {
        for (int q = 0; q < g; ++q) before += s_part[q * p.experts + e];
        if (g == per - 1) s_first[e] = before + sum;
    }
    __syncthreads();
    const int n = s_first[threadIdx.x];   // pairs of expert threadIdx.x
    const int first = scan_threads(n, s_warp);
    s_first[threadIdx.x] = first;
    if (threadIdx.x < p.experts) p.offsets[threadIdx.x + 1] = first + n;
    if (threadIdx.x == 0) p.offsets[0] = 0;
    __syncthreads();
    int row = s_first[e] + before;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        int *h = p.hist + static_cast<int64_t>(c) * p.experts + e;
        const int count = *h;
        *h = row;
        row += count;
    }
}

__global__ void __launch_bounds__(kRowThreads) moe_sort_copy_kernel(const SortParams p) {
    __shared__ int s_at[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < p.k) {
        const int64_t i = t * p.k + threadIdx.x;
        int at = p.pos[i];
        if (at >= 0 && p.hist) {   // (a rank in its chunk)
            at += p.hist[i / p.chunk * p.experts + p.idx[i]];
            p.pos[i] = at;
        }
        s_at[threadIdx.x] = at;
    }
    __syncthreads();
    copy_row(p, t, s_at, threadIdx.x, kRowThreads, true);
}

struct UnsortParams {
    const int32_t *pos;
    const float *w;
    const void *ys, *res, *dy;
    void *y, *dys;
    float *dw;
    int pairs, k, nvec;
};

// A sorted row a token's slot names, or -1.
__device__ __forceinline__ int place(const UnsortParams &p, int64_t i) {
    const int at = p.pos[i];
    return at >= 0 && at < p.pairs ? at : -1;
}

// CTA (t, piece): vectors of y_t.  Eight rows are requested before they are added.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_unsort_kernel(const UnsortParams p) {
    constexpr int EPV = 16 / sizeof(T);
    __shared__ int s_at[32];
    __shared__ float s_w[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < p.k) {
        const int at = place(p, t * p.k + threadIdx.x);
        s_at[threadIdx.x] = at;
        s_w[threadIdx.x] = at < 0 ? 0.f : p.w ? p.w[t * p.k + threadIdx.x] : 1.f;
    }
    __syncthreads();
    for (int c = blockIdx.y * kRowThreads + threadIdx.x; c < p.nvec; c += gridDim.y * kRowThreads) {
        const int64_t i = t * p.nvec + c;
        float sum[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) sum[e] = 0.f;
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < p.k && s_at[j0 + j] >= 0)
                    v[j] = __ldcs(static_cast<const uint4 *>(p.ys) + static_cast<int64_t>(s_at[j0 + j]) * p.nvec + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= p.k || s_at[j0 + j] < 0) continue;   // (a slot without a row is not read)
                float f[EPV];
                Vec16<T>::unpack(v[j], f);
                const float w = s_w[j0 + j];
#pragma unroll
                for (int e = 0; e < EPV; ++e) sum[e] = fmaf(w, f[e], sum[e]);
            }
        }
        if (p.res) {
            float f[EPV];
            Vec16<T>::unpack(__ldcs(static_cast<const uint4 *>(p.res) + i), f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum[e] += f[e];
        }
        static_cast<uint4 *>(p.y)[i] = Vec16<T>::pack(sum);
    }
}

// CTA t: dy_t goes to its k rows, weighted, and is multiplied with ys' there;
// four slots at a time, their dot products added over the CTA at the end.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_unsort_backward_kernel(const UnsortParams p) {
    constexpr int EPV = 16 / sizeof(T), J = 4;
    __shared__ int s_at[32];
    __shared__ float s_w[32], s_dot[kRowThreads / 32][J];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < p.k) {
        const int at = place(p, t * p.k + threadIdx.x);
        s_at[threadIdx.x] = at;
        s_w[threadIdx.x] = at < 0 ? 0.f : p.w[t * p.k + threadIdx.x];
    }
    __syncthreads();
    for (int j0 = 0; j0 < p.k; j0 += J) {
        float dot[J] = {};
        for (int c = threadIdx.x; c < p.nvec; c += kRowThreads) {
            uint4 v[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j0 + j < p.k && s_at[j0 + j] >= 0)
                    v[j] = __ldcs(static_cast<const uint4 *>(p.ys) + static_cast<int64_t>(s_at[j0 + j]) * p.nvec + c);
            float g[EPV];
            Vec16<T>::unpack(__ldg(static_cast<const uint4 *>(p.dy) + t * p.nvec + c), g);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j0 + j >= p.k || s_at[j0 + j] < 0) continue;
                float f[EPV];
                Vec16<T>::unpack(v[j], f);
                const float w = s_w[j0 + j];
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    dot[j] = fmaf(f[e], g[e], dot[j]);
                    f[e] = w * g[e];
                }
                __stcs(static_cast<uint4 *>(p.dys) + static_cast<int64_t>(s_at[j0 + j]) * p.nvec + c,
                       Vec16<T>::pack(f));
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if (lane == 0) s_dot[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < J && j0 + threadIdx.x < p.k) {
            float d = 0.f;
            for (int q = 0; q < kRowThreads / 32; ++q) d += s_dot[q][threadIdx.x];
            p.dw[t * p.k + j0 + threadIdx.x] = d;
        }
        __syncthreads();
    }
}

template <typename T> cudaError_t launch_unsort_typed(const UnsortParams &p, int64_t rows, cudaStream_t s) {
    LaunchScope scope(K_MOE_UNSORT, s);
    cudaError_t e;
    if (p.dy) {
        e = launch_dependent(moe_unsort_backward_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, s,
                             p);
    } else {
        const dim3 grid(static_cast<unsigned>(rows),
                        static_cast<unsigned>(std::min((p.nvec + kRowThreads - 1) / kRowThreads, 65535)));
        e = launch_dependent(moe_unsort_kernel<T>, grid, dim3(kRowThreads), 0, s, p);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_unsort_any(const UnsortParams &p, int64_t rows, int dt, cudaStream_t s) {
    switch (dt) {
        case DT_F32: return launch_unsort_typed<float>(p, rows, s);
        case DT_F16: return launch_unsort_typed<__half>(p, rows, s);
        default: return launch_unsort_typed<__nv_bfloat16>(p, rows, s);
    }
}

}  // namespace

// The chunks' counts.  Their number falls by half where a chunk grows by 1024
// pairs: what every number of pairs up to `pairs` fits into.
size_t moe_sort_workspace(int64_t pairs, int64_t experts) {
    if (pairs <= kClusterPairs) return 0;
    const int64_t full = static_cast<int64_t>(kMaxChunks) * kCountThreads, upto = std::min(pairs, full);
    return static_cast<size_t>((upto + kCountThreads - 1) / kCountThreads) * experts * sizeof(int);
}

cudaError_t launch_moe_sort(const void *x, const float *x_scales, const int32_t *idx, void *xs, float *xs_scales,
                            int32_t *pos, int32_t *offsets, int64_t rows, int64_t row_bytes, int64_t nscales,
                            int experts, int k, void *workspace, cudaStream_t s) {
    SortParams p{};
    p.idx = idx;
    p.pairs = static_cast<int>(rows * k);
    p.k = k;
    p.experts = experts;
    p.pos = pos;
    p.offsets = offsets;
    p.hist = static_cast<int *>(workspace);
    p.chunk = static_cast<int>(chunk_pairs(p.pairs));
    p.chunks = (p.pairs + p.chunk - 1) / p.chunk;
    p.x = static_cast<const uint4 *>(x);
    p.xs = static_cast<uint4 *>(xs);
    p.x_scales = x_scales;
    p.xs_scales = xs_scales;
    p.nvec = static_cast<int>(row_bytes / 16);
    p.nscales = static_cast<int>(nscales);
    cudaError_t e;
    if (p.pairs <= kSmallPairs) {
        const int threads = std::max(128, (p.pairs + 31) / 32 * 32);
        const dim3 grid(static_cast<unsigned>((p.nvec + threads - 1) / threads), static_cast<unsigned>(rows + 1));
        LaunchScope scope(K_MOE_SORT, s);
        e = launch_dependent(moe_sort_small_kernel, grid, dim3(static_cast<unsigned>(threads)), 0, s, p);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    if (p.pairs <= kClusterPairs) {
        p.hist = nullptr;
        p.chunk = (p.pairs + kCluster - 1) / kCluster;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kCluster);
        cfg.blockDim = dim3(kCountThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(experts) * 32;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        LaunchScope scope(K_MOE_SORT, s);
        e = cudaLaunchKernelEx(&cfg, moe_sort_cluster_kernel, p);
    } else {
        LaunchScope scope(K_MOE_SORT, s);
        e = launch_dependent(moe_sort_count_kernel, dim3(static_cast<unsigned>(p.chunks)), dim3(kCountThreads),
                             static_cast<size_t>(experts) * 32, s, p);
    }
    if (e == cudaSuccess && p.hist) {
        LaunchScope scope(K_MOE_SORT, s);
        e = launch_dependent(moe_sort_scan_kernel, dim3(1), dim3(1024), 0, s, p);
    }
    if (e == cudaSuccess) {
        LaunchScope scope(K_MOE_SORT, s);
        e = launch_dependent(moe_sort_copy_kernel, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, s, p);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_moe_unsort(const void *ys, const int32_t *pos, const float *w, const void *res, void *y,
                              int64_t rows, int64_t d, int k, int dt, cudaStream_t s) {
    UnsortParams p{};
    p.pos = pos;
    p.w = w;
    p.ys = ys;
    p.res = res;
    p.y = y;
    p.pairs = static_cast<int>(rows * k);
    p.k = k;
    p.nvec = static_cast<int>(d / (dt == DT_F32 ? 4 : 8));
    return launch_unsort_any(p, rows, dt, s);
}

cudaError_t launch_moe_unsort_backward(const void *dy, const void *ys, const int32_t *pos, const float *w, void *dys,
                                       float *dw, int64_t rows, int64_t d, int k, int dt, cudaStream_t s) {
    UnsortParams p{};
    p.pos = pos;
    p.w = w;
    p.ys = ys;
    p.dy = dy;
    p.dys = dys;
    p.dw = dw;
    p.pairs = static_cast<int>(rows * k);
    p.k = k;
    p.nvec = static_cast<int>(d / (dt == DT_F32 ? 4 : 8));
    return launch_unsort_any(p, rows, dt, s);
}

}  // namespace ffn
