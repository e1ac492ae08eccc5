// linear_e4m3_stream.cu -- products of e4m3 codes with block scales for few rows
// an expert: a stream of weights.
//
// Bound by HBM: every weight is read once.  The WEIGHT rows are the M operand
// (128, one scale block of them) and up to kTile rows of x the N operand, so
// that one row of x costs 16 columns and not 128 rows.  The reduction is cut over a
// cluster of up to 8 CTAs, which gives many short units for few weight rows; the
// CTAs hand each other their parts through distributed shared memory (each
// finishes 128 / splits of the features, adding the parts in the cluster's
// order: the same bits every run), so that a call needs neither a workspace
// nor a second launch.
//
// Two widths: tiles of 32 rows leave room for two CTAs on an SM, whose starts
// and ends overlap; tiles of 128 rows (linear only: with two matrices the pairs are
// faster from there on) take one.
//
// Roles: warp 0 loads, warp 1 issues the MMAs, the warps from 4 on read each block's
// sums and add them up in registers (lane = weight row, column = row of x; gate/up:
// four warps a matrix, linear: each four every second or fourth 16 columns).  The
// columns' scales, times the weight's, go through shared memory.  Every wait is bounded (1 s).
// Tensor memory is given back before a CTA waits for its cluster.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "linear_e4m3.cuh"
#include "moe.cuh"

namespace ffn {
namespace {

using e4::GATEUP;
using e4::LINEAR;
using e4::Params;

template <int MODE, int TILE> struct Config {
    static constexpr int kMats = MODE == GATEUP ? 2 : 1;
    static constexpr int kParts = MODE == LINEAR && TILE == 128 ? 4 : 2;    // of four warps each
    static constexpr int kEpiWarps = 4 * kParts, kThreads = 32 * (4 + kEpiWarps);
    static constexpr uint32_t kStageBytes = kMats * e4::kTileBytes + TILE * 128;
    static constexpr int kCtas = TILE == 32 ? 2 : 1;   // on an SM
    static constexpr int kStages = static_cast<int>((kCtas == 2 ? 108 * 1024 : 200 * 1024) / kStageBytes);
    static constexpr int kBufs = 4;                                         // accumulators in tensor memory
    static constexpr uint32_t kTmemCols = kMats * TILE * kBufs;
    static constexpr int kCols = MODE == GATEUP ? TILE : TILE / kParts;     // columns of a warp
    static constexpr size_t kSmem = kStages * kStageBytes + 1024;
    static constexpr uint32_t kPartBytes = kMats * TILE * 128 * 4;          // the parts a CTA receives
    static_assert(kPartBytes <= kStages * kStageBytes, "the parts take the stages' place");
    static_assert(kTmemCols * kCtas <= 512, "tensor memory");
    static_assert(kCtas * (kSmem + 4608) <= 228 * 1024 && (kCtas + 1) * kSmem > 228 * 1024, "CTAs on an SM");
};

struct UnitInfo {
    int expert, f, row0, valid, n;   // n: columns, a multiple of 16; 0: no such unit
};

// The unit's place (one warp): an expert's units run through its tiles of rows first.
template <int TILE> __device__ __forceinline__ UnitInfo find_unit(const Params &p, int unit, int lane) {
    UnitInfo u{0, 0, 0, 0, 0};
    int tiles_before = 0, rows_before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int2 r = e4::expert_rows(p, e0, lane, rows_before);
        const int tiles = (r.y - r.x + TILE - 1) / TILE;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int first = tiles_before + incl - tiles;
        const bool mine = tiles > 0 && unit >= first * p.nf && unit < (first + tiles) * p.nf;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            const int local = unit - __shfl_sync(0xffffffffu, first, src) * p.nf;
            const int nt = __shfl_sync(0xffffffffu, tiles, src);
            const int a = __shfl_sync(0xffffffffu, r.x, src), b = __shfl_sync(0xffffffffu, r.y, src);
            const int width = ((b - a + nt - 1) / nt + 15) & ~15, tt = local % nt;
            u.expert = e0 + src;
            u.f = local / nt;
            u.row0 = a + tt * width;
            u.valid = min(width, b - u.row0);
            u.n = (u.valid + 15) & ~15;   // (nt - 1 tiles of at most TILE rows leave the last one some)
            return u;
        }
        tiles_before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return u;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

template <int MODE, int TILE>
__global__ void __launch_bounds__((Config<MODE, TILE>::kThreads), (Config<MODE, TILE>::kCtas))
    e4m3_stream_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                       const __grid_constant__ moe::RowMaps maps_x, const Params p, const int splits) {
    using C = Config<MODE, TILE>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
    __shared__ __align__(8) uint64_t bar_tfull[C::kBufs], bar_tempty[C::kBufs], bar_drain;
    __shared__ __align__(16) float s_scale[C::kEpiWarps][2][C::kCols];
    __shared__ uint32_t s_amax[TILE], s_all[8][TILE];
    __shared__ UnitInfo s_unit;
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    auto bar = [](uint64_t *b) { return ptx::smem_u32(b); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(bar(&bar_full[s]), 1);
            ptx::mbar_init(bar(&bar_empty[s]), 1);
        }
        for (int a = 0; a < C::kBufs; ++a) {
            ptx::mbar_init(bar(&bar_tfull[a]), 1);
            ptx::mbar_init(bar(&bar_tempty[a]), C::kEpiWarps);
        }
        ptx::mbar_init(bar(&bar_drain), 1);
        s_abort = 0;
        s_never = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_map(&map_w0);
        if (MODE == GATEUP) ptx::tma_prefetch_map(&map_w1);
        for (int i = 0; i < 4; ++i) ptx::tma_prefetch_map(&maps_x.m[i]);
    }
    if (MODE == GATEUP)
        for (int i = threadIdx.x; i < TILE; i += C::kThreads) s_amax[i] = 0u;
    ptx::griddep_wait();   // x, its scales, offsets (and the weights, where they were just quantised)
    if (warp == 0) {
        const UnitInfo u = find_unit<TILE>(p, static_cast<int>(blockIdx.x) / splits, lane);
        if (lane == 0) s_unit = u;
    }
    __syncthreads();
    const UnitInfo t = s_unit;
    if (t.n == 0) return;   // the same for the whole cluster
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem_base), C::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = s_tmem_base;
    volatile int *abort_flag = &s_abort;
    volatile int *never = &s_never;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / splits),
              kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / splits);
    bool ok = true;
    float acc[C::kCols];
#pragma unroll
    for (int i = 0; i < C::kCols; ++i) acc[i] = 0.f;
    const int q = warp & 3, part = (warp - 4) >> 2;   // of the epilogue warps
    auto column = [&](int j) { return MODE == GATEUP ? j : 16 * C::kParts * (j >> 4) + 16 * part + (j & 15); };

    if (warp == 0) {
        // ------------------------------------------------------ producer
        int s = 0, issued = 0;
        uint32_t ph = 0;
        const int wrow = t.expert * p.out + t.f * 128;
        for (int kb = kb0; kb < kb1; ++kb) {
            const bool got = ptx::mbar_wait(bar(&bar_empty[s]), ph ^ 1u, abort_flag, e4::kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint32_t full = bar(&bar_full[s]), at = base + s * C::kStageBytes;
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(full, C::kMats * e4::kTileBytes + t.n * 128);
                ptx::tma_load_2d(at, &map_w0, full, kb * 128, wrow);
                if (MODE == GATEUP) ptx::tma_load_2d(at + e4::kTileBytes, &map_w1, full, kb * 128, wrow);
                moe::for_row_boxes(maps_x, t.n, [&](const CUtensorMap *m, int r) {
                    ptx::tma_load_2d(at + C::kMats * e4::kTileBytes + r * 128, m, full, kb * 128, t.row0 + r);
                });
            }
            __syncwarp();
            ++issued;
            if (++s == C::kStages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (!ok) *abort_flag = 1;
        // Every load has landed before the stages' place is used again, whoever else gives up and when.
        for (int i = 0; i < C::kStages; ++i)
            if (issued > i)
                ptx::mbar_wait(bar(&bar_full[i]), ((issued - i + C::kStages - 1) / C::kStages - 1) & 1u, never,
                               e4::kWaitNs);
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer
        const uint32_t idesc = e4::idesc_e4m3(128, t.n);
        int s = 0, a = 0;
        uint32_t ph = 0, pa = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            bool got = ptx::mbar_wait(bar(&bar_full[s]), ph, abort_flag, e4::kWaitNs);
            got = got && ptx::mbar_wait(bar(&bar_tempty[a]), pa ^ 1u, abort_flag, e4::kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                const uint32_t at = base + s * C::kStageBytes;
                const uint64_t bd = ptx::sdesc_k_sw128(at + C::kMats * e4::kTileBytes);
#pragma unroll
                for (int m = 0; m < C::kMats; ++m) {
                    const uint64_t ad = ptx::sdesc_k_sw128(at + m * e4::kTileBytes);
                    const uint32_t d = tmem + (a * C::kMats + m) * TILE;
#pragma unroll
                    for (int k = 0; k < 4; ++k) e4::mma_e4m3(d, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                }
                ptx::tc_commit(bar(&bar_empty[s]));
                ptx::tc_commit(bar(&bar_tfull[a]));
            }
            __syncwarp();
            if (++s == C::kStages) {
                s = 0;
                ph ^= 1u;
            }
            if (++a == C::kBufs) {
                a = 0;
                pa ^= 1u;
            }
        }
        if (ptx::elect_one()) ptx::tc_commit(bar(&bar_drain));   // every MMA ends before TMEM is freed
        ptx::mbar_wait(bar(&bar_drain), 0, never, e4::kWaitNs);
    } else if (MODE == LINEAR && warp == 2 && p.res) {
        // the residual that this CTA will add, on its way to L2
        const int es = p.dt == DT_F32 ? 4 : 2, rows = 128 / splits, f0 = t.f * 128 + rank * rows;
        for (int c = lane; c < t.valid && f0 < p.out; c += 32) {
            const char *line = static_cast<const char *>(p.res) + (static_cast<int64_t>(t.row0 + c) * p.out + f0) * es;
            for (int b = 0; b < min(rows, p.out - f0) * es; b += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(line + b));
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------- sums
        constexpr int kPer = (C::kCols + 31) / 32;   // scales of a lane
        const float *ws = (MODE == GATEUP && part ? p.ws[1] : p.ws[0]) +
                          (static_cast<int64_t>(t.expert) * p.nf + t.f) * p.nkb;
        const float *xs[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = lane + 32 * i, c = column(j);
            xs[i] = j < C::kCols && c < t.valid ? p.xs + static_cast<int64_t>(t.row0 + c) * p.nkb : nullptr;
        }
        float next[kPer], wnext = kb0 < kb1 ? __ldg(ws + kb0) : 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) next[i] = xs[i] && kb0 < kb1 ? __ldg(xs[i] + kb0) : 0.f;
        int a = 0;
        uint32_t pa = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            float *sc = s_scale[warp - 4][kb & 1];   // (the other half is read no more since the last __syncwarp)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < C::kCols) sc[lane + 32 * i] = next[i] * wnext;
            if (kb + 1 < kb1) {
                wnext = __ldg(ws + kb + 1);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (xs[i]) next[i] = __ldg(xs[i] + kb + 1);
            }
            __syncwarp();
            const bool got = ptx::mbar_wait(bar(&bar_tfull[a]), pa, abort_flag, e4::kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t taddr =
                tmem + (static_cast<uint32_t>(q * 32) << 16) + (a * C::kMats + (MODE == GATEUP ? part : 0)) * TILE;
#pragma unroll
            for (int j = 0; j < C::kCols; j += 16) {
                if (column(j) < t.n) {
                    uint32_t r[16];
                    ptx::tmem_ld_32x32b_x16(taddr + column(j), r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(sc + j + i);
                        acc[j + i] = fmaf(__uint_as_float(r[i]), f.x, acc[j + i]);
                        acc[j + i + 1] = fmaf(__uint_as_float(r[i + 1]), f.y, acc[j + i + 1]);
                        acc[j + i + 2] = fmaf(__uint_as_float(r[i + 2]), f.z, acc[j + i + 2]);
                        acc[j + i + 3] = fmaf(__uint_as_float(r[i + 3]), f.w, acc[j + i + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(&bar_tempty[a]));
            if (++a == C::kBufs) {
                a = 0;
                pa ^= 1u;
            }
        }
    }
    if (!ok) {
        if (lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
        *abort_flag = 1;
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kTmemCols);
    }
    ptx::cluster_sync();   // no CTA loads or multiplies any more

    // ------------------------------------------ the parts to their features' CTA
    const int rows = 128 / splits;   // features that a CTA finishes
    // part [source][matrix][column / 4][feature], four columns together
    auto part_at = [&](int src, int mat, int col4, int r) {
        return 16u * static_cast<uint32_t>(((src * C::kMats + mat) * (TILE / 4) + col4) * rows + r);
    };
    if (warp >= 4) {
        const int row = 32 * q + lane, dst = row / rows, r = row - dst * rows;
        const uint32_t to = ptx::mapa_shared(base + part_at(rank, MODE == GATEUP ? part : 0, 0, r), dst);
#pragma unroll
        for (int j = 0; j < C::kCols; j += 4)
            if (column(j) < t.valid)
                st_cluster4(to + part_at(0, 0, column(j) >> 2, 0), acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
    ptx::cluster_sync();

    // four columns of a feature a thread
    float4 *parts = reinterpret_cast<float4 *>(smem_raw + (base - ptx::smem_u32(smem_raw)));
    const int f0 = t.f * 128 + rank * rows;
    const int items = (t.valid + 3) / 4 * rows;
    for (int i0 = 32 * warp; i0 < items; i0 += C::kThreads) {   // whole warps
        const int i = i0 + lane, r = i & (rows - 1), c4 = i / rows;
        const bool in = i < items && f0 + r < p.out;
        float v[C::kMats][4];
#pragma unroll
        for (int m = 0; m < C::kMats; ++m) {
            v[m][0] = v[m][1] = v[m][2] = v[m][3] = 0.f;
            if (i < items)
                for (int src = 0; src < splits; ++src) {
                    const float4 f = parts[part_at(src, m, c4, r) >> 4];
                    v[m][0] += f.x;
                    v[m][1] += f.y;
                    v[m][2] += f.z;
                    v[m][3] += f.w;
                }
        }
        if constexpr (MODE == LINEAR) {
            if (!in) continue;
            auto store = [&](auto *y) {
                using T = typename std::remove_reference<decltype(*y)>::type;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (4 * c4 + e >= t.valid) break;
                    const int64_t at = static_cast<int64_t>(t.row0 + 4 * c4 + e) * p.out + f0 + r;
                    if (p.res) v[0][e] += to_f32(static_cast<const T *>(p.res)[at]);
                    y[at] = from_f32<T>(v[0][e]);
                }
            };
            if (p.dt == DT_BF16) store(static_cast<__nv_bfloat16 *>(p.y));
            else if (p.dt == DT_F16) store(static_cast<__half *>(p.y));
            else store(static_cast<float *>(p.y));
        } else {
            float h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = in ? e4::swiglu(v[0][e], v[C::kMats - 1][e]) : 0.f;
                uint32_t m = abs_bits(h[e]);
                const int seg = min(rows, 32);
                for (int o = seg >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (i < items && (lane & (seg - 1)) == 0) atomicMax(&s_amax[4 * c4 + e], m);
            }
            if (i < items)   // (in the place that only this thread read)
                parts[part_at(0, 0, c4, r) >> 4] = make_float4(h[0], h[1], h[2], h[3]);
        }
    }
    if constexpr (MODE == GATEUP) {
        __syncthreads();
        for (int i = threadIdx.x; i < t.valid * splits; i += C::kThreads) {
            const int c = i / splits, dst = i - c * splits;
            st_cluster(ptx::mapa_shared(ptx::smem_u32(&s_all[rank][c]), dst), s_amax[c]);
        }
        ptx::cluster_sync();
        // four features of a row a thread
        const float *h = reinterpret_cast<const float *>(parts);
        for (int i = 4 * threadIdx.x; i < t.valid * rows; i += 4 * C::kThreads) {
            const int r = i & (rows - 1), c = i / rows;
            uint32_t m = 0u;
            for (int src = 0; src < splits; ++src) m = max(m, s_all[src][c]);
            const float amax = floor_amax(__uint_as_float(m)), k = kE4m3Max / amax;
            const int64_t row = t.row0 + c;
            if (rank == 0 && r == 0) p.ys[row * p.nf + t.f] = amax / kE4m3Max;
            const float *from = h + (part_at(0, 0, c >> 2, r) >> 2) + (c & 3);
            if (f0 + r < p.out)   // (out is a multiple of 8)
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.y) + row * p.out + f0 + r) =
                    e4m3x4(from[0] * k, from[4] * k, from[8] * k, from[12] * k);
        }
    }
}

bool map_codes(CUtensorMap *m, const void *ptr, int64_t in, int64_t rows, uint32_t box_rows) {
    return encode_tma_2d(m, ptr, CU_TENSOR_MAP_DATA_TYPE_UINT8, in, rows, in, 128, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, int TILE>
cudaError_t launch(int splits, const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in, const Params &p,
                   cudaStream_t s) {
    using C = Config<MODE, TILE>;
    const auto kern = &e4m3_stream_kernel<MODE, TILE>;
    static std::atomic<int> configured_device{-1};   // (host threads may call at the same time)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device.load(std::memory_order_acquire) != dev) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
        if (e != cudaSuccess) return e;
        configured_device.store(dev, std::memory_order_release);
    }
    CUtensorMap m0, m1;
    moe::RowMaps mx;
    const int64_t wrows = static_cast<int64_t>(p.experts) * p.out;
    // (a map takes the host about a microsecond: none that the kernel does not use)
    bool good = map_codes(&m0, w0, in, wrows, 128);
    if (MODE == GATEUP) good = good && map_codes(&m1, w1, in, wrows, 128);
    else m1 = m0;
    for (int i = 3; i >= 0; --i) {   // boxes of 16, 32, ... rows up to the tile
        if ((128 >> i) <= TILE) good = good && map_codes(&mx.m[i], x, in, p.rows, 128u >> i);
        else mx.m[i] = mx.m[i + 1];
    }
    if (!good) return cudaErrorInvalidValue;
    const int64_t units = moe::max_tiles(p.rows, p.experts, TILE) * p.nf;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    LaunchScope scope(MODE == GATEUP ? K_GATEUP_E4M3 : K_LINEAR_E4M3, s);
    e = cudaLaunchKernelEx(&cfg, kern, m0, m1, mx, p, splits);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_e4m3_stream(e4::Mode mode, bool wide, int splits, const uint8_t *x, const uint8_t *w0,
                               const uint8_t *w1, int64_t in, const Params &p, cudaStream_t s) {
    if (mode == GATEUP) return launch<GATEUP, 32>(splits, x, w0, w1, in, p, s);
    return wide ? launch<LINEAR, 128>(splits, x, w0, w1, in, p, s) : launch<LINEAR, 32>(splits, x, w0, w1, in, p, s);
}

// Which kernel, from the sizes alone (of the experts' rows only the mean is known
// here: 64 experts of 2048 x 1408, 626 rows evenly or 500 of them one expert's, which
// reads its weights 16 times, 72.6 and 72.8 us gate/up; 1536 rows, 24 each or 1473 of
// one, 81.4 and 96.7).  Up to 32 rows an expert the stream of weights: dense 4096 ->
// 14336 gate/up, 32 rows 27.3 us, pairs 32.7, 48 rows (two tiles) 37.5 and 32.8; over
// 64 experts of 2048 x 1408 with 24 rows 80.6 and 83.5, with 48 rows 110 and 84.4.
// Beyond that gate/up runs on the pairs, linear there or in tiles of 128 rows, which
// cut the reduction where few units leave the pairs idle: by the estimates below, us.
// Linear 14336 -> 4096, pairs / tiles of 128: 48 rows 47.3 / 15.0, 128 rows 48.4 /
// 21.2, 256 rows 48.8 / 35.5, 512 rows 49.4 / 64.5; 4096 -> 14336, 64 rows 18.3 /
// 18.2, 128 rows 19.8 / 27.1; 64 experts 1408 -> 2048, 48 rows 46.4 / 77.8.  The pairs'
// units have 256 features, or 128 where that takes as few rounds: 14336 -> 4096, 512
// rows 49.5 / 38.5, 640 rows 50.9 / 72.5, 1024 rows 51.5 / 72.9; 512 rows of 2048 ->
// 2048 12.0 / 9.5; 777 rows of 1024 -> 520 8.9 / 7.0.
cudaError_t launch_e4m3_product(e4::Mode mode, const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in,
                                Params p, cudaStream_t s) {
    p.nf = (p.out + 127) / 128;
    p.nkb = static_cast<int>((in + 127) / 128);
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    const int64_t sms = sm_count(), used = std::min<int64_t>(p.rows, p.experts), mean = (p.rows + used - 1) / used;
    auto units = [&](int tile) { return used * ((mean + tile - 1) / tile) * p.nf; };
    // The most parts of the reduction whose CTAs all run at once, two blocks each: 4096 ->
    // 14336 gate/up, 1 row, 112 units in 1, 2, 4, 8 parts 24.9, 23.5, 29.3, 42.2 us;
    // linear 14336 -> 4096, 32 units 36.8, 20.7, 12.7, 11.7.
    auto parts = [&](int tile, int64_t slots) {
        int n = 8;
        while (n > 1 && (n * units(tile) > slots || 2 * n > p.nkb)) n >>= 1;
        return n;
    };
    if (mean <= 32) return launch_e4m3_stream(mode, false, parts(32, 2 * sms), x, w0, w1, in, p, s);
    if (mode == LINEAR) {
        const int n = parts(128, sms);
        const double block = 0.13 + 0.0027 * static_cast<double>(std::min<int64_t>(mean, 128));
        const double wide = 2. + static_cast<double>((units(128) * n + sms - 1) / sms) * (p.nkb / n * block + 6.);
        auto pairs = [&](int features, double block, double end) {
            const int64_t u = used * ((mean + 255) / 256) * ((p.out + features - 1) / features);
            return 3. + static_cast<double>((u + sms / 2 - 1) / (sms / 2)) * (p.nkb * block + end);
        };
        const double full = pairs(256, 0.42, 2.), narrow = pairs(128, 0.31, 1.5);
        if (wide < std::min(full, narrow)) return launch_e4m3_stream(mode, true, n, x, w0, w1, in, p, s);
        return launch_e4m3_pair(mode, narrow < full, x, w0, w1, in, p, s);
    }
    return launch_e4m3_pair(mode, false, x, w0, w1, in, p, s);
}

}  // namespace ffn
