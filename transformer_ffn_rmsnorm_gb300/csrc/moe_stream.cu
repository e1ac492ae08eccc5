// moe_stream.cu -- the routed block's two products with 16-bit weights where
// experts have few tokens: a stream of weights.
//
//   gate/up:  h[r, f]    = silu(W_gate[e] x_t)_f * (W_up[e] x_t)_f    for sorted row r, its token t
//   down:     part[s][r, o] = sum of (W_down[e] h_r)_o over split s   (fp32)
//
// Bound by HBM: every weight of the experts in use is read once.  Beside
// moe_gemm.cu's CTA pairs of 256 rows the unit of work is 128 weight rows in
// one CTA (gate/up: 64 rows of W_gate stacked on the same 64 of W_up, one MMA
// for both), so that the few units spread over all multiprocessors -- one
// token of 6 experts with 1408 features makes 132 units on 152 SMs instead of
// 36 on 76 pairs -- and the down product's reduction is split where that
// fills the last wave (moe_down_splits).  Four stages of 128 values keep 128
// KB of weights in flight per SM.
//
// Roles: warp 0 loads, warp 1 issues the MMAs, warps 4-7 are the epilogue.
// Every wait is bounded (1 s) as in gemm_tcgen05.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe.cuh"

namespace ffn {
namespace {

using moe::Plan;
using moe::Unit;

constexpr int kK = 128, kTile = kMoeCutStream.tile, kGran = kMoeCutStream.gran;
constexpr uint32_t kABytes = 128 * 64 * 2, kBBytes = kTile * 64 * 2;   // of 64 values
constexpr uint32_t kSubBytes = kABytes + kBBytes, kStageBytes = 2 * kSubBytes;
constexpr int kStages = 4;
constexpr size_t kSmemBytes = kStages * kStageBytes + 1024;
static_assert(kSmemBytes > 114 * 1024 && kSmemBytes < 218 * 1024, "one CTA per SM: each allocates tensor memory");
constexpr uint32_t kTmemCols = 2 * kTile;   // two accumulators
constexpr int kThreads = 32 * 8;
constexpr uint64_t kWaitNs = 1000000000ull;

enum Mode { GATEUP = 0, DOWN = 1 };

struct Params {
    const int *header;
    const int4 *tiles;
    int nf;                // feature tiles of 64 (gate/up) or 128 rows
    int wrows;             // weight rows of an expert (ffn or d)
    int nst;               // stages of 128 values over K
    int splits;            // of the reduction (down)
    int64_t split_stride;  // floats from one split of part to the next
    void *out;
    float acc_scale;
    moe::Levels levels;    // of h, where it is fp16
    unsigned *err;
};

template <int MODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    moe_stream_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                      const __grid_constant__ moe::RowMaps maps_b, const Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int kFRows = MODE == GATEUP ? 64 : 128;   // features of a unit
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages], bar_tfull[2], bar_tempty[2], bar_drain;
    __shared__ float s_swap[MODE == GATEUP ? 2 : 1][2][8][64];
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [](uint64_t *b) { return ptx::smem_u32(b); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(&bar_full[s]), 1);
            ptx::mbar_init(bar(&bar_empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar(&bar_tfull[a]), 1);
            ptx::mbar_init(bar(&bar_tempty[a]), 4);
        }
        ptx::mbar_init(bar(&bar_drain), 1);
        s_abort = 0;
        s_never = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_map(&map_w0);
        if (MODE == GATEUP) ptx::tma_prefetch_map(&map_w1);
        for (int i = 0; i < 4; ++i) ptx::tma_prefetch_map(&maps_b.m[i]);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = s_tmem_base;
    volatile int *abort_flag = &s_abort;
    volatile int *never = &s_never;
    const int u0 = blockIdx.x, ustep = gridDim.x;
    uint32_t produced = 0;
    bool ok = true;

    ptx::griddep_wait();   // the plan, x, h: written by kernels before this one
    // unit v is split v % splits of tile unit v / splits: stages [lo, hi)
    const int units = __ldcg(p.header) * p.nf * p.splits;
    auto lo_of = [&](int v) { return p.nst * (v % p.splits) / p.splits; };
    auto hi_of = [&](int v) { return p.nst * (v % p.splits + 1) / p.splits; };
    auto walk_units = [&]() { return moe::Walk<kGran>(p.tiles, p.nf, p.splits, units, u0, ustep); };

    if (warp == 0) {
        // ------------------------------------------------------ producer
        int s = 0;
        uint32_t ph = 0;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            if constexpr (MODE == DOWN && !BF16) {
                if (t.odd && !moe::level_tile(p.levels, p.tiles, t, lane, abort_flag, kWaitNs)) {
                    ok = false;
                    break;
                }
            }
            const int wrow = t.expert * p.wrows + t.f * kFRows;
            for (int g = lo_of(u), ge = hi_of(u); g < ge; ++g) {
                const bool got = ptx::mbar_wait(bar(&bar_empty[s]), ph ^ 1u, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t full = bar(&bar_full[s]), st = base + s * kStageBytes;
                if (ptx::elect_one()) {
                    ptx::mbar_arrive_expect_tx(full, 2 * (kABytes + t.n * 128));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {   // 64 values each; past the row's end zero fill
                        const int k0 = g * kK + j * 64;
                        const uint32_t at = st + j * kSubBytes;
                        ptx::tma_load_2d(at, &map_w0, full, k0, wrow);
                        if (MODE == GATEUP) ptx::tma_load_2d(at + kABytes / 2, &map_w1, full, k0, wrow);
                        moe::for_row_boxes(maps_b, t.n, [&](const CUtensorMap *m, int r) {
                            ptx::tma_load_2d(at + kABytes + r * 128, m, full, k0, t.row0 + r);
                        });
                    }
                }
                __syncwarp();
                ++produced;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer
        int s = 0, acc = 0;
        uint32_t ph = 0, pacc = 0;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            const uint32_t idesc = ptx::idesc_f16(128, t.n, BF16);
            bool got = ptx::mbar_wait(bar(&bar_tempty[acc]), pacc ^ 1u, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t d = tmem + acc * kTile;
            const int g0 = lo_of(u);
            for (int g = g0, ge = hi_of(u); g < ge; ++g) {
                got = ptx::mbar_wait(bar(&bar_full[s]), ph, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t at = base + s * kStageBytes + j * kSubBytes;
                        const uint64_t ad = ptx::sdesc_k_sw128(at), bd = ptx::sdesc_k_sw128(at + kABytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 bytes of k further: 2 in the address field
                            ptx::tc_mma_f16(d, ad + 2 * k, bd + 2 * k, idesc, (g - g0) | j | k);
                    }
                    ptx::tc_commit(bar(&bar_empty[s]));
                    if (g == ge - 1) ptx::tc_commit(bar(&bar_tfull[acc]));
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if (++acc == 2) {
                acc = 0;
                pacc ^= 1u;
            }
        }
        if (ptx::elect_one()) ptx::tc_commit(bar(&bar_drain));   // every MMA ends before TMEM is freed
        ptx::mbar_wait(bar(&bar_drain), 0, never, kWaitNs);
    } else if (warp >= 4) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;
        int acc = 0;
        uint32_t pacc = 0;
        auto walk = walk_units();
        if constexpr (MODE == DOWN && !BF16)
            moe::level_ahead(p.levels, p.tiles, blockIdx.x * 4 + q, gridDim.x * 4, lane);
        for (int u = u0; u < units; u += ustep) {
            const Unit t = walk.at(u);
            const bool got = ptx::mbar_wait(bar(&bar_tfull[acc]), pacc, abort_flag, kWaitNs);
            if (!moe::epilogue_vote(got, 1)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * kTile;
            if constexpr (MODE == GATEUP)
                moe::swiglu_epilogue<T, false>(taddr, q, lane, t, t.f * 64, p.wrows, static_cast<T *>(p.out), s_swap,
                                               0, 16, 1, p.acc_scale, p.levels, p.tiles);
            else
                moe::store_epilogue(taddr, t, t.f * 128 + 32 * q + lane, 0, 16, p.wrows,
                                    static_cast<float *>(p.out) + (u % p.splits) * p.split_stride, p.acc_scale,
                                    BF16 ? nullptr : p.levels.scale);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(&bar_tempty[acc]));
            if (++acc == 2) {
                acc = 0;
                pacc ^= 1u;
            }
        }
    }
    if (!ok) {
        if (lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
        *abort_flag = 1;
    }

    __syncthreads();
    // loads still in flight (only after an abandoned wait) land before shared memory is released
    if (warp == 0 && lane == 0)
        for (uint32_t s = 0; s < kStages; ++s)
            if (produced > s)
                ptx::mbar_wait(bar(&bar_full[s]), ((produced - s + kStages - 1) / kStages - 1) & 1u, never, kWaitNs);
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

bool map_16(CUtensorMap *m, const void *ptr, bool bf16, int64_t inner, int64_t rows, uint32_t box_rows) {
    return encode_tma_2d(m, ptr, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, inner,
                         rows, inner * 2, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, bool BF16>
cudaError_t launch(const Plan &plan, const void *w0, const void *w1, const void *b, int splits, int64_t pairs,
                   int64_t experts, int64_t wrows, int64_t K, void *out, float acc_scale, cudaStream_t s) {
    constexpr int kFRows = MODE == GATEUP ? 64 : 128;
    const auto kern = &moe_stream_kernel<MODE, BF16>;
    static std::atomic<int> configured_device{-1};   // (host threads may call at the same time)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device.load(std::memory_order_acquire) != dev) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
        if (e != cudaSuccess) return e;
        configured_device.store(dev, std::memory_order_release);
    }
    CUtensorMap m0, m1;
    moe::RowMaps mb;
    bool good = map_16(&m0, w0, BF16, K, experts * wrows, kFRows) && map_16(&m1, w1, BF16, K, experts * wrows, kFRows);
    for (int i = 0; i < 4; ++i) good = good && map_16(&mb.m[i], b, BF16, K, pairs, 128u >> i);
    if (!good) return cudaErrorInvalidValue;
    Params p{};
    p.header = plan.header;
    p.tiles = reinterpret_cast<const int4 *>(plan.tiles);
    p.nf = static_cast<int>((wrows + kFRows - 1) / kFRows);
    p.wrows = static_cast<int>(wrows);
    p.nst = static_cast<int>((K + kK - 1) / kK);
    p.splits = splits;
    p.split_stride = pairs * wrows;
    p.out = out;
    p.acc_scale = acc_scale;
    p.levels = moe::levels_of(plan, b, K);
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    const int64_t grid = std::min<int64_t>(sm_count(), moe::max_tiles(pairs, experts, kTile) * p.nf * splits);
    LaunchScope scope(MODE == GATEUP ? K_MOE_GATEUP : K_MOE_DOWN, s);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, s, m0, m1, mb, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_gateup_stream(int op, const Plan &plan, const void *xs, const void *wg, const void *wu, void *h,
                                     int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                                     cudaStream_t s) {
    return op == DT_BF16
               ? launch<GATEUP, true>(plan, wg, wu, xs, 1, pairs, experts, ffn, d, h, acc_scale, s)
               : launch<GATEUP, false>(plan, wg, wu, xs, 1, pairs, experts, ffn, d, h, acc_scale, s);
}

cudaError_t launch_moe_down_stream(int op, const Plan &plan, const void *h, const void *wd, float *part, int splits,
                                   int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                                   cudaStream_t s) {
    return op == DT_BF16
               ? launch<DOWN, true>(plan, wd, wd, h, splits, pairs, experts, d, ffn, part, acc_scale, s)
               : launch<DOWN, false>(plan, wd, wd, h, splits, pairs, experts, d, ffn, part, acc_scale, s);
}

}  // namespace ffn
