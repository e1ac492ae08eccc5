// moe_gemm.cu -- the routed block's two products with 16-bit weights, on the
// 5th-generation tensor cores.
//
//   gate/up:  h[r, f]    = silu(W_gate[e] x_t)_f * (W_up[e] x_t)_f   for sorted row r, its token t
//   down:     part[r, o] = (W_down[e] h_r)_o                         (fp32)
//
// CTA pairs (tcgen05 .cta_group::2): a unit of work is 256 weight rows (128
// in each CTA; gate/up: 64 rows of W_gate stacked on the same 64 of W_up)
// against one token tile of n <= 256 columns of one expert.  The
// weights are the M operand; the tokens' sorted rows (of x or of h) are the N
// operand, each CTA holding half of the columns in boxes of 128, 64, 32 and 16 rows.
//
// What bounds it: the tensor pipe.  The 256 x 256 tile takes 64 bytes a cycle and
// SM from L2, and its accumulator half of tensor memory, so that a unit's
// epilogue runs under the next unit's MMAs.  (Gate and up in two accumulators
// of 256 columns would take 48 bytes a cycle, but fill tensor memory: the
// epilogue then stood between the units, 7000 cycles after 30000 at d = 2048.
// Tiles of 128 tokens instead, which leave room, were slower still: 80 bytes.)
//
// Roles: warp 0 loads, warp 1 issues the MMAs (the even CTA's), warps 2-9 read
// the accumulators (lane = weight row, column = token): for a fixed column a
// warp's 32 lanes store 32 neighbouring features.  Every wait is bounded as in
// gemm_tcgen05.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe.cuh"
#include "pair_end.cuh"

namespace ffn {
namespace {

using moe::Plan;
using moe::Unit;

constexpr int kBM = 128, kBK = 64, kTile = kMoeCutPair.tile;
constexpr uint32_t kABytes = kBM * kBK * 2;                // one CTA's weight rows of a k block
constexpr uint32_t kBBytes = (kTile / 2) * kBK * 2;        // room for its half of the tokens
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint64_t kWaitNs = 1000000000ull;

enum Mode { GATEUP = 0, DOWN = 1 };

// A stage holds two blocks of 64 k values: weight rows, tokens.
constexpr int kSub = 2;
constexpr uint32_t kSubBytes = kABytes + kBBytes, kStageBytes = kSub * kSubBytes;
constexpr int kStages = 3;
constexpr size_t kSmemBytes = kStages * kStageBytes + 1024;
static_assert(kSmemBytes > 114 * 1024 && kSmemBytes < 210 * 1024,
              "one CTA per SM (each allocates all of tensor memory), beside 16 KB of static shared memory");

struct Params {
    const int *header;
    const int4 *tiles;
    int nf;            // feature tiles of 128 (gate/up) or 256 rows
    int wrows;         // weight rows of an expert (ffn or d)
    int nkb;           // 64-wide k blocks
    void *out;         // h (operand type) or part (fp32), [pairs x wrows]
    float acc_scale;
    moe::Levels levels;    // of h, where it is fp16
    unsigned *err;
};

template <int MODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ moe::RowMaps maps_b, const Params p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int kFRows = MODE == GATEUP ? 128 : 256;   // features of a unit
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages];
    __shared__ __align__(8) uint64_t bar_tfull[2], bar_tempty[2], bar_drain;
    __shared__ float s_swap[MODE == GATEUP ? kEpiWarps / 4 : 1][MODE == GATEUP ? 2 : 1][2][8][64];
    __shared__ uint32_t s_tmem_base, s_bytes[kStages];   // s_bytes: of the CTA's last load into a stage
    __shared__ PairEnd s_end;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    auto sA = [&](int s, int j) { return base + s * kStageBytes + j * kSubBytes; };
    auto sB = [&](int s, int j) { return sA(s, j) + kABytes; };
    auto full = [&](int s) { return ptx::smem_u32(&bar_full[s]); };
    auto empty = [&](int s) { return ptx::smem_u32(&bar_empty[s]); };
    auto tfull = [&](int a) { return ptx::smem_u32(&bar_tfull[a]); };
    auto tempty = [&](int a) { return ptx::smem_u32(&bar_tempty[a]); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(tfull(a), 1);
            ptx::mbar_init(tempty(a), 2 * kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
        s_abort = 0;
        s_never = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_map(&map_w0);
        if (MODE == GATEUP) ptx::tma_prefetch_map(&map_w1);
        for (int i = 0; i < 4; ++i) ptx::tma_prefetch_map(&maps_b.m[i]);
    }
    // Both CTAs run before either allocates: the allocation is the pair's, and
    // one that the even CTA began before the odd one had started (a CTA of the
    // kernel before still on its SM) left the odd one waiting in it for good.
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // both CTAs' barriers are initialised before either reports to the other
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = s_tmem_base;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    auto lead = [&](uint32_t bar) { return ptx::mapa_shared(bar, 0); };   // the pair's barriers live in the even CTA
    volatile int *abort_flag = &s_abort;
    volatile int *never = &s_never;
    const int nst = (p.nkb + kSub - 1) / kSub;
    const int u0 = blockIdx.x >> 1, ustep = gridDim.x >> 1;
    uint32_t produced = 0;

    ptx::griddep_wait();   // the plan, x, h: all written by kernels before this one
    const int units = __ldcg(p.header) * p.nf;
    auto walk_units = [&]() { return moe::Walk<kMoeCutPair.gran>(p.tiles, p.nf, 1, units, u0, ustep); };

    if (warp == 0) {
        // ------------------------------------------------------ producer
        bool ok = true;
        auto walk = walk_units();
        int s = 0;
        uint32_t ph = 0;
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            if constexpr (MODE == DOWN && !BF16) {
                if (t.odd && !moe::level_tile(p.levels, p.tiles, t, lane, abort_flag, kWaitNs)) {
                    ok = false;
                    break;
                }
            }
            const int half = t.n >> 1;   // this CTA's columns, a multiple of 16
            const int wrow = t.expert * p.wrows + t.f * kFRows + static_cast<int>(rank) * (kFRows / 2);
            const int brow = t.row0 + static_cast<int>(rank) * half;
            for (int ks = 0; ks < nst; ++ks) {
                const bool got = ptx::mbar_wait(empty(s), ph ^ 1u, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                if (ptx::elect_one()) {
                    const uint32_t bar = lead(full(s));
                    const uint32_t bytes = kSub * (kABytes + half * (kBK * 2));
                    s_bytes[s] = bytes;
                    if (leader) ptx::mbar_arrive_expect_tx(full(s), 2 * bytes);
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        const int k0 = (ks * kSub + j) * kBK;   // a block past K is zero fill
                        ptx::tma_load_2d_pair(sA(s, j), &map_w0, bar, k0, wrow);
                        if (MODE == GATEUP) ptx::tma_load_2d_pair(sA(s, j) + kABytes / 2, &map_w1, bar, k0, wrow);
                        moe::for_row_boxes(maps_b, half, [&](const CUtensorMap *m, int r) {
                            ptx::tma_load_2d_pair(sB(s, j) + r * 128, m, bar, k0, brow + r);
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
        if (!ok && lane == 0) {
            atomicOr(p.err, DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    } else if (warp == 1 && leader) {
        // -------------------------------------------------------- MMA issuer
        bool ok = true;
        auto walk = walk_units();
        int s = 0, acc = 0;
        uint32_t ph = 0, acc_ph = 0;
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            const uint32_t idesc = ptx::idesc_f16(256, t.n, BF16);
            bool got = ptx::mbar_wait(tempty(acc), acc_ph ^ 1u, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t d0 = tmem + acc * 256;
            for (int ks = 0; ks < nst; ++ks) {
                got = ptx::mbar_wait(full(s), ph, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        const uint64_t ad = ptx::sdesc_k_sw128(sA(s, j)), bd = ptx::sdesc_k_sw128(sB(s, j));
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)   // 32 bytes of k further: 2 in the address field
                            ptx::tc_mma_f16_pair(d0, ad + 2 * k, bd + 2 * k, idesc, (ks | j | k) != 0);
                    }
                    ptx::tc_commit_pair(empty(s), 0x3);
                    if (ks == nst - 1) ptx::tc_commit_pair(tfull(acc), 0x3);
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
                acc_ph ^= 1u;
            }
        }
        if (!ok && lane == 0) {
            atomicOr(p.err, DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        // every MMA ends before TMEM is freed
        if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(&bar_drain), 0x1);
        ptx::mbar_wait(ptx::smem_u32(&bar_drain), 0, never, kWaitNs);
    } else if (warp >= 2) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;                 // this warp may read TMEM lanes 32q .. 32q+31
        const int part = (warp - 2) >> 2;       // which of every two 16-column chunks
        bool ok = true;
        auto walk = walk_units();
        if constexpr (MODE == DOWN && !BF16)
            moe::level_ahead(p.levels, p.tiles, blockIdx.x * kEpiWarps + warp - 2, gridDim.x * kEpiWarps, lane);
        int acc = 0;
        uint32_t acc_ph = 0;
        for (int u = u0; u < units; u += ustep) {
            const Unit t = walk.at(u);
            const bool got = ptx::mbar_wait(tfull(acc), acc_ph, abort_flag, kWaitNs);
            if (!moe::epilogue_vote(got, 1 + part)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
            const int f0 = t.f * kFRows + static_cast<int>(rank) * (kFRows / 2);
            if constexpr (MODE == GATEUP) {
                moe::swiglu_epilogue<T, false>(taddr, q, lane, t, f0, p.wrows, static_cast<T *>(p.out), s_swap[part],
                                               16 * part, 16 * (kEpiWarps / 4), 1 + part, p.acc_scale, p.levels,
                                               p.tiles);
            } else {
                moe::store_epilogue(taddr, t, f0 + q * 32 + lane, 16 * part, 16 * (kEpiWarps / 4), p.wrows,
                                    static_cast<float *>(p.out), p.acc_scale, BF16 ? nullptr : p.levels.scale);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) ptx::mbar_arrive(tempty(acc));
                else ptx::mbar_arrive_cluster(lead(tempty(acc)));
            }
            if (++acc == 2) {
                acc = 0;
                acc_ph ^= 1u;
            }
        }
        if (!ok && lane == 0) {
            atomicOr(p.err, DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }

    end_pair<kStages>(s_end, rank, produced, abort_flag, never, kWaitNs, full, [&](int s, int r) {
        return ld_cluster(ptx::mapa_shared(ptx::smem_u32(&s_bytes[s]), r));
    });
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

bool map_16(CUtensorMap *m, const void *ptr, bool bf16, int64_t inner, int64_t rows, uint32_t box_rows) {
    return encode_tma_2d(m, ptr, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, inner,
                         rows, inner * 2, kBK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool map_rows(moe::RowMaps *m, const void *ptr, bool bf16, int64_t inner, int64_t rows) {
    for (int i = 0; i < 4; ++i)
        if (!map_16(&m->m[i], ptr, bf16, inner, rows, 128u >> i)) return false;
    return true;
}

template <int MODE, bool BF16>
cudaError_t launch(const Plan &plan, const CUtensorMap &w0, const CUtensorMap &w1, const void *rows, int64_t pairs,
                   int64_t experts, int64_t wrows, int64_t K, void *out, float acc_scale, cudaStream_t s) {
    constexpr int kFRows = MODE == GATEUP ? 128 : 256;
    const auto kern = &moe_gemm_kernel<MODE, BF16>;
    static std::atomic<int> configured_device{-1}, pair_slots{0};   // (host threads may call at the same time)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    int slots = 0;   // co-resident CTA pairs
    if (configured_device.load(std::memory_order_acquire) == dev) {
        slots = pair_slots.load(std::memory_order_relaxed);
    } else {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2 * static_cast<unsigned>(sm_count()));
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&slots, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (slots < 1) return cudaErrorLaunchOutOfResources;
        pair_slots.store(slots, std::memory_order_relaxed);
        configured_device.store(dev, std::memory_order_release);
    }
    moe::RowMaps b;
    if (!map_rows(&b, rows, BF16, K, pairs)) return cudaErrorInvalidValue;
    Params p{};
    p.header = plan.header;
    p.tiles = reinterpret_cast<const int4 *>(plan.tiles);
    p.nf = static_cast<int>((wrows + kFRows - 1) / kFRows);
    p.wrows = static_cast<int>(wrows);
    p.nkb = static_cast<int>((K + kBK - 1) / kBK);
    p.out = out;
    p.acc_scale = acc_scale;
    p.levels = moe::levels_of(plan, rows, K);
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    const int64_t most = moe::max_tiles(pairs, experts, kTile) * p.nf;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(slots, most)));
    cfg.stream = s;
    cfg.numAttrs = 2;
    LaunchScope scope(MODE == GATEUP ? K_MOE_GATEUP : K_MOE_DOWN, s);
    e = cudaLaunchKernelEx(&cfg, kern, w0, w1, b, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_gateup(int op, const Plan &plan, const void *xs, const void *wg, const void *wu, void *h,
                              int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s) {
    const bool bf = op == DT_BF16;
    CUtensorMap w0, w1;
    if (!map_16(&w0, wg, bf, d, experts * ffn, kBM / 2) || !map_16(&w1, wu, bf, d, experts * ffn, kBM / 2))
        return cudaErrorInvalidValue;
    return bf ? launch<GATEUP, true>(plan, w0, w1, xs, pairs, experts, ffn, d, h, acc_scale, s)
              : launch<GATEUP, false>(plan, w0, w1, xs, pairs, experts, ffn, d, h, acc_scale, s);
}

cudaError_t launch_moe_down(int op, const Plan &plan, const void *h, const void *wd, float *part, int64_t pairs,
                            int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s) {
    const bool bf = op == DT_BF16;
    CUtensorMap w;
    if (!map_16(&w, wd, bf, ffn, experts * d, kBM)) return cudaErrorInvalidValue;
    return bf ? launch<DOWN, true>(plan, w, w, h, pairs, experts, d, ffn, part, acc_scale, s)
              : launch<DOWN, false>(plan, w, w, h, pairs, experts, d, ffn, part, acc_scale, s);
}

}  // namespace ffn
