// moe_gemm_q4.cu -- the routed block's two products with Q4 weights, on the
// 5th-generation tensor cores with the weights dequantised into tensor memory.
//
//   gate/up:  h[r, f]    = silu(W_gate[e] x_t)_f * (W_up[e] x_t)_f    w = (u - 8) s
//   down:     part[r, o] = (W_down[e] h_r)_o                          (fp32)
//
// A unit of work is 128 weight rows (gate/up: 64 rows of W_gate and the same
// 64 of W_up) of one expert against one token tile of n <= 128 columns, the
// weights on the M side as in moe_gemm.cu.  The weights travel HBM -> shared
// memory as 4 bits (a stage is 256 values: TMA, 128 bytes of a row; their
// scales, whose row pitch need not be a multiple of 16 bytes, by cp.async),
// from there through registers, where they become fp16, into tensor memory
// (tcgen05.st), and tcgen05.mma takes its A operand from there.  Through shared
// memory the fp16 form would cost 4 bytes a weight (stored and read back)
// beside the 0.6 of the 4-bit form; so it costs none.
//
// What bounds it: few tokens: HBM, if the dequantisation keeps up.  A stage
// (128 rows of 256 values, 18 KB) is 860 cycles of this SM's share of HBM; its
// dequantisation is four warps of about 520 instructions, and the wait, the
// loads, the arithmetic and the store of one warp follow one another, so two
// groups of four warps take stages in turn, one of each group to a scheduler.
// Stages of 128 values cost the issuing warp and the barriers as much a stage
// (16 tokens, 4096 -> 14336, 8 experts: gate/up 143 us, 115 with 256; down 80
// and 68).  More tokens: the activations from L2 (64 KB a stage at 128
// columns), then the tensor pipe (3000 tokens: 1052 -> 978 and 553 -> 518 us;
// rows of 1408 values, whose sixth stage is half empty, down 167 -> 173).
//
// Arithmetic: a nibble pair becomes fp16 1024 + u (or 1024 + 16 u, the high
// nibbles where they stand), u - 8 exactly by one subtraction (one fma), and
// (u - 8) s by one product, rounded once to fp16 (11 bits of the at most 14;
// exact where it is subnormal).  The nibbles of bytes 0 and 2, and 1 and 3,
// come out as pairs, so the operands' k order within every four is 0, 2, 1, 3:
// the plan writes x and the gate/up epilogue writes h in that order.
//
// Roles: warp 0 loads nibbles, warp 3 scales, warp 2 tokens; warp 1 issues the
// MMAs; warps 4-11 dequantise (warp w fills TMEM lanes 32 (w % 4) .. of every
// second stage); warps 12-15 are the epilogue.  Every wait is bounded (1 s) as
// in gemm_tcgen05.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "moe.cuh"

namespace ffn {
namespace {

using moe::Plan;
using moe::Unit;

constexpr int kRows = 128, kK = 256, kTile = kMoeCutQ4.tile, kGran = kMoeCutQ4.gran;
constexpr uint32_t kRawBytes = kRows * 128, kScaleBytes = kRows * 16;   // nibbles and scales of a stage (256 values)
// Two rings: the stages (A in tensor memory, tokens in shared memory, one
// barrier for both) and the raw slots (nibbles and scales).  Where no tile of
// the call is wider than 64 columns they are three and six long, else two and
// four: what 512 columns of tensor memory and 227 KB hold.
constexpr int kNarrow = 64;
constexpr int kMaxStages = 3, kMaxRaw = 6, kMinStages = 2, kMinRaw = 4;
constexpr uint32_t rings_bytes(int tile, int stages, int raw) {
    return stages * tile * kK * 2 + raw * (kRawBytes + kScaleBytes);
}
constexpr size_t kSmemBytes =
    std::max(rings_bytes(kNarrow, kMaxStages, kMaxRaw), rings_bytes(kTile, kMinStages, kMinRaw)) + 1024;
static_assert(kSmemBytes > 114 * 1024 && kSmemBytes < 218 * 1024,
              "one CTA per SM (each allocates all of tensor memory), beside 8 KB of static shared memory");
constexpr uint32_t kACols = 128;   // tensor memory columns of a stage's A, after the two accumulators
constexpr int kDequantWarps = 4, kGroups = 2, kEpiWarps = 4;   // warps of a stage; groups of them taking turns
constexpr int kThreads = 32 * (4 + kGroups * kDequantWarps + kEpiWarps);
// A wait tells phases apart by parity alone, so no group may come to a barrier
// a phase too early.  A group that comes for stage m has stored stage m -
// kGroups, for which the MMAs had consumed every stage up to m - kGroups -
// slots: the slot's use before the last (m - 2 slots) and the raw slot's last
// use (m - raws) must be among those.
static_assert(kGroups <= kMinStages && kGroups <= kMaxStages && kGroups + kMaxStages <= kMaxRaw &&
                  kGroups + kMinStages <= kMinRaw,
              "waits by parity");
constexpr uint64_t kWaitNs = 1000000000ull;

enum Mode { GATEUP = 0, DOWN = 1 };

struct Params {
    const int *header;
    const int4 *tiles;
    const uint16_t *s0, *s1;   // scales of W_gate and W_up, or of W_down
    int nf;                    // feature tiles of 64 (gate/up) or 128 rows
    int wrows;                 // weight rows of an expert (ffn or d)
    int ngrp;                  // 128-value groups of a row; a stage is two
    int splits;                // of the reduction (down)
    int64_t split_stride;      // floats from one split of part to the next
    void *out;
    moe::Levels levels;    // of h, where it is fp16
    unsigned *err;
};

template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// arrives on bar once this thread's cp.async so far have landed (the barrier counts the arrival)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Eight nibbles (a word of the device layout) as (u - 8) s in fp16 pairs:
// o[0], o[1] bytes 0/2 and 1/3 of the low nibbles, o[2], o[3] of the high ones.
__device__ __forceinline__ void dequant_word(uint32_t w, __half2 s, uint32_t (&o)[4]) {
    const __half2 lo8 = __half2half2(__ushort_as_half(0x6408));        // 1032
    const __half2 hi_m = __half2half2(__ushort_as_half(0x2C00));       // 1/16
    const __half2 hi_a = __half2half2(__ushort_as_half(0xD480));       // -72
    const uint32_t v = w >> 8;
    uint32_t r[4];
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(r[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(r[1]) : "r"(v));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(r[2]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(r[3]) : "r"(v));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h = *reinterpret_cast<__half2 *>(&r[i]);
        h = i < 2 ? __hsub2(h, lo8) : __hfma2(h, hi_m, hi_a);
        h = __hmul2(h, s);
        o[i] = *reinterpret_cast<uint32_t *>(&h);
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_q4_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                       const __grid_constant__ moe::RowMaps maps_b, const Params p) {
    constexpr int kFRows = MODE == GATEUP ? 64 : 128;   // features of a unit
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_rfull[kMaxRaw], bar_rempty[kMaxRaw];
    __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages];
    __shared__ __align__(8) uint64_t bar_tfull[2], bar_tempty[2], bar_drain;
    __shared__ float s_swap[MODE == GATEUP ? 2 : 1][2][8][64];
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [](uint64_t *b) { return ptx::smem_u32(b); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxRaw; ++s) {
            ptx::mbar_init(bar(&bar_rfull[s]), 1 + 32);        // the nibbles' bytes, the scale warp's lanes
            ptx::mbar_init(bar(&bar_rempty[s]), kDequantWarps);
        }
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(bar(&bar_full[s]), 1 + kDequantWarps);   // the tokens' bytes, the weights' warps
            ptx::mbar_init(bar(&bar_empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar(&bar_tfull[a]), 1);
            ptx::mbar_init(bar(&bar_tempty[a]), kEpiWarps);
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
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem_base), 512);
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
    uint32_t produced = 0;   // stages whose loads this warp issued (warps 0 and 2)
    bool ok = true;

    ptx::griddep_wait();   // the plan, x, h: written by kernels before this one
    // unit v is split v % splits of tile unit v / splits: stages [lo, hi); an
    // odd row's last stage has 128 values
    const int units = __ldcg(p.header) * p.nf * p.splits;
    const int nst = (p.ngrp + 1) / 2;
    auto lo_of = [&](int v) { return nst * (v % p.splits) / p.splits; };
    auto hi_of = [&](int v) { return nst * (v % p.splits + 1) / p.splits; };
    auto half_of = [&](int st) { return 2 * st + 1 == p.ngrp; };
    const bool narrow = __ldcg(p.header + 1) <= kNarrow;
    const int slots = narrow ? kMaxStages : kMinStages, raws = narrow ? kMaxRaw : kMinRaw;
    const uint32_t acc_cols = narrow ? kNarrow : kTile, a_col = 2 * acc_cols;
    // 64 values of a stage's tokens (at most kNarrow or kTile columns); all of them
    const uint32_t b_sub = (narrow ? kNarrow : kTile) * 128, b_slot = 4 * b_sub;
    const uint32_t raw_off = slots * b_slot, scale_off = raw_off + raws * kRawBytes;
    auto walk_units = [&]() { return moe::Walk<kGran>(p.tiles, p.nf, p.splits, units, u0, ustep); };

    if (warp == 0) {
        // ------------------------------------------------------ nibbles
        int s = 0;
        uint32_t ph = 0;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            const int wrow = t.expert * p.wrows + t.f * kFRows;
            for (int r = lo_of(u), re = hi_of(u); r < re; ++r) {
                const bool got = ptx::mbar_wait(bar(&bar_rempty[s]), ph ^ 1u, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                if (ptx::elect_one()) {
                    const uint32_t full = bar(&bar_rfull[s]), dst = base + raw_off + s * kRawBytes;
                    ptx::mbar_arrive_expect_tx(full, kRawBytes);
                    ptx::tma_load_2d(dst, &map_w0, full, r * 128, wrow);   // past the row's end zero fill
                    if (MODE == GATEUP) ptx::tma_load_2d(dst + kRawBytes / 2, &map_w1, full, r * 128, wrow);
                }
                __syncwarp();
                ++produced;
                if (++s == raws) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------ scales
        const bool wide = (p.ngrp & 1) == 0;   // rows of scales start on 16 bytes
        int s = 0;
        uint32_t ph = 0;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            const uint16_t *src[4];   // of this lane's rows lane, lane + 32, ...
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int f = t.f * kFRows + (MODE == GATEUP ? 32 * (i & 1) : 32 * i) + lane;
                const uint16_t *m = MODE == GATEUP && i >= 2 ? p.s1 : p.s0;
                src[i] = m + (static_cast<int64_t>(t.expert) * p.wrows + min(f, p.wrows - 1)) * (4 * p.ngrp);
            }
            for (int r = lo_of(u), re = hi_of(u); r < re; ++r) {
                const bool got = ptx::mbar_wait(bar(&bar_rempty[s]), ph ^ 1u, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = base + scale_off + s * kScaleBytes + lane * 16;
                const bool last = half_of(r);   // no more scales in the row
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (wide) {
                        cp_async<16>(dst + i * 512, src[i] + 8 * r);
                    } else {
                        cp_async<8>(dst + i * 512, src[i] + 8 * r);
                        if (!last) cp_async<8>(dst + i * 512 + 8, src[i] + 8 * r + 4);
                    }
                }
                cp_async_arrive(bar(&bar_rfull[s]));
                if (++s == raws) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 2) {
        // ------------------------------------------------------ tokens
        int s = 0;
        uint32_t ph = 0;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            if constexpr (MODE == DOWN) {
                if (t.odd && !moe::level_tile(p.levels, p.tiles, t, lane, abort_flag, kWaitNs)) {
                    ok = false;
                    break;
                }
            }
            for (int g = lo_of(u), ge = hi_of(u); g < ge; ++g) {
                const bool got = ptx::mbar_wait(bar(&bar_empty[s]), ph ^ 1u, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                if (ptx::elect_one()) {
                    const uint32_t full = bar(&bar_full[s]), dst = base + s * b_slot;
                    const int nsub = half_of(g) ? 2 : 4;
                    ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(t.n) * 128 * nsub);
                    moe::for_row_boxes(maps_b, t.n, [&](const CUtensorMap *m, int r) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)   // 64 values each; past the row's end zero fill
                            if (j < nsub)
                                ptx::tma_load_2d(dst + j * b_sub + r * 128, m, full, g * kK + j * 64, t.row0 + r);
                    });
                }
                __syncwarp();
                ++produced;
                if (++s == slots) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer
        // (256 values at a time, and the next stage's barrier is looked at
        // before this stage's MMAs are issued: going round once costs some 400
        // cycles beside the MMAs, what 128 values may take)
        int s = 0, acc = 0;
        uint32_t ph = 0, pacc = 0;
        bool ready = false;
        auto walk = walk_units();
        for (int u = u0; u < units && ok; u += ustep) {
            const Unit t = walk.at(u);
            const uint32_t idesc = ptx::idesc_f16(128, t.n, false);
            bool got = ptx::mbar_wait(bar(&bar_tempty[acc]), pacc ^ 1u, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint32_t d = tmem + acc * acc_cols;
            const int g0 = lo_of(u), ge = hi_of(u);
            for (int g = g0; g < ge; ++g) {
                if (!__all_sync(0xffffffffu, ready)) {
                    got = ptx::mbar_wait(bar(&bar_full[s]), ph, abort_flag, kWaitNs);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                }
                ptx::tc_fence_after();
                const int at = s;
                if (++s == slots) {
                    s = 0;
                    ph ^= 1u;
                }
                ready = ptx::mbar_test(bar(&bar_full[s]), ph);
                if (ptx::elect_one()) {
                    const uint32_t a = tmem + a_col + at * kACols;
                    const uint64_t bd = ptx::sdesc_k_sw128(base + at * b_slot);
                    const uint32_t sub = b_sub >> 4;
#pragma unroll
                    for (int k = 0; k < 8; ++k)   // 32 bytes of k further: 2 in the address field
                        mma_ts(d, a + 8 * k, bd + (k >> 2) * sub + 2 * (k & 3), idesc, g != g0 || k != 0);
                    if (!half_of(g)) {
#pragma unroll
                        for (int k = 8; k < 16; ++k)
                            mma_ts(d, a + 8 * k, bd + (k >> 2) * sub + 2 * (k & 3), idesc, true);
                    }
                    ptx::tc_commit(bar(&bar_empty[at]));
                    if (g == ge - 1) ptx::tc_commit(bar(&bar_tfull[acc]));
                }
                __syncwarp();
            }
            if (!ok) break;
            if (++acc == 2) {
                acc = 0;
                pacc ^= 1u;
            }
        }
        if (ptx::elect_one()) ptx::tc_commit(bar(&bar_drain));   // every MMA ends before TMEM is freed
        ptx::mbar_wait(bar(&bar_drain), 0, never, kWaitNs);
    } else if (warp < 4 + kGroups * kDequantWarps) {
        // ------------------------------------------------------ dequantisation
        // this warp's rows are 32q .. 32q + 31; its group takes every kGroups-th stage
        const int q = warp & 3, group = (warp - 4) / kDequantWarps;
        const int row = 32 * q + lane;
        const uint32_t a0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + a_col;
        int turn = 0, s = 0, slot = 0;   // of the next stage: whose it is, its raw and its ring slot
        uint32_t ph = 0, pslot = 0;
        for (int u = u0; u < units && ok; u += ustep) {
            for (int g = lo_of(u), ge = hi_of(u); g < ge; ++g) {
                const bool mine = turn == group;
                const int cs = s, cslot = slot;
                const uint32_t cph = ph, cpslot = pslot;
                if (++turn == kGroups) turn = 0;
                if (++s == raws) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++slot == slots) {
                    slot = 0;
                    pslot ^= 1u;
                }
                if (!mine) continue;
                bool got = ptx::mbar_wait(bar(&bar_rfull[cs]), cph, abort_flag, kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                const uint32_t src = base + raw_off + cs * kRawBytes + row * 128;
                const uint32_t to = a0 + cslot * kACols;
                const int halves = half_of(g) ? 1 : 2;
                uint32_t sc[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(sc[0]), "=r"(sc[1]), "=r"(sc[2]), "=r"(sc[3])
                             : "r"(base + scale_off + cs * kScaleBytes + row * 16));
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {   // 128 values
                    if (hh >= halves) break;
                    uint4 w[4];   // words of canonical bytes 4t .. 4t + 3 of the four blocks
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[t].x), "=r"(w[t].y), "=r"(w[t].z), "=r"(w[t].w)
                                     : "r"(src + (((4 * hh + t) ^ (row & 7)) << 4)));
                    uint32_t o[2][32];
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk) {
                        const __half2 sp = *reinterpret_cast<const __half2 *>(&sc[2 * hh + (blk >> 1)]);
                        const __half2 s2 = blk & 1 ? __high2half2(sp) : __low2half2(sp);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            uint32_t v[4];
                            dequant_word(blk == 0 ? w[t].x : blk == 1 ? w[t].y : blk == 2 ? w[t].z : w[t].w, s2, v);
                            uint32_t *x = &o[blk >> 1][16 * (blk & 1) + 2 * t];
                            x[0] = v[0];
                            x[1] = v[1];
                            x[8] = v[2];
                            x[9] = v[3];
                        }
                    }
                    if (hh == 0) {   // (the first half's arithmetic before the wait)
                        got = ptx::mbar_wait(bar(&bar_empty[cslot]), cpslot ^ 1u, abort_flag, kWaitNs);
                        if (!__all_sync(0xffffffffu, got)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                    }
                    __syncwarp();
                    tmem_st_x32(to + 64 * hh, o[0]);
                    tmem_st_x32(to + 64 * hh + 32, o[1]);
                }
                if (!ok) break;
                tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // (the raw slot only here, where what was loaded from it has
                    // been used: released right after the second half's loads,
                    // with the first half's stores still in flight, it was
                    // filled again before they were served, in up to a tenth
                    // of the calls)
                    ptx::mbar_arrive(bar(&bar_full[cslot]));
                    ptx::mbar_arrive(bar(&bar_rempty[cs]));
                }
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;
        int acc = 0;
        uint32_t pacc = 0;
        auto walk = walk_units();
        if constexpr (MODE == DOWN)
            moe::level_ahead(p.levels, p.tiles, blockIdx.x * kEpiWarps + q, gridDim.x * kEpiWarps, lane);
        for (int u = u0; u < units; u += ustep) {
            const Unit t = walk.at(u);
            const bool got = ptx::mbar_wait(bar(&bar_tfull[acc]), pacc, abort_flag, kWaitNs);
            const bool stay = moe::epilogue_vote(got, 1);
            if (!stay) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * acc_cols;
            if constexpr (MODE == GATEUP)
                moe::swiglu_epilogue<__half, true>(taddr, q, lane, t, t.f * 64, p.wrows, static_cast<__half *>(p.out),
                                                   s_swap, 0, 16, 1, 1.f, p.levels, p.tiles);
            else
                moe::store_epilogue(taddr, t, t.f * 128 + 32 * q + lane, 0, 16, p.wrows,
                                    static_cast<float *>(p.out) + (u % p.splits) * p.split_stride, 1.f,
                                    p.levels.scale);
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
        for (int s = 0; s < raws; ++s)
            if (produced > static_cast<uint32_t>(s))
                ptx::mbar_wait(bar(&bar_rfull[s]), ((produced - s + raws - 1) / raws - 1) & 1u, never, kWaitNs);
    if (warp == 2 && lane == 0)
        for (int s = 0; s < slots; ++s)
            if (produced > static_cast<uint32_t>(s))
                ptx::mbar_wait(bar(&bar_full[s]), ((produced - s + slots - 1) / slots - 1) & 1u, never, kWaitNs);
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

bool map_rows(moe::RowMaps *m, const void *ptr, int64_t inner, int64_t rows) {
    for (int i = 0; i < 4; ++i)
        if (!encode_tma_2d(&m->m[i], ptr, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, inner, rows, inner * 2, 64, 128u >> i,
                           CU_TENSOR_MAP_SWIZZLE_128B))
            return false;
    return true;
}

template <int MODE>
cudaError_t launch(const Plan &plan, const CUtensorMap &w0, const CUtensorMap &w1, const void *rows,
                   const uint16_t *s0, const uint16_t *s1, int splits, int64_t pairs, int64_t experts, int64_t wrows,
                   int64_t K, void *out, cudaStream_t s) {
    const auto kern = &moe_gemm_q4_kernel<MODE>;
    static std::atomic<int> configured_device{-1};   // (host threads may call at the same time)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device.load(std::memory_order_acquire) != dev) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
        if (e != cudaSuccess) return e;
        configured_device.store(dev, std::memory_order_release);
    }
    constexpr int kFRows = MODE == GATEUP ? 64 : 128;
    moe::RowMaps b;
    if (!map_rows(&b, rows, K, pairs)) return cudaErrorInvalidValue;
    Params p{};
    p.header = plan.header;
    p.tiles = reinterpret_cast<const int4 *>(plan.tiles);
    p.s0 = s0;
    p.s1 = s1;
    p.nf = static_cast<int>((wrows + kFRows - 1) / kFRows);
    p.wrows = static_cast<int>(wrows);
    p.ngrp = static_cast<int>((K + 127) / 128);
    p.splits = splits;
    p.split_stride = pairs * wrows;
    p.out = out;
    p.levels = moe::levels_of(plan, rows, K);
    p.err = device_status_word();
    if (!p.err) return cudaErrorUnknown;
    const int64_t grid = std::min<int64_t>(sm_count(), moe::max_tiles(pairs, experts, kTile) * p.nf * splits);
    LaunchScope scope(MODE == GATEUP ? K_MOE_GATEUP : K_MOE_DOWN, s);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, s, w0, w1, b, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// nibbles: 128 bytes of box_rows rows, rows of whole 128-value groups
bool map_q4(CUtensorMap *m, const uint8_t *qs, int64_t K, int64_t rows, uint32_t box_rows) {
    const int64_t pitch = 64 * ((K + 127) / 128);
    return encode_tma_2d(m, qs, CU_TENSOR_MAP_DATA_TYPE_UINT8, pitch, rows, pitch, 128, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}
}  // namespace

cudaError_t launch_moe_gateup_q4(const Plan &plan, const void *xs, const uint8_t *qg, const uint16_t *sg,
                                 const uint8_t *qu, const uint16_t *su, void *h, int64_t pairs, int64_t d, int64_t ffn,
                                 int64_t experts, cudaStream_t s) {
    CUtensorMap w0, w1;
    if (!map_q4(&w0, qg, d, experts * ffn, 64) || !map_q4(&w1, qu, d, experts * ffn, 64)) return cudaErrorInvalidValue;
    return launch<GATEUP>(plan, w0, w1, xs, sg, su, 1, pairs, experts, ffn, d, h, s);
}

cudaError_t launch_moe_down_q4(const Plan &plan, const void *h, const uint8_t *qd, const uint16_t *sd, float *part,
                               int splits, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, cudaStream_t s) {
    CUtensorMap w;
    if (!map_q4(&w, qd, ffn, experts * d, 128)) return cudaErrorInvalidValue;
    return launch<DOWN>(plan, w, w, h, sd, sd, splits, pairs, experts, d, ffn, part, s);
}

}  // namespace ffn
