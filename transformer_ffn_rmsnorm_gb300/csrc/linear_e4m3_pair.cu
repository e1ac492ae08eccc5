// linear_e4m3_pair.cu -- products of e4m3 codes with block scales for many rows.
//
// CTA pairs (tcgen05 .cta_group::2): a unit of work is 256 rows of x (128 in each
// CTA, the M operand) against 256 weight rows (linear: 256 features; gate/up:
// the 128 features of one scale block, gate's rows from the even CTA's memory, up's
// from the odd one's).  A block of 128 values is multiplied in two halves of N = 128,
// each into one of four accumulators, which together are all of tensor memory; a
// gate/up half holds 64 features' gate and up columns, so that they meet in a thread.
// Linear with few units takes narrow ones, of 128 features in halves of N = 64 on
// eight accumulators: 0.31 us a block against 0.42, for half the work.
//
// What bounds it: each block's sums have to leave tensor memory before the block
// after next may use their place.  The tensor pipe needs 512 cycles a block and SM,
// the additions 256 of the FMA pipe (two an instruction); but the way of a half --
// instructions issued, sums done, seen, read and added, their leave sent back across
// the pair, seen -- is about 1300 cycles, of which two halves' 512 are hidden: 790
// cycles a block.  Nothing else is near its limit: of the cycles the tensor pipe is
// active in 60 %, instructions issue in 52, the FMA pipe works in 24, and tensor memory
// is read at 30 % of its peak, three quarters of it the pipe's own accumulators.
// (4096 tokens, 4096 -> 11008 gate/up: 273 to 283 us.  An earlier form took 349; with nothing read or
// added 252, with one such handshake in 16 blocks 195.  16 warps of 64
// columns, whose sums do not fit beside what else the registers hold, 441; one warp
// issuing both halves' MMAs 387.)
//
// With x on the M side a thread's sums share one row, so that one factor serves all
// of its columns; on the N side every column would need its own from shared memory,
// which the operands fill.
//
// Roles: warp 0 loads, warps 1 and 2 issue the MMAs of a half each (the even CTA's),
// warp 3 brings the scales of the CTA's rows to shared memory four blocks at a time
// (and what the unit is), warps 4-11 add the sums (lane = row of x; four warps for
// each half) and finish the unit while the next one's first blocks run.  Every wait
// is bounded (1 s).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "linear_e4m3.cuh"
#include "moe.cuh"
#include "pair_end.cuh"

namespace ffn {
namespace {

using e4::GATEUP;
using e4::LINEAR;
using e4::Params;

constexpr int kRows = 256;                                 // of x in a unit
constexpr int kEpiWarps = 8, kThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
// What follows from N, the columns of a half (64: linear's narrow units).
template <int MODE, int N> struct Config {
    static_assert(N == 128 || (MODE == LINEAR && N == 64), "a half");
    static constexpr int kFeatures = MODE == GATEUP ? 128 : 2 * N;   // of a unit
    static constexpr int kDepth = static_cast<int>(kTmemCols) / (2 * N);   // accumulators of a half
    static constexpr uint32_t kHalfBytes = N / 2 * 128;                // one CTA's weight rows of a half
    static constexpr uint32_t kStageBytes = e4::kTileBytes + 2 * kHalfBytes;
    static constexpr int kStages = static_cast<int>(12 * e4::kTileBytes / kStageBytes);
    static constexpr size_t kSmem = kStages * kStageBytes + 1024;
    static_assert(kSmem > 114 * 1024 && kSmem < 210 * 1024, "one CTA per SM: each allocates all of tensor memory");
};
// Registers of a thread after the warpgroups have shared them out: 168 at launch.  (Where a
// role spilled, the issuers at 56 and the sums at 208, a block took up to twice the time.)
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(4 * 32 * kFewRegs + kEpiWarps * 32 * kManyRegs <= kThreads * 168, "register split");
constexpr int kScaleBlocks = 4;   // blocks whose scales are handed over together
constexpr int kBand = 16;   // tiles of rows that go through all features together: what they read stays in L2

struct Unit {
    int expert, f, row0, valid;
};

// Says that a block's sums have been read.  They are in tensor memory and ordered by
// the fence before; no write of memory is released, so the arrival does not wait
// for those on their way (a release at the cluster's scope did, a third of the time).
__device__ __forceinline__ void arrive_read(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
// two fp32 multiply-adds
__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
// 32 bytes, a whole sector of L2, at an address that is a multiple of it
__device__ __forceinline__ void st_sector(void *at, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// 32 bytes of y, v (plus res's, if there is one) rounded to T, of which `left`
// elements, a multiple of 8, are y's.  Rows begin on multiples of 16 bytes.
template <typename T>
__device__ __forceinline__ void store_sector(T *to, const uint4 *res, bool add, float *v, int left) {
    constexpr int N = 32 / sizeof(T);
    uint4 o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) f[e] = v[i * N / 2 + e];
        if (add) {
            float r[N / 2];
            Vec16<T>::unpack(res[i], r);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) f[e] += r[e];
        }
        o[i] = Vec16<T>::pack(f);
    }
    if ((reinterpret_cast<uintptr_t>(to) & 31) == 0 && left >= N) {
        const uint32_t w[8] = {o[0].x, o[0].y, o[0].z, o[0].w, o[1].x, o[1].y, o[1].z, o[1].w};
        st_sector(to, w);
    } else {
        if (left > 0) *reinterpret_cast<uint4 *>(to) = o[0];
        if (left > N / 2) *reinterpret_cast<uint4 *>(to + N / 2) = o[1];
    }
}

// max(a, |b|), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}
template <int MODE, int N>
__global__ void __launch_bounds__(kThreads, 1)
    e4m3_pair_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                     const __grid_constant__ CUtensorMap map_x, const Params p) {
    using C = Config<MODE, N>;
    constexpr int kFeatures = C::kFeatures, kStages = C::kStages, kDepth = C::kDepth;
    constexpr uint32_t kStageBytes = C::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages];
    __shared__ __align__(8) uint64_t bar_tfull[2 * kDepth], bar_tempty[2 * kDepth], bar_drain;
    __shared__ __align__(8) uint64_t bar_sfull[2], bar_sempty[2];
    __shared__ float s_xs[2][kScaleBlocks][128], s_ws[2][kScaleBlocks][2];
    __shared__ int4 s_unit[2];   // f, row0, valid of the unit that the slot of scales begins
    // the experts' first tiles and rows, and the rows of their last tiles less one
    __shared__ int s_first[moe::kMaxExperts + 1], s_row0[moe::kMaxExperts];
    __shared__ uint8_t s_last[moe::kMaxExperts];
    __shared__ float s_amax[MODE == GATEUP ? 2 : 1][128];
    __shared__ uint32_t s_tmem_base;
    __shared__ PairEnd s_end;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [](uint64_t *b) { return ptx::smem_u32(b); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(&bar_full[s]), 1);
            ptx::mbar_init(bar(&bar_empty[s]), 2);   // both halves
        }
        for (int a = 0; a < 2 * kDepth; ++a) {   // accumulator 2 * (block % kDepth) + half
            ptx::mbar_init(bar(&bar_tfull[a]), 1);
            ptx::mbar_init(bar(&bar_tempty[a]), kEpiWarps);   // half of the warps, of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(&bar_sfull[i]), 1);
            ptx::mbar_init(bar(&bar_sempty[i]), kEpiWarps);
        }
        ptx::mbar_init(bar(&bar_drain), 2);
        s_abort = 0;
        s_never = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_map(&map_w0);
        if (MODE == GATEUP) ptx::tma_prefetch_map(&map_w1);
        ptx::tma_prefetch_map(&map_x);
    }
    // Both CTAs run before either allocates (the allocation is the pair's).
    __syncwarp();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::griddep_wait();   // x, its scales, offsets (and the weights, where they were just quantised)
    if (warp == 0) {       // the experts' tiles
        int before = 0, rows_before = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int2 r = e4::expert_rows(p, e0, lane, rows_before);
            const int tiles = (r.y - r.x + kRows - 1) / kRows;
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < p.experts) {
                s_first[e] = before + incl - tiles;
                s_row0[e] = r.x;
                s_last[e] = static_cast<uint8_t>((r.y - r.x + kRows - 1) % kRows);
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) s_first[p.experts] = before;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // both CTAs' barriers are initialised before either reports to the other
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = s_tmem_base;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    auto lead = [&](uint32_t b) { return ptx::mapa_shared(b, 0); };   // the pair's barriers live in the even CTA
    volatile int *abort_flag = &s_abort;
    volatile int *never = &s_never;
    const int nfu = (p.out + kFeatures - 1) / kFeatures;
    const int units = s_first[p.experts] * nfu;
    const int u0 = blockIdx.x >> 1, ustep = gridDim.x >> 1;
    uint32_t produced = 0;
    auto unit_of = [&](int u) {
        int lo = 0, hi = p.experts - 1;   // the last expert whose first unit is at or before u
        const int tile = u / nfu;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_first[mid] <= tile) lo = mid;
            else hi = mid - 1;
        }
        Unit t;
        t.expert = lo;
        const int nt = s_first[lo + 1] - s_first[lo];
        int local = u - s_first[lo] * nfu;
        const int band = local / (kBand * nfu), nb = min(kBand, nt - band * kBand);
        local -= band * kBand * nfu;
        t.f = local / nb;
        const int tt = band * kBand + local - t.f * nb;
        t.row0 = s_row0[lo] + tt * kRows;
        t.valid = tt == nt - 1 ? s_last[lo] + 1 : kRows;
        return t;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        // (each role's register share is set inside its branch: code after a join has the smaller one)
        if (warp == 0) {
            // ------------------------------------------------------ producer
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;
            for (int u = u0; u < units && ok; u += ustep) {
                const Unit t = unit_of(u);
                const int xrow = t.row0 + static_cast<int>(rank) * 128;
                // N / 2 weight rows of each half: gate/up: the CTA's matrix's next; linear: the CTA's part of N
                const int wrow =
                    t.expert * p.out + t.f * kFeatures + (MODE == GATEUP ? 0 : static_cast<int>(rank) * (N / 2));
                const CUtensorMap *mw = MODE == GATEUP && rank ? &map_w1 : &map_w0;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    const bool got = ptx::mbar_wait(bar(&bar_empty[s]), ph ^ 1u, abort_flag, e4::kWaitNs);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    if (ptx::elect_one()) {
                        const uint32_t full = lead(bar(&bar_full[s])), at = base + s * kStageBytes;
                        if (leader) ptx::mbar_arrive_expect_tx(bar(&bar_full[s]), 2 * kStageBytes);
                        ptx::tma_load_2d_pair(at, &map_x, full, kb * 128, xrow);
                        ptx::tma_load_2d_pair(at + e4::kTileBytes, mw, full, kb * 128, wrow);
                        ptx::tma_load_2d_pair(at + e4::kTileBytes + C::kHalfBytes, mw, full, kb * 128,
                                              wrow + (MODE == GATEUP ? 64 : N));
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
        } else if (leader && warp <= 2) {
            // -------------------------------------------------------- MMA issuers
            // One warp for each half of a block.  What a block needs besides its accumulator is
            // looked at before that, so that the instructions follow its release at once.
            constexpr uint32_t idesc = e4::idesc_e4m3(256, N);
            const int half = warp - 1;
            const uint64_t ad0 = ptx::sdesc_k_sw128(base),
                           bd0 = ptx::sdesc_k_sw128(base + e4::kTileBytes + half * C::kHalfBytes);
            bool ok = true;
            int s = 0, a = 0;
            uint32_t ph = 0, pa = 0;
            for (int u = u0; u < units && ok; u += ustep) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    const int acc = 2 * a + half;
                    const uint64_t ad = ad0 + s * (kStageBytes >> 4), bd = bd0 + s * (kStageBytes >> 4);
                    bool got = ptx::mbar_wait(bar(&bar_full[s]), ph, abort_flag, e4::kWaitNs);
                    got = got && ptx::mbar_wait(bar(&bar_tempty[acc]), pa ^ 1u, abort_flag, e4::kWaitNs);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 bytes of k further: 2 in the address field
                            e4::mma_e4m3_pair(tmem + acc * N, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                        ptx::tc_commit_pair(bar(&bar_tfull[acc]), 0x3);
                        ptx::tc_commit_pair(bar(&bar_empty[s]), 0x3);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (kDepth == 2) a ^= 1;
                    else a = (a + 1) & (kDepth - 1);
                    if (a == 0) pa ^= 1u;
                }
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            if (ptx::elect_one()) ptx::tc_commit_pair(bar(&bar_drain), 0x1);   // every MMA ends before TMEM is freed
            ptx::mbar_wait(bar(&bar_drain), 0, never, e4::kWaitNs);
        } else if (warp == 3) {
            // -------------------------------------------------------- scales
            // of the CTA's rows (four a lane) and of the unit's two weight blocks
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;
            for (int u = u0; u < units && ok; u += ustep) {
                const Unit t = unit_of(u);
                const float *xs = p.xs + static_cast<int64_t>(t.row0) * p.nkb;
                const int first = static_cast<int>(rank) * 128 + lane, last = t.valid - 1;
                int at[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) at[i] = min(first + 32 * i, last) * p.nkb;
                // lane 0: gate or the first half's block, lane 1: up or the second's
                const int nb = MODE == GATEUP ? t.f : min(N == 128 ? 2 * t.f + (lane & 1) : t.f, p.nf - 1);
                const float *ws = (MODE == GATEUP && (lane & 1) ? p.ws[1] : p.ws[0]) +
                                  (static_cast<int64_t>(t.expert) * p.nf + nb) * p.nkb;
                for (int k0 = 0; k0 < p.nkb; k0 += kScaleBlocks) {
                    const bool got = ptx::mbar_wait(bar(&bar_sempty[s]), ph ^ 1u, abort_flag, e4::kWaitNs);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j0 = 0; j0 < kScaleBlocks; j0 += 2) {
                        float v[2][4], w[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int kb = min(k0 + j0 + j, p.nkb - 1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[j][i] = __ldg(xs + at[i] + kb);
                            w[j] = __ldg(ws + kb);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) s_xs[s][j0 + j][32 * i + lane] = v[j][i];
                            if (lane < 2) s_ws[s][j0 + j][lane] = w[j];
                        }
                    }
                    if (lane == 0 && k0 == 0) s_unit[s] = make_int4(t.f, t.row0, t.valid, 0);
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(&bar_sfull[s]));
                    s ^= 1;
                    if (s == 0) ph ^= 1u;
                }
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // ---------------------------------------------------------- sums
        const int q = warp & 3, half = (warp - 4) >> 2;
        // addresses of the half's accumulators and their barriers lie 2 N columns and 16 bytes apart
        const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * N;
        const uint32_t tfull = bar(&bar_tfull[half]), tempty = lead(bar(&bar_tempty[half]));
        const uint32_t sfull = bar(&bar_sfull[0]), sempty = bar(&bar_sempty[0]);
        const float *my_xs = &s_xs[0][0][32 * q + lane], *my_ws = &s_ws[0][0][MODE == GATEUP ? 0 : half];
        uint32_t a = 0, pa = 0;             // of the next block: accumulator, its parity
        uint32_t ring = 0, pring = 0;       // its place in the ring of scales, the ring's parity
        for (int u = u0; u < units; u += ustep) {
            uint64_t acc[N / 2];   // two columns each; gate/up: 64 of gate, then 64 of up
#pragma unroll
            for (int i = 0; i < N / 2; ++i) acc[i] = 0ull;
            bool ok = true, done = false;   // done: this block's sums are known to be there
            int tf = 0, trow0 = 0, tvalid = 0;
            for (int kb = p.nkb; kb > 0; --kb) {
                bool got = true;
                if ((ring & (kScaleBlocks - 1)) == 0)
                    got = ptx::mbar_wait(sfull + 8 * (ring / kScaleBlocks), pring, abort_flag, e4::kWaitNs);
                if (kb == p.nkb) {   // (after an abandoned wait the unit is not known, and not used)
                    const int4 t = s_unit[ring / kScaleBlocks];
                    tf = t.x;
                    trow0 = t.y;
                    tvalid = t.z;
                    if (MODE == LINEAR && p.res && got) {   // its lines of this lane's row on the way to L2
                        const int r = static_cast<int>(rank) * 128 + 32 * q + lane, es = p.dt == DT_F32 ? 4 : 2;
                        const int col0 = tf * kFeatures + half * N, cols = min(N, p.out - col0);
                        const char *line = static_cast<const char *>(p.res) +
                                           (static_cast<int64_t>(trow0 + r) * p.out + col0) * es;
                        for (int b = 0; r < tvalid && b < cols * es; b += 128)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(line + b));
                    }
                }
                const float x = my_xs[ring * 128], w0 = my_ws[ring * 2];
                const uint32_t s0 = __float_as_uint(x * w0),
                               s1 = MODE == GATEUP ? __float_as_uint(x * my_ws[ring * 2 + 1]) : s0;
                const uint64_t two0 = pack2(s0, s0), two1 = pack2(s1, s1);
                got = got && (done || ptx::mbar_wait(tfull + 16 * a, pa, abort_flag, e4::kWaitNs));
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t taddr = trow + 2 * N * a;
                // 32 columns at a time, loaded under the additions before (of 16: gate/up 279 -> 301 us)
                constexpr int kCols = 32;
                uint32_t r[2][kCols];
                ptx::tmem_ld_cols<kCols>(taddr, r[0]);
#pragma unroll
                for (int c = 0; c < N / kCols; ++c) {
                    ptx::tmem_ld_wait();
                    if (c < N / kCols - 1) {
                        ptx::tmem_ld_cols<kCols>(taddr + kCols * (c + 1), r[(c + 1) & 1]);
                    } else {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_read(tempty + 16 * a);
                        if (kDepth == 2) {   // (a comparison here: gate/up 274 -> 278 us)
                            pa ^= a;
                            a ^= 1u;
                        } else {
                            a = (a + 1) & (kDepth - 1);
                            pa ^= a == 0 ? 1u : 0u;
                        }
                        done = ptx::mbar_test(tfull + 16 * a, pa);
                    }
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i)
                        fma2(acc[kCols / 2 * c + i], pack2(r[c & 1][2 * i], r[c & 1][2 * i + 1]),
                             c < 64 / kCols ? two0 : two1);
                }
                const uint32_t slot = ring / kScaleBlocks;
                ++ring;
                if (kb == 1) ring = (ring + kScaleBlocks - 1) & ~static_cast<uint32_t>(kScaleBlocks - 1);
                if ((ring & (kScaleBlocks - 1)) == 0) {   // (the warp has met since it read the scales)
                    if (lane == 0) ptx::mbar_arrive(sempty + 8 * slot);
                    if (ring == 2 * kScaleBlocks) {
                        ring = 0;
                        pring ^= 1u;
                    }
                }
            }
            const int local = static_cast<int>(rank) * 128 + 32 * q + lane;   // this lane's row of the unit
            const int64_t row = trow0 + local;
            if constexpr (MODE == LINEAR) {
                if (!ok) {
                    if (lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    break;
                }
                const int col0 = tf * kFeatures + half * N;
                auto store = [&](auto *y) {
                    using T = typename std::remove_reference<decltype(*y)>::type;
                    constexpr int M = 32 / sizeof(T), kAhead = 4;   // columns of a sector; sectors requested together
                    T *to = y + row * p.out + col0;
                    const T *from = static_cast<const T *>(p.res) + row * p.out + col0;
                    const int left = p.out - col0;
#pragma unroll
                    for (int c0 = 0; c0 < N; c0 += kAhead * M) {
                        uint4 r[2 * kAhead];
#pragma unroll
                        for (int i = 0; i < 2 * kAhead; ++i)
                            r[i] = p.res && c0 + i * (M / 2) < left
                                       ? *reinterpret_cast<const uint4 *>(from + c0 + i * (M / 2))
                                       : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const int c = c0 + i * M;
                            float v[M];
#pragma unroll
                            for (int e = 0; e < M; e += 2) unpack2(acc[(c + e) / 2], v[e], v[e + 1]);
                            store_sector<T>(to + c, r + 2 * i, p.res != nullptr, v, left - c);
                        }
                    }
                };
                if (local < tvalid) {
                    if (p.dt == DT_BF16) store(static_cast<__nv_bfloat16 *>(p.y));
                    else if (p.dt == DT_F16) store(static_cast<__half *>(p.y));
                    else store(static_cast<float *>(p.y));
                }
            } else {
                // The two warps of a lane's row, 64 features each, meet (named barrier 1 + q).
                int both;
                asm volatile(
                    "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\tbar.red.and.pred b, %2, 64, a;\n\t"
                    "selp.b32 %0, 1, 0, b;\n\t}"
                    : "=r"(both)
                    : "r"(ok ? 1 : 0), "r"(1 + q)
                    : "memory");
                if (!both) {
                    if (lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    break;
                }
                const int f0 = tf * 128 + half * 64;
                float h[64], m = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float g[2], v[2];
                    unpack2(acc[i], g[0], g[1]);
                    unpack2(acc[32 + i], v[0], v[1]);
                    h[2 * i] = e4::swiglu(g[0], v[0]);
                    h[2 * i + 1] = e4::swiglu(g[1], v[1]);
                    m = max_nan(max_nan(m, h[2 * i]), h[2 * i + 1]);
                }
                if (f0 + 64 > p.out) {   // features that are the next expert's rows, or none
                    m = 0.f;
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        h[i] = f0 + i < p.out ? h[i] : 0.f;
                        m = max_nan(m, h[i]);
                    }
                }
                s_amax[half][32 * q + lane] = m;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
                m = max_nan(m, s_amax[half ^ 1][32 * q + lane]);   // (read before the next unit's vote)
                const float amax = floor_amax(m), k = kE4m3Max / amax;
                if (local < tvalid) {
                    if (half == 0) p.ys[row * p.nf + tf] = amax / kE4m3Max;
                    uint8_t *to = static_cast<uint8_t *>(p.y) + row * p.out + f0;
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = e4m3x4(h[c + 4 * i] * k, h[c + 4 * i + 1] * k, h[c + 4 * i + 2] * k,
                                          h[c + 4 * i + 3] * k);
                        if ((reinterpret_cast<uintptr_t>(to) & 31) == 0 && f0 + c + 32 <= p.out) {
                            st_sector(to + c, w);
                        } else {   // rows of whole 8 bytes
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (f0 + c + 8 * i < p.out)
                                    *reinterpret_cast<uint2 *>(to + c + 8 * i) = make_uint2(w[2 * i], w[2 * i + 1]);
                        }
                    }
                }
            }
        }
    }

    end_pair<kStages>(s_end, rank, produced, abort_flag, never, e4::kWaitNs, [&](int s) { return bar(&bar_full[s]); },
                      [](int, int) { return kStageBytes; });
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

bool map_codes(CUtensorMap *m, const void *ptr, int64_t in, int64_t rows, uint32_t box_rows) {
    return encode_tma_2d(m, ptr, CU_TENSOR_MAP_DATA_TYPE_UINT8, in, rows, in, 128, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, int N>
cudaError_t launch(const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in, const Params &p,
                   cudaStream_t s) {
    using C = Config<MODE, N>;
    const auto kern = &e4m3_pair_kernel<MODE, N>;
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
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.attrs = attr;
    int slots = 0;   // co-resident CTA pairs
    if (configured_device.load(std::memory_order_acquire) == dev) {
        slots = pair_slots.load(std::memory_order_relaxed);
    } else {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2 * static_cast<unsigned>(sm_count()));
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&slots, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (slots < 1) return cudaErrorLaunchOutOfResources;
        pair_slots.store(slots, std::memory_order_relaxed);
        configured_device.store(dev, std::memory_order_release);
    }
    CUtensorMap m0, m1, mx;
    const int64_t wrows = static_cast<int64_t>(p.experts) * p.out;
    if (!map_codes(&m0, w0, in, wrows, N / 2) || !map_codes(&mx, x, in, p.rows, 128)) return cudaErrorInvalidValue;
    m1 = m0;
    if (MODE == GATEUP && !map_codes(&m1, w1, in, wrows, N / 2)) return cudaErrorInvalidValue;
    const int64_t most = moe::max_tiles(p.rows, p.experts, kRows) * ((p.out + C::kFeatures - 1) / C::kFeatures);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(slots, most)));
    cfg.stream = s;
    cfg.numAttrs = 2;
    LaunchScope scope(MODE == GATEUP ? K_GATEUP_E4M3 : K_LINEAR_E4M3, s);
    e = cudaLaunchKernelEx(&cfg, kern, m0, m1, mx, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_e4m3_pair(e4::Mode mode, bool narrow, const uint8_t *x, const uint8_t *w0, const uint8_t *w1,
                             int64_t in, const Params &p, cudaStream_t s) {
    if (mode == GATEUP) return launch<GATEUP, 128>(x, w0, w1, in, p, s);
    return narrow ? launch<LINEAR, 64>(x, w0, w1, in, p, s) : launch<LINEAR, 128>(x, w0, w1, in, p, s);
}

}  // namespace ffn
