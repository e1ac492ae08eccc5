// linear_e4m3_pair.cu -- products of e4m3 codes with block scales for many rows.
//
// CTA pairs (tcgen05 .cta_group::2): a unit of work is 256 rows of x (128 in each
// CTA, the M operand) against 256 weight rows (linear: 256 features; gate/up:
// the 128 features of one scale block, gate's rows in the even CTA's half of the N
// operand, up's in the odd one's).  A block of 128 values is four instructions into
// one of two accumulators, which together are all of tensor memory.
//
// What bounds it: the tensor pipe, 512 cycles a block and SM, under which the
// epilogue warps read the block's 128 x 256 sums (256 cycles of tensor-memory
// reads) and add them, times the row's and the weight block's scale, to registers
// (128 a thread; two additions an instruction).  With x on the M side a thread's
// sums share one row, so that one factor serves all 128 of them; on the N side
// every column would need its own from shared memory, which the operands fill.
//
// Roles: warp 0 loads, warp 1 issues the MMAs (the even CTA's), warps 4-11 add the
// sums (lane = row of x; four warps for each half of the columns) and finish the
// unit while the next one's first two blocks run.  Every wait is bounded (1 s).
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

constexpr int kRows = 256;                                 // of x in a unit
constexpr uint32_t kStageBytes = 2 * e4::kTileBytes;       // one CTA's rows of x and of the weights
constexpr int kStages = 5;
constexpr int kEpiWarps = 8, kThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kOutBytes = kEpiWarps * 4096;           // where rows are turned for the stores
constexpr size_t kSmem = kStages * kStageBytes + kOutBytes + 1024;
static_assert(kSmem > 114 * 1024 && kSmem < 212 * 1024, "one CTA per SM: each allocates all of tensor memory");
constexpr uint32_t kTmemCols = 512;
// Registers of a thread after the warpgroups have shared them out: 168 at launch.
constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(4 * 32 * kFewRegs + kEpiWarps * 32 * kManyRegs <= kThreads * 168, "register split");
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
__device__ __forceinline__ void sts128(uint32_t at, float a, float b, float c, float d) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ float4 lds128(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    e4m3_pair_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                     const __grid_constant__ CUtensorMap map_x, const Params p) {
    constexpr int kFeatures = MODE == GATEUP ? 128 : 256;   // of a unit
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages], bar_tfull[2], bar_tempty[2], bar_drain;
    __shared__ int s_first[moe::kMaxExperts + 1], s_row0[moe::kMaxExperts], s_rows[moe::kMaxExperts];
    __shared__ uint32_t s_amax[MODE == GATEUP ? 2 : 1][128];
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort, s_never;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t out_base = base + kStages * kStageBytes;
    auto bar = [](uint64_t *b) { return ptx::smem_u32(b); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(&bar_full[s]), 1);
            ptx::mbar_init(bar(&bar_empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar(&bar_tfull[a]), 1);
            ptx::mbar_init(bar(&bar_tempty[a]), 2 * kEpiWarps);
        }
        ptx::mbar_init(bar(&bar_drain), 1);
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
        int before = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            int2 r = make_int2(0, 0);
            if (e < p.experts) r = e4::expert_rows(p, e);
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
                s_rows[e] = r.y - r.x;
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
        t.valid = min(kRows, s_rows[lo] - tt * kRows);
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
                const int wrow = t.expert * p.out + t.f * kFeatures + (MODE == GATEUP ? 0 : static_cast<int>(rank) * 128);
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
            constexpr uint32_t idesc = e4::idesc_e4m3(256, 256);
            bool ok = true;
            int s = 0, a = 0;
            uint32_t ph = 0, pa = 0;
            for (int u = u0; u < units && ok; u += ustep) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    bool got = ptx::mbar_wait(bar(&bar_tempty[a]), pa ^ 1u, abort_flag, e4::kWaitNs);
                    got = got && ptx::mbar_wait(bar(&bar_full[s]), ph, abort_flag, e4::kWaitNs);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint32_t at = base + s * kStageBytes;
                        const uint64_t ad = ptx::sdesc_k_sw128(at), bd = ptx::sdesc_k_sw128(at + e4::kTileBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 bytes of k further: 2 in the address field
                            e4::mma_e4m3_pair(tmem + a * 256, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                        ptx::tc_commit_pair(bar(&bar_empty[s]), 0x3);
                        ptx::tc_commit_pair(bar(&bar_tfull[a]), 0x3);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    a ^= 1;
                    if (a == 0) pa ^= 1u;
                }
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            if (ptx::elect_one()) ptx::tc_commit_pair(bar(&bar_drain), 0x1);   // every MMA ends before TMEM is freed
            ptx::mbar_wait(bar(&bar_drain), 0, never, e4::kWaitNs);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // ---------------------------------------------------------- sums
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t own = out_base + static_cast<uint32_t>(warp - 4) * 4096u;   // this warp's place to turn rows
        int a = 0;
        uint32_t pa = 0;
        for (int u = u0; u < units; u += ustep) {
            const Unit t = unit_of(u);
            const int local = static_cast<int>(rank) * 128 + 32 * q + lane;   // this lane's row of the unit
            const int nb = MODE == GATEUP ? t.f : min(2 * t.f + part, p.nf - 1);
            const float *xs = p.xs + static_cast<int64_t>(t.row0 + (local < t.valid ? local : 0)) * p.nkb;
            const float *ws = (MODE == GATEUP && part ? p.ws[1] : p.ws[0]) +
                              (static_cast<int64_t>(t.expert) * p.nf + nb) * p.nkb;
            // scales two blocks ahead
            float x0 = __ldg(xs), w0 = __ldg(ws), x1 = 0.f, w1 = 0.f;
            if (p.nkb > 1) {
                x1 = __ldg(xs + 1);
                w1 = __ldg(ws + 1);
            }
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
            bool ok = true;
            for (int kb = 0; kb < p.nkb; ++kb) {
                const uint32_t sb = __float_as_uint(x0 * w0);
                const uint64_t s2 = pack2(sb, sb);
                x0 = x1;
                w0 = w1;
                if (kb + 2 < p.nkb) {
                    x1 = __ldg(xs + kb + 2);
                    w1 = __ldg(ws + kb + 2);
                }
                const bool got = ptx::mbar_wait(bar(&bar_tfull[a]), pa, abort_flag, e4::kWaitNs);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + a * 256 + part * 128;
                uint32_t r[2][16];   // (32 at a time spill)
                ptx::tmem_ld_32x32b_x16(taddr, r[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    ptx::tmem_ld_wait();
                    if (c < 7) {
                        ptx::tmem_ld_32x32b_x16(taddr + 16 * (c + 1), r[(c + 1) & 1]);
                    } else {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_read(lead(bar(&bar_tempty[a])));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fma2(acc[8 * c + i], pack2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), s2);
                }
                a ^= 1;
                if (a == 0) pa ^= 1u;
            }
            if constexpr (MODE == LINEAR) {
                if (!ok) {
                    if (lane == 0) atomicOr(p.err, DEVERR_TIMEOUT);
                    *abort_flag = 1;
                    break;
                }
                // 32 columns at a time through shared memory, 16 bytes of a row at (their place ^ row) % 8
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v[4];
                        unpack2(acc[16 * c + 2 * j], v[0], v[1]);
                        unpack2(acc[16 * c + 2 * j + 1], v[2], v[3]);
                        sts128(own + lane * 128 + ((j ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
                    const int col = t.f * 256 + part * 128 + c * 32 + (lane & 7) * 4;
                    auto store = [&](auto *y) {
                        using T = typename std::remove_reference<decltype(*y)>::type;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int row = 4 * i + (lane >> 3), at_row = static_cast<int>(rank) * 128 + 32 * q + row;
                            const float4 f = lds128(own + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                            if (at_row >= t.valid || col >= p.out) continue;   // (out is a multiple of 8)
                            const int64_t at = static_cast<int64_t>(t.row0 + at_row) * p.out + col;
                            float v[4] = {f.x, f.y, f.z, f.w};
                            struct alignas(4 * sizeof(T)) Four {
                                T e[4];
                            } o;
                            if (p.res) {
                                const Four r4 = *reinterpret_cast<const Four *>(static_cast<const T *>(p.res) + at);
#pragma unroll
                                for (int e = 0; e < 4; ++e) v[e] += to_f32(r4.e[e]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) o.e[e] = from_f32<T>(v[e]);
                            *reinterpret_cast<Four *>(y + at) = o;
                        }
                    };
                    if (p.dt == DT_BF16) store(static_cast<__nv_bfloat16 *>(p.y));
                    else if (p.dt == DT_F16) store(static_cast<__half *>(p.y));
                    else store(static_cast<float *>(p.y));
                    __syncwarp();
                }
            } else {
                // The two warps of a lane's row meet (named barrier 1 + q): the gate's
                // finishes features 0-63 of the block, the up's 64-127.
                auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory"); };
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
                const uint32_t other = out_base + static_cast<uint32_t>((warp - 4) ^ 4) * 4096u;
                float h[64];
                uint32_t m = 0u;
#pragma unroll
                for (int c = 0; c < 2; ++c) {   // 32 features
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v[4];
                        unpack2(part ? acc[16 * c + 2 * j] : acc[32 + 16 * c + 2 * j], v[0], v[1]);
                        unpack2(part ? acc[16 * c + 2 * j + 1] : acc[32 + 16 * c + 2 * j + 1], v[2], v[3]);
                        sts128(own + j * 512 + lane * 16, v[0], v[1], v[2], v[3]);
                    }
                    meet();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 f = lds128(other + j * 512 + lane * 16);
                        const float theirs[4] = {f.x, f.y, f.z, f.w};
                        float mine[4];
                        unpack2(part ? acc[32 + 16 * c + 2 * j] : acc[16 * c + 2 * j], mine[0], mine[1]);
                        unpack2(part ? acc[32 + 16 * c + 2 * j + 1] : acc[16 * c + 2 * j + 1], mine[2], mine[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = 32 * c + 4 * j + e;
                            h[i] = e4::swiglu(part ? theirs[e] : mine[e], part ? mine[e] : theirs[e]);
                            if (t.f * 128 + 64 * part + i >= p.out) h[i] = 0.f;   // (the next expert's rows)
                            m = max(m, abs_bits(h[i]));
                        }
                    }
                    if (c == 1) s_amax[part][32 * q + lane] = m;
                    meet();
                }
                m = max(m, s_amax[part ^ 1][32 * q + lane]);
                const float amax = floor_amax(__uint_as_float(m)), k = kE4m3Max / amax;
                if (part == 0 && local < t.valid) p.ys[static_cast<int64_t>(t.row0 + local) * p.nf + t.f] = amax / kE4m3Max;
                // codes: 128 bytes a row, both warps' in the gate's place, turned as in linear
                const uint32_t codes = out_base + static_cast<uint32_t>(q) * 4096u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 16 * j + 4 * e;
                        w[e] = e4m3x4(h[i] * k, h[i + 1] * k, h[i + 2] * k, h[i + 3] * k);
                    }
                    sts128(codes + lane * 128 + (((4 * part + j) ^ (lane & 7)) << 4), __uint_as_float(w[0]),
                           __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
                }
                meet();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * part + 4 * i + (lane >> 3),
                              at_row = static_cast<int>(rank) * 128 + 32 * q + row;
                    const float4 f = lds128(codes + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    const int col = t.f * 128 + (lane & 7) * 16;
                    if (at_row >= t.valid || col >= p.out) continue;
                    uint8_t *to = static_cast<uint8_t *>(p.y) + static_cast<int64_t>(t.row0 + at_row) * p.out + col;
                    if ((p.out & 15) == 0) {
                        *reinterpret_cast<float4 *>(to) = f;
                    } else {   // rows of whole 8 bytes
                        *reinterpret_cast<float2 *>(to) = make_float2(f.x, f.y);
                        if (col + 8 < p.out) *reinterpret_cast<float2 *>(to + 8) = make_float2(f.z, f.w);
                    }
                }
                meet();
            }
        }
    }

    __syncthreads();
    if (warp == 0 && lane == 0 && leader) {
        // loads still in flight (only after an abandoned wait) land before shared memory is released
        for (uint32_t s = 0; s < kStages; ++s)
            if (produced > s)
                ptx::mbar_wait(bar(&bar_full[s]), ((produced - s + kStages - 1) / kStages - 1) & 1u, never, e4::kWaitNs);
    }
    __syncthreads();
    ptx::cluster_sync();   // neither CTA leaves while the other may still use its memory or barriers
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

bool map_codes(CUtensorMap *m, const void *ptr, int64_t in, int64_t rows) {
    return encode_tma_2d(m, ptr, CU_TENSOR_MAP_DATA_TYPE_UINT8, in, rows, in, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE>
cudaError_t launch(const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in, const Params &p,
                   cudaStream_t s) {
    constexpr int kFeatures = MODE == GATEUP ? 128 : 256;
    const auto kern = &e4m3_pair_kernel<MODE>;
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
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    int slots = 0;   // co-resident CTA pairs
    if (configured_device.load(std::memory_order_acquire) == dev) {
        slots = pair_slots.load(std::memory_order_relaxed);
    } else {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
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
    if (!map_codes(&m0, w0, in, wrows) || !map_codes(&m1, w1, in, wrows) || !map_codes(&mx, x, in, p.rows))
        return cudaErrorInvalidValue;
    const int64_t most = moe::max_tiles(p.rows, p.experts, kRows) * ((p.out + kFeatures - 1) / kFeatures);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(slots, most)));
    cfg.stream = s;
    cfg.numAttrs = 2;
    LaunchScope scope(MODE == GATEUP ? K_GATEUP_E4M3 : K_LINEAR_E4M3, s);
    e = cudaLaunchKernelEx(&cfg, kern, m0, m1, mx, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_e4m3_pair(e4::Mode mode, const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in,
                             const Params &p, cudaStream_t s) {
    return mode == GATEUP ? launch<GATEUP>(x, w0, w1, in, p, s) : launch<LINEAR>(x, w0, w1, in, p, s);
}

}  // namespace ffn
