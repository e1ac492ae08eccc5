// moe.cuh -- shared by the kernels of the routed (mixture-of-experts) block.
//
//   y_t = [res_t +] sum_j w_tj * W_down[e] ( silu(W_gate[e] x_t) * (W_up[e] x_t) ),  e = idx_tj
//
// One call: the plan sorts the (token, slot) pairs by expert and copies their
// rows of x in that order; the gate/up and the down product run over the
// experts' tiles; the last kernel adds each token's weighted results in slot
// order.
//
// The products put the WEIGHT rows on the M side of the tensor-core
// instruction and an expert's tokens on its N side.  N may be any multiple of
// 32 (16 without CTA pairs), so an expert with c tokens wastes fewer than 32
// columns where tokens on the M side would waste up to a whole 256-row tile,
// and the same scheme runs from one token (a stream of weights) to long prompts.
#pragma once

#include <type_traits>

#include "ffn_internal.cuh"

namespace ffn {
namespace moe {

// A token tile: `cols` columns or, the expert's last one, fewer.  The tiles
// of one expert are numbered first .. first + count - 1; the expert's rows in
// sorted order are row0 .. row0 + rows - 1.
struct Tile {
    int expert, first, count, cols;
    int row0, rows;
    unsigned done, odd;   // see Levels: groups of rows levelled; 0, or 1 + twice the groups taken
};

struct Plan {
    int *header;       // [0] token tiles, [1] columns of the widest tile, [2] whether a tile is odd
    Tile *tiles;
    int *hist;         // [chunks][experts] pairs of each expert (more than 256 pairs)
    int *pos;          // sorted row of pair (token, slot), or -1 (no expert)
    float *scale;      // of sorted row r: its down product is multiplied by this (null with level)
    uint4 *level;      // of 32 features of h, a byte each, in whole vectors a row (see Levels; null without)
    int nlevel;        // vectors of a row
};

// How a product cuts its work: token tiles of at most `tile` columns, ending
// on multiples of `gran`.
struct Cut {
    int tile, gran;
};

constexpr int kMaxExperts = 1024;

__host__ __device__ constexpr int64_t max_tiles(int64_t pairs, int64_t experts, int tile) {
    return pairs / tile + (pairs < experts ? pairs : experts);
}

// The unit of work u of a product with nf feature tiles: an expert's units
// run through its token tiles first, so that the feature tile's weights are
// read from HBM once and from L2 by the other token tiles.
struct Unit {
    int expert, f, tt, row0, valid, n;   // tt: which token tile of the expert
    int tile;                            // its place in the table
    bool odd;                            // whether its rows have to be levelled
};
template <int GRAN>
__device__ __forceinline__ Unit unit_of(int u, int nf, const int4 &a, const int4 &b) {
    Unit r;
    const int local = u - a.y * nf;
    r.expert = a.x;
    r.f = local / a.z;
    r.tt = local - r.f * a.z;
    r.tile = a.y + r.tt;
    r.odd = b.w != 0;
    r.row0 = b.x + r.tt * a.w;
    r.valid = min(a.w, b.y - r.tt * a.w);
    r.n = (r.valid + GRAN - 1) & ~(GRAN - 1);
    return r;
}

// A role's walk over its units: the next unit's table entry is requested when
// the current one is handed out, so that its latency (an L2 access) passes
// under the current unit's stages.
template <int GRAN> struct Walk {
    const int4 *tiles;
    int nf, splits, units, step;
    int4 a, b;
    __device__ __forceinline__ void fetch(int v) {
        if (v >= units) return;
        const int4 *t = tiles + 2 * (v / splits / nf);
        a = __ldcg(t);
        b = __ldcg(t + 1);
    }
    __device__ __forceinline__ Walk(const int4 *t, int n, int s, int total, int first, int by)
        : tiles(t), nf(n), splits(s), units(total), step(by), a(make_int4(0, 0, 1, 0)), b(a) {
        fetch(first);
    }
    __device__ __forceinline__ Unit at(int v) {
        const Unit u = unit_of<GRAN>(v / splits, nf, a, b);
        fetch(v + step);
        return u;
    }
};

// The sorted rows a tile reads, loaded in boxes of 128, 64, 32 and 16 rows:
// `rows` (a multiple of 16, at most 128) are the boxes of its set bits.
struct RowMaps {
    CUtensorMap m[4];
};
template <typename F>
__device__ __forceinline__ void for_row_boxes(const RowMaps &maps, int rows, F load) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (rows & (128 >> i)) load(&maps.m[i], rows & ~((256 >> i) - 1));
}

// silu(gate) * up * scale in fp32.  The division is the approximate one (2 ulp,
// and 0 for a denominator beyond 2^126, where silu is below 1e-36), and so is the
// exponential (2 + 1.17 |gate| ulp, 105 at the end of its range): together at
// most 1.3e-5 of the value, a fortieth of fp16's half step, and a third of the
// instructions of the accurate forms in epilogues that the MMAs wait for.
__device__ __forceinline__ float swiglu(float gate, float up, float scale) {
    return __fdividef(gate, 1.0f + __expf(-gate)) * (up * scale);
}

// ---- the range of h in fp16
//
// fp16 has 11 bits from 2^-14 to 2^16 only, and nothing is known of h's size
// before it is computed.  So h is stored a block at a time -- 32 features of a
// row, what one warp of the epilogue holds of a column -- times 2^(16 level):
// level 0 where the block's largest value is in [2^-12, 2^15), 1 down to 2^-28,
// -1 up to 2^31 and so on.  One scale has to hold for a whole row, as the down
// product adds over its features: the row's is the lowest level of its blocks,
// and blocks of a higher one are multiplied down to it (what that rounds away is
// below half of 2^-24, where the row has a value of 2^-12 or more).  The down
// product's epilogue undoes the row's scale.
//
// The plan sets every level to 0; the gate/up product writes the others and
// marks their tiles as odd.  In the down product whoever needs an odd tile takes
// groups of eight of its rows and levels them until none is left, and then waits
// for those that others took, who are running; its epilogue warps, idle at
// first, begin with all odd tiles.  A tile of ordinary values costs the check
// of h and nothing else (4096 tokens, 6 of 64 experts of 2048 x 1408, fp16: 428
// us with it and 427 without; with every value of x 1 / 300 as large, all rows
// of level 1, gate/up takes 19 and down 30 us more, and at 1 / 100, where
// nearly every row has blocks of two levels, 19 and 126).  A scale fixed ahead,
// 2^-8, cost nothing either but lost h below 2^-17 altogether.
struct Levels {
    uint4 *level;      // [pairs][vectors], a byte a block of 32 features
    int nlevel;        // vectors of a row
    float *scale;      // [pairs], 1 from the plan
    __half *h;         // [pairs x cols], for the down product
    int cols;
    int *header;
};
inline Levels levels_of(const Plan &p, const void *h, int64_t cols) {
    return {p.level, p.nlevel, p.scale, static_cast<__half *>(const_cast<void *>(h)),
            static_cast<int>(cols), p.header};
}
constexpr unsigned short kLevelLow = 0x0c00, kLevelHigh = 0x7800;   // fp16: 2^-12, 2^15
constexpr int kLevelStep = 16, kMaxLevel = 7, kNoLevel = 127;           // kNoLevel: all zero, fits any row
__device__ __forceinline__ float level_scale(int level) {               // -7 .. 7
    return __uint_as_float(static_cast<uint32_t>(127 + kLevelStep * level) << 23);
}
// Of a block whose largest magnitude has these bits.  Level 0 begins where the
// value rounded to fp16 is 2^-12 (at 2^-12 - 2^-24), as in the epilogue's check
// of eight columns at once: a row's levels do not depend on the rows beside it.
__device__ __forceinline__ int level_of(uint32_t bits) {
    if (bits == 0u) return kNoLevel;
    if (bits >= 0x7f800000u) return 0;   // infinity, NaN: nothing to keep
    const int e = static_cast<int>(bits >> 23);   // biased by 127
    if (bits < 0x397ff000u) return min((114 - e) / kLevelStep + 1, kMaxLevel);
    if (e >= 142) return max(-((e - 142) / kLevelStep + 1), -kMaxLevel);
    return 0;
}

// ---- epilogues (four warps, q = warp % 4, lane: weight row 32 q + lane of the
// accumulator; columns are the tile's rows)

// Lanes 0-63 of the accumulator hold gate, 64-127 up of the 64 features from
// f0.  Of every 16 columns (from c0, `step` on) the gate warps finish the
// first eight and the up warps the others; each side hands over what the
// other needs, through `swap` and named barrier `id`.  PERM: h's columns 1
// and 2 of every four exchanged.  h feeds the next product, in its operand type.
// For bf16 that is one term, 8 bits, where the dense block has two: there the
// normalised input is rounded as well, here it comes as bf16, and what h's
// rounding (half a step is 2^-8) adds to y, about 0.17 % rms, is what y's own
// adds; a second term would double the down product's MMAs and loads of h.
template <typename T, bool PERM>
__device__ __forceinline__ void swiglu_epilogue(uint32_t taddr, int q, int lane, const Unit &t, int f0, int wrows, T *h,
                                                float (*swap)[2][8][64], int c0, int step, int id, float acc_scale,
                                                const Levels &lv, const int4 *tiles) {
    constexpr bool LEVELS = std::is_same<T, __half>::value;   // (bf16 has the range of fp32)
    const int fl = 32 * (q & 1) + lane, mat = q >> 1;
    const int f = f0 + fl;
    const int at = PERM ? (f & ~3) | ((f & 1) << 1) | ((f >> 1) & 1) : f;
    const bool live = f < wrows, block = f - lane < wrows;   // block: some lane is live
    T *dst = h + static_cast<int64_t>(t.row0) * wrows + at;
    bool odd = false;
    for (int c = c0, pp = 0; c < t.n; c += step, pp ^= 1) {
        uint32_t r[16];
        ptx::tmem_ld_32x32b_x16(taddr + c, r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) swap[pp][mat][i][fl] = __uint_as_float(mat ? r[i] : r[8 + i]);
        asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
        const int cm = c + 8 * mat;
        float hv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = swap[pp][mat ^ 1][i][fl];
            const float mine = __uint_as_float(mat ? r[8 + i] : r[i]);
            hv[i] = swiglu((mat ? other : mine) * acc_scale, mat ? mine : other, acc_scale);
        }
        T *to = dst + static_cast<int64_t>(cm) * wrows;
        if constexpr (LEVELS) {
            if (cm + 8 > t.valid) {   // columns that are none
#pragma unroll
                for (int i = 0; i < 8; ++i) hv[i] = cm + i < t.valid ? hv[i] : 1.f;
            }
            __half2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __floats2half2_rn(hv[2 * i], hv[2 * i + 1]);
            // a lane all of whose values are in [2^-12, 2^15), none with one
            // beyond: every block is of level 0 (the usual case)
            __half2 least = __habs2(v[0]), most = least;
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                least = __hmin2(least, __habs2(v[i]));
                most = __hmax2(most, __habs2(v[i]));
            }
            const bool usual =
                __any_sync(0xffffffffu, live && __hbge2(least, __half2half2(__ushort_as_half(kLevelLow)))) &&
                !__any_sync(0xffffffffu, live && !__hblt2(most, __half2half2(__ushort_as_half(kLevelHigh))));
            int mine = 0;   // lane i: the level of column i
            if (!usual && block) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t bits = live ? __float_as_uint(hv[i]) & 0x7fffffffu : 0u;
                    const int level = level_of(__reduce_max_sync(0xffffffffu, bits));
                    if (level != 0 && level != kNoLevel) {
                        hv[i] *= level_scale(level);
                        odd = true;
                    }
                    mine = lane == i ? level : mine;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __floats2half2_rn(hv[2 * i], hv[2 * i + 1]);
                if (mine != 0 && cm + lane < t.valid) {   // (lanes 0 to 7)
                    uint4 *of_row = lv.level + static_cast<int64_t>(t.row0 + cm + lane) * lv.nlevel;
                    reinterpret_cast<int8_t *>(of_row)[f >> 5] = static_cast<int8_t>(mine);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (live && cm + i < t.valid) *to = i & 1 ? __high2half(v[i >> 1]) : __low2half(v[i >> 1]);
                to += wrows;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (live && cm + i < t.valid) *to = from_f32<T>(hv[i]);
                to += wrows;
            }
        }
    }
    if (LEVELS && odd && !t.odd && lane == 0) {
        reinterpret_cast<Tile *>(const_cast<int4 *>(tiles))[t.tile].odd = 1u;
        lv.header[2] = 1;
    }
}

// Takes groups of eight rows of an odd tile and brings them to one level each,
// until none is left (a converged warp).
__device__ __forceinline__ void level_groups(const Levels &lv, Tile *tile, int row0, int valid, int lane) {
    const unsigned groups = static_cast<unsigned>(valid + 7) / 8;
    while (true) {
        unsigned g = 0u;
        if (lane == 0) g = atomicAdd(&tile->odd, 2u) >> 1;
        g = __shfl_sync(0xffffffffu, g, 0);
        if (g >= groups) break;
        // the levels of eight rows, four lanes a row
        const int r = 8 * static_cast<int>(g) + (lane >> 2);
        int lowest = kNoLevel, highest = -kNoLevel;
        if (r < valid) {
            const uint4 *lvl = lv.level + static_cast<int64_t>(row0 + r) * lv.nlevel;
#pragma unroll 4
            for (int c = lane & 3; c < lv.nlevel; c += 4) {
                const uint4 v = __ldcg(lvl + c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                if ((v.x | v.y | v.z | v.w) == 0u) {   // (so are the bytes past the row's last block)
                    lowest = min(lowest, 0);
                    highest = max(highest, 0);
                    continue;
                }
#pragma unroll
                for (int b = 0; b < 16; ++b) {
                    const int level = static_cast<int8_t>(w[b >> 2] >> (8 * (b & 3)));
                    if (512 * c + 32 * b >= lv.cols || level == kNoLevel) continue;
                    lowest = min(lowest, level);
                    highest = max(highest, level);
                }
            }
        }
        for (int o = 1; o < 4; o <<= 1) {
            lowest = min(lowest, __shfl_xor_sync(0xffffffffu, lowest, o));
            highest = max(highest, __shfl_xor_sync(0xffffffffu, highest, o));
        }
        if ((lane & 3) == 0 && lowest != 0 && lowest != kNoLevel) lv.scale[row0 + r] = level_scale(-lowest);
        // the rows of unequal levels, one after the other
        unsigned todo = __ballot_sync(0xffffffffu, (lane & 3) == 0 && lowest < highest);
        while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            const int to = __shfl_sync(0xffffffffu, lowest, i);
            const int64_t at = row0 + 8 * static_cast<int>(g) + (i >> 2);
            const signed char *lvl = reinterpret_cast<const signed char *>(lv.level + at * lv.nlevel);
            uint4 *row = reinterpret_cast<uint4 *>(lv.h + at * lv.cols);   // (whole vectors)
#pragma unroll 4
            for (int c = lane; c < lv.cols / 8; c += 32) {
                const int level = __ldcg(lvl + (c >> 2));
                const uint4 v = __ldcg(row + c);
                if (level != kNoLevel && level > to) {
                    const float scale = level_scale(max(to - level, -kMaxLevel));
                    float f[8];
                    Vec16<__half>::unpack(v, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= scale;
                    row[c] = Vec16<__half>::pack(f);
                }
            }
        }
        asm volatile("fence.proxy.async;" ::: "memory");   // the copy engine reads the rows
        __threadfence();
        __syncwarp();
        if (lane == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(&tile->done) : "memory");
    }
}

// Before a warp of the down product loads an odd tile.  False if the wait for
// the groups that others took was given up.
__device__ __forceinline__ bool level_tile(const Levels &lv, const int4 *tiles, const Unit &t, int lane,
                                           volatile int *abort, uint64_t limit_ns) {
    Tile *tile = reinterpret_cast<Tile *>(const_cast<int4 *>(tiles)) + t.tile;
    auto finished = [&]() {
        unsigned n;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(&tile->done) : "memory");
        return __all_sync(0xffffffffu, 8u * n >= static_cast<unsigned>(t.valid));
    };
    if (!finished()) {
        level_groups(lv, tile, t.row0, t.valid, lane);
        const uint64_t t0 = ptx::globaltimer_ns();
        while (!finished())
            if (__any_sync(0xffffffffu, *abort != 0 || ptx::globaltimer_ns() - t0 > limit_ns)) return false;
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    return true;
}

// Warp w of n idle ones: the odd tiles from one of its own on.  At most 128, as
// accumulators wait for it for no more than a second; that is all of 77000, and
// the others are levelled by who loads them.
__device__ __forceinline__ void level_ahead(const Levels &lv, const int4 *tiles, int w, int n, int lane) {
    if (__ldcg(lv.header + 2) == 0) return;
    const int count = __ldcg(lv.header);
    const int first = static_cast<int>(static_cast<int64_t>(count) * w / n);
    for (int i = 0; i < min(count, 128); ++i) {
        const int at = first + i < count ? first + i : first + i - count;
        const int4 a = __ldcg(tiles + 2 * at), b = __ldcg(tiles + 2 * at + 1);
        const int valid = min(a.w, b.y - (at - a.y) * a.w);
        if (b.w == 0 || (b.w >> 1) * 8 >= valid) continue;   // of level 0, or all taken
        level_groups(lv, reinterpret_cast<Tile *>(const_cast<int4 *>(tiles)) + at, b.x + (at - a.y) * a.w, valid, lane);
    }
}

// The down product's results of 16 columns (ODD: of rows with scales).
template <bool ODD>
__device__ __forceinline__ void store_columns(uint32_t taddr, float *dst, const float *scale, bool live, int columns,
                                              int wrows, float acc_scale) {
    uint32_t r[16];
    ptx::tmem_ld_32x32b_x16(taddr, r);
    const int lane = threadIdx.x & 31;
    float mine = acc_scale;   // lane i: of column i
    if (ODD && lane < min(columns, 16)) mine *= __ldcg(scale + lane);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s = ODD ? __shfl_sync(0xffffffffu, mine, i) : acc_scale;
        if (live && i < columns) *dst = __uint_as_float(r[i]) * s;
        dst += wrows;
    }
}
// Columns c0, c0 + step, ... (16 each) of a unit, feature f of this lane.
__device__ __forceinline__ void store_epilogue(uint32_t taddr, const Unit &t, int f, int c0, int step, int wrows,
                                               float *part, float acc_scale, const float *scale) {
    float *dst = part + static_cast<int64_t>(t.row0) * wrows + f;
    for (int c = c0; c < t.n; c += step) {
        float *to = dst + static_cast<int64_t>(c) * wrows;
        const bool live = f < wrows;
        if (t.odd && scale) store_columns<true>(taddr + c, to, scale + t.row0 + c, live, t.valid - c, wrows, acc_scale);
        else store_columns<false>(taddr + c, to, nullptr, live, t.valid - c, wrows, acc_scale);
    }
}

// Whether all four warps of named barrier `id` passed their wait (they stay
// or leave together).
__device__ __forceinline__ bool epilogue_vote(bool got, int id) {
    int all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\tbar.red.and.pred b, %2, 128, a;\n\t"
        "selp.b32 %0, 1, 0, b;\n\t}"
        : "=r"(all)
        : "r"(got ? 1 : 0), "r"(id)
        : "memory");
    return all != 0;
}

}  // namespace moe

size_t moe_plan_bytes(int64_t pairs, int64_t experts, int tile);
// what every number of pairs up to `pairs` fits into
size_t moe_plan_bytes_upto(int64_t pairs, int64_t experts, int tile);
moe::Plan moe_plan_carve(void *base, int64_t pairs, int64_t experts, int tile);
// Sorts the pairs of idx [rows x k] into token tiles and writes their rows of
// x [rows x d] (type dt) in sorted order to xs [pairs x d]: as they are, or as
// fp16 (to_f16), there with columns 1 and 2 of every four exchanged (perm).
cudaError_t launch_moe_plan(const int32_t *idx, int64_t rows, int k, int experts, moe::Cut cut, const moe::Plan &plan,
                            const void *x, void *xs, int64_t d, int dt, bool to_f16, bool perm, cudaStream_t s);
// y = [res +] sum over slots of w * (sum over splits of part[split][pos]);
// part fp32 [splits x pairs x d].
cudaError_t launch_moe_combine(const moe::Plan &plan, const float *w, const float *part, int splits, const void *res,
                               void *y, int64_t rows, int k, int64_t d, int dt, cudaStream_t s);

// 16-bit weights (op: the operands' type), many tokens: CTA pairs (moe_gemm.cu).
constexpr moe::Cut kMoeCutPair = {256, 32};
cudaError_t launch_moe_gateup(int op, const moe::Plan &plan, const void *xs, const void *wg, const void *wu, void *h,
                              int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s);
cudaError_t launch_moe_down(int op, const moe::Plan &plan, const void *h, const void *wd, float *part, int64_t pairs,
                            int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s);

// 16-bit weights, few tokens: single CTAs streaming weights (moe_stream.cu).
constexpr moe::Cut kMoeCutStream = {64, 16};
cudaError_t launch_moe_gateup_stream(int op, const moe::Plan &plan, const void *xs, const void *wg, const void *wu,
                                     void *h, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                                     cudaStream_t s);
cudaError_t launch_moe_down_stream(int op, const moe::Plan &plan, const void *h, const void *wd, float *part,
                                   int splits, int64_t pairs, int64_t d, int64_t ffn, int64_t experts,
                                   float acc_scale, cudaStream_t s);

// Q4 weights (moe_gemm_q4.cu): xs is fp16 with perm; h is written in the same order.
constexpr moe::Cut kMoeCutQ4 = {128, 16};
cudaError_t launch_moe_gateup_q4(const moe::Plan &plan, const void *xs, const uint8_t *qg, const uint16_t *sg,
                                 const uint8_t *qu, const uint16_t *su, void *h, int64_t pairs, int64_t d, int64_t ffn,
                                 int64_t experts, cudaStream_t s);
cudaError_t launch_moe_down_q4(const moe::Plan &plan, const void *h, const uint8_t *qd, const uint16_t *sd, float *part,
                               int splits, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, cudaStream_t s);

// Splits of the down product's reduction on the single-CTA kernels (units of
// 128 weight rows, counted in stages of 128 values; the Q4 kernel cuts between
// its stages of 256): at most kMoeMaxSplits, none shorter than 4 stages, 1 beyond
// kMoeSplitPairs pairs.  A function of the sizes alone, so that the workspace
// query and the call agree.
constexpr int kMoeMaxSplits = 8;
constexpr int64_t kMoeSplitPairs = 1024;
int moe_down_splits(int64_t pairs, int64_t experts, int64_t d, int64_t ffn);

}  // namespace ffn
