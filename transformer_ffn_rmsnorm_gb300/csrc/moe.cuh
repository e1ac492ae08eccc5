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

#include "ffn_internal.cuh"

namespace ffn {
namespace moe {

// A token tile: `cols` columns or, the expert's last one, fewer.  The tiles
// of one expert are numbered first .. first + count - 1; the expert's rows in
// sorted order are row0 .. row0 + rows - 1.
struct Tile {
    int expert, first, count, cols;
    int row0, rows, pad0, pad1;
};

struct Plan {
    int *header;       // [0] token tiles, [1] columns of the widest tile
    Tile *tiles;
    int *hist;         // [chunks][experts] pairs of each expert (more than 256 pairs)
    int *pos;          // sorted row of pair (token, slot), or -1 (no expert)
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
};
template <int GRAN>
__device__ __forceinline__ Unit unit_of(int u, int nf, const int4 &a, const int4 &b) {
    Unit r;
    const int local = u - a.y * nf;
    r.expert = a.x;
    r.f = local / a.z;
    r.tt = local - r.f * a.z;
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
// and 0 for a denominator beyond 2^126, where silu is below 1e-36): next to the
// 16-bit rounding of h nothing, and a third of the instructions of the
// correctly rounded reciprocal, in epilogues that the MMAs wait for.
__device__ __forceinline__ float swiglu(float gate, float up, float scale) {
    return __fdividef(gate, 1.0f + __expf(-gate)) * (up * scale);
}

// ---- epilogues (four warps, q = warp % 4, lane: weight row 32 q + lane of the
// accumulator; columns are the tile's rows)

// Lanes 0-63 of the accumulator hold gate, 64-127 up of the 64 features from
// f0.  Of every 16 columns (from c0, `step` on) the gate warps finish the
// first eight and the up warps the others; each side hands over what the
// other needs, through `swap` and named barrier `id`.  PERM: h's columns 1
// and 2 of every four exchanged.  h feeds the next product: one rounding to
// its operand type.
template <typename T, bool PERM>
__device__ __forceinline__ void swiglu_epilogue(uint32_t taddr, int q, int lane, const Unit &t, int f0, int wrows, T *h,
                                                float (*swap)[2][8][64], int c0, int step, int id, float acc_scale,
                                                float out_scale) {
    const int fl = 32 * (q & 1) + lane, mat = q >> 1;
    const int f = f0 + fl;
    const int at = PERM ? (f & ~3) | ((f & 1) << 1) | ((f >> 1) & 1) : f;
    const bool live = f < wrows;
    T *dst = h + static_cast<int64_t>(t.row0) * wrows + at;
    for (int c = c0, pp = 0; c < t.n; c += step, pp ^= 1) {
        uint32_t r[16];
        ptx::tmem_ld_32x32b_x16(taddr + c, r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) swap[pp][mat][i][fl] = __uint_as_float(mat ? r[i] : r[8 + i]);
        asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
        T *to = dst + static_cast<int64_t>(c + 8 * mat) * wrows;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = swap[pp][mat ^ 1][i][fl];
            const float mine = __uint_as_float(mat ? r[8 + i] : r[i]);
            const float hv = swiglu((mat ? other : mine) * acc_scale, mat ? mine : other, acc_scale * out_scale);
            if (live && c + 8 * mat + i < t.valid) *to = from_f32<T>(hv);
            to += wrows;
        }
    }
}

__device__ __forceinline__ void store_epilogue(uint32_t taddr, int q, int lane, const Unit &t, int wrows, float *part,
                                               float acc_scale) {
    const int f = t.f * 128 + 32 * q + lane;
    float *dst = part + static_cast<int64_t>(t.row0) * wrows + f;
    for (int c = 0; c < t.n; c += 16) {
        uint32_t r[16];
        ptx::tmem_ld_32x32b_x16(taddr + c, r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (f < wrows && c + i < t.valid)
                dst[static_cast<int64_t>(c + i) * wrows] = __uint_as_float(r[i]) * acc_scale;
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
                              int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale, float out_scale,
                              cudaStream_t s);
cudaError_t launch_moe_down(int op, const moe::Plan &plan, const void *h, const void *wd, float *part, int64_t pairs,
                            int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s);

// 16-bit weights, few tokens: single CTAs streaming weights (moe_stream.cu).
constexpr moe::Cut kMoeCutStream = {64, 16};
cudaError_t launch_moe_gateup_stream(int op, const moe::Plan &plan, const void *xs, const void *wg, const void *wu,
                                     void *h, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                                     float out_scale, cudaStream_t s);
cudaError_t launch_moe_down_stream(int op, const moe::Plan &plan, const void *h, const void *wd, float *part,
                                   int splits, int64_t pairs, int64_t d, int64_t ffn, int64_t experts,
                                   float acc_scale, cudaStream_t s);

// Q4 weights (moe_gemm_q4.cu): xs is fp16 with perm; h is written in the same order.
constexpr moe::Cut kMoeCutQ4 = {128, 16};
cudaError_t launch_moe_gateup_q4(const moe::Plan &plan, const void *xs, const uint8_t *qg, const uint16_t *sg,
                                 const uint8_t *qu, const uint16_t *su, void *h, int64_t pairs, int64_t d, int64_t ffn,
                                 int64_t experts, float out_scale, cudaStream_t s);
cudaError_t launch_moe_down_q4(const moe::Plan &plan, const void *h, const uint8_t *qd, const uint16_t *sd, float *part,
                               int splits, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                               cudaStream_t s);

// Splits of the down product's reduction on the single-CTA kernels (units of
// 128 weight rows, stages of 128 values): at most 8, none shorter than 4
// stages.  A function of the sizes alone, so that the workspace query and the
// call agree.
int moe_down_splits(int64_t pairs, int64_t experts, int64_t d, int64_t ffn);

}  // namespace ffn
