// moe.cuh -- shared by the kernels of the routed (mixture-of-experts) block.
//
//   y_t = [res_t +] sum_j w_tj * W_down[e] ( silu(W_gate[e] x_t) * (W_up[e] x_t) ),  e = idx_tj
//
// One call is four kernels: the plan sorts the (token, slot) pairs by expert;
// the gate/up and the down product run over the experts' tiles; the last one
// adds each token's weighted results in slot order.
//
// The products put the WEIGHT rows on the M side of the tensor-core
// instruction and an expert's tokens on its N side.  N may be any multiple of
// 32, so an expert with c tokens wastes fewer than 32 columns where tokens on
// the M side would waste up to a whole 256-row tile, and the same kernel runs
// from one token (a stream of weights) to long prompts.
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
    int *row_token;    // token of each sorted row
    int *pos;          // sorted row of pair (token, slot), or -1 (no expert)
};

constexpr int kMaxExperts = 1024;

__host__ __device__ constexpr int64_t max_tiles(int64_t pairs, int64_t experts, int tile) {
    return pairs / tile + (pairs < experts ? pairs : experts);
}

// The unit of work u of a product with nf feature tiles: an expert's units
// run through its token tiles first, so that the feature tile's weights are
// read from HBM once and from L2 by the other token tiles.
struct Unit {
    int expert, f, row0, valid, n;
};
__device__ __forceinline__ Unit unit_of(int u, int nf, const int4 &a, const int4 &b) {
    Unit r;
    const int local = u - a.y * nf;
    r.expert = a.x;
    r.f = local / a.z;
    const int tt = local - r.f * a.z;
    r.row0 = b.x + tt * a.w;
    r.valid = min(a.w, b.y - tt * a.w);
    r.n = (r.valid + 31) & ~31;
    return r;
}

}  // namespace moe

size_t moe_plan_bytes(int64_t pairs, int64_t experts, int tile);
moe::Plan moe_plan_carve(void *base, int64_t pairs, int64_t experts, int tile);
// Sorts the pairs of idx [rows x k] into token tiles of at most `tile`
// columns (a multiple of 32) and, with x16, writes x (bf16 or fp16, type dt)
// as fp16 there; perm: columns 1 and 2 of every four exchanged.
cudaError_t launch_moe_plan(const int32_t *idx, int64_t rows, int k, int experts, int tile, const moe::Plan &plan,
                            const void *x, void *x16, int64_t d, int dt, bool perm, cudaStream_t s);
// y = [res +] sum over slots of w * part[pos]; part fp32 [pairs x d].
cudaError_t launch_moe_combine(const moe::Plan &plan, const float *w, const float *part, const void *res, void *y,
                               int64_t rows, int k, int64_t d, int dt, cudaStream_t s);

// The products with 16-bit weights (moe_gemm.cu); op: the operands' type.
constexpr int kMoeTile = 256;
cudaError_t launch_moe_gateup(int op, const moe::Plan &plan, const void *x, const void *wg, const void *wu, void *h,
                              int64_t rows, int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                              float out_scale, cudaStream_t s);
cudaError_t launch_moe_down(int op, const moe::Plan &plan, const void *h, const void *wd, float *part, int64_t pairs,
                            int64_t d, int64_t ffn, int64_t experts, float acc_scale, cudaStream_t s);

// The products with Q4 weights (moe_gemm_q4.cu): x16 is x in fp16, columns 1
// and 2 of every four exchanged; h is written in the same order.
constexpr int kMoeQ4Tile = 128;
cudaError_t launch_moe_gateup_q4(const moe::Plan &plan, const void *x16, const uint8_t *qg, const uint16_t *sg,
                                 const uint8_t *qu, const uint16_t *su, void *h, int64_t rows, int64_t pairs, int64_t d,
                                 int64_t ffn, int64_t experts, float out_scale, cudaStream_t s);
cudaError_t launch_moe_down_q4(const moe::Plan &plan, const void *h, const uint8_t *qd, const uint16_t *sd, float *part,
                               int64_t pairs, int64_t d, int64_t ffn, int64_t experts, float acc_scale,
                               cudaStream_t s);

}  // namespace ffn
