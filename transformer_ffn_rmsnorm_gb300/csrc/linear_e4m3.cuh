// linear_e4m3.cuh -- shared by the products of e4m3 codes with scales for each 128
// values:
//
//   linear:  y[r, o] = [res[r, o] +] P(W)[r, o]
//   gate/up: h[r, f] = silu(P(W_gate)[r, f]) * P(W_up)[r, f], stored as e4m3 codes
//            with a scale for each 128 features
//   P(W)[r, o] = sum_b sx[r, b] * sw[o / 128, b] * sum_{i in block b} qx[r, i] * qw[o, i]
//
// The tensor cores multiply the codes (tcgen05 kind::f8f6f4, exact products, fp32
// sums) a block of 128 values at a time into tensor memory; the scales differ from
// block to block, so that each block's sums are read out and added to fp32
// registers times their two scales.  W is one matrix, or one of each expert, the
// rows of x then in the order of their experts (offsets[e] .. offsets[e + 1] - 1).
#pragma once

#include "e4m3.cuh"

namespace ffn {
namespace e4 {

enum Mode { LINEAR = 0, GATEUP = 1 };

struct Params {
    const float *xs;          // [rows x nkb]
    const float *ws[2];       // [experts x nf x nkb] (linear: one)
    const int32_t *offsets;   // [experts + 1], or null: one expert, all rows
    int rows, experts;
    int out;                  // weight rows of an expert
    int nf, nkb;              // blocks of 128 of out and of the reduction
    void *y;                  // linear: [rows x out] of type dt; gate/up: codes
    const void *res;          // linear: as y, or null
    float *ys;                // gate/up: [rows x nf]
    int dt;
    unsigned *err;
};

constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kTileBytes = 128 * 128;   // 128 rows of 128 codes

// Rows first .. end - 1 of expert e0 + lane (a converged warp; `before`: where the
// experts before e0 end, carried from one call to the next).  Whatever offsets holds,
// they are inside 0 .. rows and no row is two experts'.
__device__ __forceinline__ int2 expert_rows(const Params &p, int e0, int lane, int &before) {
    if (!p.offsets) return make_int2(0, lane == 0 ? p.rows : 0);
    const int e = e0 + lane;
    int first = 0, end = 0;
    if (e < p.experts) {
        first = min(max(__ldcg(p.offsets + e), 0), p.rows);
        end = min(max(__ldcg(p.offsets + e + 1), first), p.rows);
    }
    int most = end;   // of the experts up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, most, o);
        if (lane >= o) most = max(most, v);
    }
    most = max(most, before);
    const int ahead = __shfl_up_sync(0xffffffffu, most, 1);
    first = max(first, lane ? ahead : before);
    before = __shfl_sync(0xffffffffu, most, 31);
    return make_int2(first, max(first, end));
}

// Instruction descriptor, kind::f8f6f4: e4m3 operands, K-major, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 2^x and 1 / x, approximate (2 and 1 ulp), subnormal results as 0
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// silu(gate) * up = gate / (1 + 2^(-gate log2 e)) * up, within (5 + |gate|) 2^-23 of
// the value (the exponent is off by an ulp of itself), 2.5e-6 where silu is not
// vanishing, |gate| < 16, next to half a step of e4m3, 6e-2; 0 below gate = -87.3
// (a denominator beyond 2^126), where |silu| is 1e-36 and less.  (With the forms
// that keep subnormals, whose fix-ups are as many instructions again, gate/up of
// 4096 tokens 4096 -> 11008 took 279 us instead of 274.)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float swiglu(float gate, float up) {
    return gate * rcp_approx(1.0f + exp2_approx(gate * -kLog2e)) * up;
}

}  // namespace e4

// x codes [rows x in], w codes [experts x out x in]; p but nf, nkb, err filled in
cudaError_t launch_e4m3_product(e4::Mode mode, const uint8_t *x, const uint8_t *w0, const uint8_t *w1, int64_t in,
                                e4::Params p, cudaStream_t s);
// wide: tiles of 128 rows (linear only), else 32
cudaError_t launch_e4m3_stream(e4::Mode mode, bool wide, int splits, const uint8_t *x, const uint8_t *w0,
                               const uint8_t *w1, int64_t in, const e4::Params &p, cudaStream_t s);
// narrow: units of 128 features (linear only), else 256 (gate/up: 128 of both)
cudaError_t launch_e4m3_pair(e4::Mode mode, bool narrow, const uint8_t *x, const uint8_t *w0, const uint8_t *w1,
                             int64_t in, const e4::Params &p, cudaStream_t s);

cudaError_t launch_quantize_e4m3(const void *x, uint8_t *q, float *scales, int64_t batch, int64_t rows, int64_t d,
                                 int64_t group, bool blocks, bool transpose, int dt, cudaStream_t s);

}  // namespace ffn
