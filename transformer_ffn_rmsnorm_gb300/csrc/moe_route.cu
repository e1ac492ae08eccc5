// moe_route.cu -- each token's experts and their weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),   order_e = s_e + b_e, or l_e without a bias
//   groups: a group's score is the sum of its two largest s_e + b_e; the
//           topk_groups groups of the largest score stay
//   idx = the k largest order_e, descending;  w_j = s_(idx_j) [/ sum_j] * scale
// Ties go to the lower index.  A logit of -inf or NaN is never chosen.
//
// One warp per token: lane l holds experts l, l + 32, ... in registers,
// sorted (up to 8 of them; more are scanned each time), and the k largest
// come out one by one: a warp maximum over the lanes' largest, a warp minimum
// over the indices that have it.  Bound by issue and, in a single wave, by the
// latency of one token's reductions: 630 warp instructions a token at 16384 x
// 128 bf16, 8 of them (issue 67 % active, 38 % of the warps), 1886 at 4097 x 256
// with groups and a bias (55 %, 35 %); HBM and L2 are below 6 %.
//
// The chosen set is that of the formula in 64 bits although the scores are
// computed in 32.  Without a bias nothing has to be computed: the order is
// the order of the logits.  With one, a 32-bit order is within DELTA + 2^-24
// |order| of the exact one, so a maximum that no other candidate approaches
// within twice that is the exact maximum; only where one does are the
// candidates computed in 64 bits and compared again.  (FP64 runs at a small
// fraction of the FP32 rate on this GPU: a 64-bit exponential for every
// score would be most of the kernel.)  Groups are decided the same way.
//   DELTA, in units of 2^-24 of s <= 1 (the approximate division is within 2
//   ulp, 4 units): sigmoid: expf 2, its sum with 1 one, the division 4: 7,
//   taken as 8.  softmax: l - max rounds by |l - max| 2^-24, which moves
//   exp(l - max) by at most 1 (x e^-x < 1), expf 2; the denominator adds terms
//   with those errors over at most 10 levels (a lane's 32 in pairs, then 32
//   lanes): 13; the division 4: 20, taken as 32.
#include "ffn_internal.cuh"

namespace ffn {
namespace {

constexpr int kRouteWarps = 4;
constexpr float kDeltaSoftmax = 1.0f / (1 << 19);
constexpr float kDeltaSigmoid = 1.0f / (1 << 21);
constexpr float kDeltaRel = 1.0f / (1 << 23);

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *w;
    int64_t rows;
    int experts, k, groups, topk_groups;
    float scale;
    bool sigmoid, renorm;
};

// a float's bits as an unsigned integer of the same order
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(0xffffffffu, ordered(v))); }

// NaN counts as -inf (never chosen), +inf as the largest finite value
__device__ __forceinline__ float clean_logit(float l) {
    // (fmaxf gives the other operand for NaN; + 0 makes -0 the equal +0 for ordered())
    return fminf(fmaxf(l, -INFINITY), 3.402823466e38f) + 0.f;
}
__device__ __forceinline__ float clean_bias(float b) { return fminf(fmaxf(b, -1e30f), 1e30f); }

// a token's scores in 64 bits
struct Exact {
    bool sigmoid;
    double top, sum;
    __device__ double score(float l) const {
        return sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : exp(static_cast<double>(l) - top) / sum;
    }
};

// the two largest of two pairs (a >= b in each)
template <typename R> __device__ __forceinline__ void merge_two(R &a, R &b, R c, R d) {
    if (c > a) {
        b = a > d ? a : d;
        a = c;
    } else if (c > b) {
        b = c;
    }
}

// Sum of the two largest values of each group (one if it has one, -inf if
// none), the score of group g in lane g.  value(e) is expert e's; sub lanes
// (a power of two) share a group's entries.
template <typename R, typename V>
__device__ __forceinline__ R group_scores(int groups, int per, int lane, V value) {
    const R none = static_cast<R>(-INFINITY);
    int sub = 1;
    while (2 * sub * groups <= 32) sub <<= 1;
    const int g = lane / sub;
    R a = none, b = none;
    if (g < groups)
        for (int j = lane % sub; j < per; j += sub) {
            const R v = value(g * per + j);
            if (v > a) {
                b = a;
                a = v;
            } else if (v > b) {
                b = v;
            }
        }
    for (int o = 1; o < sub; o <<= 1) {
        const R c = __shfl_xor_sync(0xffffffffu, a, o), d = __shfl_xor_sync(0xffffffffu, b, o);
        merge_two(a, b, c, d);
    }
    const R sum = a == none ? none : (b == none ? a : a + b);
    const R mine = __shfl_sync(0xffffffffu, sum, lane * sub < 32 ? lane * sub : 0);
    return lane < groups ? mine : none;
}

// The mask of the `keep` groups of the largest score, group g's in lane g
// (ties to the lower index; never a group without an eligible expert).
template <typename R>
__device__ __forceinline__ uint32_t keep_groups(R score, int groups, int keep, int lane) {
    const R none = static_cast<R>(-INFINITY);
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const R other = __shfl_sync(0xffffffffu, score, g);
        rank += other > score || (other == score && g < lane);
    }
    return __ballot_sync(0xffffffffu, lane < groups && score > none && rank < keep);
}

// (72 registers up to 256 experts: 28 warps an SM, 4097 x 256 in one wave; 96
// registers 17.9, 72 15.9, 64 16.6 us with the launch)
template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kRouteWarps, EPL <= 8 ? 7 : 4) moe_route_kernel(const RouteParams p) {
    extern __shared__ float s_scores[];   // [kRouteWarps][experts], with groups only
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (row >= p.rows) return;
    const T *lrow = static_cast<const T *>(p.logits) + row * p.experts;
    const int E = p.experts;

    float l[EPL];   // logits; then the order, -inf once chosen or not eligible
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < E ? clean_logit(to_f32(lrow[e])) : -INFINITY;
        top = fmaxf(top, l[i]);
    }
    top = warp_max(top);
    const bool grouped = p.groups > 1, scored = p.bias != nullptr || grouped;
    // softmax denominator: not needed where the weights are renormalised over
    // the chosen (the largest of them is then at least 1/E of the whole)
    float denom = 1.f;
    const bool need_sum = !p.sigmoid && (scored || !p.renorm);
    if (need_sum && top > -INFINITY) {
        float t[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) t[i] = expf(l[i] - top);
        // in pairs, so that no sum is deeper than five additions
#pragma unroll
        for (int i = 0; i < EPL / 2; ++i) t[i] += t[i + EPL / 2];
        if constexpr (EPL >= 4) {
#pragma unroll
            for (int i = 0; i < EPL / 4; ++i) t[i] += t[i + EPL / 4];
        }
        if constexpr (EPL >= 8) {
#pragma unroll
            for (int i = 0; i < EPL / 8; ++i) t[i] += t[i + EPL / 8];
        }
        if constexpr (EPL >= 16) {
#pragma unroll
            for (int i = 0; i < EPL / 16; ++i) t[i] += t[i + EPL / 16];
        }
        if constexpr (EPL >= 32) {
#pragma unroll
            for (int i = 0; i < EPL / 32; ++i) t[i] += t[i + EPL / 32];
        }
        denom = t[0];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, o);
    }
    auto score32 = [&](float z) {
        return p.sigmoid ? __fdividef(1.f, 1.f + expf(-z)) : __fdividef(expf(z - top), denom);
    };
    auto bias_of = [&](int e) { return p.bias ? clean_bias(__ldg(p.bias + e)) : 0.f; };

    Exact ex;
    ex.sigmoid = p.sigmoid;
    ex.top = static_cast<double>(top);
    ex.sum = 0.0;
    auto prepare_exact = [&]() {   // the denominator in 64 bits, once, if anything is close
        if (p.sigmoid || ex.sum > 0.0) return;
        double t = 0.0;
        for (int e = lane; e < E; e += 32) t += exp(static_cast<double>(clean_logit(to_f32(lrow[e]))) - ex.top);
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        ex.sum = t;
    };
    auto exact_order = [&](int e) {
        return ex.score(clean_logit(to_f32(lrow[e]))) + static_cast<double>(bias_of(e));
    };

    const float delta = p.sigmoid ? kDeltaSigmoid : kDeltaSoftmax;
    if (scored && top > -INFINITY) {
        float most = 0.f;   // largest |order|
        float *sc = s_scores + static_cast<size_t>(warp) * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            if (e < E) {
                const float o = l[i] > -INFINITY ? score32(l[i]) + bias_of(e) : -INFINITY;
                if (grouped) sc[e] = o;
                if (o > -INFINITY) most = fmaxf(most, fabsf(o));
                if (p.bias) l[i] = o;   // the order; without a bias the logits keep it exactly
            }
        }
        if (grouped) {
            __syncwarp();
            const int per = E / p.groups;
            const float inv_per = 1.f / static_cast<float>(per);
            auto approx = [&](int e) -> float { return sc[e]; };
            auto exact = [&](int e) -> double {
                if (!(sc[e] > -INFINITY)) return -INFINITY;
                return exact_order(e);
            };
            const float gs = group_scores<float>(p.groups, per, lane, approx);
            uint32_t kept = keep_groups<float>(gs, p.groups, p.topk_groups, lane);
            const bool mine = (kept >> lane) & 1u;
            const float lo = -warp_max(mine ? -gs : -INFINITY);                          // smallest kept
            const float hi = warp_max(!mine && lane < p.groups ? gs : -INFINITY);        // largest dropped
            // a score is a sum of two orders, and two scores are compared
            if (kept && hi > -INFINITY && lo - hi <= 4.f * (delta + kDeltaRel * (warp_max(most) + fabsf(lo)))) {
                prepare_exact();
                const double gd = group_scores<double>(p.groups, per, lane, exact);
                kept = keep_groups<double>(gd, p.groups, p.topk_groups, lane);
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * 32 + lane;
                // e / per: e + 1/2 is at least 1 / (2 per) from a multiple, far more than the product's rounding
                const int g = static_cast<int>((static_cast<float>(e) + 0.5f) * inv_per);
                if (e < E && !((kept >> g) & 1u)) l[i] = -INFINITY;
            }
        }
    }

    constexpr bool SORTED = EPL <= 8;
    constexpr uint32_t kDead = 0x007fffffu;   // ordered(-inf): chosen or not eligible
    uint32_t key[EPL];
    int id[EPL];   // register i holds expert id[i] * 32 + lane
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = ordered(l[i]);
        id[i] = i;
    }
    if constexpr (SORTED) {
        // largest first, the lower index first among equals (odd-even merge network)
        auto order_pair = [&](int x, int y) {
            const bool swap = key[y] > key[x] || (key[y] == key[x] && id[y] < id[x]);
            const uint32_t kx = key[x], ky = key[y];
            const int ix = id[x], iy = id[y];
            key[x] = swap ? ky : kx;
            key[y] = swap ? kx : ky;
            id[x] = swap ? iy : ix;
            id[y] = swap ? ix : iy;
        };
#pragma unroll
        for (int i = 0; i + 1 < EPL; i += 2) order_pair(i, i + 1);
        if constexpr (EPL >= 4) {
#pragma unroll
            for (int i = 0; i + 3 < EPL; i += 4) {
                order_pair(i, i + 2);
                order_pair(i + 1, i + 3);
                order_pair(i + 1, i + 2);
            }
        }
        if constexpr (EPL == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) order_pair(i, i + 4);
            order_pair(2, 4);
            order_pair(3, 5);
            order_pair(1, 2);
            order_pair(3, 4);
            order_pair(5, 6);
        }
    }
    int my_idx = -1;   // lane j keeps the j-th choice
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = key[0];
        int at = id[0];
        if constexpr (!SORTED) {
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
        }
        const uint32_t top_key = __reduce_max_sync(0xffffffffu, best);
        if (top_key <= kDead) break;   // nothing eligible is left
        unsigned pick =
            __reduce_min_sync(0xffffffffu, best == top_key ? static_cast<unsigned>(at * 32 + lane) : 0xffffffffu);
        if (p.bias) {
            const float m = unordered(top_key);
            const uint32_t near = ordered(m - 2.f * (delta + kDeltaRel * fabsf(m)));
            bool close;   // whether a second candidate is near the maximum
            if constexpr (SORTED) {
                const unsigned heads = __ballot_sync(0xffffffffu, key[0] >= near);
                close = (heads & (heads - 1u)) != 0u || __any_sync(0xffffffffu, key[1] >= near);
            } else {
                unsigned n = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) n += key[i] >= near;
                close = __reduce_add_sync(0xffffffffu, n) > 1u;
            }
            if (close) {
                prepare_exact();
                double bd = -INFINITY;
                unsigned be = 0xffffffffu;
                for (int i = 0; i < EPL; ++i) {
                    uint32_t v = kDead;
                    int vi = 0;
#pragma unroll
                    for (int q = 0; q < EPL; ++q)
                        if (q == i) {
                            v = key[q];
                            vi = id[q];
                        }
                    if (v >= near) {
                        const unsigned e = static_cast<unsigned>(vi * 32 + lane);
                        const double o = exact_order(static_cast<int>(e));
                        if (o > bd || (o == bd && e < be)) {
                            bd = o;
                            be = e;
                        }
                    }
                }
                for (int o = 16; o > 0; o >>= 1) {
                    const double od = __shfl_xor_sync(0xffffffffu, bd, o);
                    const unsigned oe = __shfl_xor_sync(0xffffffffu, be, o);
                    if (od > bd || (od == bd && oe < be)) {
                        bd = od;
                        be = oe;
                    }
                }
                pick = be;
            }
        }
        if (lane == j) my_idx = static_cast<int>(pick);
        if ((pick & 31u) == static_cast<unsigned>(lane)) {   // taken out of its lane
            const int gone = static_cast<int>(pick >> 5);
            if constexpr (SORTED) {
                bool after = false;
#pragma unroll
                for (int i = 0; i + 1 < EPL; ++i) {
                    after = after || id[i] == gone;
                    if (after) {
                        key[i] = key[i + 1];
                        id[i] = id[i + 1];
                    }
                }
                key[EPL - 1] = kDead;
                id[EPL - 1] = -1;
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i == gone) key[i] = kDead;
            }
        }
        __syncwarp();
    }

    float s = 0.f;
    if (my_idx >= 0) s = score32(clean_logit(to_f32(lrow[my_idx])));
    if (p.renorm) {
        float sum = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s = s / fmaxf(sum, 7.888609052210118e-31f);   // 2^-100
    }
    if (lane < p.k) {
        p.idx[row * p.k + lane] = my_idx;
        p.w[row * p.k + lane] = s * p.scale;
    }
}

template <typename T, int EPL>
cudaError_t launch_epl(const RouteParams &p, cudaStream_t s) {
    const size_t smem = p.groups > 1 ? static_cast<size_t>(kRouteWarps) * p.experts * sizeof(float) : 0;
    const int64_t blocks = (p.rows + kRouteWarps - 1) / kRouteWarps;
    LaunchScope scope(K_MOE_ROUTE, s);
    const cudaError_t e = launch_dependent(moe_route_kernel<T, EPL>, dim3(static_cast<unsigned>(blocks)),
                                           dim3(32 * kRouteWarps), smem, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const RouteParams &p, cudaStream_t s) {
    const int epl = (p.experts + 31) / 32;
    if (epl <= 2) return launch_epl<T, 2>(p, s);
    if (epl <= 4) return launch_epl<T, 4>(p, s);
    if (epl <= 8) return launch_epl<T, 8>(p, s);
    if (epl <= 16) return launch_epl<T, 16>(p, s);
    return launch_epl<T, 32>(p, s);
}

}  // namespace

cudaError_t launch_moe_route(const void *logits, const float *bias, int32_t *idx, float *w, int64_t rows, int experts,
                             int k, int groups, int topk_groups, float scale, bool sigmoid, bool renorm, int dt,
                             cudaStream_t s) {
    RouteParams p{logits, bias, idx, w, rows, experts, k, groups, topk_groups, scale, sigmoid, renorm};
    switch (dt) {
        case DT_F32: return launch_typed<float>(p, s);
        case DT_F16: return launch_typed<__half>(p, s);
        default: return launch_typed<__nv_bfloat16>(p, s);
    }
}

}  // namespace ffn
