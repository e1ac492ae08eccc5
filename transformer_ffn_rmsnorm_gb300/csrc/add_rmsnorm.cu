// add_rmsnorm.cu -- r = x + res, then the RMSNorm of r, in one pass:
//
//   r[t,c] = round(x[t,c] + res[t,c])                      (fp32 sum, one rounding)
//   v[t,c] = r[t,c] * rsqrt(mean_c(r[t,c]^2) + eps) * g[c]
//   n[t,c] = round(v[t,c])                                 or, in 8 bits,
//   a = max(max |v| over the row or group, 2^-100),  scale = a / 448,
//   q[t,c] = e4m3(v[t,c] * (448 / a))
//
// Bound by HBM: x and res are read once, r and n (or q and the scales)
// written once.  A CTA takes one row and holds it in registers as 16-byte
// vectors (r already rounded, so that the norm is the norm of what is
// stored); sum of squares and, for a scale per row, max |r g| go through one
// barrier together -- rsqrt(...) > 0 scales that maximum exactly as it scales
// v, so no second reduction is needed.  A group of 32, 64 or 128 columns is
// 4 to 32 neighbouring lanes and its maximum a few shuffles.
//
// NaN and infinities: the maxima are taken over the bit patterns of |v| as
// unsigned integers, where NaN is largest, so a NaN reaches the scale (and
// q); a row with an infinity has v = NaN there and 0 elsewhere, as the
// formula says.
#include "ffn_internal.cuh"

namespace ffn {
namespace {

constexpr float kE4m3Max = 448.f;
// A row whose squares pass fp32's range is summed again times 2^-96 (fp32 and
// bf16 values reach 3e38): exact, and far above where squares vanish.
constexpr float kDown = 1.2621774483536189e-29f;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max(a, 2^-100) with NaN kept (both are bit patterns of non-negative floats)
__device__ __forceinline__ float floor_amax(float a) {
    const uint32_t b = __float_as_uint(a), lo = __float_as_uint(7.888609052210118e-31f);
    return __uint_as_float(b > lo ? b : lo);
}

// two values to e4m3 (lo in the low byte), nearest even, finite values clamped to +-448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

enum Out { OUT_N = 0, OUT_ROW = 1, OUT_GROUP = 2 };

struct AddNormParams {
    const void *x, *res, *g;   // res may be null (r = x)
    void *r, *out;             // r may be null (not stored)
    float *scales;
    int64_t rows;
    int d, group, ngroups;     // group: columns per scale
    float eps;
};

// One row per CTA; thread t holds vectors t, t + blockDim.x, ... (VPT of them).
template <typename T, int VPT, int OUT>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const AddNormParams p) {
    constexpr int EPV = 16 / sizeof(T);
    constexpr bool KEEP_G = VPT <= 2;   // g in registers beside the row, or read again (longer rows)
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const int nvec = p.d / EPV;
    const uint4 *xr = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) + row * p.d);
    const uint4 *er = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.res) + row * p.d);
    uint4 *rr = p.r ? reinterpret_cast<uint4 *>(static_cast<T *>(p.r) + row * p.d) : nullptr;
    const uint4 *gv = reinterpret_cast<const uint4 *>(p.g);

    uint4 v[VPT], e[VPT], gr[KEEP_G ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int vi = i * blockDim.x + threadIdx.x;
        const bool in = vi < nvec;
        v[i] = in ? __ldcs(xr + vi) : make_uint4(0, 0, 0, 0);
        e[i] = in && p.res ? __ldcs(er + vi) : make_uint4(0, 0, 0, 0);
        if constexpr (KEEP_G) gr[i] = in ? __ldg(gv + vi) : make_uint4(0, 0, 0, 0);
    }
    auto g_of = [&](int i, float (&w)[EPV]) {
        if constexpr (KEEP_G) {
            Vec16<T>::unpack(gr[i], w);
        } else {
            const int vi = i * blockDim.x + threadIdx.x;
            Vec16<T>::unpack(vi < nvec ? __ldg(gv + vi) : make_uint4(0, 0, 0, 0), w);
        }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int vi = i * blockDim.x + threadIdx.x;
        if (p.res) {
            float f[EPV], a[EPV];
            Vec16<T>::unpack(v[i], f);
            Vec16<T>::unpack(e[i], a);
#pragma unroll
            for (int j = 0; j < EPV; ++j) f[j] += a[j];
            v[i] = Vec16<T>::pack(f);
        }
        if (rr && vi < nvec) __stcs(rr + vi, v[i]);
    }
    float ss, scale = 1.f;
    uint32_t mx;
    while (true) {
        ss = 0.f;
        mx = 0u;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float f[EPV];
            Vec16<T>::unpack(v[i], f);
#pragma unroll
            for (int j = 0; j < EPV; ++j) {
                f[j] *= scale;
                ss = fmaf(f[j], f[j], ss);
            }
            if constexpr (OUT == OUT_ROW) {
                float w[EPV];
                g_of(i, w);
#pragma unroll
                for (int j = 0; j < EPV; ++j) mx = max(mx, abs_bits(f[j] * w[j]));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (OUT == OUT_ROW) mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) {
            s_sum[warp] = ss;
            s_max[warp] = mx;
        }
        __syncthreads();
        ss = lane < nwarps ? s_sum[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (OUT == OUT_ROW) mx = __reduce_max_sync(0xffffffffu, lane < nwarps ? s_max[lane] : 0u);
        if (ss != INFINITY || scale != 1.f) break;   // the same in every thread
        scale = kDown;
        __syncthreads();
    }
    const float inv = rsqrtf(ss / static_cast<float>(p.d) + p.eps * scale * scale);

    if constexpr (OUT == OUT_N) {
        uint4 *nr = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * p.d);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vi = i * blockDim.x + threadIdx.x;
            float f[EPV], w[EPV];
            Vec16<T>::unpack(v[i], f);
            g_of(i, w);
#pragma unroll
            for (int j = 0; j < EPV; ++j) f[j] = f[j] * scale * inv * w[j];   // the order of ffn_rmsnorm
            if (vi < nvec) __stcs(nr + vi, Vec16<T>::pack(f));
        }
    } else {
        float k = 0.f;   // 448 / a
        if constexpr (OUT == OUT_ROW) {
            const float a = floor_amax(__uint_as_float(mx) * inv);
            k = kE4m3Max / a;
            if (threadIdx.x == 0) p.scales[row] = a / kE4m3Max;
        }
        uint8_t *qr = static_cast<uint8_t *>(p.out) + row * p.d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vi = i * blockDim.x + threadIdx.x;
            float f[EPV], w[EPV];
            Vec16<T>::unpack(v[i], f);
            g_of(i, w);
#pragma unroll
            for (int j = 0; j < EPV; ++j) f[j] = f[j] * scale * w[j] * inv;
            if constexpr (OUT == OUT_GROUP) {
                uint32_t m = 0u;
#pragma unroll
                for (int j = 0; j < EPV; ++j) m = max(m, abs_bits(f[j]));
                const int lanes = p.group / EPV;   // 4 to 32, a power of two
                for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float a = floor_amax(__uint_as_float(m));
                k = kE4m3Max / a;
                if (vi < nvec && (lane & (lanes - 1)) == 0) p.scales[row * p.ngroups + vi / lanes] = a / kE4m3Max;
            }
            uint32_t q[EPV / 4];
#pragma unroll
            for (int j = 0; j < EPV / 4; ++j)
                q[j] = e4m3x2(f[4 * j] * k, f[4 * j + 1] * k) | (e4m3x2(f[4 * j + 2] * k, f[4 * j + 3] * k) << 16);
            if (vi < nvec) {
                if constexpr (EPV == 8) __stcs(reinterpret_cast<uint2 *>(qr) + vi, make_uint2(q[0], q[1]));
                else __stcs(reinterpret_cast<uint32_t *>(qr) + vi, q[0]);
            }
        }
    }
}

// Rows that are not whole 16-byte vectors, or longer than a CTA's registers
// hold: one CTA per row, an element at a time, the row read again in each
// pass (r is recomputed from x and res where it is not stored; every element
// is read and written by one thread, so r may take x's or res's place).
template <typename T, int OUT>
__global__ void __launch_bounds__(256) add_rmsnorm_generic_kernel(const AddNormParams p) {
    __shared__ float s_sum[8];
    __shared__ uint32_t s_max[8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x, base = row * p.d;
    const T *x = static_cast<const T *>(p.x) + base;
    const T *res = p.res ? static_cast<const T *>(p.res) + base : nullptr;
    const T *g = static_cast<const T *>(p.g);
    T *r = p.r ? static_cast<T *>(p.r) + base : nullptr;
    auto sum_of = [&](int c) {
        return res ? to_f32(from_f32<T>(to_f32(x[c]) + to_f32(res[c]))) : to_f32(x[c]);
    };
    auto stored = [&](int c) { return r ? to_f32(r[c]) : sum_of(c); };
    if (r) {
        for (int c = threadIdx.x; c < p.d; c += blockDim.x) r[c] = from_f32<T>(sum_of(c));
        __syncthreads();   // r is read below by other threads
    }
    float ss, scale = 1.f;
    uint32_t mx;
    while (true) {
        ss = 0.f;
        mx = 0u;
        for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
            const float f = stored(c) * scale;
            ss = fmaf(f, f, ss);
            if (OUT == OUT_ROW) mx = max(mx, abs_bits(f * to_f32(g[c])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) {
            s_sum[warp] = ss;
            s_max[warp] = mx;
        }
        __syncthreads();
        ss = 0.f;
        mx = 0u;
        for (int w = 0; w < 8; ++w) {
            ss += s_sum[w];
            mx = max(mx, s_max[w]);
        }
        __syncthreads();
        if (ss != INFINITY || scale != 1.f) break;
        scale = kDown;
    }
    const float inv = rsqrtf(ss / static_cast<float>(p.d) + p.eps * scale * scale);
    if (OUT == OUT_N) {
        T *n = static_cast<T *>(p.out) + base;
        for (int c = threadIdx.x; c < p.d; c += blockDim.x) n[c] = from_f32<T>(stored(c) * scale * inv * to_f32(g[c]));
        return;
    }
    uint8_t *q = static_cast<uint8_t *>(p.out) + base;
    if (OUT == OUT_ROW) {
        const float a = floor_amax(__uint_as_float(mx) * inv), k = kE4m3Max / a;
        if (threadIdx.x == 0) p.scales[row] = a / kE4m3Max;
        for (int c = threadIdx.x; c < p.d; c += blockDim.x)
            q[c] = static_cast<uint8_t>(e4m3x2(stored(c) * scale * to_f32(g[c]) * inv * k, 0.f) & 0xffu);
        return;
    }
    // a warp per group; the values a thread reads here another thread stored
    // (r is read after the barrier), the group's lanes stay together
    for (int gi = warp; gi < p.ngroups; gi += 8) {
        const int c0 = gi * p.group, c1 = min(p.d, c0 + p.group);
        uint32_t m = 0u;
        for (int c = c0 + lane; c < c1; c += 32) m = max(m, abs_bits(stored(c) * scale * to_f32(g[c]) * inv));
        m = __reduce_max_sync(0xffffffffu, m);
        const float a = floor_amax(__uint_as_float(m)), k = kE4m3Max / a;
        if (lane == 0) p.scales[row * p.ngroups + gi] = a / kE4m3Max;
        for (int c = c0 + lane; c < c1; c += 32)
            q[c] = static_cast<uint8_t>(e4m3x2(stored(c) * scale * to_f32(g[c]) * inv * k, 0.f) & 0xffu);
    }
}

template <typename T, int OUT>
cudaError_t launch_out(const AddNormParams &p, cudaStream_t s) {
    constexpr int EPV = 16 / sizeof(T);
    LaunchScope scope(K_ADD_RMSNORM, s);
    const dim3 grid(static_cast<unsigned>(p.rows));
    const int nvec = p.d / EPV;
    cudaError_t e;
    if (p.d % EPV || nvec > 4 * 1024) {
        e = launch_dependent(add_rmsnorm_generic_kernel<T, OUT>, grid, dim3(256), 0, s, p);
    } else {
        // few rows: as many threads as the row has vectors (shortest path to
        // the answer); many rows: four vectors a thread, which keeps most bytes in
        // flight for a CTA's barrier (16384 x 4096 fp16 to e4m3: one vector
        // 106, two 73, four 69 us; copy speed is 69).  At 64 registers a
        // thread: with g kept as well (128) four were slower than two.
        // Measured at 4096 columns; rows of 256 make CTAs of one warp.
        int vpt = p.rows <= 2 * static_cast<int64_t>(sm_count()) ? 1 : 4;
        while (nvec > vpt * 1024) vpt <<= 1;
        const dim3 block(static_cast<unsigned>(((nvec + vpt - 1) / vpt + 31) / 32 * 32));
        switch (vpt) {
            case 1: e = launch_dependent(add_rmsnorm_kernel<T, 1, OUT>, grid, block, 0, s, p); break;
            case 2: e = launch_dependent(add_rmsnorm_kernel<T, 2, OUT>, grid, block, 0, s, p); break;
            default: e = launch_dependent(add_rmsnorm_kernel<T, 4, OUT>, grid, block, 0, s, p); break;
        }
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const AddNormParams &p, bool quant, cudaStream_t s) {
    if (!quant) return launch_out<T, OUT_N>(p, s);
    return p.ngroups == 1 && p.group >= p.d ? launch_out<T, OUT_ROW>(p, s) : launch_out<T, OUT_GROUP>(p, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void *x, const void *res, const void *g, void *r, void *out, float *scales,
                               int64_t rows, int64_t d, int64_t group, float eps, int dt, bool quant,
                               cudaStream_t s) {
    AddNormParams p{};
    p.x = x;
    p.res = res;
    p.g = g;
    p.r = r;
    p.out = out;
    p.scales = scales;
    p.rows = rows;
    p.d = static_cast<int>(d);
    p.group = static_cast<int>(group ? group : d);
    p.ngroups = (p.d + p.group - 1) / p.group;
    p.eps = eps;
    switch (dt) {
        case DT_F32: return launch_typed<float>(p, quant, s);
        case DT_F16: return launch_typed<__half>(p, quant, s);
        default: return launch_typed<__nv_bfloat16>(p, quant, s);
    }
}

}  // namespace ffn
