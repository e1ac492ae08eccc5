// quantize.cu -- a matrix to e4m3 codes and fp32 scales:
//
//   a = max(max |x| over the block, 2^-100),  scale = a / 448,  q = e4m3(x * (448 / a))
//
// with a block of 32, 64 or 128 columns of one row (activations, gradients:
// what a product reads along its reduction) or of 128 x 128 (weights).  The
// codes of 128 x 128 blocks may be written transposed, with their scales: the
// operand of dX = dY W, whose blocks are the same ones.
//
// Bound by HBM: x is read once and held in registers between its maximum and its
// codes.  A row's block is 2 to 16 neighbouring lanes with two 16-byte vectors each,
// its maximum a few shuffles, and a thread has four vectors in flight.  A 128 x 128
// block is one CTA's.
#include "e4m3.cuh"

namespace ffn {
namespace {

struct QuantParams {
    const void *x;
    uint8_t *q;
    float *scales;
    int64_t rows, total;   // total: pairs of vectors, each row filled up to whole groups
    int d, group, ngroups;
};

// The largest magnitude of a vector (max_of), or of several (max of those), as bits
// that order magnitudes: a 16-bit type's own, two at a time, widened only at the end.
template <typename T> struct Magnitude {
    __device__ static __forceinline__ uint32_t max_of(const uint4 &v) {
        const uint32_t k = 0x7fff7fffu, m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
        return max(m >> 16, m & 0xffffu);
    }
    __device__ static __forceinline__ float value(uint32_t bits) {
        const unsigned short b = static_cast<unsigned short>(bits);
        return to_f32(*reinterpret_cast<const T *>(&b));
    }
};
template <> struct Magnitude<float> {
    __device__ static __forceinline__ uint32_t max_of(const uint4 &v) {
        const uint32_t k = 0x7fffffffu;
        return max(max(v.x & k, v.y & k), max(v.z & k, v.w & k));
    }
    __device__ static __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }
};

template <int EPV> __device__ __forceinline__ void store_codes(uint8_t *to, const float (&f)[EPV], float k) {
    if constexpr (EPV == 8)
        __stcs(reinterpret_cast<uint2 *>(to), make_uint2(e4m3x4(f[0] * k, f[1] * k, f[2] * k, f[3] * k),
                                                         e4m3x4(f[4] * k, f[5] * k, f[6] * k, f[7] * k)));
    else
        __stcs(reinterpret_cast<uint32_t *>(to), e4m3x4(f[0] * k, f[1] * k, f[2] * k, f[3] * k));
}

constexpr int kRowThreads = 256, kRowPairs = 2;

// Rows of whole vectors, a thread two in a row at a time (one at a time, the divisions and
// shuffles for a block kept the schedulers busy 70 % of the time).  FLAT: rows of whole
// groups too, so that the matrix is one run of groups; else a row's pairs of vectors are
// counted up to whole groups.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const QuantParams p) {
    constexpr int EPV = 16 / sizeof(T);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, lanes = p.group / (2 * EPV);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kRowThreads * kRowPairs) + threadIdx.x;
    const int per_row = p.ngroups * lanes;
    uint4 v[kRowPairs][2];
    int64_t at[kRowPairs];   // first element
    int have[kRowPairs];     // vectors of the pair that are the row's
#pragma unroll
    for (int b = 0; b < kRowPairs; ++b) {
        const int64_t i = i0 + b * kRowThreads;
        if (FLAT) {
            at[b] = i * (2 * EPV);
            have[b] = i < p.total ? 2 : 0;
        } else {
            const int64_t row = i / per_row;
            const int c = static_cast<int>(i - row * per_row) * (2 * EPV);
            at[b] = row * p.d + c;
            have[b] = i < p.total ? min(max((p.d - c) / EPV, 0), 2) : 0;
        }
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) + at[b]);
#pragma unroll
        for (int j = 0; j < 2; ++j) v[b][j] = j < have[b] ? __ldcs(x + j) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < kRowPairs; ++b) {
        uint32_t m = max(Magnitude<T>::max_of(v[b][0]), Magnitude<T>::max_of(v[b][1]));
        for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float a = floor_amax(Magnitude<T>::value(m)), k = kE4m3Max / a;
        const int64_t i = i0 + b * kRowThreads;
        if (i < p.total && (lane & (lanes - 1)) == 0) p.scales[i / lanes] = a / kE4m3Max;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float f[EPV];
            Vec16<T>::unpack(v[b][j], f);
            if (j < have[b]) store_codes<EPV>(p.q + at[b] + j * EPV, f, k);
        }
    }
}

// Any row length: a warp per group, an element at a time.
template <typename T>
__global__ void __launch_bounds__(256) quantize_any_kernel(const QuantParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (g >= p.rows * p.ngroups) return;
    const int64_t row = g / p.ngroups;
    const int c0 = static_cast<int>(g - row * p.ngroups) * p.group, n = min(p.group, p.d - c0);
    const T *x = static_cast<const T *>(p.x) + row * p.d + c0;
    float f[4];
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = lane + 32 * j < n ? to_f32(x[lane + 32 * j]) : 0.f;
        m = max(m, abs_bits(f[j]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const float a = floor_amax(__uint_as_float(m)), k = kE4m3Max / a;
    if (lane == 0) p.scales[g] = a / kE4m3Max;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < n) p.q[row * p.d + c0 + lane + 32 * j] = static_cast<uint8_t>(e4m3x2(f[j] * k, 0.f));
}

// A 128 x 128 block of one matrix of a batch; d a multiple of 16 (and rows,
// where the codes are transposed).  The transposed block goes through shared
// memory by bytes; its pitch of 129 spreads a warp's 16 columns over the banks.
constexpr int kBlockThreads = 256, kPitch = 129;

template <typename T, bool TRANSPOSE>
__global__ void __launch_bounds__(kBlockThreads) quantize_blocks_kernel(const QuantParams p) {
    constexpr int EPV = 16 / sizeof(T), VPR = kE4m3Block / EPV, STEP = kBlockThreads / VPR, N = kE4m3Block / STEP;
    __shared__ uint32_t s_max[kBlockThreads / 32];
    __shared__ uint8_t s_code[TRANSPOSE ? kE4m3Block * kPitch : 1];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t nbr = (p.rows + kE4m3Block - 1) / kE4m3Block, mat = blockIdx.x / (nbr * p.ngroups);
    const int64_t in_mat = blockIdx.x - mat * nbr * p.ngroups, br = in_mat / p.ngroups;
    const int bc = static_cast<int>(in_mat - br * p.ngroups);
    const int64_t r0 = br * kE4m3Block, base = mat * p.rows * p.d;
    const int c0 = bc * kE4m3Block, col = threadIdx.x % VPR * EPV, row = threadIdx.x / VPR;
    const int nr = static_cast<int>(min(static_cast<int64_t>(kE4m3Block), p.rows - r0)),
              nc = min(kE4m3Block, p.d - c0);
    const T *x = static_cast<const T *>(p.x) + base + r0 * p.d + c0;
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = row + i * STEP;
        v[i] = r < nr && col < nc ? __ldcs(reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(r) * p.d + col))
                                  : make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, Magnitude<T>::max_of(v[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBlockThreads / 32; ++w) m = max(m, s_max[w]);
    const float a = floor_amax(Magnitude<T>::value(m)), k = kE4m3Max / a;
    if (threadIdx.x == 0)
        p.scales[mat * nbr * p.ngroups + (TRANSPOSE ? bc * nbr + br : in_mat)] = a / kE4m3Max;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = row + i * STEP;
        float f[EPV];
        Vec16<T>::unpack(v[i], f);
        if constexpr (TRANSPOSE) {
#pragma unroll
            for (int j = 0; j < EPV; j += 2) {
                const uint32_t two = e4m3x2(f[j] * k, f[j + 1] * k);
                s_code[(col + j) * kPitch + r] = static_cast<uint8_t>(two & 0xffu);
                s_code[(col + j + 1) * kPitch + r] = static_cast<uint8_t>(two >> 8);
            }
        } else if (r < nr && col < nc) {
            store_codes<EPV>(p.q + base + (r0 + r) * p.d + c0 + col, f, k);
        }
    }
    if constexpr (TRANSPOSE) {
        __syncthreads();
        // 16 codes a thread; eight neighbouring threads write a row of 128
        for (int i = threadIdx.x; i < kE4m3Block * 8; i += kBlockThreads) {
            const int c = i >> 3, r = (i & 7) * 16;
            if (c >= nc || r >= nr) continue;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t *s = s_code + c * kPitch + r + 4 * j;
                w[j] = s[0] | (s[1] << 8) | (s[2] << 16) | (static_cast<uint32_t>(s[3]) << 24);
            }
            __stcs(reinterpret_cast<uint4 *>(p.q + base + (c0 + c) * p.rows + r0 + r),
                   make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

template <typename T>
cudaError_t launch_typed(QuantParams p, int64_t batch, bool blocks, bool transpose, cudaStream_t s) {
    constexpr int EPV = 16 / sizeof(T);
    LaunchScope scope(K_QUANTIZE, s);
    cudaError_t e;
    if (blocks) {
        const dim3 grid(static_cast<unsigned>(batch * ((p.rows + kE4m3Block - 1) / kE4m3Block) * p.ngroups));
        e = transpose ? launch_dependent(quantize_blocks_kernel<T, true>, grid, dim3(kBlockThreads), 0, s, p)
                      : launch_dependent(quantize_blocks_kernel<T, false>, grid, dim3(kBlockThreads), 0, s, p);
    } else if (p.d % EPV) {
        const dim3 grid(static_cast<unsigned>((p.rows * p.ngroups + 7) / 8));
        e = launch_dependent(quantize_any_kernel<T>, grid, dim3(256), 0, s, p);
    } else {
        p.total = p.rows * p.ngroups * (p.group / (2 * EPV));
        const dim3 grid(static_cast<unsigned>((p.total + kRowThreads * kRowPairs - 1) / (kRowThreads * kRowPairs)));
        e = p.d % p.group == 0
                ? launch_dependent(quantize_rows_kernel<T, true>, grid, dim3(kRowThreads), 0, s, p)
                : launch_dependent(quantize_rows_kernel<T, false>, grid, dim3(kRowThreads), 0, s, p);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_e4m3(const void *x, uint8_t *q, float *scales, int64_t batch, int64_t rows, int64_t d,
                                 int64_t group, bool blocks, bool transpose, int dt, cudaStream_t s) {
    QuantParams p{};
    p.x = x;
    p.q = q;
    p.scales = scales;
    p.rows = blocks ? rows : batch * rows;
    p.d = static_cast<int>(d);
    p.group = static_cast<int>(group);
    p.ngroups = static_cast<int>((d + group - 1) / group);
    switch (dt) {
        case DT_F32: return launch_typed<float>(p, batch, blocks, transpose, s);
        case DT_F16: return launch_typed<__half>(p, batch, blocks, transpose, s);
        default: return launch_typed<__nv_bfloat16>(p, batch, blocks, transpose, s);
    }
}

}  // namespace ffn
