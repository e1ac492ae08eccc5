// selftest.cu -- exercises the bounded wait every streaming kernel relies on,
// without a fault: one CTA in which a role waits on an mbarrier phase that
// nothing ever completes.  It gives up after the limit, records
// FFN_ERR_TIMEOUT in the device status word and raises the CTA's abort flag;
// a second role, waiting with a far longer limit on another such barrier, is
// released by that flag within about a millisecond (the suspend hint of the
// wait), exactly the path the GEMM and decode kernels take when a copy or a
// peer never arrives.  The kernel then returns normally: the context stays
// usable.
//
// And the end of a CTA pair after one of its CTAs has given up (pair_end.cuh): two
// producers that stop at different places, and nobody who takes what they load.
#include <algorithm>

#include "ffn_internal.cuh"
#include "pair_end.cuh"

namespace ffn {
namespace {

__global__ void __launch_bounds__(64) bounded_wait_probe_kernel(uint64_t limit_ns, unsigned *err) {
    __shared__ __align__(8) uint64_t bar_a, bar_b;
    __shared__ int s_abort;
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&bar_a), 1);
        ptx::mbar_init(ptx::smem_u32(&bar_b), 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    volatile int *abort_flag = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        // warp 0: gives up after limit_ns; warp 1: would wait 1000x longer
        const uint64_t limit = warp == 0 ? limit_ns : 1000 * limit_ns;
        const uint32_t bar = ptx::smem_u32(warp == 0 ? &bar_a : &bar_b);
        if (!ptx::mbar_wait(bar, 0, abort_flag, limit)) {
            atomicOr(err, DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }
    __syncthreads();
}

constexpr uint64_t kProbeWaitNs = 1000000000ull;

// Load number i of CTA r brings rows 32 (2 i + r) .. of src (rows of 128 bytes) to slot i %
// kPairProbeSlots.  Whole rounds that both CTAs load are waited for, as the MMAs would; what the
// last slots hold when the pair ends is compared with src, byte for byte, into wrong[r].
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(128)
    pair_end_probe_kernel(const __grid_constant__ CUtensorMap map, const uint8_t *src, int32_t *wrong, int even,
                          int odd, unsigned *err) {
    constexpr int kSlots = kPairProbeSlots;
    constexpr uint32_t kBytes = kPairProbeBytes;
    __shared__ __align__(128) uint8_t s_slot[kSlots][kBytes];
    __shared__ __align__(8) uint64_t bar_full[kSlots];
    __shared__ PairEnd s_end;
    __shared__ int s_abort, s_never;
    const uint32_t rank = ptx::cluster_ctarank();
    auto full = [&](int s) { return ptx::smem_u32(&bar_full[s]); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) ptx::mbar_init(full(s), 1);
        s_abort = 1;   // a role has given up
        s_never = 0;
        ptx::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kSlots * static_cast<int>(kBytes) / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(s_slot)[i] = 0xffffffffu;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (before the copies write there)
    __syncthreads();
    ptx::cluster_sync();
    const int loads = rank ? odd : even, rounds = min(even, odd) / kSlots;
    uint32_t produced = 0;
    for (int i0 = 0; i0 <= rounds * kSlots; i0 += kSlots) {
        if (threadIdx.x == 0)
            for (int i = i0; i < min(i0 + kSlots, loads); ++i, ++produced) {
                const int s = i - i0;
                if (rank == 0) ptx::mbar_arrive_expect_tx(full(s), 2 * kBytes);
                ptx::tma_load_2d_pair(ptx::smem_u32(s_slot[s]), &map, ptx::mapa_shared(full(s), 0), 0,
                                      32 * (2 * i + static_cast<int>(rank)));
            }
        __syncwarp();
        if (i0 == rounds * kSlots) break;
        if (rank == 0 && threadIdx.x == 0)
            for (int s = 0; s < kSlots; ++s)
                if (!ptx::mbar_wait(full(s), (i0 / kSlots) & 1u, &s_never, kProbeWaitNs)) atomicOr(err, DEVERR_TIMEOUT);
        __syncwarp();
        ptx::cluster_sync();
    }
    end_pair<kSlots>(s_end, rank, produced, &s_abort, &s_never, kProbeWaitNs, full, [](int, int) { return kBytes; });
    int bad = 0;
    for (int s = 0; s < kSlots && s < loads; ++s) {
        const int i = s + (loads - 1 - s) / kSlots * kSlots;   // the last load into the slot
        const uint8_t *from = src + static_cast<int64_t>(2 * i + static_cast<int>(rank)) * kBytes;
        for (uint32_t b = threadIdx.x; b < kBytes; b += blockDim.x) bad += s_slot[s][b] != from[b];
    }
    if (bad) atomicAdd(wrong + rank, bad);
}

}  // namespace

cudaError_t launch_pair_end_probe(const uint8_t *src, int32_t *wrong, int even, int odd, cudaStream_t s) {
    unsigned *err = device_status_word();
    if (!err) return cudaErrorUnknown;
    CUtensorMap map;
    const int most = std::max(even, odd);
    if (!encode_tma_2d(&map, src, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, 64 * std::max(most, 1), 128, 128, 32,
                       CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    LaunchScope scope(K_SELFTEST, s);
    pair_end_probe_kernel<<<2, 128, 0, s>>>(map, src, wrong, even, odd, err);
    return cudaGetLastError();
}

cudaError_t launch_bounded_wait_probe(uint64_t limit_ns, cudaStream_t s) {
    unsigned *err = device_status_word();
    if (!err) return cudaErrorUnknown;
    LaunchScope scope(K_SELFTEST, s);
    bounded_wait_probe_kernel<<<1, 64, 0, s>>>(limit_ns, err);
    return cudaGetLastError();
}

}  // namespace ffn
