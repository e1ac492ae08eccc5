// pair_end.cuh -- the end of a kernel on CTA pairs one of whose roles may have given up.
//
// Both CTAs of a pair load their parts of a ring's slots and count the bytes on the even
// CTA's barriers, which the even CTA arms with the bytes of both.  A slot is given back
// to both at once, after the MMAs that needed both parts, so that of each slot the two
// have issued equally many loads or, where one has given up, one of them one more.
// Neither CTA may end, and give its shared memory away, before all of these have landed.
#pragma once

#include "ffn_internal.cuh"

namespace ffn {

struct PairEnd {   // in shared memory, at the same place in both CTAs
    uint32_t produced[2];
    int abort[2];
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Called by every thread of both CTAs when its role has ended; thread 0 knows the CTA's
// `produced`, the slots that it has filled one after the other.  full(s): the address of slot s's
// barrier; bytes(s, r): what CTA r's last load into slot s brings (the two parts are alike in
// size).
template <int STAGES, typename Full, typename Bytes>
__device__ __forceinline__ void end_pair(PairEnd &end, uint32_t rank, uint32_t produced, const volatile int *abort_flag,
                                         volatile int *never, uint64_t limit_ns, const Full &full, const Bytes &bytes) {
    __syncthreads();   // the CTA issues nothing more, and has given up or not
    if (threadIdx.x == 0) {
        const int gave_up = *abort_flag;
#pragma unroll
        for (uint32_t r = 0; r < 2; ++r) {
            st_cluster(ptx::mapa_shared(ptx::smem_u32(&end.produced[rank]), r), produced);
            st_cluster(ptx::mapa_shared(ptx::smem_u32(&end.abort[rank]), r), static_cast<uint32_t>(gave_up));
        }
    }
    __syncwarp();
    ptx::cluster_sync();   // neither CTA uses the other's memory or barriers any more
    // Where no one has given up, every load was waited for before its MMAs.
    if (!(end.abort[0] | end.abort[1])) return;
    if (rank == 0 && threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            const uint32_t first = static_cast<uint32_t>(s);
            auto fills = [&](uint32_t n) { return n > first ? (n - first + STAGES - 1) / STAGES : 0u; };
            const uint32_t mine = fills(end.produced[0]), theirs = fills(end.produced[1]);
            if (mine < theirs) ptx::mbar_arrive_expect_tx(full(s), bytes(s, 1));   // armed for their part alone
            if (mine > theirs) ptx::mbar_complete_tx(full(s), bytes(s, 0));        // their part is not to come
            const uint32_t last = max(mine, theirs);
            if (last) ptx::mbar_wait(full(s), (last - 1) & 1u, never, limit_ns);
        }
    }
    __syncwarp();
    ptx::cluster_sync();
}

}  // namespace ffn
