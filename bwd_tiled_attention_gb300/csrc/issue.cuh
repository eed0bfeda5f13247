// issue.cuh -- waits that end a kernel with an error, and the MMA issuer's two forms.
#pragma once
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

__device__ __forceinline__ void raise_abort(volatile int* flag, WsHeader* hdr, int code) {
    *flag = 1;
    atomicOr(&hdr->error, code);
}

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* flag,
                                              WsHeader* hdr) {
    if (mbar_wait(bar, parity, flag)) return true;
    raise_abort(flag, hdr, kErrTimeout);
    return false;
}

// Whole-warp wait: every lane leaves with the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* flag,
                                          WsHeader* hdr) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, flag, hdr));
}

// The same; PASS: the phase is mostly there, and the common case is one branch of the whole
// warp (the windowed forward's issuer, N = 32768, W = 4096: 803 us against 838).
template <bool PASS>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* flag,
                                          WsHeader* hdr) {
    if (PASS && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return warp_wait(bar, parity, flag, hdr);
}

// How the MMAs are issued: by one thread, or (WARP) by a converged warp of which one lane
// issues, so that descriptors and addresses stay in uniform registers.  Windowed kernels are
// compiled with the latter: backward of 32768 tokens, 16 heads of 128, W = 4096, 2338 us against
// 2450, d = 256 forward of 3.5k tokens 129 against 152.  The deterministic backward up to
// d = 128 is not: 3762 against 3823 (d = 64 846 against 857, d = 96 1137 against 1127).  Above, it is
// (d = 192 3121 against 3281, d = 256 3830 against 3909).
template <bool WARP>
struct Issuer {
    uint32_t lead = WARP ? elect_lead() : 1;
    __device__ __forceinline__ void ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) const {
        if constexpr (WARP) warp_mma_ss(lead, d, a, b, id, acc);
        else mma_ss(d, a, b, id, acc);
    }
    __device__ __forceinline__ void ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) const {
        if constexpr (WARP) warp_mma_ts(lead, d, a, b, id, acc);
        else mma_ts(d, a, b, id, acc);
    }
    __device__ __forceinline__ void commit(uint32_t bar) const {
        if constexpr (WARP) warp_mma_commit(lead, bar);
        else mma_commit(bar);
    }
    __device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) const {
        if constexpr (WARP) return make_sdesc(addr, lbo, sbo);
        else return make_sdesc_here(addr, lbo, sbo);
    }
    __device__ __forceinline__ bool any(bool x) const { return WARP ? __any_sync(0xffffffffu, x) : x; }
    __device__ __forceinline__ bool test(uint32_t bar, uint32_t parity) const {
        const bool in = mbar_test_wait(bar, parity);
        return WARP ? __all_sync(0xffffffffu, in) : in;
    }
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* flag, WsHeader* hdr) const {
        return WARP ? warp_wait<true>(bar, parity, flag, hdr) : wait_or_abort(bar, parity, flag, hdr);
    }
    __device__ __forceinline__ int2 uniform(int2 x) const {
        return WARP ? make_int2(__shfl_sync(0xffffffffu, x.x, 0), __shfl_sync(0xffffffffu, x.y, 0)) : x;
    }
};

}  // namespace
}  // namespace fa
