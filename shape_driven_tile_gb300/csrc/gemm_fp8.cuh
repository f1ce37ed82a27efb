// gemm_fp8.cuh -- what the kernels of gemm_fp8 share: arguments, the fp8 MMA, waits that ask ahead.
//
//   C[m][n] = sum_b ws[n / 128][b] * as[m][b] * sum_{k in block b} a[m][k] * w[n][k]
//
// with blocks of 128 along k.  Both scales change with the block, so the accumulator of the
// tensor cores holds one block's sum only: each 128-deep partial product is read from tensor
// memory, multiplied by as * ws and added to fp32 registers, while the tensor cores work on
// the next block in another accumulator.  (The scaled forms of the MMA take powers of two per
// 32 values, which fp32 scales are not.)  An fp8 product is exact in fp32 and a block adds 128
// of them in the MMA's fp32; the sum over blocks is one fused multiply-add a block in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_kernel.cuh"
#include "ptx.cuh"
#include "sdt.h"

namespace sdt {

constexpr int kFp8Block = 128;  // k-values per scale: one 128-byte swizzle row of fp8

struct Fp8Args {
    const float *a_scales, *w_scales;
    void *C;
    int64_t as_row, as_block, ws_row, ws_block;  // elements
    int64_t ldc;
    int M, N, num_kb;        // num_kb: 128-deep blocks of k
    int num_m_tiles, num_n_tiles;
    int splits;              // CTAs of the cluster that share a tile's blocks (swapped form)
    // two-CTA form: m-tiles per raster band; items [0, tail_start) are whole tiles, those from
    // there to num_items halves of the tiles left for a partly empty round
    int raster_group, tail_start, num_items;
    uint32_t idesc;          // types of the MMA's operands
    int c_dtype;
    unsigned long long timeout_ns;
    int *status;
};

// D[tmem] (+)= A[smem desc] . B[smem desc], fp8 operands, K = 32.
__device__ __forceinline__ void umma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A bounded wait that reads the timer only after many failed polls: these kernels' roles wait for
// one another every block, for a few hundred cycles.  RELAXED: what is waited for is that another
// CTA's reads of tensor memory are over, no memory of its; an acquire at cluster scope would
// refresh the SM's cache each time.
template <bool RELAXED = false>
__device__ __forceinline__ bool mbar_wait_soon(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    const auto complete = [&] {
        if (!RELAXED) return mbar_try_wait(bar, parity);
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
#pragma unroll 1
    for (int polls = 0; polls < 256; ++polls)
        if (complete()) return true;
    const uint64_t deadline = global_timer_ns() + limit_ns;
    uint32_t polls = 0;
    while (!complete())
        if ((++polls & 63u) == 0 && global_timer_ns() > deadline) return false;
    return true;
}

// The same for a whole warp, which leaves it converged.
template <bool RELAXED = false>
__device__ __forceinline__ bool warp_wait_soon(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait_soon<RELAXED>(bar, parity, limit_ns));
}

// Whether the phase is complete, without waiting.  Even a wait for a complete phase takes some 150
// cycles, so every role asks for its next barrier before it works on the present one, and waits
// only if the answer was no.
template <bool RELAXED = false>
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (RELAXED)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}
// After a peek: true at once if it saw the phase complete, otherwise a bounded wait.  Whole warp.
template <bool RELAXED = false>
__device__ __forceinline__ bool warp_wait_peeked(bool peeked, uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, peeked) || warp_wait_soon<RELAXED>(bar, parity, limit_ns);
}

// One lane of a converged warp.  A warp that issues copies or MMAs runs its loop as a whole and
// elects a lane for the instructions alone: addresses and descriptors then stay in uniform
// registers, which these instructions take them from.  (As one lane's own loop, a block's four
// MMAs and their barriers took 650 cycles, its two or three copies 600.)
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// acc[0..1] += v[0..1] * scale, two values an instruction (on one GPU 8192^3 takes 369 us, with one at a time
// 378; 4096^3 56.4, 58.3).
__device__ __forceinline__ void fma2(float *acc, const uint32_t *v, float2 scale) {
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), scale, make_float2(acc[0], acc[1]));
    acc[0] = r.x;
    acc[1] = r.y;
}

// The two halves of a meeting of the cluster; the relaxed first half publishes nothing.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Hint: bring a box into L2.
__device__ __forceinline__ void tma_prefetch_l2_2d(const CUtensorMap *map, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace sdt
