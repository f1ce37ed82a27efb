// gemm_fp8.cuh -- what the kernels of gemm_fp8 share: arguments, the fp8 MMA, packed fp32
// arithmetic, scales in shared memory, output types.
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
    int raster_group;        // pair form: m-tiles per raster band
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

// Two fp32 values in a 64-bit register: one instruction multiplies and adds both.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x), "r"(y));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace sdt
