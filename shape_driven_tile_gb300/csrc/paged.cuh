// paged.cuh -- what the paged key-value cache operators share: the cache as the kernels
// see it, division by a run-time constant, checked arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "host_common.cuh"

namespace sdt {

constexpr int kPagedMaxHeadDim = 256;
constexpr int kPagedGroup = 32;  // values per scale of a q8 cache

// Codes of the device status word (low 4 bits, beside WaitSite's): the kernel met a page or
// slot outside the cache, or a length outside its table; it left that access out.
enum PagedSite : int { kSitePage = 8, kSiteSlot = 9, kSiteLength = 10 };

// n / d and n % d for 0 <= n < 2^31 by one widening product: with 2^(l-1) < d <= 2^l and
// m = floor(2^(31+l) / d) + 1, m d exceeds 2^(31+l) by at most 2^l, so n m / 2^(31+l)
// exceeds n / d by less than 1 / d.
struct FastDiv {
    uint32_t d, m, shift;
    __host__ static FastDiv of(uint32_t d) {
        uint32_t l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        return {d, static_cast<uint32_t>((uint64_t(1) << (31 + l)) / d + 1), 31 + l};
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> shift);
    }
};

// One tensor of the cache ([page][token][head][d], any order in memory with d contiguous).
// Strides are held in units of UNIT bytes as 32 bits, so that an address is three wide
// multiply-adds and a shifted add; offsets are 64 bits.
template <int UNIT>
struct PagedRows {
    char *base;
    uint32_t page, token, head;
    __device__ __forceinline__ char *at(uint32_t p, uint32_t t, uint32_t h) const {
        return base + (static_cast<uint64_t>(p) * page + static_cast<uint64_t>(t) * token + static_cast<uint64_t>(h) * head) * UNIT;
    }
};
using KvRows = PagedRows<16>;    // keys and values
using ScaleRows = PagedRows<4>;  // q8 scales

__device__ __forceinline__ void paged_status(int *status, int code) { atomicCAS(status, 0, code); }

// Checks a cache descriptor; SDT_OK or a negative status with the last error set.
int check_cache(const sdt_paged_cache *c);
// The cache's tensors (after check_cache).
KvRows rows_k(const sdt_paged_cache &c), rows_v(const sdt_paged_cache &c);
ScaleRows rows_ks(const sdt_paged_cache &c), rows_vs(const sdt_paged_cache &c);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace sdt
