// paged_attn_launch.cuh -- launch of the paged attention kernel, instantiated per head width
// and query type (paged_attn_d*.cu).
#pragma once

#include <algorithm>
#include <atomic>

#include "launch.cuh"
#include "paged_attn.cuh"
#include "paged_attn_plan.cuh"

namespace sdt {

// CTAs per SM of a variant with q_rows query rows; asked of the runtime once per device.
template <typename T, int DP, int NH, int WH, int NW, bool Q8>
static cudaError_t resident_ctas(int device, int q_rows, int *ctas) {
    using C = AttnCfg<DP, NH, WH, NW, Q8>;
    static std::atomic<int> known[kMaxDevices][C::ROWS + 1];
    *ctas = known[device][q_rows].load(std::memory_order_acquire);
    if (*ctas) return cudaSuccess;
    auto kern = paged_attn_kernel<T, DP, NH, WH, NW, Q8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::ROWS));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kern, C::THREADS, C::smem(q_rows));
    if (e != cudaSuccess) return e;
    *ctas = std::max(1, std::min(*ctas, paged_attn_ctas(NW)));
    known[device][q_rows].store(*ctas, std::memory_order_release);
    return cudaSuccess;
}

template <typename T, int DP, int NH, int WH, int NW, bool Q8>
static cudaError_t launch_variant(PagedAttnArgs a, const PagedAttnLaunch &l) {
    using C = AttnCfg<DP, NH, WH, NW, Q8>;
    a.q_rows = std::min(a.group, C::ROWS);
    int ctas = 0;
    cudaError_t e = resident_ctas<T, DP, NH, WH, NW, Q8>(l.device, a.q_rows, &ctas);
    if (e != cudaSuccess) return e;
    const int64_t keys = (l.max_keys + C::TK - 1) / C::TK;
    const int64_t units = std::max<int64_t>(keys, 1) * a.batch * a.kv_heads * a.head_blocks;  // no mix of lengths has more
    const int64_t slots = static_cast<int64_t>(l.sm_count) * ctas;
    const int64_t items = static_cast<int64_t>(a.batch) * a.kv_heads * a.head_blocks;
    if (!C::SPLITS || !paged_attn_splits(items, keys, slots)) a.split = nullptr;
    e = launch_kernel(paged_attn_kernel<T, DP, NH, WH, NW, Q8>, dim3(static_cast<unsigned>(std::min(units, slots))),
                      dim3(C::THREADS), C::smem(a.q_rows), l.stream, 1, a);
    if (e == cudaSuccess && a.split)
        e = launch_paged_attn_join(a, std::is_same_v<T, __half>, DP, C::ROWS, static_cast<int>(items), l.stream);
    return e;
}

template <typename T, int DP, bool Q8>
static cudaError_t launch_of(const PagedAttnArgs &a, const PagedAttnLaunch &l) {
    const PagedAttnVariant v = l.variant;  // (every variant that paged_attn_variant names for this width)
    if constexpr (DP == 256) {
        if constexpr (!Q8)
            if (v.nh == 2) return launch_variant<T, DP, 2, 4, 4, Q8>(a, l);
        if (v.wh == 4) return launch_variant<T, DP, 1, 4, 4, Q8>(a, l);
        if (v.wh == 2) return launch_variant<T, DP, 1, 2, 4, Q8>(a, l);
    } else if (v.nh == 2) {
        if (v.wh == 4) return launch_variant<T, DP, 2, 4, 4, Q8>(a, l);
        return v.wh == 2 ? launch_variant<T, DP, 2, 2, 4, Q8>(a, l) : launch_variant<T, DP, 2, 1, 4, Q8>(a, l);
    }
    if constexpr (!(Q8 && DP == 128))
        if (v.nw == 1) return launch_variant<T, DP, 1, 1, 1, Q8>(a, l);
    return launch_variant<T, DP, 1, 1, 4, Q8>(a, l);
}

template <typename T, int DP>
cudaError_t launch_paged_attn(const PagedAttnArgs &a, const PagedAttnLaunch &l) {
    return l.q8 ? launch_of<T, DP, true>(a, l) : launch_of<T, DP, false>(a, l);
}

}  // namespace sdt
