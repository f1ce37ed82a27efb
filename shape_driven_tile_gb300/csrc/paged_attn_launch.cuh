// paged_attn_launch.cuh -- launch of the paged attention kernel, instantiated per head width
// and query type (paged_attn_d*.cu).
#pragma once

#include "launch.cuh"
#include "paged_attn.cuh"
#include "paged_attn_plan.cuh"

namespace sdt {

template <typename T, int DP, int WH, bool Q8>
static cudaError_t launch_variant(const PagedAttnArgs &a, const PagedAttnLaunch &l) {
    using C = AttnCfg<DP, WH, Q8>;
    auto kern = paged_attn_kernel<T, DP, WH, Q8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t keys = (l.max_keys + C::TK - 1) / C::TK;
    const int64_t units = (keys < 1 ? 1 : keys) * a.batch * a.kv_heads * a.head_blocks;  // no mix of lengths has more
    const int64_t slots = static_cast<int64_t>(l.sm_count) * C::CTAS;
    return launch_kernel(kern, dim3(static_cast<unsigned>(units < slots ? units : slots)), dim3(kAttnThreads), C::SMEM,
                         l.stream, 1, a);
}

template <typename T, int DP>
cudaError_t launch_paged_attn(const PagedAttnArgs &a, const PagedAttnLaunch &l) {
    if (l.q8) return l.wh == 1 ? launch_variant<T, DP, 1, true>(a, l) : l.wh == 2 ? launch_variant<T, DP, 2, true>(a, l) : launch_variant<T, DP, 4, true>(a, l);
    return l.wh == 1 ? launch_variant<T, DP, 1, false>(a, l) : l.wh == 2 ? launch_variant<T, DP, 2, false>(a, l) : launch_variant<T, DP, 4, false>(a, l);
}

}  // namespace sdt
