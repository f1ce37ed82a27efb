// paged_attn_plan.cuh -- which variant of the paged attention kernel a call takes.
#pragma once

#include "paged.cuh"

namespace sdt {

struct PagedAttnArgs;

struct PagedAttnLaunch {
    int wh;            // warps of a CTA that share keys, 16 query heads each
    bool q8;
    int sm_count;
    int64_t max_keys;  // of one request
    cudaStream_t stream;
};

// Warps on the same keys: enough for the query heads of one key head, so that keys are read
// once for up to 64 of them.
inline int paged_attn_wh(int64_t group) { return group <= 16 ? 1 : group <= 32 ? 2 : 4; }
// Head width the kernel is built for.
inline int paged_attn_width(int64_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

template <typename T, int DP>
cudaError_t launch_paged_attn(const PagedAttnArgs &a, const PagedAttnLaunch &l);

}  // namespace sdt
