// paged_attn_plan.cuh -- which variant of the paged attention kernel a call takes.
#pragma once

#include "paged.cuh"

namespace sdt {

struct PagedAttnArgs;

struct PagedAttnVariant {
    int nh;  // a warp's query heads / 8
    int wh;  // warps of a CTA that share keys, with query heads of their own
    int nw;  // warps of a CTA
};

struct PagedAttnLaunch {
    PagedAttnVariant variant;
    bool q8;
    int device, sm_count;
    int64_t max_keys;  // of one request
    cudaStream_t stream;
};

// Head width the kernel is built for.
inline int paged_attn_width(int64_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

// CTAs of nw warps per SM, at most.
inline int paged_attn_ctas(int nw) { return nw == 1 ? 12 : 3; }

// `group` query heads per key head; keys are read once for up to 64 of them.  `items`:
// requests x key heads.
inline PagedAttnVariant paged_attn_variant(int64_t group, int64_t items, int64_t head_dim, bool q8, int sm_count) {
    if (group > 32) return {2, 4, 4};
    if (group > 16) return {2, 2, 4};
    if (group > 8) return {2, 1, 4};
    const int width = paged_attn_width(head_dim);
    const bool many = items >= static_cast<int64_t>(sm_count) * (width == 256 ? 6 : 12);
    return {1, 1, many && !(q8 && width == 128) ? 1 : 4};
}

template <typename T, int DP>
cudaError_t launch_paged_attn(const PagedAttnArgs &a, const PagedAttnLaunch &l);

}  // namespace sdt
