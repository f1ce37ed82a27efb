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

// `group` query heads per key head; keys are read once for up to 64 of them (q8 of 256: 32).
// `items`: requests x key heads.
//
// Up to 8 heads: one warp has them.  Many items take CTAs of one warp, whose items end without a
// barrier: 256 requests x 16 heads of 64 in fp16, up to 1000 tokens, 32.9 us (four warps 43.0), q8 40.6
// (45.7), 128 x 8 heads of 256 39.8 (51.6); with fewer items the pieces of split ones cost more
// (128 x 8 heads of 128, up to 60 tokens, 15.3 us, four warps 10.1), and q8 of 128 is bound by
// arithmetic that four warps with larger units do less of (46.8, 41.4).
// More heads: a warp takes 16 where o fits its registers (heads of 128, 16 a key head, 16 requests of
// 8192, 8 key heads, in q8: 71.3 us, 8 a warp 113.4), and 8 of 256-wide ones (90.5 us, 16 a warp 103.9;
// q8 90.1, 136.2);
// beyond 32 of those reading the keys once is worth more (64 a key head: 115.4 us, 8 a warp 149.9).
inline PagedAttnVariant paged_attn_variant(int64_t group, int64_t items, int64_t head_dim, bool q8, int sm_count) {
    const int width = paged_attn_width(head_dim);
    if (width == 256 && group > 8) {
        if (group <= 16) return {1, 2, 4};
        if (group <= 32 || q8) return {1, 4, 4};
        return {2, 4, 4};
    }
    if (group > 32) return {2, 4, 4};
    if (group > 16) return {2, 2, 4};
    if (group > 8) return {2, 1, 4};
    const bool many = items >= static_cast<int64_t>(sm_count) * (width == 256 ? 6 : 12);
    return {1, 1, many && !(q8 && width == 128) ? 1 : 4};
}

// Whether an item's pieces are joined by a kernel of their own: where a piece is large (kAttnSplitValues)
// and one CTA would join eight or more.  `keys`: units of the longest request, `slots`: CTAs.
// 4 requests of 4096 tokens, 4 key heads for 64 queries of 128: 13.9 us on the GPU (19.5 joined by the
// last CTA to arrive); one key head for 64 queries of 256 and 32768 tokens 28.7 (81.7).  The second launch
// costs 2 to 3 us of host time.  Pieces of 1024 values, which most calls of few requests have, are left
// to the last CTA for that: split they take 10.6 us (14.4; 1 query head, 32768 tokens), 7.3 (10.0; 8 to a
// key head, 2048), 83.6 (84.8; 64 to 8, 131071), but also 27.2 (26.7; 4 requests of 8192, 32 to 8) and
// 7.0 (6.5; 32 to 8, 512), where the host's time is most of the call.
constexpr int kAttnSplitItems = 256;  // items that the workspace has room for then
inline bool paged_attn_splits(int64_t items, int64_t keys, int64_t slots) {
    return items * 8 <= slots && items <= kAttnSplitItems && keys >= 8;
}
cudaError_t launch_paged_attn_join(const PagedAttnArgs &a, bool f16, int width, int rows, int items, cudaStream_t stream);

template <typename T, int DP>
cudaError_t launch_paged_attn(const PagedAttnArgs &a, const PagedAttnLaunch &l);

}  // namespace sdt
