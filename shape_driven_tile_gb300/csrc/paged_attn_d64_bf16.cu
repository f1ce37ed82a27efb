// paged_attn_d64_bf16.cu -- paged_attn kernels for head widths up to 64, bf16 queries.
#include "paged_attn_launch.cuh"

namespace sdt {
template cudaError_t launch_paged_attn<__nv_bfloat16, 64>(const PagedAttnArgs &, const PagedAttnLaunch &);
}  // namespace sdt
