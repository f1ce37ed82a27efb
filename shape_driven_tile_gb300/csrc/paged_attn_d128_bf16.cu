// paged_attn_d128_bf16.cu -- paged_attn kernels for head widths up to 128, bf16 queries.
#include "paged_attn_launch.cuh"

namespace sdt {
template cudaError_t launch_paged_attn<__nv_bfloat16, 128>(const PagedAttnArgs &, const PagedAttnLaunch &);
}  // namespace sdt
