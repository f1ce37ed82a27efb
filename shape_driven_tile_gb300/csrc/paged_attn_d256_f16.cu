// paged_attn_d256_f16.cu -- paged_attn kernels for head widths up to 256, f16 queries.
#include "paged_attn_launch.cuh"

namespace sdt {
template cudaError_t launch_paged_attn<__half, 256>(const PagedAttnArgs &, const PagedAttnLaunch &);
}  // namespace sdt
