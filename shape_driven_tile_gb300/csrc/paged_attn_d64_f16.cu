// paged_attn_d64_f16.cu -- paged_attn kernels for head widths up to 64, f16 queries.
#include "paged_attn_launch.cuh"

namespace sdt {
template cudaError_t launch_paged_attn<__half, 64>(const PagedAttnArgs &, const PagedAttnLaunch &);
}  // namespace sdt
