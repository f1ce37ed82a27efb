// paged_attn_d128_f16.cu -- paged_attn kernels for head widths up to 128, f16 queries.
#include "paged_attn_launch.cuh"

namespace sdt {
template cudaError_t launch_paged_attn<__half, 128>(const PagedAttnArgs &, const PagedAttnLaunch &);
}  // namespace sdt
