// tensor_map.cuh -- the library's cache of TMA tensor maps (gemm_host.cu).
#pragma once

#include <cuda.h>

#include <cstdint>

namespace sdt {

// A 2-D map of `outer` rows of `inner` contiguous elements (types by their SDT_DTYPE codes)
// with a box of box_inner elements by box_outer rows; SDT_OK or a negative status.
int tensor_map_2d(const void *ptr, int dtype, uint64_t inner, uint64_t outer, uint64_t row_stride_bytes, int box_outer,
                  CUtensorMap *out, int box_inner = 64, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

}  // namespace sdt
