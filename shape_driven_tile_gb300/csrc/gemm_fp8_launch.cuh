// gemm_fp8_launch.cuh -- the launchers of gemm_fp8's kernels (a cudaError_t each).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sdt {

struct Fp8Args;

template <int BT>
int launch_fp8_swap(const CUtensorMap &tmW, const CUtensorMap &tmX, const Fp8Args &args, cudaStream_t stream);

template <int WIDTH>
int launch_fp8_pair(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmC, const Fp8Args &args, int pairs,
                    cudaStream_t stream);

}  // namespace sdt
