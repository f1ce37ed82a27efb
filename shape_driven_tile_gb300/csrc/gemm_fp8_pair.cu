// The two-CTA form of gemm_fp8.
#include "gemm_fp8_pair.cuh"

#include "gemm_fp8_launch.cuh"
#include "gemm_launch.cuh"

namespace sdt {

template <int WIDTH>
int launch_fp8_pair(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmC, const Fp8Args &args, int pairs,
                    cudaStream_t stream) {
    using Cfg = Fp8PairCfg<WIDTH>;
    static std::atomic<int> configured[64];
    if (int e = ensure_smem(gemm_fp8_pair_kernel<WIDTH>, Cfg::SMEM_BYTES, configured)) return e;
    // The epilogue's warps wait until the launch's registers cover their share: a build whose kernel starts with
    // fewer (the compiler may give fewer than the block's size allows) is not launched.
    static std::atomic<bool> covered{false};
    if (!covered.load(std::memory_order_relaxed)) {
        cudaFuncAttributes has;
        if (cudaError_t e = cudaFuncGetAttributes(&has, gemm_fp8_pair_kernel<WIDTH>)) return e;
        if (has.numRegs * Cfg::THREADS < Cfg::SPLIT_REGS) return cudaErrorLaunchOutOfResources;
        covered.store(true, std::memory_order_relaxed);
    }
    return launch_kernel(gemm_fp8_pair_kernel<WIDTH>, dim3(2 * static_cast<unsigned>(pairs)), dim3(Cfg::THREADS), size_t(Cfg::SMEM_BYTES),
                         stream, 2, tmA, tmB, tmC, args);
}

template int launch_fp8_pair<256>(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, const Fp8Args &, int, cudaStream_t);
template int launch_fp8_pair<192>(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, const Fp8Args &, int, cudaStream_t);

}  // namespace sdt
