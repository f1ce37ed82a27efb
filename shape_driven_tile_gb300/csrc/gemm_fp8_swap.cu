// The swapped form of gemm_fp8 for each token width.
#include "gemm_fp8_swap.cuh"

#include "gemm_fp8_launch.cuh"
#include "gemm_launch.cuh"

namespace sdt {

template <int BT>
int launch_fp8_swap(const CUtensorMap &tmW, const CUtensorMap &tmX, const Fp8Args &args, cudaStream_t stream) {
    using Cfg = SwapCfg<BT>;
    static std::atomic<int> configured[64];
    if (int e = ensure_smem(gemm_fp8_swap_kernel<BT>, Cfg::SMEM_MOST, configured)) return e;
    const unsigned grid = static_cast<unsigned>(args.num_m_tiles) * static_cast<unsigned>(args.num_n_tiles) *
                          static_cast<unsigned>(args.splits);
    return launch_kernel(gemm_fp8_swap_kernel<BT>, dim3(grid), dim3(Cfg::THREADS),
                         size_t(BT == 128 && args.splits == 1 ? Cfg::SMEM_ALONE : Cfg::SMEM_BYTES), stream,
                         static_cast<unsigned>(args.splits), tmW, tmX, args);
}

template int launch_fp8_swap<16>(const CUtensorMap &, const CUtensorMap &, const Fp8Args &, cudaStream_t);
template int launch_fp8_swap<32>(const CUtensorMap &, const CUtensorMap &, const Fp8Args &, cudaStream_t);
template int launch_fp8_swap<64>(const CUtensorMap &, const CUtensorMap &, const Fp8Args &, cudaStream_t);
template int launch_fp8_swap<128>(const CUtensorMap &, const CUtensorMap &, const Fp8Args &, cudaStream_t);

}  // namespace sdt
