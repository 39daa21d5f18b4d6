// launch_group_few.cu -- the products over groups of few rows.
#include "kernel_group_few.cuh"
#include "launch_group.h"

namespace tcg {

namespace {

template <int MP, int CS, bool MAJB>
cudaError_t few_launch_impl(const GroupMaps &maps, const GroupArgs &args, int grid, cudaStream_t stream)
{
    using Cfg = FewCfg<MP, CS>;
    auto kfn = group_few_kernel<MP, CS, MAJB>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kfn), Cfg::SMEM_ALLOC, done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_ALLOC;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.numAttrs = 1;
    if (CS > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = CS;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, kfn, maps, args);
}

template <int MP>
cudaError_t few_launch(int cs, bool b_major, const GroupMaps &maps, const GroupArgs &args, int grid,
                       cudaStream_t stream)
{
    if (cs == 2)
        return b_major ? few_launch_impl<MP, 2, true>(maps, args, grid, stream)
                       : few_launch_impl<MP, 2, false>(maps, args, grid, stream);
    return b_major ? few_launch_impl<MP, 1, true>(maps, args, grid, stream)
                   : few_launch_impl<MP, 1, false>(maps, args, grid, stream);
}

}  // namespace

cudaError_t launch_group_few(int mp, int cs, bool b_major, const GroupMaps &maps, const GroupArgs &args, int grid,
                             cudaStream_t stream)
{
    switch (mp) {
    case 16: return few_launch<16>(cs, b_major, maps, args, grid, stream);
    case 32: return few_launch<32>(cs, b_major, maps, args, grid, stream);
    case 64: return few_launch<64>(cs, b_major, maps, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
