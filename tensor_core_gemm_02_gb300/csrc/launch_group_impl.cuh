// launch_group_impl.cuh -- the group kernel's launch, for the launch_group_*.cu.
#pragma once

#include "launch_group.h"

namespace tcg {

template <int BN, int STAGES, bool PAIR, int KIND, int MAJ, bool SYM, int PREC, int CS = 1>
cudaError_t group_launch_impl(const GroupMaps &maps, const GroupArgs &args, int grid, cudaStream_t stream)
{
    using Cfg = GroupCfg<BN, STAGES, PAIR, KIND, PREC, CS>;
    auto kfn = group_gemm_kernel<BN, STAGES, PAIR, KIND, MAJ, SYM, PREC, CS>;
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
    if (PAIR || CS > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, kfn, maps, args);
}

// The forms, with ring depths as deep as shared memory allows (the plain forms').
template <int KIND, int MAJ, bool SYM>
cudaError_t group_launch_forms(int bn, bool pair, const GroupMaps &maps, const GroupArgs &args, int grid,
                               cudaStream_t stream)
{
    constexpr int kLess = KIND == kKindBatch ? 1 : 0;  // (C's buffers)
    if (pair)
        return bn == 256 ? group_launch_impl<256, 6 - kLess, true, KIND, MAJ, SYM, kPrecAcc>(maps, args, grid, stream)
                         : cudaErrorInvalidValue;
    if (bn == 128)
        return group_launch_impl<128, 6 - kLess, false, KIND, MAJ, SYM, kPrecAcc>(maps, args, grid, stream);
    if (bn == 64)
        return group_launch_impl<64, 8, false, KIND, MAJ, SYM, kPrecAcc>(maps, args, grid, stream);
    if constexpr (!SYM) {
        if (bn == 256)
            return group_launch_impl<256, 4 - kLess, false, KIND, MAJ, SYM, kPrecAcc>(maps, args, grid, stream);
    }
    return cudaErrorInvalidValue;
}

// The forms that keep float32 sums in registers (bn 256: CTA pairs).
template <int KIND, int MAJ, bool SYM, int PREC>
cudaError_t group_launch_sums(int bn, const GroupMaps &maps, const GroupArgs &args, int grid, cudaStream_t stream)
{
    constexpr int kDeep = PREC == kPrecSplit ? 2 : 1;
    if constexpr (PREC == kPrecSums) {
        if (bn == 256)
            return group_launch_impl<256, 5, true, KIND, MAJ, SYM, PREC>(maps, args, grid, stream);
    }
    if (bn == 128)
        return group_launch_impl<128, 6 / kDeep, false, KIND, MAJ, SYM, PREC>(maps, args, grid, stream);
    if (bn == 64)
        return group_launch_impl<64, 8 / kDeep, false, KIND, MAJ, SYM, PREC>(maps, args, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tcg
