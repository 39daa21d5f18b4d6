// launch_skinny_gated.cu -- the swap-AB stream-K kernel's gated-form
// instantiations (16-bit operands, or both FP4 on the block-scaled MMA), and those
// for B stored K x N.
#include <cuda_runtime.h>

#include "kernel_skinny.cuh"
#include "launch.h"

namespace tcg {

namespace {

template <typename Cfg, typename K, typename... Maps>
cudaError_t launch_with(K kfn, std::atomic<uint64_t> &done, const GemmArgs &args, int grid,
                        cudaStream_t stream, const Maps &...maps)
{
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kfn), Cfg::SMEM_ALLOC, done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_ALLOC;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kfn, maps..., args);
}

template <int MP, bool MX>
cudaError_t launch_skinny_gated_impl(const GemmMaps &maps, const TileMapsTwo &two, const GemmArgs &args,
                                     int grid, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_with<SkinnyCfg<MP, 1, false, MX, true>>(skinny_gated_kernel<MP, 1, MX>, done, args, grid,
                                                          stream, maps.a, maps.b, maps.c, maps.sfa, two.b2,
                                                          two.sfb2);
}

template <int MP>
cudaError_t launch_skinny_trans_impl(const GemmMaps &maps, const TileMapsTwo &two, const GemmArgs &args,
                                     int grid, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_with<SkinnyCfg<MP, 1>>(skinny_trans_kernel<MP, 1>, done, args, grid, stream, maps.a,
                                         maps.b, two.b2, two.a2);
}

}  // namespace

cudaError_t launch_skinny_gated(int mp, bool mx, const GemmMaps &maps, const TileMapsTwo &two,
                                const GemmArgs &args, int grid, cudaStream_t stream)
{
    switch (mp) {
    case 16: return mx ? launch_skinny_gated_impl<16, true>(maps, two, args, grid, stream)
                       : launch_skinny_gated_impl<16, false>(maps, two, args, grid, stream);
    case 32: return mx ? launch_skinny_gated_impl<32, true>(maps, two, args, grid, stream)
                       : launch_skinny_gated_impl<32, false>(maps, two, args, grid, stream);
    case 64: return mx ? launch_skinny_gated_impl<64, true>(maps, two, args, grid, stream)
                       : launch_skinny_gated_impl<64, false>(maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_skinny_trans(int mp, const GemmMaps &maps, const TileMapsTwo &two, const GemmArgs &args,
                                int grid, cudaStream_t stream)
{
    switch (mp) {
    case 16: return launch_skinny_trans_impl<16>(maps, two, args, grid, stream);
    case 32: return launch_skinny_trans_impl<32>(maps, two, args, grid, stream);
    case 64: return launch_skinny_trans_impl<64>(maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
