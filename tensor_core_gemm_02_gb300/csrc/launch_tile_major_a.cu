// launch_tile_major_a.cu -- the tile kernel's instantiations for A stored K x M
// (a translation unit of its own, so the storages compile in parallel), and the
// dispatch over the three storages (the others in launch_tile_major_{b,ab}.cu).
#include "launch_tile_impl.cuh"

namespace tcg {

template cudaError_t launch_tile_major_impl<kMajA>(int, bool, int, const GemmMaps &, const TileMapsTwo &,
                                                 const GemmArgs &, int, cudaStream_t);

cudaError_t launch_tile_major(int maj, int bn, bool pair, int nsub, const GemmMaps &maps,
                              const TileMapsTwo &two, const GemmArgs &args, int grid,
                              cudaStream_t stream)
{
    switch (maj) {
    case kMajA: return launch_tile_major_impl<kMajA>(bn, pair, nsub, maps, two, args, grid, stream);
    case kMajB: return launch_tile_major_impl<kMajB>(bn, pair, nsub, maps, two, args, grid, stream);
    case kMajA | kMajB:
        return launch_tile_major_impl<kMajA | kMajB>(bn, pair, nsub, maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
