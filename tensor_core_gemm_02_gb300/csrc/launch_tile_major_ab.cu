// launch_tile_major_ab.cu -- the tile kernel's instantiations for A stored K x M and B stored K x N
// (a translation unit of its own, so the storages compile in parallel).
#include "launch_tile_impl.cuh"

namespace tcg {

template cudaError_t launch_tile_major_impl<kMajA | kMajB>(int, bool, int, const GemmMaps &, const TileMapsTwo &,
                                                 const GemmArgs &, int, cudaStream_t);

}  // namespace tcg
