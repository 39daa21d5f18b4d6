// launch_tile_major_b.cu -- the tile kernel's instantiations for B stored K x N
// (a translation unit of its own, so the storages compile in parallel).
#include "launch_tile_impl.cuh"

namespace tcg {

template cudaError_t launch_tile_major_impl<kMajB>(int, bool, int, const GemmMaps &, const TileMapsTwo &,
                                                 const GemmArgs &, int, cudaStream_t);

}  // namespace tcg
