// launch_tile_gated.cu -- the tile kernel's gated-form instantiations for 16-bit
// operands.
#include "launch_tile_impl.cuh"

namespace tcg {

cudaError_t launch_tile_gated(int bn, bool pair, bool rows, const GemmMaps &maps, const TileMapsTwo &two,
                              const GemmArgs &args, int grid, cudaStream_t stream)
{
    return rows ? launch_tile_gated_rows(bn, pair, maps, two, args, grid, stream)
                : launch_tile_gated_impl<kModeGated>(bn, pair, maps, two, args, grid, stream);
}

}  // namespace tcg
