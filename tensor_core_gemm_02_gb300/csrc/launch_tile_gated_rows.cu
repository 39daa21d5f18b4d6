// launch_tile_gated_rows.cu -- the 16-bit gated form's instantiations for outputs
// whose rows are not whole 16 bytes apart (a translation unit of its own).
#include "launch_tile_impl.cuh"

namespace tcg {

cudaError_t launch_tile_gated_rows(int bn, bool pair, const GemmMaps &maps, const TileMapsTwo &two,
                                   const GemmArgs &args, int grid, cudaStream_t stream)
{
    return launch_tile_gated_impl<kModeGatedRows>(bn, pair, maps, two, args, grid, stream);
}

}  // namespace tcg
