// launch_tile_gated_mx.cu -- the tile kernel's gated-form instantiations for
// packed FP4 operands.
#include "launch_tile_impl.cuh"

namespace tcg {

int tile_gated_mx_stages(int bn) { return bn == 256 ? 4 : (bn == 128 ? 5 : 0); }

cudaError_t launch_tile_gated_mx(int bn, bool rows, const GemmMaps &maps, const TileMapsTwo &two,
                                 const GemmArgs &args, int grid, cudaStream_t stream)
{
    return rows ? launch_tile_gated_mx_impl<kModeGatedRows>(bn, maps, two, args, grid, stream)
                : launch_tile_gated_mx_impl<kModeGated>(bn, maps, two, args, grid, stream);
}

}  // namespace tcg
