// launch_tile_gated_mx.cu -- the tile kernel's gated-form instantiations for
// packed FP4 operands (ring depths as the plain FP4 forms of the same tiles).
#include "launch_tile_impl.cuh"

namespace tcg {

cudaError_t launch_tile_gated_mx(int bn, const GemmMaps &maps, const TileMapsTwo &two,
                                 const GemmArgs &args, int grid, cudaStream_t stream)
{
    switch (bn) {
    case 256: return tile_launch2_impl<256, 3, false, 1, kModeGated, 1, 0>(maps, two, args, grid, stream);
    case 128: return tile_launch2_impl<128, 5, false, 1, kModeGated, 1, 0>(maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
