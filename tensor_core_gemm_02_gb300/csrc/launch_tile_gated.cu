// launch_tile_gated.cu -- the tile kernel's gated-form instantiations for 16-bit
// operands (ring depths as the plain forms of the same tiles).
#include "launch_tile_impl.cuh"

namespace tcg {

cudaError_t launch_tile_gated(int bn, bool pair, const GemmMaps &maps, const TileMapsTwo &two,
                              const GemmArgs &args, int grid, cudaStream_t stream)
{
    if (pair)
        return bn == 256 ? tile_launch2_impl<256, 6, true, 1, kModeGated, 0, 0>(maps, two, args, grid, stream)
                         : cudaErrorInvalidValue;
    switch (bn) {
    case 256: return tile_launch2_impl<256, 4, false, 1, kModeGated, 0, 0>(maps, two, args, grid, stream);
    case 128: return tile_launch2_impl<128, 6, false, 1, kModeGated, 0, 0>(maps, two, args, grid, stream);
    case 64: return tile_launch2_impl<64, 8, false, 1, kModeGated, 0, 0>(maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
