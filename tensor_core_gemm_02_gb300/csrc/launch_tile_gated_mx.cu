// launch_tile_gated_mx.cu -- the tile kernel's gated-form instantiations for
// packed FP4 operands (single CTAs; rings as deep as shared memory allows).
#include "launch_tile_impl.cuh"

namespace tcg {

int tile_gated_mx_stages(int bn) { return bn == 256 ? 4 : (bn == 128 ? 5 : 0); }

cudaError_t launch_tile_gated_mx(int bn, const GemmMaps &maps, const TileMapsTwo &two,
                                 const GemmArgs &args, int grid, cudaStream_t stream)
{
    switch (bn) {
    case 256: return tile_launch2_impl<256, 4, false, 1, kModeGated, 1, 0>(maps, two, args, grid, stream);
    case 128: return tile_launch2_impl<128, 5, false, 1, kModeGated, 1, 0>(maps, two, args, grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
