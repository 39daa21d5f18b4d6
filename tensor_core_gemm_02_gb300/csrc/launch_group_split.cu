// launch_group_split.cu -- the group kernel over stacks of equal sizes, operands in two parts.
#include "launch_group_impl.cuh"

namespace tcg {

namespace {

template <int MAJ, bool SYM>
cudaError_t split_launch(int bn, int cs, const GroupMaps &maps, const GroupArgs &args, int grid, cudaStream_t stream)
{
    if (cs == 2)
        return bn == 64 ? group_launch_impl<64, 3, false, kKindBatch, MAJ, SYM, kPrecSplit, 2>(maps, args, grid, stream)
                        : cudaErrorInvalidValue;
    return group_launch_sums<kKindBatch, MAJ, SYM, kPrecSplit>(bn, maps, args, grid, stream);
}

}  // namespace

cudaError_t launch_group_split(int bn, int cs, int maj, bool sym, const GroupMaps &maps, const GroupArgs &args, int grid,
                               cudaStream_t stream)
{
    if (sym)
        return maj == 0   ? split_launch<0, true>(bn, cs, maps, args, grid, stream)
               : maj == 3 ? split_launch<3, true>(bn, cs, maps, args, grid, stream)
                          : cudaErrorInvalidValue;
    return maj == 0   ? split_launch<0, false>(bn, cs, maps, args, grid, stream)
           : maj == 2 ? split_launch<2, false>(bn, cs, maps, args, grid, stream)
                      : cudaErrorInvalidValue;
}

}  // namespace tcg
