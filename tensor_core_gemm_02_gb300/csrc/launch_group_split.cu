// launch_group_split.cu -- the group kernel over stacks of equal sizes, operands in two parts.
#include "launch_group_impl.cuh"

namespace tcg {

cudaError_t launch_group_split(int bn, int maj, bool sym, const GroupMaps &maps, const GroupArgs &args, int grid,
                               cudaStream_t stream)
{
    if (sym)
        return maj == 0   ? group_launch_sums<kKindBatch, 0, true, kPrecSplit>(bn, maps, args, grid, stream)
               : maj == 3 ? group_launch_sums<kKindBatch, 3, true, kPrecSplit>(bn, maps, args, grid, stream)
                          : cudaErrorInvalidValue;
    return maj == 0   ? group_launch_sums<kKindBatch, 0, false, kPrecSplit>(bn, maps, args, grid, stream)
           : maj == 2 ? group_launch_sums<kKindBatch, 2, false, kPrecSplit>(bn, maps, args, grid, stream)
                      : cudaErrorInvalidValue;
}

}  // namespace tcg
