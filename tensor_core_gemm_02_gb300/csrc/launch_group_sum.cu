// launch_group_sum.cu -- the group kernel's sums over each group's rows.
#include "launch_group_impl.cuh"

namespace tcg {

cudaError_t launch_group_sum(int bn, bool pair, const GroupMaps &maps, const GroupArgs &args, int grid,
                             cudaStream_t stream)
{
    return group_launch_forms<kKindSum, 3, false>(bn, pair, maps, args, grid, stream);
}

}  // namespace tcg
