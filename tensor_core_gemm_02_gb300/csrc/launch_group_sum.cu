// launch_group_sum.cu -- the group kernel's sums over each group's rows.
#include "launch_group_impl.cuh"

namespace tcg {

cudaError_t launch_group_sum(int bn, bool pair, int prec, const GroupMaps &maps, const GroupArgs &args,
                             int grid, cudaStream_t stream)
{
    return prec == kPrecSums ? group_launch_sums<kKindSum, 3, false, kPrecSums>(bn, maps, args, grid, stream)
                             : group_launch_forms<kKindSum, 3, false>(bn, pair, maps, args, grid, stream);
}

}  // namespace tcg
