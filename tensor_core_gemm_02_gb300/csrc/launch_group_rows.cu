// launch_group_rows.cu -- the group kernel over rows grouped by offsets.
#include "launch_group_impl.cuh"

namespace tcg {

cudaError_t launch_group_rows(int bn, bool pair, bool b_major, int prec, const GroupMaps &maps,
                              const GroupArgs &args, int grid, cudaStream_t stream)
{
    if (prec == kPrecSums)
        return b_major ? group_launch_sums<kKindRows, 2, false, kPrecSums>(bn, maps, args, grid, stream)
                       : group_launch_sums<kKindRows, 0, false, kPrecSums>(bn, maps, args, grid, stream);
    return b_major ? group_launch_forms<kKindRows, 2, false>(bn, pair, maps, args, grid, stream)
                   : group_launch_forms<kKindRows, 0, false>(bn, pair, maps, args, grid, stream);
}

}  // namespace tcg
