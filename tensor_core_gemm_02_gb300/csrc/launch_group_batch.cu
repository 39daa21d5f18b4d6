// launch_group_batch.cu -- the group kernel over stacks of equal sizes, operands in one part.
#include "launch_group_impl.cuh"

namespace tcg {

// (launch_group_split.cu)
cudaError_t launch_group_split(int bn, int cs, int maj, bool sym, const GroupMaps &maps, const GroupArgs &args, int grid,
                               cudaStream_t stream);

cudaError_t launch_group_batch(int bn, bool pair, int maj, bool sym, int prec, int cs, const GroupMaps &maps,
                               const GroupArgs &args, int grid, cudaStream_t stream)
{
    if (prec == kPrecSplit)
        return launch_group_split(bn, cs, maj, sym, maps, args, grid, stream);
    if (sym)
        return maj == 0   ? group_launch_forms<kKindBatch, 0, true>(bn, pair, maps, args, grid, stream)
               : maj == 3 ? group_launch_forms<kKindBatch, 3, true>(bn, pair, maps, args, grid, stream)
                          : cudaErrorInvalidValue;
    return maj == 0   ? group_launch_forms<kKindBatch, 0, false>(bn, pair, maps, args, grid, stream)
           : maj == 2 ? group_launch_forms<kKindBatch, 2, false>(bn, pair, maps, args, grid, stream)
                      : cudaErrorInvalidValue;
}

}  // namespace tcg
