// group_gather.cu -- the rows that an index names, one behind another, for products over groups.
//
// W[i] = table[idx[i]] for the rows i of all groups (those before the first and behind the last one's
// are not read); an index that is not a row of the table gives zeros and is recorded.  The products
// fetch gathered rows by TMA themselves where they are few: a gather of four rows takes the TMA unit
// about 67 clocks, so 128 rows' piece of 64 columns takes 2150, four times the MMAs of a 256 x 256 tile
// that read it (16384 rows, 4096 x 4096: 1038 us against 282 of rows that lie in order, and 326 with
// this kernel in front).  Bound by memory: a warp a row, 16 bytes a lane, four loads in flight (those
// 44 us, its launch among them, move 268 MB: 6.1 TB/s).  W's rows begin on 128-byte lines.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_group.h"

namespace tcg {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    group_gather_kernel(const uint16_t *table, int32_t table_rows, int64_t lda, const int32_t *idx,
                        const int32_t *offsets, int32_t groups, int32_t M, int32_t K, uint16_t *W, int64_t ldw,
                        uint32_t *status)
{
    const int32_t lane = static_cast<int32_t>(threadIdx.x) % 32;
    const int32_t warps = static_cast<int32_t>(gridDim.x) * (kThreads / 32);
    const int32_t first = static_cast<int32_t>(blockIdx.x) * (kThreads / 32) + static_cast<int32_t>(threadIdx.x) / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t lo = max(0, __ldcg(offsets)), hi = min(M, __ldcg(offsets + groups));
    const int32_t whole = K / 8;  // pieces of 16 bytes
    for (int64_t i = static_cast<int64_t>(lo) + first; i < hi; i += warps) {
        const int32_t r = __ldcg(idx + i);
        const bool there = r >= 0 && r < table_rows;
        if (!there && lane == 0)
            record_error(status, kStatusIndex, 0);
        const uint16_t *from = table + (there ? r : 0) * lda;
        uint16_t *to = W + i * ldw;
        for (int32_t c0 = 0; c0 < whole; c0 += 128) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t c = c0 + 32 * j + lane;
                v[j] = there && c < whole ? __ldcg(reinterpret_cast<const uint4 *>(from) + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t c = c0 + 32 * j + lane;
                if (c < whole)
                    reinterpret_cast<uint4 *>(to)[c] = v[j];
            }
        }
        const int32_t c = 8 * whole + lane;  // the row's last elements
        if (c < K)
            to[c] = there ? __ldcg(from + c) : static_cast<uint16_t>(0);
    }
}

}  // namespace

cudaError_t launch_group_gather(const void *table, int32_t table_rows, int64_t lda, const int32_t *idx,
                                const int32_t *offsets, int32_t groups, int32_t M, int32_t K, void *W, int64_t ldw,
                                uint32_t *status, int sm_count, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int64_t blocks = (static_cast<int64_t>(M) + kThreads / 32 - 1) / (kThreads / 32), most = 8 * sm_count;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, group_gather_kernel, static_cast<const uint16_t *>(table), table_rows, lda, idx,
                              offsets, groups, M, K, static_cast<uint16_t *>(W), ldw, status);
}

}  // namespace tcg
