// group_rows.cu -- the rows of each group: a stable counting sort of group ids.
//
// order lists the positions 0 .. M - 1 by ids[i], equal ones in their order; ids outside
// [0, groups) come last, in a bucket of their own.  offsets[g] is the number of ids below g.
//
// A warp takes a run of consecutive ids, 32 at a time: __match_any_sync names the lanes with
// a lane's id, so the lowest of them adds their number to the warp's count (first pass) or
// its place (second pass), and a lane's own place is that plus the number of such lanes
// before it.  No atomics: the order of nothing depends on timing.  Between the passes the
// counts of a thread block's 32 warps become places, bucket by bucket.  Up to 65536 ids one
// block does it all; more are cut into chunks, a first kernel counts each chunk's, and every
// block of the second adds up the counts before its own.
//
// Bound by latency: two passes over the ids, each 32 ids a warp and step.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_group.h"

namespace tcg {

namespace {

constexpr int kSortWarps = 32;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr int kAhead = 8;  // loads of ids in flight

__device__ __forceinline__ int32_t bucket_of(const int32_t *ids, int64_t i, int64_t end, int32_t groups)
{
    const int32_t v = i < end ? __ldcg(ids + i) : groups;
    return v < 0 || v > groups ? groups : v;
}

// f(position, bucket, whether there is such a position) for the ids [lo, hi), 32 at a time
template <class F>
__device__ __forceinline__ void for_ids(const int32_t *ids, int64_t lo, int64_t hi, int32_t groups,
                                        uint32_t lane, F f)
{
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kAhead) {
        int32_t b[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            b[j] = bucket_of(ids, i0 + 32 * j + lane, hi, groups);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + 32 * j < hi)
                f(i0 + 32 * j + lane, b[j], i0 + 32 * j + lane < hi);
    }
}

// counts[w (groups + 1) + b]: this warp's ids in bucket b
__device__ __forceinline__ void count_ids(const int32_t *ids, int64_t lo, int64_t hi, int32_t groups,
                                          uint32_t lane, int32_t *mine)
{
    for_ids(ids, lo, hi, groups, lane, [&](int64_t, int32_t b, bool there) {
        const uint32_t live = __ballot_sync(0xffffffffu, there);
        if (there) {
            const uint32_t same = __match_any_sync(live, b);
            if (lane == static_cast<uint32_t>(__ffs(same)) - 1u)
                mine[b] += __popc(same);
        }
        __syncwarp();
    });
}

// The chunk [lo, hi) of thread block `chunk`, cut into its warps' runs.
struct Run {
    int64_t lo, hi;
};
__device__ __forceinline__ Run warp_run(int64_t lo, int64_t hi, uint32_t warp)
{
    const int64_t steps = (hi - lo + 31) / 32;
    const int64_t per = (steps + kSortWarps - 1) / kSortWarps * 32;
    const int64_t a = lo + per * warp;
    return Run{a < hi ? a : hi, a + per < hi ? a + per : hi};
}

__global__ void __launch_bounds__(kSortThreads)
    group_count_kernel(const int32_t *ids, int64_t M, int64_t chunk, int32_t groups, int32_t *counts)
{
    extern __shared__ int32_t sh[];
    const int32_t nb = groups + 1;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    grid_dependency_wait();
    for (int32_t i = threadIdx.x; i < nb * kSortWarps; i += kSortThreads)
        sh[i] = 0;
    __syncthreads();
    const int64_t lo = chunk * blockIdx.x, hi = lo + chunk < M ? lo + chunk : M;
    const Run r = warp_run(lo, hi, warp);
    count_ids(ids, r.lo, r.hi, groups, lane, sh + warp * nb);
    __syncthreads();
    for (int32_t b = threadIdx.x; b < nb; b += kSortThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w)
            sum += sh[w * nb + b];
        counts[static_cast<int64_t>(blockIdx.x) * nb + b] = sum;
    }
}

__global__ void __launch_bounds__(kSortThreads)
    group_place_kernel(const int32_t *ids, int64_t M, int64_t chunk, int32_t groups, int32_t choices,
                       const int32_t *counts, int32_t *offsets, int32_t *order, int32_t *rows)
{
    extern __shared__ int32_t sh[];
    __shared__ int32_t warp_sum[kSortWarps];
    const int32_t nb = groups + 1;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int32_t i = threadIdx.x; i < nb * kSortWarps; i += kSortThreads)
        sh[i] = 0;
    __syncthreads();
    const int64_t lo = chunk * blockIdx.x, hi = lo + chunk < M ? lo + chunk : M;
    const Run r = warp_run(lo, hi, warp);
    count_ids(ids, r.lo, r.hi, groups, lane, sh + warp * nb);
    __syncthreads();
    // counts -> places: bucket b starts behind all ids of lower buckets and, within it, behind
    // the chunks and warps before
    int32_t carry = 0;
    for (int32_t b0 = 0; b0 < nb; b0 += kSortThreads) {
        const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
        int32_t here = 0, before = 0, all = 0;
        if (b < nb) {
            for (int w = 0; w < kSortWarps; ++w)
                here += sh[w * nb + b];
            all = here;
            if (gridDim.x > 1) {
                all = 0;
                for (uint32_t c = 0; c < gridDim.x; ++c) {
                    const int32_t n = __ldcg(counts + static_cast<int64_t>(c) * nb + b);
                    before += c < blockIdx.x ? n : 0;
                    all += n;
                }
            }
        }
        int32_t sum = all;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int32_t x = __shfl_up_sync(0xffffffffu, sum, d);
            if (static_cast<int>(lane) >= d)
                sum += x;
        }
        if (lane == 31)
            warp_sum[warp] = sum;
        __syncthreads();
        int32_t lower = carry, total = 0;
        for (uint32_t w = 0; w < kSortWarps; ++w) {
            const int32_t x = warp_sum[w];
            lower += w < warp ? x : 0;
            total += x;
        }
        carry += total;
        const int32_t start = lower + sum - all;
        if (b < nb) {
            if (blockIdx.x == 0)
                offsets[b] = start;
            int32_t at = start + before;
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t n = sh[w * nb + b];
                sh[w * nb + b] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    int32_t *mine = sh + warp * nb;
    for_ids(ids, r.lo, r.hi, groups, lane, [&](int64_t i, int32_t b, bool there) {
        const uint32_t live = __ballot_sync(0xffffffffu, there);
        if (there) {
            const uint32_t same = __match_any_sync(live, b);
            const int32_t at = mine[b] + __popc(same & ((1u << lane) - 1u));
            __syncwarp(live);
            if (lane == static_cast<uint32_t>(__ffs(same)) - 1u)
                mine[b] += __popc(same);
            order[at] = static_cast<int32_t>(i);
            if (rows)
                rows[at] = static_cast<int32_t>(i) / choices;
        }
        __syncwarp();
    });
}

}  // namespace

cudaError_t launch_group_rows_sort(const int32_t *ids, int64_t M, int32_t groups, int32_t choices,
                                   int32_t *offsets, int32_t *order, int32_t *rows, int32_t *counts,
                                   int32_t chunks, cudaStream_t stream)
{
    const uint32_t smem = static_cast<uint32_t>((groups + 1) * kSortWarps * sizeof(int32_t));
    static std::atomic<uint64_t> done_count{0}, done_place{0};
    cudaError_t e;
    if ((e = allow_smem(reinterpret_cast<const void *>(group_count_kernel), 1025 * 128, done_count)) !=
            cudaSuccess ||
        (e = allow_smem(reinterpret_cast<const void *>(group_place_kernel), 1025 * 128, done_place)) !=
            cudaSuccess)
        return e;
    const int64_t chunk = chunks > 1 ? (M + chunks - 1) / chunks : M;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(chunks), 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (chunks > 1 && (e = cudaLaunchKernelEx(&cfg, group_count_kernel, ids, M, chunk, groups, counts)) != cudaSuccess)
        return e;
    return cudaLaunchKernelEx(&cfg, group_place_kernel, ids, M, chunk, groups, choices,
                              static_cast<const int32_t *>(counts), offsets, order, rows);
}

}  // namespace tcg
