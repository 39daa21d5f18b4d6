// group_rows.cu -- the rows of each group: a stable counting sort of group ids.
//
// order lists the positions 0 .. M - 1 by ids[i], equal ones in their order; ids outside
// [0, groups) come last, in a bucket of their own.  offsets[g] is the number of ids below g.
//
// A warp takes a run of consecutive ids, 32 at a time.  First pass: each id counts one in its
// warp's bucket (shared-memory atomics; a count does not depend on their order).  Then the
// counts become places, bucket by bucket: behind all ids of lower buckets and, within one,
// behind the thread blocks and warps before.  Second pass: the lanes with a lane's id are
// those whose bits agree (a ballot a bit), a lane's place is its warp's next one plus the
// number of such lanes before it, and the lowest of them moves the warp's next place on.  The
// order of nothing depends on timing.  (__match_any_sync instead of the ballots, in one block:
// 16384 ids of 64 groups 27 us.)
//
// Up to 32 a warp one thread block does it all, up to 131072 ids a cluster of eight, whose
// blocks read one another's counts; more are cut into chunks, whose counts a first kernel
// leaves in memory.  Bound by latency: a few dependent steps, each a round trip to shared
// memory or L2 (16384 ids of 64 groups 10.8 us, the call's host time 9 to 10).
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

// The ids [lo, hi) of a thread block, cut into its warps' runs.
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

// First pass: counts[w nb + b], warp w's ids in bucket b, and all[b] their sum over the warps.
__device__ __forceinline__ void count_ids(const int32_t *ids, const Run &r, int32_t groups, int32_t *counts,
                                          int32_t *all)
{
    const int32_t nb = groups + 1;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    for (int32_t i = threadIdx.x; i < nb * kSortWarps; i += kSortThreads)
        counts[i] = 0;
    __syncthreads();
    for_ids(ids, r.lo, r.hi, groups, lane, [&](int64_t, int32_t b, bool there) {
        if (there)
            atomicAdd(counts + warp * nb + b, 1);
    });
    __syncthreads();
    for (int32_t b = threadIdx.x; b < nb; b += kSortThreads) {
        int32_t sum = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w)
            sum += counts[w * nb + b];
        all[b] = sum;
    }
}

__global__ void __launch_bounds__(kSortThreads)
    group_count_kernel(const int32_t *ids, int64_t M, int64_t chunk, int32_t groups, int32_t *counts)
{
    extern __shared__ int32_t sh[];
    const int32_t nb = groups + 1;
    grid_dependency_wait();
    const int64_t lo = chunk * blockIdx.x < M ? chunk * blockIdx.x : M, hi = lo + chunk < M ? lo + chunk : M;
    count_ids(ids, warp_run(lo, hi, threadIdx.x / 32u), groups, sh,
              counts + static_cast<int64_t>(blockIdx.x) * nb);
}

// CLUSTER: the grid is one cluster, whose blocks read one another's counts; otherwise
// (several blocks) `counts` has every block's.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSortThreads)
    group_place_kernel(const int32_t *ids, int64_t M, int64_t chunk, int32_t groups, int32_t choices,
                       const int32_t *counts, int32_t *offsets, int32_t *order, int32_t *rows)
{
    extern __shared__ int32_t sh[];
    __shared__ int32_t warp_sum[kSortWarps];
    const int32_t nb = groups + 1;
    int32_t *all = sh + nb * kSortWarps;
    const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t lo = chunk * blockIdx.x < M ? chunk * blockIdx.x : M, hi = lo + chunk < M ? lo + chunk : M;
    const Run r = warp_run(lo, hi, warp);
    count_ids(ids, r, groups, sh, all);
    if (CLUSTER)
        cluster_sync_all();
    else
        __syncthreads();
    int32_t carry = 0;
    for (int32_t b0 = 0; b0 < nb; b0 += kSortThreads) {
        const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
        int32_t before = 0, total_b = 0;  // ids of the bucket in the blocks before, and in all
        if (b < nb) {
#pragma unroll 8
            for (uint32_t c = 0; c < gridDim.x; ++c) {
                const int32_t n = gridDim.x == 1 ? all[b]
                                  : CLUSTER      ? static_cast<int32_t>(ld_shared_cluster_u32(mapa_shared(smem_u32(all + b), c)))
                                                 : __ldcg(counts + static_cast<int64_t>(c) * nb + b);
                before += c < blockIdx.x ? n : 0;
                total_b += n;
            }
        }
        int32_t sum = total_b;
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
#pragma unroll
        for (uint32_t w = 0; w < kSortWarps; ++w) {
            const int32_t x = warp_sum[w];
            lower += w < warp ? x : 0;
            total += x;
        }
        carry += total;
        const int32_t start = lower + sum - total_b;
        if (b < nb) {
            if (blockIdx.x == 0)
                offsets[b] = start;
            int32_t at = start + before;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t n = sh[w * nb + b];
                sh[w * nb + b] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    int32_t *mine = sh + warp * nb;
    const int bits = 32 - __clz(groups);  // of a bucket's number, at most `groups`
    for_ids(ids, r.lo, r.hi, groups, lane, [&](int64_t i, int32_t b, bool there) {
        uint32_t same = __ballot_sync(0xffffffffu, there);
        for (int k = 0; k < bits; ++k) {
            const uint32_t bit = __ballot_sync(0xffffffffu, (b >> k) & 1);
            same &= ((b >> k) & 1) ? bit : ~bit;
        }
        const int32_t at = mine[b] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (there) {
            if (lane == static_cast<uint32_t>(__ffs(same)) - 1u)
                mine[b] += __popc(same);
            order[at] = static_cast<int32_t>(i);
            if (rows)
                rows[at] = static_cast<int32_t>(i) / choices;
        }
        __syncwarp();
    });
    if (CLUSTER)
        cluster_sync_all();  // (every block has read this one's counts)
}

}  // namespace

cudaError_t launch_group_rows_sort(const int32_t *ids, int64_t M, int32_t groups, int32_t choices,
                                   int32_t *offsets, int32_t *order, int32_t *rows, int32_t *counts,
                                   int32_t chunks, cudaStream_t stream)
{
    const uint32_t most = 1025 * (kSortWarps + 1) * sizeof(int32_t);
    static std::atomic<uint64_t> done_count{0}, done_place{0}, done_cluster{0};
    const bool cluster = chunks == 1 && M > kSortThreads;
    const int64_t blocks = cluster ? 8 : chunks;
    auto place = cluster ? group_place_kernel<true> : group_place_kernel<false>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(place), most, cluster ? done_cluster : done_place);
    if (e != cudaSuccess)
        return e;
    if (chunks > 1 && (e = allow_smem(reinterpret_cast<const void *>(group_count_kernel), most, done_count)) != cudaSuccess)
        return e;
    const int64_t chunk = (M + blocks - 1) / blocks;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<uint32_t>((groups + 1) * (kSortWarps + 1) * sizeof(int32_t));
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 8;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (chunks > 1 && (e = cudaLaunchKernelEx(&cfg, group_count_kernel, ids, M, chunk, groups, counts)) != cudaSuccess)
        return e;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, place, ids, M, chunk, groups, choices, static_cast<const int32_t *>(counts),
                              offsets, order, rows);
}

}  // namespace tcg
