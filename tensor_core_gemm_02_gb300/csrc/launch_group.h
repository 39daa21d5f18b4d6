// launch_group.h -- host-side interface between the entry points for groups
// (api_group.cu) and their kernels' launchers.
#pragma once

#include "kernel_group.cuh"
#include "launch.h"

namespace tcg {

// A form of the group kernel: single CTAs with 128 x bn tiles (bn 64, 128, 256), or
// (pair) CTA pairs with 256 x 256 ones.  maj: bit 0 A stored with K outermost, bit 1 B.
// grid counts CTAs.  prec: kPrecAcc, or sums kept in registers (bn 64 or 128, or pairs).
cudaError_t launch_group_rows(int bn, bool pair, bool b_major, int prec, const GroupMaps &maps, const GroupArgs &args,
                              int grid, cudaStream_t stream);
// Few rows a group: tiles of mp (16, 32, 64) rows, each tile's sum shared by cs (1, 2) CTAs.
// maps.a: boxes of mp rows (or a table's rows); maps.b: of 128 rows, or 64 x 64.
cudaError_t launch_group_few(int mp, int cs, bool b_major, const GroupMaps &maps, const GroupArgs &args, int grid,
                             cudaStream_t stream);
cudaError_t launch_group_sum(int bn, bool pair, int prec, const GroupMaps &maps, const GroupArgs &args,
                             int grid, cudaStream_t stream);
// (symmetric results: maj 0 or 3; others: maj 0 or 2; prec: kPrecAcc or kPrecSplit,
// the latter with bn 64 also on cs = 2 CTAs a tile)
cudaError_t launch_group_batch(int bn, bool pair, int maj, bool sym, int prec, int cs, const GroupMaps &maps,
                               const GroupArgs &args, int grid, cudaStream_t stream);

// W[i] = table[idx[i]] (M rows of K 16-bit elements, 16-byte aligned rows in both) for the rows that
// the groups' offsets name; zeros, and an error recorded, where idx[i] is not a row of the table.
cudaError_t launch_group_gather(const void *table, int32_t table_rows, int64_t lda, const int32_t *idx,
                                const int32_t *offsets, int32_t groups, int32_t M, int32_t K, void *W, int64_t ldw,
                                uint32_t *status, int sm_count, cudaStream_t stream);

// The stable order of M ids by value: offsets (groups + 1), order and rows (each M; rows
// may be NULL: order[i] / choices).  counts: `chunks` x (groups + 1) int32 (unused for one
// chunk).
constexpr int64_t kGroupRowsChunk = 16384;  // ids a thread block sorts, where there are chunks
constexpr int64_t kGroupRowsOne = 131072;   // up to this many, one launch does
cudaError_t launch_group_rows_sort(const int32_t *ids, int64_t M, int32_t groups, int32_t choices,
                                   int32_t *offsets, int32_t *order, int32_t *rows, int32_t *counts,
                                   int32_t chunks, cudaStream_t stream);

// Sums of squares of `count` matrices X (M x N of type kOut...), in `parts` parts each, to
// partial; and X scale / (sqrt(the parts' sum) + eps) as float16 Xs and, lo elements behind it, the rest.
int orthogonalize_parts(int64_t M, int64_t N);
cudaError_t launch_square_sums(const void *X, int64_t ldx, int64_t stride_x, int type, int32_t M, int32_t N,
                               int32_t count, float *partial, int parts, cudaStream_t stream);
cudaError_t launch_normalize(const void *X, int64_t ldx, int64_t stride_x, int type, int32_t M, int32_t N,
                             int32_t count, const float *partial, int parts, float scale, float eps,
                             uint16_t *Xs, int64_t lds, int64_t stride_s, int64_t lo, cudaStream_t stream);

// All steps on `count` small matrices in one launch, a matrix by `cluster` (1 or 8) thread blocks; s <= 64
// and l its sides, the shared memory of a block at most kSmallShared bytes.
constexpr size_t kSmallShared = 220 * 1024;
struct SmallArgs {
    const void *X;
    int64_t ldx, stride_x;
    int32_t type;
    void *Y;
    int64_t ldy, stride_y;
    int32_t out;
    int32_t s, l, tall;  // tall: X is l x s
    int32_t steps, cluster;
    float a, b, c, eps;
    int32_t lc, px, ps;  // (the launch's: columns of a block, pitches)
};
size_t orthogonalize_small_shared(int64_t s, int64_t l, int cluster);
cudaError_t launch_orthogonalize_small(SmallArgs a, int64_t count, cudaStream_t stream);

// Symmetric matrices P (s x s, float16, and, lo != 0, their low parts lo elements behind) from `parts`
// float32 matrices each, whose sums' elements on and below the diagonal are P's.
cudaError_t launch_join_parts(const float *Q, int64_t ldq, int64_t stride_q, int32_t parts, int32_t s, int32_t count,
                              uint16_t *P, int64_t ldp, int64_t stride_p, int64_t lo, cudaStream_t stream);

}  // namespace tcg
