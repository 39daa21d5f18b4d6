// launch.h -- host-side interface between the C ABI (api.cu) and the kernel
// launchers (launch_*.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

// Launch with programmatic dependent launch allowed (1) or not (0): a GEMM
// may then start its set-up while the previous kernel in the stream ends.
#ifndef TCG_PDL
#define TCG_PDL 1
#endif
// skinny kernel, FP4 B: whole waves of tiles go to CTAs whole (0: every tile shared)
#ifndef TCG_SKINNY_WHOLE
#define TCG_SKINNY_WHOLE 1
#endif

namespace tcg {

// Let `kfn` use `bytes` of dynamic shared memory, once per device (`done`: the
// devices that have it, one bit each, kept by the caller per kernel).
inline cudaError_t allow_smem(const void *kfn, uint32_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if ((done.load(std::memory_order_relaxed) & bit) != 0)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

struct GemmMaps {
    CUtensorMap a;    // A tiles, or the gather table (box of one row); FP4: A's codes
    CUtensorMap b;    // B tiles; FP4: B's codes
    CUtensorMap c;    // C boxes (float32), unused when C is not read
    CUtensorMap d;    // D boxes
    CUtensorMap sfa;  // FP4 operands: A's block scales (K/32 rows of M bytes)
    CUtensorMap sfb;  // FP4 operands: B's block scales (K/32 rows of N bytes)
};

// Tile kernel forms: 128 x bn tiles on single CTAs (mc = 1), or on clusters of
// mc = 4 CTAs sharing each A box by multicast; 256 x (nsub * bn) tiles on CTA
// pairs with tcgen05 cta_group::2.  grid counts CTAs.
int tile_stages(int bn, bool pair, int nsub, int mc);
// clusters (pairs, or groups of mc) of a form that can be resident at once on
// the current device; 0 if unknown
int tile_max_clusters(int bn, bool pair, int nsub, int mc);
// mode: 0 plain epilogue, 1 scattered rows, 2 reduce-add into D, 3 seeded
// accumulators (kModePlain ... kModeSeed)
cudaError_t launch_tile(int mode, int bn, bool pair, int nsub, int mc, const GemmMaps &maps,
                        const GemmArgs &args, int grid, cudaStream_t stream);

// The tile kernel with FP4 E2M1 operands and UE8M0 block scales (plain
// epilogue): single CTAs with 128 x bn tiles (bn 128 or 256), or CTA pairs with
// 256 x 256 tiles (pair = true, bn 256).  mx 1: codes packed two per byte,
// kind::mxf4; mx 2: codes in the 16U4_ALIGN16B image, kind::mxf8f6f4.
// maps.a / maps.b: the codes (128-byte boxes of 128 / bn rows -- pairs: bn / 2
// -- with 128-byte swizzle); maps.sfa / maps.sfb: the scales (uint8 boxes of
// 128 / bn columns by K_stage / 32 rows).  tile_mx_kstage: K elements per
// stage; tile_mx_max_pairs: pairs that can be resident at once (0 if unknown).
int tile_mx_stages(int mx, int bn, bool pair);
int tile_mx_kstage(int mx);
int tile_mx_max_pairs(int mx);
inline int tile_max_pairs_or(int mx, int fallback)
{
    const int r = tile_mx_max_pairs(mx);
    return r > 0 ? r : fallback;
}
cudaError_t launch_tile_mx(int mx, int bn, bool pair, const GemmMaps &maps, const GemmArgs &args,
                           int grid, cudaStream_t stream);

// Gated form (D = act(A Bg^T) * (A Bu^T)): single CTAs with 128 x bn accumulator
// tiles (bn 64, 128, 256), or CTA pairs with 256 x 256 ones; D tiles are bn / 2
// wide.  maps.b / two.b2: Bg / Bu in boxes of bn / 2 rows; maps.d, two.d2,
// two.d3: D, G, U.  The mx form takes packed FP4 codes (maps.sfa, maps.sfb,
// two.sfb2: scales of A, Bg and Bu; single CTAs, bn 128 or 256).  rows: D, or
// a kept G or U, has no descriptor (rows not whole 16 bytes apart).
cudaError_t launch_tile_gated(int bn, bool pair, bool rows, const GemmMaps &maps, const TileMapsTwo &two,
                              const GemmArgs &args, int grid, cudaStream_t stream);
int tile_gated_mx_stages(int bn);
cudaError_t launch_tile_gated_rows(int bn, bool pair, const GemmMaps &maps, const TileMapsTwo &two,
                                   const GemmArgs &args, int grid, cudaStream_t stream);
cudaError_t launch_tile_gated_mx(int bn, bool rows, const GemmMaps &maps, const TileMapsTwo &two,
                                 const GemmArgs &args, int grid, cudaStream_t stream);

// Operands stored K x M (maj bit 0) or K x N (bit 1), boxes of 64 columns x 64 K
// rows; two: the second source along K or M.  Forms: single CTAs (bn 64, 128,
// 256) and CTA pairs (256 x 256, or 256 x 512 with nsub = 2).
cudaError_t launch_tile_major(int maj, int bn, bool pair, int nsub, const GemmMaps &maps,
                              const TileMapsTwo &two, const GemmArgs &args, int grid,
                              cudaStream_t stream);

// D[i][j] = fma.rn(alpha, sum_p W[p part_rows + i][j], beta C[i][j]) for i < M, j <
// N, the parts p < parts added in order: W float32, ldw apart; D of type out.
cudaError_t launch_add_parts(const float *W, int64_t ldw, int64_t part_rows, int32_t parts, const float *C,
                             int64_t ldc, void *D, int64_t ldd, int out, float alpha, float beta, int32_t M,
                             int32_t N, cudaStream_t stream);

// dG = dD * U * act'(G), dU = dD * act(G) over M x N, 16-bit (bf16 or f16)
// matrices; dG may be G and dU may be U.
cudaError_t launch_gated_slope(const void *dD, int64_t lddd, const void *G, int64_t ldg,
                               const void *U, int64_t ldu, void *dG, int64_t lddg, void *dU,
                               int64_t lddu, int32_t M, int32_t N, bool bf16, int32_t act,
                               cudaStream_t stream);

// X (M x K; type kOutF32 / kOutBF16 / kOutF16) -> E2M1 codes Q (rows of K / 2
// bytes) and UE8M0 scales S (K / 32 rows of M bytes); Y (NULL: none): the
// values they stand for, in X's type.
cudaError_t launch_quantize_e2m1(const void *X, int64_t ldx, int type, uint8_t *Q, int64_t ldq,
                                 uint8_t *S, int64_t lds, void *Y, int64_t ldy, int32_t M, int32_t K,
                                 cudaStream_t stream);

// Warp-level tiny-GEMM kernel: one 16 x 8 block of D per warp.
int tiny_warps_per_cta();
cudaError_t launch_tiny(const void *A, int64_t lda, const void *B, int64_t ldb,
                        const GemmArgs &args, int grid, cudaStream_t stream);

int skinny_stages(int mp);
// The same kernel with FP4 B: maps.b = the codes (uint8, 128-byte boxes of
// 128 rows, 128-byte swizzle), maps.c = the block scales (uint8, 128 x 8
// boxes); bf16 A.
int skinny_w4_stages(int mp);
int skinny_w4_kstage();  // K elements per stage (and per stream-K unit) of the FP4 form
// FP4 codes (N rows of K/2 bytes, ldq apart) and scales (K/32 rows of N bytes,
// lds apart) -> bf16 N x K rows, ldo elements apart; K a multiple of 32.
cudaError_t launch_dequant_fp4(const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                               int64_t lds, int32_t N, int32_t K, uint16_t *out, int64_t ldo,
                               cudaStream_t stream);
cudaError_t launch_skinny_w4(int mp, const GemmMaps &maps, const GemmArgs &args, int grid,
                             cudaStream_t stream);
int skinny_kstage();  // K elements per pipeline stage (and per stream-K unit)
// Both operands FP4 (packed codes, UE8M0 scales per 32), M <= 64: maps.a / maps.b
// the codes of A / B (uint8, 128-byte boxes of mp / 128 rows, 128-byte
// swizzle), maps.c / maps.sfa the scales of B / A (uint8 boxes of 128 / mp
// columns by K_stage / 32 rows); block-scaled MMA kind::mxf4.
int skinny_mx_kstage();
int skinny_mx_stages(int mp);
cudaError_t launch_skinny_mx(int mp, const GemmMaps &maps, const GemmArgs &args, int grid,
                             cudaStream_t stream);
cudaError_t launch_skinny(int mp, const GemmMaps &maps, const GemmArgs &args, int grid,
                          cudaStream_t stream);
// The gated form of the 16-bit and (mx) both-FP4 kernels: maps.b / two.b2: Bg / Bu
// in boxes of 64 rows; (mx) maps.c / two.sfb2: their scales in boxes of 64
// columns, maps.sfa: A's.  Tiles are 64 columns of D.
cudaError_t launch_skinny_gated(int mp, bool mx, const GemmMaps &maps, const TileMapsTwo &two,
                                const GemmArgs &args, int grid, cudaStream_t stream);
// B stored K x N (boxes of 64 columns x 64 K rows); two.a2, two.b2: the second
// source along K (args.k2_block), if any.
cudaError_t launch_skinny_trans(int mp, const GemmMaps &maps, const TileMapsTwo &two, const GemmArgs &args,
                                int grid, cudaStream_t stream);

// Stream-K split of the skinny kernel: the CTA that owns linear k-block x
// when W blocks are shared by G CTAs as [W g / G, W (g+1) / G).
inline int64_t skinny_owner_host(int64_t x, int64_t W, int64_t G) { return ((x + 1) * G - 1) / W; }

// Tiles of the skinny kernel shared block by block when T tiles run on G
// CTAs.  bf16 / f16 B: all of them.  FP4 B: the T mod G left over after
// whole waves (each CTA takes floor(T / G) tiles whole), plus one wave more
// when fewer than G / 4 are left over, so that no tile is cut into more than
// about five parts.  The shared tiles are tiles 0 .. S-1; T - S is always a
// multiple of G.
inline int64_t skinny_sk_tiles(int64_t T, int64_t G, bool w4)
{
    if (!w4 || !TCG_SKINNY_WHOLE)
        return T;
    const int64_t waves = T / G;
    int64_t S = T - waves * G;
    if (S != 0 && waves > 0 && 4 * S < G)
        S += G;
    return S;
}

// Most CTAs that contribute to one shared tile (workspace slots per tile)
// when `tiles` tiles of nkb K blocks are shared by G CTAs.
inline int32_t skinny_max_parts_of(int64_t tiles, int64_t nkb, int64_t G)
{
    if (tiles == 0)
        return 1;
    const int64_t W = tiles * nkb;
    if (tiles > 65536) {
        // shares are at least W / G blocks long, so a tile of nkb blocks holds at
        // most (nkb - 1) / (W / G) + 1 share boundaries
        const int64_t shortest = W / G;
        return static_cast<int32_t>((nkb - 1) / shortest + 2);
    }
    int64_t most = 1;
    for (int64_t t = 0; t < tiles; ++t) {
        const int64_t parts = skinny_owner_host((t + 1) * nkb - 1, W, G) -
                              skinny_owner_host(t * nkb, W, G) + 1;
        most = parts > most ? parts : most;
    }
    return static_cast<int32_t>(most);
}

// The same, remembering the last few answers: two divisions a tile are microseconds of
// a call whose kernel takes ten, and a model's calls come in a few sizes.
inline int32_t skinny_max_parts(int64_t tiles, int64_t nkb, int64_t G)
{
    struct Answer {
        int64_t tiles, nkb, G;
        int32_t parts;
    };
    static thread_local Answer last[16] = {};
    Answer &a = last[static_cast<uint64_t>(tiles * 31 + nkb * 7 + G) % 16];
    if (a.parts == 0 || a.tiles != tiles || a.nkb != nkb || a.G != G)
        a = Answer{tiles, nkb, G, skinny_max_parts_of(tiles, nkb, G)};
    return a.parts;
}

}  // namespace tcg
