// kernel_group.cuh -- persistent warp-specialised tcgen05 products over groups.
//
//   KIND_ROWS   D[i] = alpha A[i] B_g^T for the rows i of group g: the rows of A and D
//               are grouped by offsets that only the device knows, B is a stack.
//               Tiles are cut group by group: a group of r rows has ceil(r / TILE_M)
//               block rows, so a tile never mixes groups.  Its boxes of A may reach
//               into the next group's rows (loaded, multiplied, never stored).
//   KIND_SUM    D_g = alpha A_g^T B_g over the rows of group g (both operands stored
//               with the sum's index outermost): every group has the same tiles, and
//               its own number of K blocks.  The last block of a group ends inside a
//               box, whose other rows belong to the next group and may hold anything
//               (also NaN): a warp of its own zeroes them in shared memory before the
//               MMAs read the stage.
//   KIND_BATCH  D_g = alpha A_g B_g^T + beta C_g for a stack of equal sizes, in either
//               storage, C in 16 bits.  SYM: D_g is known to be symmetric (A A^T, or
//               the square of a symmetric matrix): only the tiles that reach the
//               diagonal or lie below it are computed, and each is stored twice.  A long sum of
//               few tiles can be cut into parts, each a tile of its own into a matrix of its own.
//
// Sums.  The tensor cores add each K step of 16 to a float32 accumulator and drop what
// does not fit, so the error of a long sum grows with its steps.  How much of that is let
// stand is a template parameter:
//   PREC_ACC    one accumulator for the whole sum (results of 16 bits).
//   PREC_SUMS   the accumulator is emptied every eight (PREC_SPLIT: four) K blocks into float32
//               registers, which round to nearest (float32 results, relative error of sums
//               over 1024 1.2e-6 -> 6e-7).
//   PREC_SPLIT  as PREC_SUMS, and both operands are pairs of float16 matrices, a high part and
//               the rest: high x high + high x low + low x high, 22 bits of each operand.  Twelve
//               MMAs a K block: two issuing warps, half of its K steps each (a lone thread's
//               ~117 cycles an MMA took longer than loading the block).  CS = 2: the CTAs of a
//               cluster share a tile's sum, half of its K blocks each, where the tiles alone
//               leave SMs idle; each finishes half of the tile's columns, with the other's sums
//               of them through its shared memory.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer (tcgen05.mma by one thread; 64 columns wide tiles have
// two, whose K blocks of 24 KB come faster than a thread's four MMAs go: a symmetric 1024 x 1024 over 2816
// 17.7 -> 16.0 us), then four or eight epilogue warps, (KIND_SUM) one that zeroes.  Two TMEM accumulators: the epilogue of one tile
// runs beside the next tile's MMAs.  PAIR: the roles on a CTA pair and one 256 x 256 tile
// (tcgen05 cta_group::2), each CTA loading its 128 rows of A and its half of B.  The
// protocol is the tile kernel's (kernel_tile.cuh).  Every wait is bounded.
//
// Bounds and figures.  KIND_ROWS and KIND_SUM of long sums are bound by the tensor cores under
// the power cap (16384 rows in eight uneven groups, 14336 x 4096 bf16: 1.19 to 1.20 ms forward,
// 1.25 to 1.26 the input's gradient, 1.20 to 1.22 the weights'; 1.5 to 1.6 PFLOP/s; tensor pipe active 90, 87
// and 82 % of cycles), of short ones by the results' way out (eight groups
// of 128 rows: 940 MB of bf16 gradients 224 us, float32 1.9 GB 290).  KIND_BATCH likewise: 4096 x
// 4096 x 14336, half of a symmetric product 148 us, the update 290 (1.66 and 1.65 PFLOP/s); where
// the tiles are few, by the rate L2 feeds an SM (at most 63 bytes a clock) and whole waves of tiles
// (operands in two parts, the update of 2816 x 1024: 16 K blocks of 64 KB take 8.5 us, two waves and the
// last epilogue 23).  Rows of D that are not 16 bytes apart go out as words (16 x 1000 x 1367 from 100
// rows each 36 us, 1368 20).
//
// Why tiles from device offsets and not from a list: a list is a second kernel before
// every call.  Each warp that needs coordinates reads the offsets (at most 1024 groups,
// 4 KB) once, keeps a prefix sum of block rows in its lanes, and finds a tile's group with
// two ballots where it is not the last one's.
#pragma once

#include "common.cuh"

namespace tcg {

enum : int { kKindRows = 0, kKindSum = 1, kKindBatch = 2 };
enum : int { kPrecAcc = 0, kPrecSums = 1, kPrecSplit = 2 };

struct GroupMaps {
    CUtensorMap a, b, d;           // stacks 3-D (inner, rows, group); one matrix's rows 2-D (D's always 3-D)
    CUtensorMap a_lo, b_lo;        // the operands' low parts (PREC_SPLIT)
    CUtensorMap c, c_lo, d_lo;     // C and its low part (where it comes by TMA), D's low part: boxes of 32 columns
};

struct GroupArgs {
    int32_t groups;
    const int32_t *offsets;  // groups + 1 row numbers (KIND_ROWS, KIND_SUM)
    int32_t rows;            // rows the offsets may name (of A and D, or the sum's)
    int32_t M, N, K;         // of one group's product (KIND_ROWS: M unused; KIND_SUM: K unused)
    int32_t num_m_blocks, num_n_blocks;
    int32_t group_m;         // tile order: block rows visited side by side
    float alpha, beta;
    int32_t out_kind, ab_bf16;
    const int32_t *idx;      // KIND_ROWS: row i of A is row idx[i] of a table (NULL: row i)
    int32_t table_rows;
    int32_t gather;          // idx is followed here (0: A is those rows already)
    int32_t d_tma;           // D goes out through TMA where a box is whole
    int32_t d_vec;           // D's rows are whole 16 bytes apart, its base 16-byte aligned
    void *D;
    int64_t ldd, stride_d;   // elements between rows, and between groups
    int32_t n_out;           // columns of D that may be written (N, or a workspace's padding too)
    const uint16_t *C;       // KIND_BATCH: f16, 16-byte aligned rows (NULL: none)
    int64_t ldc, stride_c;
    int64_t c_lo, d_lo;      // KIND_BATCH: elements from C, D to their low parts (0: none)
    int32_t parts, part_blocks;  // SYM: a tile's sum in so many parts of so many K blocks, each a matrix of D
    int32_t loads;           // there is something to multiply (K > 0; KIND_SUM: rows > 0)
    uint32_t extra_tx;
    uint32_t *status;
    uint64_t timeout_ns;
};

template <int BN_, int STAGES_, bool PAIR_, int KIND_, int PREC_, int CS_ = 1>
struct GroupCfg {
    static constexpr int CS = CS_;
    // MMA issuers: two where one thread's MMAs take longer than the loads
    static constexpr int ISS = PREC_ == kPrecSplit || (BN_ == 64 && KIND_ != kKindSum) ? 2 : 1;
    static constexpr int PARTS = PREC_ == kPrecSplit ? 2 : 1;  // boxes of an operand in a stage
    static constexpr int CHUNK = PREC_ == kPrecAcc ? 0 : (PREC_ == kPrecSums ? 8 : 4);  // K blocks an accumulator takes (0: all)
    static constexpr bool PAIR = PAIR_;
    static constexpr int BM = 128, BN = BN_, BK = 64, STAGES = STAGES_;
    static constexpr int TILE_M = PAIR ? 256 : 128;
    static constexpr int BN_LOCAL = PAIR ? BN / 2 : BN;
    static constexpr uint32_t A_BYTES = BM * 128u, B_BYTES = BN_LOCAL * 128u;
    static constexpr uint32_t STAGE_BYTES = PARTS * (A_BYTES + B_BYTES);
    static constexpr uint32_t OFF_A = 0, OFF_B = STAGES * PARTS * A_BYTES;
    static constexpr uint32_t EPI_BUF = 32 * 128;  // 32 rows x 128 bytes
    static constexpr uint32_t OFF_EPI = STAGES * STAGE_BYTES;
    // Epilogue groups of four warps: two, half of the columns each, but for the narrowest
    // tiles.  (A warp's chain of TMEM load, conversion, shared image and store is all latency:
    // about 1 us for 64 columns.)  Four where 256 columns' sums stay in registers.
    static constexpr int EPI_GROUPS = BN >= 128 ? (BN == 256 && PREC_ != kPrecAcc ? 4 : 2) : 1;
    static constexpr int COLS = BN / EPI_GROUPS;
    // C by TMA, into the buffers that D leaves from: two a warp then, and a stage less
    static constexpr bool C_TMA = KIND_ == kKindBatch && PREC_ == kPrecAcc;
    static constexpr int EPI_BUFS = EPI_GROUPS == 1 || C_TMA ? 2 : 1;
    // (CS = 2) the other CTA's sums of a warp's rows, half of the columns
    static constexpr uint32_t RED_BYTES = CS == 2 ? 32u * COLS / 2 * 4u : 0u;
    static constexpr uint32_t OFF_RED = OFF_EPI + 4 * EPI_GROUPS * EPI_BUFS * EPI_BUF;
    static constexpr uint32_t OFF_BAR = OFF_RED + 4 * RED_BYTES;
    static constexpr uint32_t NUM_BARS = 3 * STAGES + 4 + (C_TMA ? 8 * EPI_GROUPS : 0) + (CS == 2 ? 8 : 0);
    static_assert(CS == 1 || (CS == 2 && !PAIR && PREC_ == kPrecSplit && EPI_GROUPS == 1), "shared sums");
    static constexpr int LAST_WARP = 2 + 4 * EPI_GROUPS;  // zeroes (KIND_SUM), or the second MMA issuer
    static constexpr int THREADS = 32 * (LAST_WARP + (KIND_ == kKindSum || ISS == 2 ? 1 : 0));
    static constexpr uint32_t TMEM_COLS = 2 * BN * ISS;
    static constexpr uint32_t SMEM_ALLOC = OFF_BAR + NUM_BARS * 8 + 16 + 1024;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(BN == 64 || BN == 128 || BN == 256, "tile width");
    static_assert(!PAIR || BN == 256, "pairs: 256 x 256");
    static_assert(PREC_ != kPrecSplit || (BN <= 128 && !PAIR), "a row's sums in a thread's registers");
};

// The groups' rows, as one warp knows them.  Lane l keeps the block rows of groups l per
// .. l per + per - 1.
template <int TILE_M>
struct GroupRows {
    const int32_t *off;
    int32_t groups, rows, per;
    int32_t lo[2], hi[2];  // rows of this lane's groups (up to two: with 64 groups find() loads nothing)
    int32_t first, mine;   // block rows before this lane's groups, and of them
    int32_t total;        // block rows of all groups (0 where the offsets are not valid)
    bool ok;
    // the group found last: its rows, its first block row and their number
    int32_t g_last, lo_last, hi_last, base_last, blocks_last;

    // (L2: the offsets may be the work of the kernel before, beside which this one began)
    __device__ __forceinline__ int32_t at(int32_t g) const { return __ldcg(off + g); }

    // (whole warp; offsets that fall, or leave [0, rows], make every group empty)
    __device__ __forceinline__ void init(const int32_t *offsets, int32_t n, int32_t limit, uint32_t lane)
    {
        off = offsets;
        groups = n;
        rows = limit;
        per = (n + 31) / 32;
        mine = 0;
        bool good = true;
        const int32_t g0 = static_cast<int32_t>(lane) * per;
        auto count = [&](int32_t l, int32_t h) {
            good = good && l >= 0 && l <= h && h <= limit;
            mine += good ? (h - l + TILE_M - 1) / TILE_M : 0;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool there = i < per && g0 + i < n;
            lo[i] = there ? at(g0 + i) : 0;
            hi[i] = there ? at(g0 + i + 1) : 0;
        }
        count(lo[0], hi[0]);
        count(lo[1], hi[1]);
        for (int32_t g = g0 + 2; g < min(g0 + per, n); ++g)
            count(at(g), at(g + 1));
        ok = __all_sync(0xffffffffu, good);
        int32_t sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int32_t x = __shfl_up_sync(0xffffffffu, sum, d);
            if (static_cast<int>(lane) >= d)
                sum += x;
        }
        first = sum - mine;
        total = ok ? __shfl_sync(0xffffffffu, sum, 31) : 0;
        base_last = blocks_last = 0;
        g_last = -1;
    }

    // rows [lo_last, hi_last) of group g
    __device__ __forceinline__ void load(int32_t g)
    {
        if (g == g_last)
            return;
        g_last = g;
        lo_last = ok ? at(g) : 0;
        hi_last = ok ? at(g + 1) : 0;
    }

    // (whole warp) the group of block row q < total
    __device__ __forceinline__ void find(int32_t q, uint32_t lane)
    {
        if (q >= base_last && q < base_last + blocks_last)
            return;
        const int chunk = __ffs(__ballot_sync(0xffffffffu, q >= first && q < first + mine)) - 1;
        if (per <= 2) {
            const int32_t l0 = __shfl_sync(0xffffffffu, lo[0], chunk), h0 = __shfl_sync(0xffffffffu, hi[0], chunk);
            const int32_t l1 = __shfl_sync(0xffffffffu, lo[1], chunk), h1 = __shfl_sync(0xffffffffu, hi[1], chunk);
            const int32_t start = __shfl_sync(0xffffffffu, first, chunk), b0 = (h0 - l0 + TILE_M - 1) / TILE_M;
            const bool second = q >= start + b0;
            g_last = chunk * per + (second ? 1 : 0);
            lo_last = second ? l1 : l0;
            hi_last = second ? h1 : h0;
            base_last = second ? start + b0 : start;
            blocks_last = (hi_last - lo_last + TILE_M - 1) / TILE_M;
            return;
        }
        const int32_t g = chunk * per + static_cast<int32_t>(lane);
        int32_t l = 0, h = 0;
        if (static_cast<int32_t>(lane) < per && g < groups) {
            l = at(g);
            h = at(g + 1);
        }
        const int32_t blocks = (h - l + TILE_M - 1) / TILE_M;
        int32_t sum = blocks;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int32_t x = __shfl_up_sync(0xffffffffu, sum, d);
            if (static_cast<int>(lane) >= d)
                sum += x;
        }
        const int32_t start = __shfl_sync(0xffffffffu, first, chunk) + sum - blocks;
        const int who = __ffs(__ballot_sync(0xffffffffu, q >= start && q < start + blocks)) - 1;
        g_last = chunk * per + who;
        lo_last = __shfl_sync(0xffffffffu, l, who);
        hi_last = __shfl_sync(0xffffffffu, h, who);
        base_last = __shfl_sync(0xffffffffu, start, who);
        blocks_last = __shfl_sync(0xffffffffu, blocks, who);
    }
};

template <bool V>
struct Bool {
    static constexpr bool value = V;
};

// One tile's place.
struct GroupTile {
    int32_t g;          // group
    int32_t row0, end;  // its first row (PAIR: of the pair's tile) and the end of the rows it may store
    int32_t n0;         // first column
    int32_t gd;         // matrix of D
    int32_t k0;         // first row of the sum (KIND_SUM, SYM)
    bool mirror;        // SYM: below the diagonal, stored a second time
};

// Byte offset of 16-byte chunk `chunk` of row `row` in an image of 128-byte rows (128-byte
// swizzle).
__device__ __forceinline__ uint32_t swz128(uint32_t row, uint32_t chunk)
{
    return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// The same for rows of 64 bytes (64-byte swizzle).
__device__ __forceinline__ uint32_t swz64(uint32_t row, uint32_t chunk)
{
    return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}

// Rows [0, nrows) of an image of 32 rows of 128 (64) bytes to D at (row0, col0), columns below
// N.  vec: D's rows are whole 16 bytes apart: pieces of 16 bytes, four or eight rows a pass, each
// row's bytes together.  Otherwise a row a pass, lanes along the columns: float32 elements, or 16-bit
// ones in pairs that begin where D's row has a 4-byte boundary.  (Pieces of 16 bytes taken apart
// there: 16 x 1000 x 1367 of 100 rows each 85 us.)
__device__ __forceinline__ void store_image_rows(uint32_t buf, uint32_t lane, bool narrow, int32_t nrows,
                                                 uint32_t esize, void *D, int64_t ldd, int32_t row0,
                                                 int32_t col0, int32_t N, bool vec)
{
    if (vec) {
        const uint32_t pieces = narrow ? 4u : 8u;
        const uint32_t chunk = lane % pieces;
        const int32_t per = static_cast<int32_t>(16u / esize);
        const int32_t col = col0 + static_cast<int32_t>(chunk) * per;
        for (uint32_t r = lane / pieces; static_cast<int32_t>(r) < nrows; r += 32u / pieces) {
            uint32_t w[4];
            ld_shared_v4(buf + (narrow ? swz64(r, chunk) : swz128(r, chunk)), w[0], w[1], w[2], w[3]);
            uint8_t *p = static_cast<uint8_t *>(D) + ((static_cast<int64_t>(row0) + r) * ldd + col) * esize;
            if (col + per <= N) {
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (esize == 4u) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < N)
                        reinterpret_cast<uint32_t *>(p)[i] = w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i < N)
                        reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
            }
        }
        return;
    }
    // (four rows at once, so that their loads, shuffles and stores overlap)
    const uint32_t words = narrow ? 16u : 32u;
    const uint32_t in_row = lane % words;
    uint8_t *p = static_cast<uint8_t *>(D) + (static_cast<int64_t>(row0) * ldd + col0) * esize;
    const int64_t pitch = ldd * esize;
    const int32_t left = N - col0;  // columns of the row, at most
    for (int32_t r0 = 0; r0 < nrows; r0 += 4, p += 4 * pitch) {
        uint32_t w[4];
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i) {
            const uint32_t r = static_cast<uint32_t>(r0) + i;
            w[i] = ld_shared_u32(buf + (narrow ? swz64(r, in_row / 4u) : swz128(r, in_row / 4u)) + in_row % 4u * 4u);
        }
        if (esize == 4u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st_global_u32_if(r0 + i < nrows && static_cast<int32_t>(lane) < left,
                                 reinterpret_cast<uint32_t *>(p + i * pitch) + lane, w[i]);
            continue;
        }
        const int32_t c = 2 * static_cast<int32_t>(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t *h = reinterpret_cast<uint16_t *>(p + i * pitch);
            const bool odd = (reinterpret_cast<uintptr_t>(h) & 2u) != 0;
            const uint32_t next = __shfl_down_sync(0xffffffffu, w[i], 1);
            const uint32_t pair = odd ? (w[i] >> 16) | (next << 16) : w[i];
            const int32_t e = c + (odd ? 1 : 0);  // the pair's first element
            const bool row = r0 + i < nrows && lane < words;
            const bool both = e + 1 < left && !(odd && lane == words - 1u);
            st_global_u32_if(row && both, h + e, pair);
            st_global_u16_if(row && !both && e < left, h + e, pair);
            st_global_u16_if(row && odd && lane == 0u && left > 0, h, w[i]);
        }
    }
}

template <int BN, int STAGES, bool PAIR, int KIND, int MAJ, bool SYM, int PREC, int CS = 1>
__global__ void __launch_bounds__(GroupCfg<BN, STAGES, PAIR, KIND, PREC, CS>::THREADS, 1)
    group_gemm_kernel(const __grid_constant__ GroupMaps maps, const GroupArgs args)
{
    using Cfg = GroupCfg<BN, STAGES, PAIR, KIND, PREC, CS>;
    constexpr int CL = PAIR ? 2 : CS;  // CTAs of a cluster
    constexpr bool kSums = PREC != kPrecAcc, kSplit = PREC == kPrecSplit;
    constexpr bool kRows = KIND == kKindRows, kSum = KIND == kKindSum, kBatch = KIND == kKindBatch;
    constexpr bool kMnA = (MAJ & 1) != 0, kMnB = (MAJ & 2) != 0;
    constexpr int TM = Cfg::TILE_M;
    static_assert(!SYM || kBatch, "symmetric results: equal sizes");
    static_assert(!kSplit || kBatch, "operands in two parts: equal sizes");
    static_assert(!kSum || MAJ == 3, "a sum over rows: both operands stored with them outermost");
    static_assert(!kRows || !kMnA, "grouped rows are stored row by row");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;

    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x / 32u, 0);
    const uint32_t lane = threadIdx.x % 32u;

    const uint32_t bar0 = base + Cfg::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    // (KIND_SUM) the boxes of a group's last, partial block have landed in this CTA
    auto tail_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (3 * STAGES + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (3 * STAGES + 2 + b); };
    // (CS = 2) the other CTA's sums of warp q's rows are there / have been read (arrives at
    // the writer)
    auto redf_bar = [&](uint32_t q) { return bar0 + 8u * (3 * STAGES + 4 + q); };
    auto rede_bar = [&](uint32_t q) { return bar0 + 8u * (3 * STAGES + 8 + q); };
    // (C by TMA) epilogue warp w's buffer j holds its piece of C
    auto c_bar = [&](uint32_t w, uint32_t j) { return bar0 + 8u * (3 * STAGES + 4 + 2 * w + j); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bar0 - raw) + 8 * Cfg::NUM_BARS);
    volatile uint32_t *abort_flag = tmem_slot + 1;

    const uint32_t role = PAIR ? cluster_ctarank() : 0u;
    const bool leader = role == 0u;
    const uint32_t share = CS == 2 ? cluster_ctarank() : 0u;  // which part of a shared sum
    const int32_t cta_set = static_cast<int32_t>(blockIdx.x) / CL;
    const int32_t cta_sets = static_cast<int32_t>(gridDim.x) / CL;
    auto lead = [&](uint32_t bar) { return PAIR ? mapa_shared(bar, 0u) : bar; };

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // (KIND_SUM on pairs: two arrivals, since a partial block is handed over by both
            // CTAs' zeroing warps; the leader's producer arrives twice for a whole one)
            mbar_init(full_bar(s), kSum && PAIR ? 2 : 1);
            mbar_init(empty_bar(s), Cfg::ISS);
            mbar_init(tail_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), Cfg::ISS);
            mbar_init(acce_bar(b), (PAIR ? 8 : 4) * Cfg::EPI_GROUPS);
        }
        if (CS == 2)
            for (uint32_t q = 0; q < 4u; ++q) {
                mbar_init(redf_bar(q), 1);
                mbar_init(rede_bar(q), 1);
            }
        if (Cfg::C_TMA)
            for (uint32_t w = 0; w < 4u * Cfg::EPI_GROUPS; ++w)
                for (uint32_t j = 0; j < 2u; ++j)
                    mbar_init(c_bar(w, j), 1);
        *abort_flag = 0u;
        fence_mbar_init();
        fence_proxy_async_smem();
        if (args.loads) {
            tma_prefetch_desc(&maps.a);
            tma_prefetch_desc(&maps.b);
        }
        if (args.d_tma)
            tma_prefetch_desc(&maps.d);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), Cfg::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
            tmem_relinquish();
        }
    }
    // (the offsets come while the barriers and the tensor memory are set up; without any, that is
    // done before the kernel before ends: between CTAs 500 clocks of every launch)
    GroupRows<TM> gr;
    if constexpr (!kBatch) {
        grid_dependency_wait();
        gr.init(args.offsets, args.groups, args.rows, lane);
    }
    tc_fence_before_sync();
    if (CL > 1)
        cluster_sync_all();
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    if constexpr (kBatch)
        grid_dependency_wait();
    if (threadIdx.x == 0)
        grid_launch_dependents();

    // ---- the tiles, as each warp finds them
    int32_t num_tiles;
    if constexpr (kBatch) {
        const int32_t per = SYM ? (TM / BN) * (args.num_m_blocks * (args.num_m_blocks + 1) / 2)
                                : args.num_m_blocks * args.num_n_blocks;
        num_tiles = args.groups * per * (SYM ? args.parts : 1);
    } else {
        if (!gr.ok && blockIdx.x == 0 && threadIdx.x == 0)
            record_error(args.status, kStatusIndex, 0);
        if constexpr (kRows)
            num_tiles = gr.total * args.num_n_blocks;
        else
            num_tiles = args.groups * args.num_m_blocks * args.num_n_blocks;
    }
    // (KIND_ROWS: by the whole warp)
    auto locate = [&](int32_t t) {
        GroupTile p{};
        int32_t blocks = args.num_m_blocks, r = t;
        if constexpr (kRows) {
            gr.find(t / args.num_n_blocks, lane);
            p.g = gr.g_last;
            blocks = gr.blocks_last;
            r = t - gr.base_last * args.num_n_blocks;
            p.row0 = gr.lo_last;
            p.end = gr.hi_last;
        } else if constexpr (SYM) {
            // block row mb of a matrix has the TM / BN (mb + 1) tiles up to the diagonal
            constexpr int32_t q = TM / BN;
            const int32_t per = q * (blocks * (blocks + 1) / 2);
            int32_t part = 0;
            if (args.parts > 1) {
                part = t % args.parts;
                t /= args.parts;
            }
            p.g = t / per;
            p.gd = p.g * args.parts + part;
            p.k0 = part * args.part_blocks * Cfg::BK;
            r = t - p.g * per;
            const int32_t u = r / q;
            int32_t mb = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(u) + 1.0f) - 1.0f) * 0.5f);
            while (mb * (mb + 1) / 2 > u)
                --mb;
            while ((mb + 1) * (mb + 2) / 2 <= u)
                ++mb;
            const int32_t nb = r - q * (mb * (mb + 1) / 2);
            p.row0 = mb * TM;
            p.n0 = nb * BN;
            p.end = args.M;
            p.mirror = nb / q != mb && args.parts == 1;
            return p;
        } else {
            const int32_t per = blocks * args.num_n_blocks;
            p.g = p.gd = t / per;
            r = t - p.g * per;
            p.end = args.M;
            if constexpr (kSum) {
                gr.load(p.g);
                p.k0 = gr.lo_last;
            }
        }
        const int32_t per_super = args.group_m * args.num_n_blocks;
        const int32_t first_m = r / per_super * args.group_m;
        const int32_t rows = min(blocks - first_m, args.group_m);
        const int32_t rr = r % per_super;
        p.row0 += (first_m + rr % rows) * TM;
        p.n0 = rr / rows * BN;
        return p;
    };
    const int32_t k_blocks = (args.K + Cfg::BK - 1) / Cfg::BK;
    // (CS = 2) this CTA's K blocks of a tile: from kb_first, kb_mine of them (not 0: sums of fewer
    // than eight blocks are not shared)
    const int32_t kb_first = CS == 2 ? static_cast<int32_t>(share) * (k_blocks / 2) : 0;
    const int32_t kb_mine = CS == 2 ? (share == 0u ? k_blocks / 2 : k_blocks - k_blocks / 2) : k_blocks;
    // (KIND_SUM) A partial block is loaded this many blocks before the end of its tile and
    // multiplied at the end, so that its zeros are there in time: loaded last, it held up
    // every tile (four groups of 1025 rows, 4096 x 4096: 101.8 us against 87 of 1024).
    constexpr int32_t kEarly = 3;
    static_assert(!kSum || STAGES > kEarly, "the blocks after a partial one fit beside it");
    // K blocks of tile t (KIND_SUM: of its group) that this CTA multiplies
    auto blocks_of = [&](int32_t t, int32_t &rem) -> int32_t {
        rem = 0;
        if constexpr (CS == 2)
            return kb_mine;
        if constexpr (kSum) {
            gr.load(t / (args.num_m_blocks * args.num_n_blocks));
            const int32_t n = gr.hi_last - gr.lo_last;
            rem = n % Cfg::BK;
            return (n + Cfg::BK - 1) / Cfg::BK;
        }
        if (SYM && args.parts > 1)
            return min(args.part_blocks, k_blocks - t % args.parts * args.part_blocks);
        return k_blocks;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int s = 0;
        uint32_t ph = 0;
        int pending = 0;
        [[maybe_unused]] uint32_t tails = 0, tail_ph = 0;  // (bit per stage) last use partial; parity of tail_bar
        bool first = true, alive = true;
        for (int32_t t = cta_set; t < num_tiles && alive; t += cta_sets) {
            const GroupTile p = locate(t);
            int32_t rem;
            const int32_t nkb = blocks_of(t, rem);
            const int32_t m0 = p.row0 + static_cast<int32_t>(role) * Cfg::BM;
            const int32_t n0 = p.n0 + static_cast<int32_t>(role) * Cfg::BN_LOCAL;
            const int32_t ga = kBatch ? p.g : 0, gb = kSum ? 0 : p.g;
            int32_t rows[4] = {0, 0, 0, 0};
            if (kRows && args.gather) {
                // lane l fetches rows 4 l .. 4 l + 3, four per gather4; rows past the group's,
                // and those whose index is not a row of the table, fetch row 0
                int32_t v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {  // (at once: each is a round trip to L2)
                    const int32_t m = m0 + 4 * static_cast<int32_t>(lane) + r;
                    v[r] = m < p.end ? __ldcg(args.idx + m) : 0;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (v[r] < 0 || v[r] >= args.table_rows)
                        record_error(args.status, kStatusIndex, 0);
                    else
                        rows[r] = v[r];
                }
            }
            // K block kb into the next stage; false if the kernel is aborting.  (Partial or not is
            // a constant: as a condition at run time it cost a pair's main loop a quarter, 14336 x 4096
            // summed over 4096 347 us against 246.)
            auto fetch = [&](auto partial, int32_t kb) -> bool {
                constexpr bool part = kSum && decltype(partial)::value;
                if (!warp_wait_bounded<true>(empty_bar(s), ph ^ 1u, abort_flag, args.status, args.timeout_ns,
                                             kWhereProducerEmpty)) {
                    return false;
                }
                const uint32_t sa = base + Cfg::OFF_A + s * (Cfg::PARTS * Cfg::A_BYTES);
                const uint32_t sb = base + Cfg::OFF_B + s * (Cfg::PARTS * Cfg::B_BYTES);
                const int32_t k = p.k0 + (kb_first + kb) * Cfg::BK;
                if (lane == 0) {
                    const uint32_t extra = first ? args.extra_tx : 0u;
                    if (part) {
                        mbar_arrive_expect_tx(tail_bar(s), Cfg::STAGE_BYTES + extra);
                    } else if (leader) {
                        mbar_arrive_expect_tx(full_bar(s), (PAIR ? 2u : 1u) * Cfg::STAGE_BYTES + extra);
                        if (kSum && PAIR)
                            mbar_arrive(full_bar(s));
                    }
                }
                first = false;
                __syncwarp();
                // (a partial block is counted in this CTA, whose zeroing warp waits for it)
                const uint32_t bar = part ? tail_bar(s) : lead(full_bar(s));
                auto load = [&](auto stacked, uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y, int32_t z) {
                    if constexpr (decltype(stacked)::value) {
                        if (PAIR && !part)
                            tma_load_3d_pair(dst, m, bar, x, y, z);
                        else
                            tma_load_3d(dst, m, bar, x, y, z);
                    } else {
                        if (PAIR && !part)
                            tma_load_2d_pair(dst, m, bar, x, y);
                        else
                            tma_load_2d(dst, m, bar, x, y);
                    }
                };
                constexpr Bool<kBatch> kStackA{};   // (A is a stack, or rows of one matrix)
                constexpr Bool<!kSum> kStackB{};
                if (kRows && args.gather) {
                    if (PAIR)
                        tma_gather4_pair(sa + lane * 512u, &maps.a, bar, k, rows[0], rows[1], rows[2], rows[3]);
                    else
                        tma_gather4(sa + lane * 512u, &maps.a, bar, k, rows[0], rows[1], rows[2], rows[3]);
                } else if (lane == 0) {
#pragma unroll
                    for (int part2 = 0; part2 < Cfg::PARTS; ++part2) {
                        const CUtensorMap *m = part2 == 0 ? &maps.a : &maps.a_lo;
                        const uint32_t to = sa + part2 * Cfg::A_BYTES;
                        if constexpr (kMnA) {
                            for (int j = 0; j < Cfg::BM / 64; ++j)
                                load(kStackA, to + j * 8192u, m, m0 + 64 * j, k, ga);
                        } else {
                            load(kStackA, to, m, k, m0, ga);
                        }
                    }
                }
                if (lane == 0) {
#pragma unroll
                    for (int part2 = 0; part2 < Cfg::PARTS; ++part2) {
                        const CUtensorMap *m = part2 == 0 ? &maps.b : &maps.b_lo;
                        const uint32_t to = sb + part2 * Cfg::B_BYTES;
                        if constexpr (kMnB) {
                            for (int j = 0; j < Cfg::BN_LOCAL / 64; ++j)
                                load(kStackB, to + j * 8192u, m, n0 + 64 * j, k, gb);
                        } else {
                            load(kStackB, to, m, k, n0, gb);
                        }
                    }
                }
                if constexpr (kSum)
                    tails = part ? tails | (1u << s) : tails & ~(1u << s);
                if (part)
                    tail_ph ^= 1u << s;
                pending = min(pending + 1, STAGES);
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
                return true;
            };
            const int32_t whole = kSum && rem != 0 ? nkb - 1 : nkb;
            const int32_t early = kSum && rem != 0 ? max(0, whole - kEarly) : whole;
            for (int32_t kb = 0; kb < early && alive; ++kb)
                alive = fetch(Bool<false>{}, kb);
            if constexpr (kSum) {
                if (rem != 0 && alive)
                    alive = fetch(Bool<true>{}, whole);
                for (int32_t kb = early; kb < whole && alive; ++kb)
                    alive = fetch(Bool<false>{}, kb);
            }
        }
        if (!alive) {
            // every copy issued lands before the shared memory is released (bounded; the
            // leader's barriers count both CTAs' bytes)
            int ds = s;
            uint32_t dph = ph;
            for (int i = 0; i < pending; ++i) {
                if (--ds < 0) {
                    ds = STAGES - 1;
                    dph ^= 1u;
                }
                if ((tails >> ds) & 1u)
                    wait_drain(tail_bar(ds), ((tail_ph >> ds) & 1u) ^ 1u, 10000000ull);
                else if (leader)
                    wait_drain(full_bar(ds), dph, 10000000ull);
            }
        }
    } else if (warp == 1 || (Cfg::ISS == 2 && warp == Cfg::LAST_WARP)) {
        // ------------------------------------------------------------ MMA issuers
        if (lane == 0 && leader) {
            // (two issuers: the first or the second half of every block's K steps, into an
            // accumulator of its own)
            const int e = Cfg::ISS == 2 && warp != 1 ? 1 : 0;
            const uint32_t idesc = idesc_f16_f32acc(args.ab_bf16 != 0, TM, BN, kMnA, kMnB);
            int s = 0, ab = 0;
            uint32_t ph = 0, aph = 0;
            bool alive = true;
            auto commit_to = [&](uint32_t bar) {
                if (PAIR)
                    tc_commit_pair_multicast(bar, 3);
                else
                    tc_commit(bar);
            };
            for (int32_t t = cta_set; t < num_tiles && alive; t += cta_sets) {
                int32_t rem;
                const int32_t nkb = blocks_of(t, rem);
                auto wait_acc = [&]() {
                    const bool got = wait_bounded<true>(acce_bar(ab), aph ^ 1u, abort_flag, args.status,
                                                        args.timeout_ns, kWhereMmaAccEmpty);
                    tc_fence_after_sync();
                    return got;
                };
                auto next_acc = [&]() {
                    commit_to(accf_bar(ab));
                    if (++ab == 2) {
                        ab = 0;
                        aph ^= 1u;
                    }
                };
                if (!wait_acc())
                    break;
                // K block kb, on stage st (phase sph of its barrier)
                auto multiply = [&](auto partial, int32_t kb, int st, uint32_t sph) -> bool {
                    constexpr bool part = kSum && decltype(partial)::value;
                    // (a chunk's sum goes to the epilogue, the next chunk starts from zero)
                    const bool begins = kSums ? kb % Cfg::CHUNK == 0 : kb == 0;
                    if (kSums && begins && kb > 0) {
                        next_acc();
                        if (!wait_acc())
                            return false;
                    }
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((ab * Cfg::ISS + e) * BN);
                    // (the peer's zeros: an acquire at cluster scope)
                    const bool got =
                        PAIR && part
                            ? wait_bounded_cluster(full_bar(st), sph, abort_flag, args.status, args.timeout_ns,
                                                   kWhereMmaFull)
                            : wait_bounded<true>(full_bar(st), sph, abort_flag, args.status, args.timeout_ns,
                                                 kWhereMmaFull);
                    if (!got)
                        return false;
                    tc_fence_after_sync();
                    const uint32_t sa = base + Cfg::OFF_A + st * (Cfg::PARTS * Cfg::A_BYTES);
                    const uint32_t sb = base + Cfg::OFF_B + st * (Cfg::PARTS * Cfg::B_BYTES);
                    constexpr uint32_t kStepA = kMnA ? 128u : 2u, kStepB = kMnB ? 128u : 2u;
                    // (of a partial block only the K steps that hold rows of the group)
                    const int steps = part ? (rem + 15) / 16 : 4;
                    // low x high and high x low first, while the sum is small
#pragma unroll
                    for (int pr = kSplit ? 0 : 2; pr < 3; ++pr) {
                        const uint32_t pa = sa + (pr == 0 ? Cfg::A_BYTES : 0u);
                        const uint32_t pb = sb + (pr == 1 ? Cfg::B_BYTES : 0u);
                        const uint64_t ad = kMnA ? sdesc_mn_sw128(pa) : sdesc_k_sw128(pa);
                        const uint64_t bd = kMnB ? sdesc_mn_sw128(pb) : sdesc_k_sw128(pb);
#pragma unroll
                        for (int k2 = 0; k2 < 4 / Cfg::ISS; ++k2) {
                            const int k = Cfg::ISS == 2 ? 2 * e + k2 : k2;
                            if (k < steps) {
                                const uint32_t acc = !begins || k2 > 0 || pr > (kSplit ? 0 : 2) ? 1u : 0u;
                                if (PAIR)
                                    tc_mma_f16_pair(d_tmem, ad + kStepA * k, bd + kStepB * k, idesc, acc);
                                else
                                    tc_mma_f16(d_tmem, ad + kStepA * k, bd + kStepB * k, idesc, acc);
                            }
                        }
                    }
                    commit_to(empty_bar(st));
                    return true;
                };
                auto next_stage = [&]() {
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                };
                const int32_t whole = kSum && rem != 0 ? nkb - 1 : nkb;
                const int32_t early = kSum && rem != 0 ? max(0, whole - kEarly) : whole;
                for (int32_t kb = 0; kb < early && alive; ++kb) {
                    alive = multiply(Bool<false>{}, kb, s, ph);
                    next_stage();
                }
                if constexpr (kSum) {
                    if (rem != 0 && alive) {
                        const int st = s;
                        const uint32_t sph = ph;
                        next_stage();
                        for (int32_t kb = early; kb < whole && alive; ++kb) {
                            alive = multiply(Bool<false>{}, kb, s, ph);
                            next_stage();
                        }
                        alive = alive && multiply(Bool<true>{}, whole, st, sph);
                    }
                }
                if (!alive)
                    break;
                next_acc();
            }
        }
        __syncwarp();
    } else if (kSum && warp == Cfg::LAST_WARP) {
        // ------------------------------------------------------------ zeroing warp
        if constexpr (kSum) {
            int s = 0;
            uint32_t tail_ph = 0;
            for (int32_t t = cta_set; t < num_tiles; t += cta_sets) {
                int32_t rem;
                const int32_t nkb = blocks_of(t, rem);
                if (rem != 0) {
                    const int at = (s + max(0, nkb - 1 - kEarly)) % STAGES;
                    if (!warp_wait_bounded(tail_bar(at), (tail_ph >> at) & 1u, abort_flag, args.status,
                                           args.timeout_ns, kWhereMmaFull))
                        break;
                    tail_ph ^= 1u << at;
                    // rows [rem, next multiple of 16) of every box: 64 columns are one row's 128
                    // bytes, so the swizzle does not matter
                    const uint32_t sa = base + Cfg::OFF_A + at * Cfg::A_BYTES;  // (one part a stage)
                    const uint32_t sb = base + Cfg::OFF_B + at * Cfg::B_BYTES;
                    const int32_t more = (rem + 15) / 16 * 16 - rem;
                    constexpr int32_t kBoxesA = Cfg::BM / 64, kBoxes = kBoxesA + Cfg::BN_LOCAL / 64;
                    for (int32_t i = static_cast<int32_t>(lane); i < more * 8; i += 32) {
                        const uint32_t o = static_cast<uint32_t>(rem * 128 + i * 16);
#pragma unroll
                        for (int j = 0; j < kBoxes; ++j)
                            st_shared_v4((j < kBoxesA ? sa + 8192u * j : sb + 8192u * (j - kBoxesA)) + o, 0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR)
                            mbar_arrive_cluster(lead(full_bar(at)));
                        else
                            mbar_arrive(full_bar(at));
                    }
                }
                s = (s + nkb) % STAGES;
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        constexpr bool kF32 = kSums && !kBatch;  // (the products over groups sum in registers for float32 only)
        constexpr int kCols = Cfg::COLS;
        constexpr bool kOne = Cfg::EPI_BUFS == 1;  // one buffer a warp
        const uint32_t q = warp & 3u, ew = (warp - 2u) / 4u * 4u + q;
        const int32_t col_g = static_cast<int32_t>((warp - 2u) / 4u) * kCols;  // first column of this group of warps
        const uint32_t buf0 = base + Cfg::OFF_EPI + Cfg::EPI_BUFS * ew * Cfg::EPI_BUF;
        const bool f32 = kF32 || args.out_kind == kOutF32;
        const uint32_t esize = f32 ? 4u : 2u;
        const bool narrow = CS == 2 && !f32;         // (images of 64-byte rows)
        const int32_t wide = f32 || narrow ? 32 : 64;  // columns of an image's row
        // TMA stores whole 16 bytes of a row: D's descriptor ends with the last whole ones
        const int32_t n_tma = args.n_out & ~(f32 ? 3 : 7);
        const uint64_t policy = l2_policy_evict_first();
        auto pack2 = [&](float x, float y) {
            return args.out_kind == kOutBF16 ? pack_bf16x2(x, y) : pack_f16x2(x, y);
        };
        int ab = 0;
        uint32_t aph = 0, slot = 0;
        [[maybe_unused]] uint32_t shared_tiles = 0;  // (CS = 2) tiles handed over so far
        [[maybe_unused]] uint32_t c_ph = 0;  // (bit j) parity of c_bar j's next phase
        bool alive = true;
        for (int32_t t = cta_set; t < num_tiles && alive; t += cta_sets) {
            const GroupTile p = locate(t);
            int32_t rem;
            const int32_t nkb = blocks_of(t, rem);
            const int32_t row0 = p.row0 + static_cast<int32_t>(role) * Cfg::BM + 32 * static_cast<int32_t>(q);
            const int32_t nrows = min(32, p.end - row0);
            const int32_t my_row = row0 + static_cast<int32_t>(lane);
            const int32_t n_g = p.n0 + col_g;  // first column of D
            const bool stores = nrows > 0 && n_g < args.N;
            bool zero = CS == 1 && nkb == 0;
            if (kRows && args.idx && my_row < p.end) {
                const int32_t v = __ldcg(args.idx + my_row);
                zero = zero || v < 0 || v >= args.table_rows;
            }
            uint8_t *d_g = static_cast<uint8_t *>(args.D) + (kRows ? 0 : p.gd * args.stride_d * esize);
            // (PREC_SPLIT) C's high and low parts for 32 columns of this lane's row
            const uint16_t *c_row =
                kBatch && args.C && my_row < p.end
                    ? args.C + p.g * args.stride_c + static_cast<int64_t>(my_row) * args.ldc + n_g
                    : nullptr;
            struct CPart {
                uint4 hi[4], lo[4];
            };
            auto load_c = [&](int32_t col, CPart &c) {
                if constexpr (kSplit) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        c.hi[i] = c.lo[i] = make_uint4(0, 0, 0, 0);
                        if (c_row && n_g + col + 8 * i < args.N) {
                            c.hi[i] = *reinterpret_cast<const uint4 *>(c_row + col + 8 * i);
                            if (args.c_lo)
                                c.lo[i] = *reinterpret_cast<const uint4 *>(c_row + args.c_lo + col + 8 * i);
                        }
                    }
                }
            };
            // alpha sum + beta C
            auto finish = [&](float(&v)[32], const CPart &c) {
                if (kSplit && args.C) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int sh = 16 * (i & 1);
                        const uint32_t w = reinterpret_cast<const uint32_t *>(c.hi)[i / 2];
                        const uint32_t wl = reinterpret_cast<const uint32_t *>(c.lo)[i / 2];
                        const float x = cvt_f16_f32(static_cast<uint16_t>(w >> sh)) +
                                        cvt_f16_f32(static_cast<uint16_t>(wl >> sh));
                        v[i] = fma_rn(args.alpha, v[i], mul_rn(args.beta, x));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = zero ? 0.f : mul_rn(args.alpha, v[i]);
                }
            };
            // a row of an image a lane, from column col of this group's, to D
            auto put = [&](int32_t col, const uint32_t(&w)[32]) {
                const int32_t col0 = n_g + col;
                if (nrows <= 0 || col0 >= args.N)
                    return;
                const uint32_t buf = buf0 + (kOne ? 0u : slot * Cfg::EPI_BUF);
                slot ^= 1u;
                if (lane == 0) {  // the last store that used the buffer has read it
                    if (kOne)
                        bulk_wait_group_read<0>();
                    else
                        bulk_wait_group_read<1>();
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!narrow || i < 4)
                        st_shared_v4(buf + (narrow ? swz64(lane, i) : swz128(lane, i)), w[4 * i], w[4 * i + 1],
                                     w[4 * i + 2], w[4 * i + 3]);
                // a whole box by TMA; rows that end with the group (KIND_ROWS; the others' boxes
                // end with their matrix), or columns past the last whole 16 bytes, by plain stores
                const bool tma = args.d_tma && (!kRows || nrows == 32) && (col0 + wide <= n_tma || n_tma == args.n_out);
                if (tma) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (kBatch)  // (read by the next product)
                            tma_store_3d(&maps.d, buf, col0, row0, p.gd);
                        else
                            tma_store_3d_hint(&maps.d, buf, col0, row0, kRows ? 0 : p.gd, policy);
                    }
                } else {
                    __syncwarp();
                    store_image_rows(buf, lane, narrow, nrows, esize, d_g, args.ldd, row0, col0, args.n_out, args.d_vec != 0);
                    __syncwarp();
                }
                if (lane == 0)  // (every use of a buffer is a group: the wait above counts them)
                    bulk_commit_group();
            };
            // 32 columns as the image of their transpose, 32 rows of 64 bytes: two neighbouring rows'
            // values from a lane and its neighbour make a word, two of its rows' words a conflict-free
            // store.  (Those words stored to D from here: 8 x 1000 x 1000 20 us against 26 with a
            // condition after each shuffle.)
            auto transpose = [&](uint32_t buf, const float (&v)[32]) {
                const uint32_t odd = lane & 1u;
#pragma unroll
                for (uint32_t k = 0; k < 16u; ++k) {
                    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * k] : v[2 * k + 1], 1);
                    const uint32_t w = odd ? pack_f16x2(other, v[2 * k + 1]) : pack_f16x2(v[2 * k], other);
                    st_shared_u32(buf + swz64(2 * k + odd, lane >> 3) + ((lane & 6u) << 1), w);
                }
            };
            // (PREC_SPLIT) 32 columns of a workspace in two parts: two images of 64-byte rows, and
            // boxes of them.  (Each lane its own row in 16-byte stores instead: 8 x 1000 x 1367 52 ->
            // 76 us.)
            auto free_buffer = [&]() {
                const uint32_t buf = buf0 + (kOne ? 0u : slot * Cfg::EPI_BUF);
                slot ^= 1u;
                if (lane == 0) {
                    if (kOne)
                        bulk_wait_group_read<0>();
                    else
                        bulk_wait_group_read<1>();
                }
                __syncwarp();
                return buf;
            };
            auto send_two = [&](uint32_t buf, int32_t x, int32_t y) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&maps.d, buf, x, y, p.g);
                    tma_store_3d(&maps.d_lo, buf + 2048u, x, y, p.g);
                    bulk_commit_group();
                }
            };
            auto put_two = [&](int32_t col, float(&v)[32], const uint32_t(&hi)[16]) {
                const int32_t col0 = n_g + col;
                if (nrows <= 0 || col0 >= args.N)
                    return;
                uint32_t buf = free_buffer();
                if (SYM && p.mirror)
                    transpose(buf, v);
                // what rounding to float16 left of the values
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] -= cvt_f16_f32(static_cast<uint16_t>(hi[i / 2] >> (16 * (i & 1))));
                if (SYM && p.mirror) {
                    transpose(buf + 2048u, v);
                    send_two(buf, row0, col0);
                    buf = free_buffer();
                }
                uint32_t lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    lo[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i) {
                    const uint32_t o = swz64(lane, i);
                    st_shared_v4(buf + o, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                    st_shared_v4(buf + 2048u + o, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                }
                send_two(buf, col0, row0);
            };
            // 64 columns from col, their sums 32 at a time from take(half, v), C's elements from
            // c (the first half's) and next(half) (those of the half after it)
            auto piece = [&](int32_t col, CPart &c, auto take, auto next) {
                uint32_t w[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    take(h, v);
                    if (!stores)
                        continue;
                    finish(v, c);
                    next(h);
                    if (f32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = __float_as_uint(v[i]);
                        put(col + 32 * h, w);
                        continue;
                    }
                    if constexpr (!kF32) {
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = pack2(v[2 * i], v[2 * i + 1]);
                        if (kSplit && args.d_lo) {
                            put_two(col + 32 * h, v, x);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[16 * h + i] = x[i];
                            if (h == 1)
                                put(col, w);
                        }
                    }
                }
            };
            auto hand_back = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && !leader)
                        mbar_arrive_cluster(lead(acce_bar(ab)));
                    else
                        mbar_arrive(acce_bar(ab));
                }
                if (++ab == 2) {
                    ab = 0;
                    aph ^= 1u;
                }
            };
            auto wait_full = [&]() {
                // (PREC_SUMS: inline, or the call would save the sums' registers)
                if constexpr (kSums)
                    alive = warp_wait_bounded_inline(accf_bar(ab), aph, abort_flag, args.status, args.timeout_ns,
                                                     kWhereEpiAccFull);
                else
                    alive = warp_wait_bounded<true>(accf_bar(ab), aph, abort_flag, args.status, args.timeout_ns,
                                                    kWhereEpiAccFull);
                tc_fence_after_sync();
                return tmem_base + ((32u * q) << 16) + static_cast<uint32_t>(ab * Cfg::ISS * BN + col_g);
            };
            // (two issuers) the second one's sums of 32 columns, added to the first one's
            auto add_second = [&](uint32_t at, uint32_t(&r)[32]) {
                if constexpr (Cfg::ISS == 2) {
                    uint32_t r2[32];
                    tc_ld_32x32b_x32(at + BN, r2);
                    tc_wait_ld(r2);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        r[i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), __uint_as_float(r2[i])));
                }
            };
            if constexpr (kSums) {
                float sums[kCols];
                // (CS = 2) the columns this CTA finishes, and C's elements there
                const int32_t half = CS == 2 ? 32 * static_cast<int32_t>(share) : 0;
                [[maybe_unused]] CPart c_early;
                if (CS == 2 && stores)
                    load_c(half, c_early);
                const int32_t fills = max(1, (nkb + Cfg::CHUNK - 1) / Cfg::CHUNK);
                for (int32_t f = 0; f < fills; ++f) {
                    const uint32_t acc = wait_full();
                    if (!alive)
                        break;
                    if constexpr (Cfg::EPI_GROUPS == 4) {  // (18 warps: about 100 registers each)
#pragma unroll
                        for (int c = 0; c < kCols / 16; ++c) {
                            uint32_t r[16];
                            tc_ld_32x32b_x16(acc + 16u * c, r);
                            tc_wait_ld(r);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                sums[16 * c + i] = f == 0 ? __uint_as_float(r[i])
                                                          : __fadd_rn(sums[16 * c + i], __uint_as_float(r[i]));
                        }
                    } else
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        uint32_t r[32];
                        tc_ld_32x32b_x32(acc + 32u * c, r);
                        tc_wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sums[32 * c + i] = f == 0 ? __uint_as_float(r[i])
                                                      : __fadd_rn(sums[32 * c + i], __uint_as_float(r[i]));
                        if constexpr (Cfg::ISS == 2) {
                            tc_ld_32x32b_x32(acc + 32u * c + BN, r);
                            tc_wait_ld(r);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                sums[32 * c + i] = __fadd_rn(sums[32 * c + i], __uint_as_float(r[i]));
                        }
                    }
                    hand_back();
                }
                if (!alive)
                    break;
                if constexpr (CS == 2) {
                    // the halves change places; each CTA finishes 32 columns
                    float v[32];
                    const uint32_t at = base + Cfg::OFF_RED + q * Cfg::RED_BYTES + lane * 4u;
                    const uint32_t to = mapa_shared(at, share ^ 1u);
                    if (shared_tiles > 0 && !warp_wait_cluster(rede_bar(q), (shared_tiles - 1u) & 1u, abort_flag,
                                                               args.status, args.timeout_ns, kWhereEpiC)) {
                        alive = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        st_shared_cluster_u32(to + 128u * static_cast<uint32_t>(i),
                                              __float_as_uint(share ? sums[i] : sums[32 + i]));
                        v[i] = share ? sums[32 + i] : sums[i];
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(mapa_shared(redf_bar(q), share ^ 1u));
                    if (!warp_wait_cluster(redf_bar(q), shared_tiles & 1u, abort_flag, args.status, args.timeout_ns,
                                           kWhereEpiC)) {
                        alive = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __fadd_rn(v[i], __uint_as_float(ld_shared_u32(at + 128u * static_cast<uint32_t>(i))));
                    __syncwarp();
                    // (not after the last tile: the writer may have ended)
                    if (lane == 0 && t + cta_sets < num_tiles)
                        mbar_arrive_cluster(mapa_shared(rede_bar(q), share ^ 1u));
                    ++shared_tiles;
                    if (!stores)
                        continue;
                    finish(v, c_early);
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i] = pack2(v[2 * i], v[2 * i + 1]);
                    if (args.d_lo) {
                        put_two(half, v, x);
                    } else {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = f32 ? __float_as_uint(v[i]) : x[i % 16];
                        put(half, w);
                    }
                    continue;
                }
                if (!stores)
                    continue;
                if constexpr (kF32) {
#pragma unroll
                    for (int col = 0; col < kCols; col += 32) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = zero ? 0u : __float_as_uint(mul_rn(args.alpha, sums[col + i]));
                        put(col, w);
                    }
                    continue;
                }
                CPart c;
                if (stores)
                    load_c(0, c);
#pragma unroll
                for (int col = 0; col < kCols; col += 64)
                    piece(
                        col, c,
                        [&](int h, float(&v)[32]) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = sums[col + 32 * h + i];
                        },
                        [&](int h) {
                            if (col + 32 * h + 32 < kCols)
                                load_c(col + 32 * h + 32, c);
                        });
            } else if constexpr (Cfg::C_TMA) {
                // KIND_BATCH.  C by TMA, 32 columns (and their low parts) a buffer, the first two while
                // the tile's MMAs run; D takes C's place and leaves from there, and (SYM) its transpose
                // from the low parts' place.  (C by loads of each lane's own row: 32 x 1000 x 1000 113
                // against 91 us.)
                {
                    const bool has_c = args.C != nullptr;
                    const int32_t units = stores ? min(kCols / 32, (args.N - n_g + 31) / 32) : 0;
                    auto load_unit = [&](int32_t u) {  // (lane 0; the buffer's last store has read it)
                        const uint32_t j = (slot + static_cast<uint32_t>(u)) & 1u, to = buf0 + j * Cfg::EPI_BUF;
                        mbar_arrive_expect_tx(c_bar(ew, j), args.c_lo ? 4096u : 2048u);
                        tma_load_3d(to, &maps.c, c_bar(ew, j), n_g + 32 * u, row0, p.g);
                        if (args.c_lo)
                            tma_load_3d(to + 2048u, &maps.c_lo, c_bar(ew, j), n_g + 32 * u, row0, p.g);
                    };
                    if (lane == 0 && has_c && units > 0) {
                        bulk_wait_group_read<0>();
                        for (int32_t u = 0; u < min(units, 2); ++u)
                            load_unit(u);
                    }
                    const uint32_t acc = wait_full();
                    int32_t landed = 0;  // pieces of C seen to have landed
#pragma unroll 1
                    for (int32_t u = 0; u < kCols / 32 && alive; ++u) {
                        const uint32_t j = (slot + static_cast<uint32_t>(u)) & 1u, buf = buf0 + j * Cfg::EPI_BUF;
                        uint32_t r[32];
                        tc_ld_32x32b_x32(acc + 32u * static_cast<uint32_t>(u), r);
                        tc_wait_ld(r);
                        add_second(acc + 32u * static_cast<uint32_t>(u), r);
                        if (u == kCols / 32 - 1)
                            hand_back();
                        if (u >= units)
                            continue;
                        if (has_c) {
                            if (!warp_wait_bounded<true>(c_bar(ew, j), (c_ph >> j) & 1u, abort_flag, args.status,
                                                         args.timeout_ns, kWhereEpiC)) {
                                alive = false;
                                break;
                            }
                            c_ph ^= 1u << j;
                            ++landed;
                        } else if (lane == 0) {
                            bulk_wait_group_read<1>();  // the store before the last has left this buffer
                        }
                        float v[32];
                        if (!has_c) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = mul_rn(args.alpha, __uint_as_float(r[i]));
                        } else
#pragma unroll
                        for (uint32_t i = 0; i < 4u; ++i) {
                            uint32_t h[4], l[4] = {0u, 0u, 0u, 0u};
                            ld_shared_v4(buf + swz64(lane, i), h[0], h[1], h[2], h[3]);
                            if (args.c_lo)
                                ld_shared_v4(buf + 2048u + swz64(lane, i), l[0], l[1], l[2], l[3]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int sh = 16 * (e & 1);
                                const float x = cvt_f16_f32(static_cast<uint16_t>(h[e / 2] >> sh)) +
                                                cvt_f16_f32(static_cast<uint16_t>(l[e / 2] >> sh));
                                v[8 * i + e] = fma_rn(args.alpha, __uint_as_float(r[8 * i + e]), mul_rn(args.beta, x));
                            }
                        }
                        // the buffer before: refilled while this piece leaves
                        if (has_c && lane == 0 && u >= 1 && u + 1 < units) {
                            bulk_wait_group_read<0>();
                            load_unit(u + 1);
                        }
                        __syncwarp();  // (every lane has read C)
                        const int32_t col = 32 * u, col0 = n_g + col;
                        if (f32) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                st_shared_v4(buf + swz128(lane, i), __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                             __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
                        } else {
                            uint32_t x[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[i] = pack2(v[2 * i], v[2 * i + 1]);
#pragma unroll
                            for (uint32_t i = 0; i < 4u; ++i)
                                st_shared_v4(buf + swz64(lane, i), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                            if (SYM) {
                                if (p.mirror)
                                    transpose(buf + 2048u, v);
                            } else if (args.d_lo) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    v[i] -= cvt_f16_f32(static_cast<uint16_t>(x[i / 2] >> (16 * (i & 1))));
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    x[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
#pragma unroll
                                for (uint32_t i = 0; i < 4u; ++i)
                                    st_shared_v4(buf + 2048u + swz64(lane, i), x[4 * i], x[4 * i + 1], x[4 * i + 2],
                                                 x[4 * i + 3]);
                            }
                        }
                        if (args.d_tma && (col0 + 32 <= n_tma || n_tma == args.n_out)) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_3d(&maps.d, buf, col0, row0, p.gd);
                                if (SYM) {
                                    if (p.mirror)
                                        tma_store_3d(&maps.d, buf + 2048u, row0, col0, p.g);
                                } else if (args.d_lo) {
                                    tma_store_3d(&maps.d_lo, buf + 2048u, col0, row0, p.g);
                                }
                            }
                        } else {
                            __syncwarp();
                            store_image_rows(buf, lane, !f32, nrows, esize, d_g, args.ldd, row0, col0, args.n_out,
                                             args.d_vec != 0);
                            fence_proxy_async_smem();  // (the buffer is a TMA load's next)
                            __syncwarp();
                        }
                        if (lane == 0)
                            bulk_commit_group();
                    }
                    if (!alive && has_c && lane == 0) {
                        // pieces of C under way land before the shared memory is released
                        for (int32_t u = landed; u < min(units, landed + 2); ++u)
                            wait_drain(c_bar(ew, (slot + static_cast<uint32_t>(u)) & 1u),
                                       (c_ph >> ((slot + static_cast<uint32_t>(u)) & 1u)) & 1u, 10000000ull);
                    }
                    slot += static_cast<uint32_t>(units);  // (the buffers in turn, also from tile to tile)
                }
            } else {
                CPart c;  // (no C)
                const uint32_t acc = wait_full();
                if (!alive)
                    break;
#pragma unroll 1
                for (int32_t col = 0; col < kCols; col += 64)
                    piece(
                        col, c,
                        [&](int h, float(&v)[32]) {
                            uint32_t r[32];
                            tc_ld_32x32b_x32(acc + static_cast<uint32_t>(col + 32 * h), r);
                            tc_wait_ld(r);
                            add_second(acc + static_cast<uint32_t>(col + 32 * h), r);
                            if (h == 1 && col + 64 >= kCols)
                                hand_back();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = __uint_as_float(r[i]);
                        },
                        [](int) {});
            }
        }
        if (lane == 0)
            bulk_wait_group_all();
        __syncwarp();
    }

    tc_fence_before_sync();
    if (PAIR) {
        if (threadIdx.x == 0 && *abort_flag)
            st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(abort_flag)), role ^ 1u), 1u);
        if (*abort_flag && !leader) {
            // copies that report to the leader's barriers get time to land here too
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 100000ull) {
            }
        }
    }
    // The other CTA's work may use this one's shared memory until here.  (CS = 2: not where all
    // went well.  Its sums have been waited for, and so has every arrival at this CTA's barriers.
    // Of a kernel of 9 us the barrier took 0.6.)
    bool together = PAIR;
    if (CS == 2) {
        __syncthreads();
        together = *abort_flag != 0u;
    }
    if (together)
        cluster_sync_all();
    else if (CS == 1)
        __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace tcg
