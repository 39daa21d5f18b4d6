// api_group.cu -- the entry points for layers of experts: gemm_group_rows, gemm_grouped,
// gemm_grouped_weights (products over groups of rows) and gemm_orthogonalize (Newton-Schulz
// steps on a stack of matrices).  include/tcgemm.h has the contracts.  Checks run before any
// CUDA call, as everywhere.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "host_internal.h"
#include "launch_group.h"

namespace tcg {
namespace host {

namespace {

constexpr int64_t kMaxGroups = 1024;  // (a warp keeps 32 groups a lane)
constexpr int64_t kMaxRows = kMaxDim - 512;  // (a tile's rows past the last one are 32-bit numbers too)
constexpr int kGroupM = 16;           // block rows per tile-order group, as the plain forms

// A form of the group kernel, with the time of a tile's K block and of its fixed part in ns
// (operand bytes from L2 to an SM set the first, the epilogue and the hand-overs the second).
struct GForm {
    int bn;
    bool pair;
    int cs;  // CTAs that share a tile's sum
    int64_t block_ns, fixed_ns;
};
// Measured, us a tile, 2 / 8 / 32 and more blocks: 128 x 256 2.35 / 4.1, pairs 3.0 / 3.6 / 12.7;
// float32 results, 128 columns 1.5 / - / 0.5 a block, pairs 6.3 / - / 26.8 (64 blocks).
constexpr GForm kForms[4] = {{64, false, 1, 200, 800}, {128, false, 1, 300, 1000}, {256, false, 1, 330, 1700},
                             {256, true, 1, 285, 2000}};
// (float32 results, sums in registers)
constexpr GForm kSumForms[3] = {{64, false, 1, 200, 700}, {128, false, 1, 480, 800}, {256, true, 1, 320, 7500}};
// (operands in two parts)
constexpr GForm kSplitForms[3] = {{64, false, 1, 440, 3500}, {128, false, 1, 600, 4500}, {64, false, 2, 440, 2000}};

// Shorter sums than these K blocks are not shared: their halves' exchange takes what they save (64 x
// 128 x 512 150 us, shared 220; 512 x 512 133, shared 108).
constexpr int64_t kSharedBlocks = 8;

// The form of the least waves x time of a tile.  tiles(tile_m, bn): tiles of the problem
// (0: the form does not apply).
template <class F>
GForm choose_form(int64_t k_blocks, int prec, int sm_count, F tiles)
{
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    const GForm *forms = prec == kPrecSplit ? kSplitForms : (prec == kPrecSums ? kSumForms : kForms);
    const int n_forms = prec == kPrecAcc ? 4 : 3;
    const GForm *best = nullptr;
    int64_t best_ns = 0;
    for (const GForm *f = forms; f != forms + n_forms; ++f) {
        const int64_t n = tiles(f->pair ? 256 : 128, f->bn), sets = sm_count / (f->pair ? 2 : f->cs);
        if (n <= 0 || sets <= 0 || (f->cs > 1 && k_blocks < kSharedBlocks))
            continue;
        if ((fk == 1 && !f->pair && f->cs == 1 && f->bn == fbn) || (fk == 3 && (f->pair || f->cs == 2)))
            return *f;
        const int64_t ns = ceil_div(n, sets) * (ceil_div(k_blocks, f->cs) * f->block_ns + f->fixed_ns);
        if (!best || ns < best_ns) {
            best = f;
            best_ns = ns;
        }
    }
    return best ? *best : forms[1];
}

// CTAs of a launch over at most `tiles` tiles.
gemm_status group_grid(const GForm &f, int64_t tiles, const DeviceInfo *dev, int *grid)
{
    int64_t sets = dev->sm_count / f.cs;
    if (f.pair) {
        sets = tcg::tile_max_clusters(256, true, 1, 1);  // (the same shared memory)
        if (sets <= 0)
            return GEMM_ERR_CUDA;
    }
    *grid = static_cast<int>((f.pair ? 2 : f.cs) * (tiles < sets ? tiles : sets));
    return GEMM_OK;
}

void fill_group(GroupArgs &a, bool bf16, int out, const DeviceInfo *dev)
{
    std::memset(&a, 0, sizeof(a));
    GemmArgs g;
    std::memset(&g, 0, sizeof(g));
    Problem q{};
    fill_common(g, q, dev);
    a.out_kind = out;
    a.ab_bf16 = bf16 ? 1 : 0;
    a.extra_tx = g.extra_tx;
    a.status = g.status;
    a.timeout_ns = g.timeout_ns;
    a.beta = 0.0f;
}

// D of a launch: `depth` matrices of rows x cols; false if the descriptor was refused.
// d_lo != 0 (16 bits): in two parts, the second d_lo elements behind the first; narrow: boxes of
// 32 columns.
bool set_out(GroupArgs &a, GroupMaps &maps, void *D, int out, int64_t rows, int64_t cols, int64_t ld,
             int64_t depth, int64_t stride, int64_t d_lo = 0, bool narrow = false)
{
    const int64_t es = out_size(out), per16 = 16 / es;
    a.D = D;
    a.ldd = ld;
    a.stride_d = stride;
    a.n_out = static_cast<int32_t>(cols);
    a.d_vec = aligned16(D) && ld * es % 16 == 0 && (depth == 1 || stride * es % 16 == 0) ? 1 : 0;
    a.d_tma = a.d_vec && cols >= per16 ? 1 : 0;
    a.d_lo = d_lo;
    auto map = [&](CUtensorMap *m, const void *p) {
        return encode_3d(m, out_type(out), p, cols / per16 * per16, rows, ld * es, depth,
                         depth == 1 ? rows * ld * es : stride * es, narrow ? 32 : static_cast<uint32_t>(128 / es), 32,
                         narrow && es == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    };
    return !a.d_tma || (map(&maps.d, D) && (!d_lo || map(&maps.d_lo, static_cast<const uint16_t *>(D) + d_lo)));
}

// A stack of `depth` matrices of rows x cols 16-bit elements as an operand: boxes of 64
// columns and box_rows rows.
bool set_operand(CUtensorMap *m, bool bf16, const void *p, int64_t cols, int64_t rows, int64_t ld, int64_t depth,
                 int64_t stride, int box_rows)
{
    return encode_3d(m, ab_type(bf16), p, cols, rows, ld * 2, depth, depth == 1 ? rows * ld * 2 : stride * 2, 64,
                     static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

// A stack of matrices among the arguments: checked as check_mats checks one, and the
// distance from one to the next, which may not be less than a matrix.
struct Stack {
    Mat m;
    int64_t depth, stride;
};
gemm_status check_stack(const Stack &s)
{
    if (s.depth == 0 || s.m.rows == 0 || s.m.cols == 0)
        return GEMM_OK;
    const gemm_status st = check_mats({s.m});
    if (st != GEMM_OK || s.depth == 1)
        return st;
    if (s.stride < (s.m.rows - 1) * s.m.ld + s.m.cols)
        return GEMM_ERR_INVALID_ARG;
    if (s.stride > INT64_MAX / 8 / s.depth)
        return GEMM_ERR_UNSUPPORTED;
    return s.m.mma && s.stride * s.m.esize % 16 != 0 ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}
Span span_of(const Stack &s)
{
    if (s.depth == 0 || s.m.rows == 0 || s.m.cols == 0)
        return Span{nullptr, 0};
    const Span one = span_of(s.m);
    return Span{one.p, one.bytes + static_cast<uint64_t>(s.depth - 1) * s.stride * s.m.esize};
}

// Few rows a group: the kernel that streams the weights, as (rows of a tile, CTAs a tile); rows
// 0 where the tile kernel runs.  Measured, us, groups x N x K of so many rows, bf16: tiles of 16 / 32 /
// 64 rows, 8 x 14336 x 4096 of 4 141 / 137 / 138, of 12 143 / 139 / 140, of 24 154 / 141 / 141, of 40 183 /
// 159 / 142 (the tile kernel 143 to 149); 2 x 2816 x 1024 of 1 6.4 / 6.7 / 7.9 (9.0).  One / two CTAs a tile:
// 2 x 4096 x 14336 (64 tiles) 42.7 / 39.2, 2 x 14336 x 4096 (224) 39.0 / 39.1, 2 x 2816 x 1024 (44) 6.4 / 6.7,
// 32 x 2816 x 1024 (704) 31.6 / 39.0: two where they have SMs of their own and a long sum to share.  (Each list of
// one run; from one GPU to another they differ by up to 4 %.)
struct Few {
    int mp, cs;
};
Few choose_few(int64_t M, int64_t N, int64_t K, int64_t groups, int sm_count)
{
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    const int64_t used = groups < M ? groups : M, rows = ceil_div(M, used);  // (of a group, on average)
    if (K == 0 || (fk != 0 && fk != 2) || (fk == 0 && rows > 48))
        return Few{0, 0};
    const int mp = rows <= 8 ? 16 : (rows <= 16 ? 32 : 64);
    const int64_t tiles = used * ceil_div(rows, mp) * ceil_div(N, 128);
    return Few{mp, 2 * tiles <= sm_count && K >= 4096 ? 2 : 1};
}

// Gathered rows of A: whether a kernel that lays them out in order comes first.  The products' own
// gathers cost about 36 ns for four rows and 64 columns where the tiles are 128 rows high, and 1.5 us a
// tile where the rows of a group are few; the kernel a launch and each row in and out.  (us, own / in
// order first: 16384 rows, 4096 x 4096 1038 / 326; 8 x 500, 4096 x 512 47.5 / 27.3; 777 rows, 2743 x 1000
// 30.8 / 19.1; 60 groups of 163, 5489 x 118 175 / 55; 43 of 4, 8640 x 298 71 / 44; 8 of 4, 14336 x 4096
// 146.4 / 144.5.)
constexpr int64_t kGatheredBytes = int64_t(8) << 30;  // of a buffer for them, at most
bool gather_first(int64_t M, int64_t K, const GForm &f, const Few &few, int64_t waves)
{
    if (ceil_div(K, 64) * 128 > kGatheredBytes / M)
        return false;
    const int64_t block_ns = f.block_ns < 32 * 36 ? 32 * 36 - f.block_ns : 0;
    const int64_t own_ns = few.mp ? waves * 1500 : waves * ceil_div(K, 64) * block_ns;
    return own_ns > 4000 + M * K / 1250;
}

// The buffer's size for so many bytes (kGatheredBytes at most): the next power of two.  A larger call then finds
// a buffer of its own size or gets one twice as large, and none is larger than kGatheredBytes.
size_t gathered_size(int64_t bytes)
{
    size_t size = 1 << 20;
    while (size < static_cast<size_t>(bytes))
        size *= 2;
    return size;
}

bool bad_flag(int f) { return f != 0 && f != 1; }

}  // namespace

}  // namespace host
}  // namespace tcg

using namespace tcg::host;
using tcg::GroupArgs;
using tcg::GroupMaps;

extern "C" {

gemm_status gemm_group_rows(int64_t M, int64_t groups, int64_t choices, const int32_t *ids, int32_t *offsets,
                            int32_t *order, int32_t *rows, void *stream)
{
    if (M < 0 || groups < 0 || choices < 1 || !offsets || (M > 0 && (!ids || !order)))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || choices > kMaxDim || groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    if (!elem_aligned(offsets, 4) || (M > 0 && (!elem_aligned(ids, 4) || !elem_aligned(order, 4) || !elem_aligned(rows, 4))))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t b = static_cast<uint64_t>(M) * 4;
    if (any_overlap({Span{offsets, static_cast<uint64_t>(groups + 1) * 4}, Span{order, b}, Span{rows, rows ? b : 0}},
                    {Span{ids, b}}))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    gemm_status st = device_info(&dev);
    if (st != GEMM_OK)
        return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    int64_t chunks = 1;
    void *counts = nullptr;
    std::unique_lock<std::mutex> hold;
    if (M > tcg::kGroupRowsOne) {
        chunks = ceil_div(M, tcg::kGroupRowsChunk);
        chunks = chunks < dev->sm_count ? chunks : dev->sm_count;
        hold = std::unique_lock<std::mutex>(buffer_mutex(dev->index, cs));
        if ((st = get_dequant_buffer(dev->index, cs, kBufGroupRows,
                                     static_cast<size_t>(chunks * (groups + 1)) * sizeof(int32_t), &counts)) != GEMM_OK)
            return st;
    }
    const cudaError_t e = tcg::launch_group_rows_sort(ids, M, static_cast<int32_t>(groups),
                                                      static_cast<int32_t>(choices), offsets, order, rows,
                                                      static_cast<int32_t *>(counts), static_cast<int32_t>(chunks), cs);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status gemm_grouped(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype_is_bf16, const void *A,
                         int64_t a_rows, int64_t lda, const int32_t *idx, const int32_t *offsets, int trans_b,
                         const void *B, int64_t ldb, int64_t stride_b, void *D, int64_t ldd, int out, float alpha,
                         void *stream)
{
    if (bad_flag(dtype_is_bf16) || bad_flag(trans_b) || M < 0 || N < 0 || K < 0 || groups < 0 || !out_ok(out) ||
        (idx && a_rows < 1))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxRows || (idx && a_rows > kMaxDim) || groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0 || groups == 0)
        return GEMM_OK;
    auto most = [&](int tm, int bn) { return (M / tm + groups) * ceil_div(N, bn); };
    if (most(16, 64) > kMaxDim)
        return GEMM_ERR_UNSUPPORTED;
    const int64_t rows = idx ? a_rows : M;
    const Mat a{A, lda, K > 0 ? rows : 0, K, 2, true}, d{D, ldd, M, N, out_size(out), false};
    const Stack b{Mat{B, ldb, trans_b ? K : N, trans_b ? N : K, 2, true}, groups, stride_b};
    if (!offsets)
        return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_mats({a, d});
    if (st != GEMM_OK || (st = check_stack(b)) != GEMM_OK)
        return st;
    if (!elem_aligned(offsets, 4) || !elem_aligned(idx, 4))
        return GEMM_ERR_ALIGNMENT;
    if (any_overlap({span_of(d)}, {span_of(a), span_of(b), Span{offsets, static_cast<uint64_t>(groups + 1) * 4},
                                   Span{idx, idx ? static_cast<uint64_t>(M) * 4 : 0}}))
        return GEMM_ERR_ALIAS;
    // a group of r rows has ceil(r / tile) block rows: on average half a tile more than its rows
    auto tiles = [&](int tm, int bn) {
        const int64_t blocks = M / tm + (groups < M ? groups : M) / 2 + 1;
        return (blocks < M ? blocks : M) * ceil_div(N, bn);
    };
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const bool bf16 = dtype_is_bf16 == 1;
    const int prec = out == GEMM_OUT_F32 ? tcg::kPrecSums : tcg::kPrecAcc;
    const Few few = choose_few(M, N, K, groups, dev->sm_count);
    GForm f = choose_form(ceil_div(K, 64), prec, dev->sm_count, tiles);
    int grid = 0;
    int64_t waves = 0;  // (the tiles in rows are known on average only)
    if (few.mp) {
        f.pair = false;
        f.bn = 128;
        const int64_t n = most(few.mp, 128), sets = dev->sm_count / few.cs;
        grid = static_cast<int>(few.cs * (n < sets ? n : sets));
        waves = ceil_div(tiles(few.mp, 128), sets);
    } else if ((st = group_grid(f, most(f.pair ? 256 : 128, f.bn), dev, &grid)) != GEMM_OK) {
        return st;
    } else {
        waves = ceil_div(tiles(f.pair ? 256 : 128, f.bn), dev->sm_count / (f.pair ? 2 : 1));
    }
    GroupMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    GroupArgs g;
    fill_group(g, bf16, out, dev);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    bool first = idx && K > 0 && gather_first(M, K, f, few, waves);
    std::unique_lock<std::mutex> hold;
    const int64_t ldw = ceil_div(K, 64) * 64;
    void *w = nullptr;
    if (first) {
        hold = std::unique_lock<std::mutex>(buffer_mutex(dev->index, cs));
        // (where there is no memory for them, the product gathers the rows itself)
        first = get_dequant_buffer(dev->index, cs, kBufGathered, gathered_size(M * ldw * 2), &w) == GEMM_OK;
    }
    if (first) {
        if (tcg::launch_group_gather(A, static_cast<int32_t>(rows), lda, idx, offsets, static_cast<int32_t>(groups),
                                     static_cast<int32_t>(M), static_cast<int32_t>(K), w, ldw, g.status,
                                     dev->sm_count, cs) != cudaSuccess)
            return GEMM_ERR_CUDA;
        A = w;
        lda = ldw;
    }
    const bool own = idx && !first;
    const bool a_ok = K == 0 || (own ? encode_2d(&maps.a, ab_type(bf16), A, K, rows, lda * 2, 64, 1,
                                                 CU_TENSOR_MAP_SWIZZLE_128B)
                                     : encode_2d(&maps.a, ab_type(bf16), A, K, M, lda * 2, 64,
                                                 static_cast<uint32_t>(few.mp ? few.mp : 128),
                                                 CU_TENSOR_MAP_SWIZZLE_128B));
    const bool b_ok = K == 0 || (trans_b ? set_operand(&maps.b, bf16, B, N, K, ldb, groups, stride_b, 64)
                                         : set_operand(&maps.b, bf16, B, K, N, ldb, groups, stride_b,
                                                       f.pair ? f.bn / 2 : f.bn));
    if (!a_ok || !b_ok || !set_out(g, maps, D, out, M, N, ldd, 1, 0))
        return GEMM_ERR_CUDA;
    g.groups = static_cast<int32_t>(groups);
    g.offsets = offsets;
    g.rows = static_cast<int32_t>(M);
    g.N = static_cast<int32_t>(N);
    g.K = static_cast<int32_t>(K);
    g.num_n_blocks = static_cast<int32_t>(ceil_div(N, f.bn));
    g.group_m = kGroupM;
    g.alpha = alpha;
    g.idx = idx;
    g.table_rows = static_cast<int32_t>(rows);
    g.gather = own ? 1 : 0;
    g.loads = K > 0 ? 1 : 0;
    if (few.mp)
        return tcg::launch_group_few(few.mp, few.cs, trans_b == 1, maps, g, grid, cs) ==
                       cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    const cudaError_t e = tcg::launch_group_rows(f.bn, f.pair, trans_b == 1, prec, maps, g, grid, cs);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status gemm_grouped_weights(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype_is_bf16, const void *dD,
                                 int64_t lddd, const void *A, int64_t lda, const int32_t *offsets, void *dB,
                                 int64_t lddb, int64_t stride_db, int out, float alpha, void *stream)
{
    if (bad_flag(dtype_is_bf16) || M < 0 || N < 0 || K < 0 || groups < 0 || !out_ok(out))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxRows || groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0 || groups == 0)
        return GEMM_OK;
    if (ceil_div(N, 128) > kMaxDim / ceil_div(K, 64) / groups)
        return GEMM_ERR_UNSUPPORTED;
    const Mat dd{dD, lddd, M, N, 2, true}, a{A, lda, M, K, 2, true};
    const Stack db{Mat{dB, lddb, N, K, out_size(out), false}, groups, stride_db};
    if (!offsets)
        return GEMM_ERR_INVALID_ARG;
    gemm_status st = check_mats({dd, a});
    if (st != GEMM_OK || (st = check_stack(db)) != GEMM_OK)
        return st;
    if (!elem_aligned(offsets, 4))
        return GEMM_ERR_ALIGNMENT;
    if (any_overlap({span_of(db)}, {span_of(dd), span_of(a), Span{offsets, static_cast<uint64_t>(groups + 1) * 4}}))
        return GEMM_ERR_ALIAS;
    auto tiles = [&](int tm, int bn) { return groups * ceil_div(N, tm) * ceil_div(K, bn); };
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const bool bf16 = dtype_is_bf16 == 1;
    const int prec = out == GEMM_OUT_F32 ? tcg::kPrecSums : tcg::kPrecAcc;
    const tcg::host::GForm f = choose_form(ceil_div(ceil_div(M, groups), 64), prec, dev->sm_count, tiles);
    int grid = 0;
    if ((st = group_grid(f, tiles(f.pair ? 256 : 128, f.bn), dev, &grid)) != GEMM_OK)
        return st;
    GroupMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    GroupArgs g;
    fill_group(g, bf16, out, dev);
    if ((M > 0 && (!encode_2d(&maps.a, ab_type(bf16), dD, N, M, lddd * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
                   !encode_2d(&maps.b, ab_type(bf16), A, K, M, lda * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))) ||
        !set_out(g, maps, dB, out, N, K, lddb, groups, stride_db))
        return GEMM_ERR_CUDA;
    g.groups = static_cast<int32_t>(groups);
    g.offsets = offsets;
    g.rows = static_cast<int32_t>(M);
    g.M = static_cast<int32_t>(N);
    g.N = static_cast<int32_t>(K);
    g.num_m_blocks = static_cast<int32_t>(ceil_div(N, f.pair ? 256 : 128));
    g.num_n_blocks = static_cast<int32_t>(ceil_div(K, f.bn));
    g.group_m = kGroupM;
    g.alpha = alpha;
    g.loads = M > 0 ? 1 : 0;
    const cudaError_t e = tcg::launch_group_sum(f.bn, f.pair, prec, maps, g, grid, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // extern "C"

namespace tcg {
namespace host {
namespace {

// A product of the Newton-Schulz steps over a stack of `count` matrices: D = alpha op(A) op(B)
// + beta C, M x N, the sum over K; operands float16.
struct BatchProduct {
    int64_t count, M, N, K;
    int maj;  // bit 0: A stored K x M, bit 1: B stored K x N
    bool sym;
    const uint16_t *A;
    int64_t lda, stride_a;
    const uint16_t *B;
    int64_t ldb, stride_b;
    const uint16_t *C;
    int64_t ldc, stride_c;
    void *D;
    int64_t ldd, stride_d;
    int out;
    bool padded;  // D is a workspace: its rows' padding is written too
    float alpha, beta;
    // elements from each matrix to its low part: of A and B operands too where `split`, of C
    // and D where not 0
    bool split;
    int64_t a_lo, b_lo, c_lo, d_lo;
    int64_t parts;  // (sym) D: so many matrices of parts of each sum; 0: whole sums
};

// Parts for the sums of `count` symmetric s x s products over l: as many as leave the tiles (of 64
// columns) to the SMs in one wave, eight K blocks each at least, where the blocks saved (of operands in
// two parts those that two CTAs a tile would not save) take longer than the launch that adds the parts,
// about 5 us.  Five steps, whole sums / parts, us: bf16 20000 x 41 472 / 165, 128 x 8192 214 / 119, 512 x
// 4096 160 / 129, 512 x 2048 118.8 / 119.9, 256 x 1024 88 / 90; float32 512 x 4096 195 / 176, 128 x 2048
// 130 / 113, 512 x 2048 143.5 / 142.7, 2816 x 1024 259 / 273.
int64_t sum_parts(int64_t count, int64_t s, int64_t l, bool split, int sm_count)
{
    const int64_t mb = ceil_div(s, 128), tiles = count * mb * (mb + 1), blocks = ceil_div(l, 64);
    int64_t parts = sm_count / tiles;
    parts = parts < blocks / 8 ? parts : blocks / 8;
    if (parts < 2)
        return 1;
    const int64_t saved_ns = split ? (blocks / 2 - blocks / parts) * kSplitForms[0].block_ns
                                   : (blocks - blocks / parts) * kForms[0].block_ns;
    if (saved_ns < (split ? 3000 : 5000))
        return 1;
    return ceil_div(blocks, ceil_div(blocks, parts));  // (no part is empty)
}

gemm_status run_batch(const BatchProduct &p, const DeviceInfo *dev, cudaStream_t stream)
{
    auto tiles = [&](int tm, int bn) -> int64_t {
        const int64_t mb = ceil_div(p.M, tm);
        if (p.sym)
            return tm < bn ? 0 : p.count * (tm / bn) * (mb * (mb + 1) / 2);
        return p.count * mb * ceil_div(p.N, bn);
    };
    const int prec = p.split ? tcg::kPrecSplit : tcg::kPrecAcc;
    const int64_t parts = p.parts > 1 ? p.parts : 1, k_blocks = ceil_div(p.K, 64);
    const GForm f = parts > 1 ? (p.split ? kSplitForms[0] : kForms[0]) : choose_form(k_blocks, prec, dev->sm_count, tiles);
    const int tm = f.pair ? 256 : 128, b_rows = f.pair ? f.bn / 2 : f.bn;
    int grid = 0;
    gemm_status st = group_grid(f, parts * tiles(tm, f.bn), dev, &grid);
    if (st != GEMM_OK)
        return st;
    GroupMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    GroupArgs g;
    fill_group(g, false, p.out, dev);
    auto map_a = [&](CUtensorMap *m, const uint16_t *x) {
        return (p.maj & 1) ? set_operand(m, false, x, p.M, p.K, p.lda, p.count, p.stride_a, 64)
                           : set_operand(m, false, x, p.K, p.M, p.lda, p.count, p.stride_a, 128);
    };
    auto map_b = [&](CUtensorMap *m, const uint16_t *x) {
        return (p.maj & 2) ? set_operand(m, false, x, p.N, p.K, p.ldb, p.count, p.stride_b, 64)
                           : set_operand(m, false, x, p.K, p.N, p.ldb, p.count, p.stride_b, b_rows);
    };
    if (!map_a(&maps.a, p.A) || !map_b(&maps.b, p.B) ||
        (p.split && (!map_a(&maps.a_lo, p.A + p.a_lo) || !map_b(&maps.b_lo, p.B + p.b_lo))))
        return GEMM_ERR_CUDA;
    const int64_t whole = ceil_div(p.N, 8) * 8, cols = !p.padded ? p.N : (whole < p.ldd ? whole : p.ldd);
    const bool c_tma = p.C && !p.split;
    auto map_c = [&](CUtensorMap *m, const uint16_t *x) {
        return encode_3d(m, ab_type(false), x, p.N, p.M, p.ldc * 2, p.count,
                         p.count == 1 ? p.M * p.ldc * 2 : p.stride_c * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    };
    if (!set_out(g, maps, p.D, p.out, p.M, cols, p.ldd, p.count * parts, p.stride_d, p.d_lo,
                 p.d_lo || !p.split || f.cs == 2) ||
        (c_tma && (!map_c(&maps.c, p.C) || (p.c_lo && !map_c(&maps.c_lo, p.C + p.c_lo)))))
        return GEMM_ERR_CUDA;
    g.c_lo = p.c_lo;
    g.groups = static_cast<int32_t>(p.count);
    g.M = static_cast<int32_t>(p.M);
    g.N = static_cast<int32_t>(p.N);
    g.K = static_cast<int32_t>(p.K);
    g.num_m_blocks = static_cast<int32_t>(ceil_div(p.M, tm));
    g.num_n_blocks = static_cast<int32_t>(ceil_div(p.N, f.bn));
    g.group_m = kGroupM;
    g.alpha = p.alpha;
    g.beta = p.beta;
    g.C = p.C;
    g.ldc = p.ldc;
    g.stride_c = p.stride_c;
    g.parts = static_cast<int32_t>(parts);
    g.part_blocks = static_cast<int32_t>(ceil_div(k_blocks, parts));
    g.loads = 1;
    const cudaError_t e = tcg::launch_group_batch(f.bn, f.pair, p.maj, p.sym, prec, f.cs, maps, g, grid, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

constexpr int64_t kSmallColumns = 1 << 16;  // (a block's elements are 32-bit numbers)
// Thread blocks a matrix for all steps in one launch (1 or 8), or 0 where the tile kernels are faster
// or the matrix does not fit.  Five steps, the tile kernels / one launch, us: bf16 1 x 38 x 24 68 / 19, 1 x
// 1070 x 18 95 / 27, 9 x 128 x 34 84 / 32, 1 x 16 x 4096 87 / 38, 100 x 721 x 20 164 / 61, 1000 x 16 x 64 234 /
// 59, 300 x 32 x 128 107 / 45, 1 x 64 x 512 79 / 77, 1 x 64 x 1024 87 / 103, 1 x 2048 x 48 101 / 116, 16 x 64 x 1024 95 / 204.
int small_blocks(int64_t count, int64_t s, int64_t l, int steps, int out, int sm_count)
{
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    if (fk != 0 || s > 64 || count > kMaxDim / 8)
        return 0;
    const int64_t s4 = ceil_div(s, 4) * 4, blocks = ceil_div(l, 64);
    // the tile kernels': launches, K blocks of X X^T (long sums are shared), waves of tiles
    const int64_t more = ceil_div(count * ceil_div(l, 128), sm_count) - 1;
    int64_t best_ns = (2 + 3 * static_cast<int64_t>(steps)) * 3600 + steps * ((blocks < 30 ? blocks : 30) * 200 + more * 4500);
    if (out == GEMM_OUT_F32)
        best_ns += best_ns / 8;
    int best = 0;
    for (int c = 1; c <= 8; c += 7) {
        const int64_t lc = ceil_div(l, c);
        const size_t shared = tcg::orthogonalize_small_shared(s, l, c);
        if (lc > kSmallColumns || shared > tcg::kSmallShared)
            continue;
        // FMAs of a block's step, 100 a ns; passes over s x s, and what a step waits for; waves (a
        // cluster wants eight free SMs of one group, two small blocks share an SM)
        const int64_t step_ns = (2 * s4 * s4 * lc + s4 * s4 * s4) / 100 + s4 * s4 * 8 / 10 + (c == 1 ? 1700 : 3500);
        const int64_t at_once = c == 8 ? sm_count / 11 : (shared <= tcg::kSmallShared / 2 ? sm_count * 7 / 5 : sm_count);
        const int64_t ns = ceil_div(count, at_once) * (steps * step_ns + 4000);
        if (ns < best_ns) {
            best = c;
            best_ns = ns;
        }
    }
    return best;
}

// Powers of two that keep the float16 iterates (elements up to 1 and a little) and their
// products with themselves (as small as the product of two of their elements) away from
// float16's subnormal numbers.
constexpr float kIterateScale = 4096.0f, kProductScale = 4096.0f;
// Workspace of a call: matrices are taken so many at a time that theirs fit, one at least.
constexpr int64_t kOrthogonalizeBytes = int64_t(1) << 30;

}  // namespace
}  // namespace host
}  // namespace tcg

extern "C" gemm_status gemm_orthogonalize(int64_t count, int64_t M, int64_t N, int type, const void *X, int64_t ldx,
                                          int64_t stride_x, int out, void *Y, int64_t ldy, int64_t stride_y,
                                          int steps, float a, float b, float c, float eps, void *stream)
{
    if (count < 0 || M < 0 || N < 0 || !out_ok(type) || !out_ok(out) || steps < 1 || steps > 100 ||
        !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !(eps >= 0.0f))
        return GEMM_ERR_INVALID_ARG;
    if (count > kMaxDim || M > kMaxRows || N > kMaxRows)
        return GEMM_ERR_UNSUPPORTED;
    if (count == 0 || M == 0 || N == 0)
        return GEMM_OK;
    if (ceil_div(M, 128) > kMaxDim / ceil_div(N, 64) || M > (int64_t(1) << 40) / N)
        return GEMM_ERR_UNSUPPORTED;
    const Stack x{Mat{X, ldx, M, N, out_size(type), false}, count, stride_x};
    const Stack y{Mat{Y, ldy, M, N, out_size(out), false}, count, stride_y};
    gemm_status st = check_stack(x);
    if (st != GEMM_OK || (st = check_stack(y)) != GEMM_OK)
        return st;
    const bool in_place = X == Y && type == out && ldx == ldy && (count == 1 || stride_x == stride_y);
    if (!in_place && any_overlap({span_of(y)}, {span_of(x)}))
        return GEMM_ERR_ALIAS;
    const bool wide = M <= N;
    const int64_t s = wide ? M : N, l = wide ? N : M;
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (const int blocks = small_blocks(count, s, l, steps, out, dev->sm_count)) {
        tcg::SmallArgs q{};
        q.X = X;
        q.ldx = ldx;
        q.stride_x = stride_x;
        q.type = type;
        q.Y = Y;
        q.ldy = ldy;
        q.stride_y = stride_y;
        q.out = out;
        q.s = static_cast<int32_t>(s);
        q.l = static_cast<int32_t>(l);
        q.tall = wide ? 0 : 1;
        q.steps = steps;
        q.cluster = blocks;
        q.a = a;
        q.b = b;
        q.c = c;
        q.eps = eps;
        return tcg::launch_orthogonalize_small(q, count, cs) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    }
    // The iterate is held in two float16 parts, since what its rounding loses in one step the
    // next ones multiply (1000 x 1367, relative to 64 bits: one part 3.1e-3, two 2.7e-4).  The
    // products take the high parts, or, in the last `exact` steps, both, as Y's type asks for
    // (emulated, with 0, 1, 2, 3 such steps: a momentum of 1000 x 1000 3.0e-4, 1.3e-4, 9.8e-5, 2.2e-5,
    // random numbers 1.3e-3, 9.5e-4, 3.8e-4, 8e-6; of 64 x 64 1.7e-3, 1.3e-3, 7.4e-4, 1.8e-4 and 2.1e-3,
    // 1.8e-3, 1.5e-3, 6.4e-4; bfloat16 rounds by 1.7e-3, float16 by 2.1e-4).  Small matrices, which
    // wait for their launches anyway, get two more.
    const int more = s < 256 ? 2 : 0;
    const int wanted = out == GEMM_OUT_F32 ? steps : (out == GEMM_OUT_F16 ? 1 + more : more);
    const int exact = wanted < steps ? wanted : steps;
    // workspace of a matrix: two iterates, the product of one with itself, and the polynomial of that;
    // rows begin on 128-byte lines, or every row of a box would be two requests to L2 (8 x 1000 x 1367
    // float16 528 us with rows of 8 elements' multiples, 427; 32 x 1000 x 1000 1357, 1055)
    const int64_t ldi = ceil_div(N, 64) * 64, ldp = ceil_div(s, 64) * 64;
    const int64_t size_i = ceil_div(M * ldi, 64) * 64, size_p = ceil_div(s * ldp, 64) * 64;
    const int parts = tcg::orthogonalize_parts(M, N);
    const int64_t each = 2 * (4 * size_i + 4 * size_p) + 4 * static_cast<int64_t>(parts);
    int64_t at_once = kOrthogonalizeBytes / each;
    const int64_t tiles_one = ceil_div(M, 128) * ceil_div(N, 64);
    at_once = at_once < count ? at_once : count;
    at_once = at_once < 65535 ? at_once : 65535;  // (a grid's second dimension)
    at_once = at_once < kMaxDim / tiles_one ? at_once : kMaxDim / tiles_one;
    at_once = at_once > 1 ? at_once : 1;
    std::unique_lock<std::mutex> hold(buffer_mutex(dev->index, cs));
    void *w = nullptr;
    // parts of the sums of X X^T (with one operand part or two), float32
    const int64_t parts_of[2] = {sum_parts(at_once, s, l, false, dev->sm_count), sum_parts(at_once, s, l, true, dev->sm_count)};
    const int64_t most_parts = parts_of[0] > parts_of[1] ? parts_of[0] : parts_of[1];
    const int64_t ldq = ceil_div(s, 4) * 4, size_q = ceil_div(s * ldq, 64) * 64;
    const int64_t bytes_q = most_parts > 1 ? at_once * most_parts * size_q * 4 : 0;
    const int64_t bytes = ceil_div(at_once * each, 256) * 256;
    if ((st = get_dequant_buffer(dev->index, cs, kBufOrthogonalize, static_cast<size_t>(bytes + bytes_q), &w)) != GEMM_OK)
        return st;
    const int64_t lo_i = at_once * size_i, lo_p = at_once * size_p;  // to the low parts
    uint16_t *iter[2] = {static_cast<uint16_t *>(w), static_cast<uint16_t *>(w) + 2 * lo_i};
    uint16_t *prod = iter[1] + 2 * lo_i, *poly = prod + 2 * lo_p;
    float *partial = reinterpret_cast<float *>(poly + 2 * lo_p);
    float *sums = reinterpret_cast<float *>(static_cast<uint8_t *>(w) + bytes);
    for (int64_t first = 0; first < count; first += at_once) {
        const int64_t n = count - first < at_once ? count - first : at_once;
        const void *xf = static_cast<const uint8_t *>(X) + first * stride_x * out_size(type);
        void *yf = static_cast<uint8_t *>(Y) + first * stride_y * out_size(out);
        if (tcg::launch_square_sums(xf, ldx, stride_x, type, static_cast<int32_t>(M), static_cast<int32_t>(N),
                                    static_cast<int32_t>(n), partial, parts, cs) != cudaSuccess ||
            tcg::launch_normalize(xf, ldx, stride_x, type, static_cast<int32_t>(M), static_cast<int32_t>(N),
                                  static_cast<int32_t>(n), partial, parts, kIterateScale, eps, iter[0], ldi, size_i,
                                  lo_i, cs) != cudaSuccess)
            return GEMM_ERR_CUDA;
        for (int i = 0; i < steps; ++i) {
            const uint16_t *xi = iter[i % 2];
            const bool last = i == steps - 1, both = i >= steps - exact;
            // P = kProductScale X X^T (or X^T X), on the smaller side
            BatchProduct p{};
            p.count = n;
            p.M = p.N = s;
            p.K = l;
            p.maj = wide ? 0 : 3;
            p.sym = true;
            p.A = p.B = xi;
            p.lda = p.ldb = ldi;
            p.stride_a = p.stride_b = size_i;
            p.D = prod;
            p.ldd = ldp;
            p.stride_d = size_p;
            p.out = GEMM_OUT_F16;
            p.padded = true;
            p.alpha = kProductScale / (kIterateScale * kIterateScale);
            p.split = both;
            p.a_lo = p.b_lo = lo_i;
            p.d_lo = both ? lo_p : 0;
            const int64_t shared = parts_of[both];
            if (shared > 1) {
                p.parts = shared;
                p.D = sums;
                p.ldd = ldq;
                p.stride_d = size_q;
                p.out = GEMM_OUT_F32;
                p.d_lo = 0;
            }
            if ((st = run_batch(p, dev, cs)) != GEMM_OK)
                return st;
            if (shared > 1) {
                if (tcg::launch_join_parts(sums, ldq, size_q, static_cast<int32_t>(shared), static_cast<int32_t>(s),
                                           static_cast<int32_t>(n), prod, ldp, size_p, both ? lo_p : 0, cs) != cudaSuccess)
                    return GEMM_ERR_CUDA;
                p.parts = 0;
                p.ldd = ldp;
                p.stride_d = size_p;
                p.out = GEMM_OUT_F16;
                p.d_lo = both ? lo_p : 0;
            }
            // Q = kProductScale (b P + c P^2)
            p.K = s;
            p.maj = 0;
            p.A = p.B = prod;
            p.lda = p.ldb = ldp;
            p.stride_a = p.stride_b = size_p;
            p.C = prod;
            p.ldc = ldp;
            p.stride_c = size_p;
            p.D = poly;
            p.alpha = c / kProductScale;
            p.beta = b;
            p.a_lo = p.b_lo = lo_p;
            p.c_lo = both ? lo_p : 0;
            if ((st = run_batch(p, dev, cs)) != GEMM_OK)
                return st;
            // X <- a X + Q X (or X Q; Q is symmetric)
            BatchProduct u{};
            u.count = n;
            u.M = M;
            u.N = N;
            u.K = s;
            u.maj = wide ? 2 : 0;
            u.A = wide ? poly : xi;
            u.lda = wide ? ldp : ldi;
            u.stride_a = wide ? size_p : size_i;
            u.B = wide ? xi : poly;
            u.ldb = wide ? ldi : ldp;
            u.stride_b = wide ? size_i : size_p;
            u.C = xi;
            u.ldc = ldi;
            u.stride_c = size_i;
            u.D = last ? yf : iter[1 - i % 2];
            u.ldd = last ? ldy : ldi;
            u.stride_d = last ? stride_y : size_i;
            u.out = last ? out : GEMM_OUT_F16;
            u.padded = !last;
            u.split = both;
            u.a_lo = wide ? lo_p : lo_i;
            u.b_lo = wide ? lo_i : lo_p;
            u.c_lo = lo_i;
            u.d_lo = last ? 0 : lo_i;
            u.alpha = last ? 1.0f / (kIterateScale * kProductScale) : 1.0f / kProductScale;
            u.beta = last ? a / kIterateScale : a;
            if ((st = run_batch(u, dev, cs)) != GEMM_OK)
                return st;
        }
    }
    return GEMM_OK;
}
