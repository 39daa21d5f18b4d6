// api_gated.cu -- the gated feed-forward entry points: gemm_gated and
// gemm_gated_e2m1 (both products, the activation and the product in one
// kernel), gemm_gated_backward, gemm_trans (operands stored K x M / K x N, the
// products of a backward pass) and gemm_quantize_e2m1 (include/tcgemm.h has
// the contracts).  Checks run before any CUDA call, as everywhere.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstring>
#include <initializer_list>

#include "host_internal.h"

namespace tcg {
namespace host {

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int kGroupM = 16;  // block rows per tile-order group, as the plain forms
// FP4: rows of A are a quarter as long, and each group reads all of B's: groups of up to
// 64 block rows that hold 16 MB of A (8192 x 14336 x 4096, 8 / 16 / 32 / 64 block rows with
// the quantiser 379 / 365 / 356 / 351 us; 8192 x 4096 x 14336, 16 / 64 alone 341 / 348;
// bf16 8192 x 14336 x 4096 1018 / 1008 / 1090 / 1085)
int32_t fp4_group_m(int64_t K)
{
    const int64_t rows = (int64_t(1) << 24) / (64 * (K > 0 ? K : 1));  // 128 rows of K / 2 bytes
    return static_cast<int32_t>(rows < kGroupM ? kGroupM : (rows > 64 ? 64 : rows));
}

struct Span {
    const void *p;
    uint64_t bytes;
};

// Whether any of the outputs overlaps an input or another output.
bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(o->p, o->bytes, i.p, i.bytes))
                return true;
        for (const Span *q = o + 1; q != outs.end(); ++q)
            if (overlap(o->p, o->bytes, q->p, q->bytes))
                return true;
    }
    return false;
}

bool out_ok(int out) { return out == GEMM_OUT_F32 || out == GEMM_OUT_BF16 || out == GEMM_OUT_F16; }
bool act_ok(int act) { return act >= GEMM_ACT_SILU && act <= GEMM_ACT_SIGMOID; }
bool elem_aligned(const void *p, int size)
{
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(size - 1)) == 0;
}

// A matrix argument: pointer, leading dimension, rows and columns of `esize`-byte
// elements; `mma`: it is a TMA operand (16-byte base and pitch).
struct Mat {
    const void *p;
    int64_t ld;
    int64_t rows, cols;
    int esize;
    bool mma;
};

gemm_status check_mats(std::initializer_list<Mat> mats)
{
    for (const Mat &m : mats)
        if (m.rows > 0 && m.cols > 0 && (!m.p || m.ld < m.cols))
            return GEMM_ERR_INVALID_ARG;
    for (const Mat &m : mats)
        if (m.ld > kMaxDim)
            return GEMM_ERR_UNSUPPORTED;
    for (const Mat &m : mats)
        if (m.rows > 0 && m.cols > 0 &&
            (m.mma ? !aligned16(m.p) || (m.ld * m.esize) % 16 != 0 : !elem_aligned(m.p, m.esize)))
            return GEMM_ERR_ALIGNMENT;
    return GEMM_OK;
}

Span span_of(const Mat &m) { return Span{m.p, span_bytes(m.rows, m.cols, m.ld, m.esize)}; }

CUtensorMapDataType out_type(int out)
{
    return out == GEMM_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                               : (out == GEMM_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
}

// Boxes of 32 rows x box_cols columns of an output matrix, up to the last column whose row ends on whole 16
// bytes (a store writes 16-byte pieces whole; the kernel stores the columns past it
// one by one)
bool encode_out(CUtensorMap *m, const void *p, int out, int64_t rows, int64_t cols, int64_t ld,
                uint32_t box_cols = 32)
{
    const int64_t per16 = 16 / out_size(out);
    cols = cols / per16 * per16;
    return encode_2d(m, out_type(out), p, cols, rows, ld * out_size(out), box_cols, 32,
                     box_cols * out_size(out) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

bool out_tma(const void *p, int64_t ld, int out, int64_t cols)
{
    return aligned16(p) && (ld * out_size(out)) % 16 == 0 && cols * out_size(out) >= 16;
}

// ---------------------------------------------------------------- gated form

struct GatedProblem {
    int64_t M, N, K;
    bool bf16, fp4;
    const void *A;
    int64_t lda;
    const void *Bg;
    int64_t ldbg;
    const void *Bu;
    int64_t ldbu;
    const uint8_t *As, *Bgs, *Bus;  // (fp4) block scales
    int64_t ldas, ldbgs, ldbus;
    void *G;
    int64_t ldg;
    void *U;
    int64_t ldu;
    void *D;
    int64_t ldd;
    int out, act;
    cudaStream_t stream;
};

gemm_status validate_gated(const GatedProblem &p, bool *empty)
{
    *empty = false;
    if (p.M < 0 || p.N < 0 || p.K < 0 || !out_ok(p.out) || !act_ok(p.act))
        return GEMM_ERR_INVALID_ARG;
    if (p.M > kMaxDim || p.N > kMaxDim || p.K > kMaxDim)
        return GEMM_ERR_UNSUPPORTED;
    if (p.fp4 && p.K % 32 != 0)
        return GEMM_ERR_UNSUPPORTED;  // whole scale blocks only
    if (p.M == 0 || p.N == 0) {
        *empty = true;
        return GEMM_OK;
    }
    const int64_t cols = p.fp4 ? p.K / 2 : p.K;
    const int es = p.fp4 ? 1 : 2;
    const Mat a{p.A, p.lda, p.M, cols, es, true}, bg{p.Bg, p.ldbg, p.N, cols, es, true},
        bu{p.Bu, p.ldbu, p.N, cols, es, true}, d{p.D, p.ldd, p.M, p.N, out_size(p.out), false};
    const int64_t sf = p.fp4 ? p.K / 32 : 0;
    const Mat as{p.As, p.ldas, sf, p.M, 1, false}, bgs{p.Bgs, p.ldbgs, sf, p.N, 1, false},
        bus{p.Bus, p.ldbus, sf, p.N, 1, false};
    const Mat g{p.G, p.ldg, p.G ? p.M : 0, p.N, 2, false}, u{p.U, p.ldu, p.U ? p.M : 0, p.N, 2, false};
    gemm_status st = check_mats({a, bg, bu, d, as, bgs, bus, g, u});
    if (st != GEMM_OK)
        return st;
    if (any_overlap({span_of(d), span_of(g), span_of(u)},
                    {span_of(a), span_of(bg), span_of(bu), span_of(as), span_of(bgs), span_of(bus)}))
        return GEMM_ERR_ALIAS;
    return GEMM_OK;
}

// Tiles of the gated form: D tiles half as wide as the accumulator tile.
void set_gated_tile_plan(gemm_plan &p, int kernel, int bn, int64_t M, int64_t N, int sm_count)
{
    p.kernel = kernel;
    p.bn = bn;
    p.bm = kernel == 3 ? 256 : 128;
    p.stages = tcg::tile_stages(bn, kernel == 3, 1, 1);
    p.tiles = ceil_div(M, p.bm) * ceil_div(N, bn / 2);
    p.splits = 1;
    const int64_t cl = kernel == 3 ? 2 : 1, sets = sm_count / cl;
    p.grid = static_cast<int32_t>(cl * (p.tiles < sets ? p.tiles : sets));
}

// Kernel arguments both forms share.
void fill_gated(GemmArgs &a, const GatedProblem &p, const DeviceInfo *dev)
{
    Problem q{};  // (the fields fill_common reads)
    q.M = p.M;
    q.N = p.N;
    q.K = p.K;
    q.bf16 = p.bf16;
    q.D = p.D;
    q.ldd = p.ldd;
    q.out = p.out;
    q.alpha = 1.0f;
    fill_common(a, q, dev);
    a.act = p.act;
    a.group_m = 1;
    a.splits = 1;
    a.k2_block = INT_MAX;
    a.m2_block = INT_MAX;
    a.d_tma = out_tma(p.D, p.ldd, p.out, p.N) ? 1 : 0;
    a.G = p.G;
    a.ldg = p.ldg;
    a.U = p.U;
    a.ldu = p.ldu;
    const int kind = p.bf16 ? GEMM_OUT_BF16 : GEMM_OUT_F16;
    a.keep_tma =
        (!p.G || out_tma(p.G, p.ldg, kind, p.N)) && (!p.U || out_tma(p.U, p.ldu, kind, p.N)) ? 1 : 0;
}

gemm_status run_gated_skinny(const GatedProblem &p, const gemm_plan &plan, const DeviceInfo *dev)
{
    const int mp = plan.bm;
    GemmMaps maps;
    TileMapsTwo two;
    std::memset(&maps, 0, sizeof(maps));
    std::memset(&two, 0, sizeof(two));
    gemm_status st;
    const int kstage = p.fp4 ? tcg::skinny_mx_kstage() : tcg::skinny_kstage();
    if (p.fp4) {
        const uint8_t *as = nullptr, *bgs = nullptr, *bus = nullptr;
        int64_t ldas = 0, ldbgs = 0, ldbus = 0;
        if ((st = tma_scales(dev, p.stream, kBufScalesA, p.As, p.ldas, p.M, p.K / 32, &as, &ldas)) != GEMM_OK ||
            (st = tma_scales(dev, p.stream, kBufScalesB, p.Bgs, p.ldbgs, p.N, p.K / 32, &bgs, &ldbgs)) != GEMM_OK ||
            (st = tma_scales(dev, p.stream, kBufScalesB2, p.Bus, p.ldbus, p.N, p.K / 32, &bus, &ldbus)) != GEMM_OK)
            return st;
        const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
        const uint32_t sf_rows = static_cast<uint32_t>(kstage / 32);
        if (!encode_2d(&maps.a, u8, p.A, p.K / 2, p.M, p.lda, 128, static_cast<uint32_t>(mp),
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&maps.b, u8, p.Bg, p.K / 2, p.N, p.ldbg, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&two.b2, u8, p.Bu, p.K / 2, p.N, p.ldbu, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&maps.c, u8, bgs, p.N, p.K / 32, ldbgs, 64, sf_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode_2d(&two.sfb2, u8, bus, p.N, p.K / 32, ldbus, 64, sf_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode_2d(&maps.sfa, u8, as, p.M, p.K / 32, ldas, static_cast<uint32_t>(mp), sf_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE))
            return GEMM_ERR_CUDA;
    } else if (!encode_2d(&maps.a, ab_type(p.bf16), p.A, p.K, p.M, p.lda * 2, 64, static_cast<uint32_t>(mp),
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
               !encode_2d(&maps.b, ab_type(p.bf16), p.Bg, p.K, p.N, p.ldbg * 2, 64, 64,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
               !encode_2d(&two.b2, ab_type(p.bf16), p.Bu, p.K, p.N, p.ldbu * 2, 64, 64,
                          CU_TENSOR_MAP_SWIZZLE_128B)) {
        return GEMM_ERR_CUDA;
    }
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    fill_gated(a, p, dev);
    a.num_m_blocks = 1;
    a.num_n_blocks = static_cast<int32_t>(plan.tiles);
    a.num_k_blocks = static_cast<int32_t>(ceil_div(p.K, kstage));
    a.num_tiles = static_cast<int32_t>(plan.tiles);
    a.sk_tiles = static_cast<int32_t>(plan.tiles);  // every tile shared block by block
    a.splits = plan.splits;
    if (plan.splits > 1) {
        Workspace w;
        const size_t bytes = static_cast<size_t>(plan.tiles) * plan.splits * 128 * mp * sizeof(float);
        if ((st = get_workspace(dev->index, p.stream, bytes, static_cast<size_t>(plan.tiles), &w)) != GEMM_OK)
            return st;
        a.workspace = w.partials;
        a.counters = w.counters;
    }
    const cudaError_t e = tcg::launch_skinny_gated(mp, p.fp4, maps, two, a, plan.grid, p.stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status run_gated(const GatedProblem &p)
{
    bool empty = false;
    gemm_status st = validate_gated(p, &empty);
    if (st != GEMM_OK || empty)
        return st;
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    std::unique_lock<std::mutex> hold;
    if (p.fp4)  // (copies of the scales)
        hold = std::unique_lock<std::mutex>(buffer_mutex(dev->index, p.stream));
    const gemm_plan plan = p.fp4 ? gated_e2m1_plan(p.M, p.N, p.K, dev->sm_count)
                                 : gated_plan(p.M, p.N, p.K, p.G || p.U, dev->sm_count);
    if (plan.kernel == 2 || plan.kernel == 15)
        return run_gated_skinny(p, plan, dev);
    const bool pair = plan.kernel == 3;
    const int bn = plan.bn;
    const uint32_t half = static_cast<uint32_t>(bn / 2);  // rows of Bg (Bu) per box
    int grid = plan.grid;
    if (pair) {
        // never more pairs than can be resident together
        const int resident = tcg::tile_max_clusters(256, true, 1, 1);
        if (resident <= 0)
            return GEMM_ERR_CUDA;
        grid = static_cast<int>(2 * (plan.tiles < resident ? plan.tiles : resident));
    }
    GemmMaps maps;
    TileMapsTwo two;
    std::memset(&maps, 0, sizeof(maps));
    std::memset(&two, 0, sizeof(two));
    const int kstage = p.fp4 ? tcg::tile_mx_kstage(1) : 64;
    if (p.K > 0 && p.fp4) {
        const uint8_t *as = nullptr, *bgs = nullptr, *bus = nullptr;
        int64_t ldas = 0, ldbgs = 0, ldbus = 0;
        if ((st = tma_scales(dev, p.stream, kBufScalesA, p.As, p.ldas, p.M, p.K / 32, &as, &ldas)) != GEMM_OK ||
            (st = tma_scales(dev, p.stream, kBufScalesB, p.Bgs, p.ldbgs, p.N, p.K / 32, &bgs, &ldbgs)) != GEMM_OK ||
            (st = tma_scales(dev, p.stream, kBufScalesB2, p.Bus, p.ldbus, p.N, p.K / 32, &bus, &ldbus)) != GEMM_OK)
            return st;
        const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
        const uint32_t sf_rows = static_cast<uint32_t>(kstage / 32);
        if (!encode_2d(&maps.a, u8, p.A, p.K / 2, p.M, p.lda, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&maps.b, u8, p.Bg, p.K / 2, p.N, p.ldbg, 128, half, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&two.b2, u8, p.Bu, p.K / 2, p.N, p.ldbu, 128, half, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&maps.sfa, u8, as, p.M, p.K / 32, ldas, 128, sf_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode_2d(&maps.sfb, u8, bgs, p.N, p.K / 32, ldbgs, half, sf_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode_2d(&two.sfb2, u8, bus, p.N, p.K / 32, ldbus, half, sf_rows, CU_TENSOR_MAP_SWIZZLE_NONE))
            return GEMM_ERR_CUDA;
    } else if (p.K > 0) {
        const CUtensorMapDataType t = ab_type(p.bf16);
        if (!encode_2d(&maps.a, t, p.A, p.K, p.M, p.lda * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&maps.b, t, p.Bg, p.K, p.N, p.ldbg * 2, 64, half, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&two.b2, t, p.Bu, p.K, p.N, p.ldbu * 2, 64, half, CU_TENSOR_MAP_SWIZZLE_128B))
            return GEMM_ERR_CUDA;
    }
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    fill_gated(a, p, dev);
    const int keep = p.bf16 ? GEMM_OUT_BF16 : GEMM_OUT_F16;
    // (the FP4 form stores 64 bytes of a row at a time)
    const uint32_t d_cols = p.fp4 && p.out == GEMM_OUT_F32 ? 16 : 32;
    if ((a.d_tma && !encode_out(&maps.d, p.D, p.out, p.M, p.N, p.ldd, d_cols)) ||
        (a.keep_tma && p.G && !encode_out(&two.d2, p.G, keep, p.M, p.N, p.ldg)) ||
        (a.keep_tma && p.U && !encode_out(&two.d3, p.U, keep, p.M, p.N, p.ldu)))
        return GEMM_ERR_CUDA;
    a.num_m_blocks = static_cast<int32_t>(ceil_div(p.M, plan.bm));
    a.num_n_blocks = static_cast<int32_t>(ceil_div(p.N, bn / 2));
    a.num_k_blocks = static_cast<int32_t>(ceil_div(p.K, kstage));
    a.num_tiles = static_cast<int32_t>(plan.tiles);
    const int32_t group_m = p.fp4 ? fp4_group_m(p.K) : kGroupM;
    a.group_m = a.num_m_blocks < group_m ? a.num_m_blocks : group_m;
    const bool rows = !a.d_tma || !a.keep_tma;
    const cudaError_t e = p.fp4 ? tcg::launch_tile_gated_mx(bn, rows, maps, two, a, grid, p.stream)
                                : tcg::launch_tile_gated(bn, pair, rows, maps, two, a, grid, p.stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// ---------------------------------------------------------------- transposed storage

// D = fma.rn(alpha, op(A) op(B), beta C).  A second source: K blocks that follow
// (A2, B2: D also gets op(A2) op(B2)), or block rows that follow (A2, D2: D2
// = op(A2) op(B)).
struct TransProblem {
    int64_t M, N, K;
    bool bf16, ta, tb;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    const float *C;
    int64_t ldc;
    void *D;
    int64_t ldd;
    int out;
    float alpha, beta;
    cudaStream_t stream;
    const void *A2 = nullptr;
    int64_t lda2 = 0;
    const void *B2 = nullptr;
    int64_t ldb2 = 0;
    void *D2 = nullptr;
    int64_t ldd2 = 0;
    // launched right behind a kernel that it does not depend on, but that waited
    // for what it does depend on: it starts on the SMs that kernel leaves idle
    bool co_tail = false;
    int parts_use = kBufParts;  // buffer for the parts of a sum (its own for each product under way)
};

// One way to run a product: the tile kernel's form, and how its sums are cut
// (parts of k_part K blocks; 1: not cut).  Time: waves of tiles (of every source and
// part) x tile_ns + extra_ns.
struct Form {
    int kernel, bn, parts;
    int64_t k_part, tiles, tile_ns, extra_ns;
};

constexpr int kMaxForms = 9;

int64_t form_ns(const Form &f, int64_t sms)
{
    const int64_t sets = f.kernel == 1 ? sms : sms / 2;
    return sets > 0 ? ceil_div(f.tiles, sets) * f.tile_ns + f.extra_ns : INT64_MAX / 4;
}

// The forms of a product, with their times in ns.  A tile takes its K blocks x the
// time of one (the operand bytes from L2 to an SM: 190, 260 and 390 for 64, 128 and 256
// columns, 280 and 532 for a pair's 256 x 256 and 256 x 512) and a fixed part, its
// epilogue as far as the next tile's MMAs do not hide it.  A product with few tiles
// and a long sum leaves most SMs idle: it may be cut, in at least 8 K blocks a part,
// and the parts' float32 results added in a second kernel (4000 and its bytes).  (Whole /
// in parts, or parts on single CTAs / on pairs: 512 x 512 x 8192 36 / 14 us, 512 x 4096 x
// 14336 60 / 53, 256 x 4096 x 14336 38 / 35.)
// Against measurements (64 / 128 / 256 columns / pairs / 512-wide pairs, us): two
// sources stacked along M, 2816 x 1024 x 2048 47 / 34 / 30 / 26 / 25; 911 x 6867 x 606
// 19.3 / 14.3 / 15.4 / 13.2 / 13.7; 460 x 6030 x 397 9.8 / 8.3 / 6.9 / 7.5 / 11.1.
int trans_forms(int64_t M, int64_t N, int64_t K, int m_sources, int k_sources, int stored, int sm_count,
                Form (&out)[kMaxForms])
{
    struct Step {
        int kernel, bn;
        int64_t block_ns, fixed_ns;
    };
    constexpr Step steps[5] = {{1, 64, 190, 300}, {1, 128, 260, 500}, {1, 256, 390, 600}, {3, 256, 280, 1500},
                               {4, 512, 532, 3000}};
    const int64_t kb = k_sources * ceil_div(K, 64);
    int n = 0;
    for (const Step &s : steps) {
        // A short sum leaves the stores to set the time: single CTAs, which start and
        // finish a tile without the pair's hand-overs (two sources stacked along M, 14336
        // x 4096 each, 16-bit: K = 16 24.8 against 34.0 us, 256 31.9 / 40.9, 1024 85.7 /
        // 72.1; both stored K x M, 2020 x 10164: K = 320 23.7 / 23.7, 384 26.5 / 24.7)
        if (s.kernel != 1 && (k_sources * K <= 320 || (s.kernel == 4 && N <= 256)))
            continue;
        // Up to 8 rows stored K x M are one 16-byte piece of each of K lines that every
        // CTA reads: fewer, wider tiles (64 / 128 / 256 columns: 3 x 6279 x 1534 23.7 / 12.7
        // / 15.2 us, 1 x 5894 x 387 11.4 / 6.0 / 6.9, 5 x 13769 x 2288 37.9 / 29.6 / 22.9)
        if (M <= 8 && (stored & 1) && (s.kernel != 1 || s.bn != (ceil_div(N, 128) <= 64 ? 128 : 256)))
            continue;
        Form f{s.kernel, s.bn, 1, kb, 0, kb * s.block_ns + s.fixed_ns, 0};
        f.tiles = m_sources * ceil_div(M, s.kernel == 1 ? 128 : 256) * ceil_div(N, s.bn);
        out[n++] = f;
        const int64_t sets = s.kernel == 1 ? sm_count : sm_count / 2;
        if (s.kernel == 4 || kb < 16 || f.tiles > sets || (M <= 8 && (stored & 1)))
            continue;
        Form cut = f;
        int64_t cut_ns = INT64_MAX;
        for (int64_t parts = 2; parts <= 16 && parts * f.tiles <= sets && kb / parts >= 8; ++parts) {
            const int64_t k_part = ceil_div(kb, parts);
            if ((parts - 1) * k_part >= kb)
                continue;  // (the last part would be empty)
            // written and read once each, mostly in L2: 4 + 4 bytes at ~6 KB a ns
            Form c = f;
            c.parts = static_cast<int>(parts);
            c.k_part = k_part;
            c.tiles = parts * f.tiles;
            c.tile_ns = k_part * s.block_ns + s.fixed_ns;
            c.extra_ns = 4000 + m_sources * M * N * 8 * parts / 6000;
            if (form_ns(c, sm_count) < cut_ns) {
                cut_ns = form_ns(c, sm_count);
                cut = c;
            }
        }
        if (cut.parts > 1)
            out[n++] = cut;
    }
    return n;
}

void set_form_plan(gemm_plan &p, const Form &f, int64_t M, int64_t N, int64_t sms)
{
    set_tile_plan(p, f.kernel, f.bn, M, N, static_cast<int>(sms));
    p.splits = f.parts;
    p.tiles = f.tiles;
    const int64_t cl = f.kernel == 1 ? 1 : 2, sets = sms / cl;
    p.grid = static_cast<int32_t>(cl * (p.tiles < sets ? p.tiles : sets));
}

void fill_trans(GemmArgs &a, const TransProblem &p, const DeviceInfo *dev)
{
    Problem q{};  // (the fields fill_common reads)
    q.M = p.M;
    q.N = p.N;
    q.K = p.K;
    q.bf16 = p.bf16;
    q.C = p.C;
    q.ldc = p.ldc;
    q.D = p.D;
    q.ldd = p.ldd;
    q.out = p.out;
    q.alpha = p.alpha;
    q.beta = p.beta;
    fill_common(a, q, dev);
}

// M <= 64 rows of A as stored, B stored K x N: the skinny kernel.
gemm_status run_trans_skinny(const TransProblem &p, const gemm_plan &plan, const DeviceInfo *dev)
{
    GemmMaps maps;
    TileMapsTwo two;
    std::memset(&maps, 0, sizeof(maps));
    std::memset(&two, 0, sizeof(two));
    const CUtensorMapDataType t = ab_type(p.bf16);
    const uint32_t mp = static_cast<uint32_t>(plan.bm);
    auto map_a = [&](CUtensorMap *m, const void *A, int64_t lda) {
        return encode_2d(m, t, A, p.K, p.M, lda * 2, 64, mp, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto map_b = [&](CUtensorMap *m, const void *B, int64_t ldb) {
        return encode_2d(m, t, B, p.N, p.K, ldb * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    // (without a second source, its descriptors are the first's)
    if (!map_a(&maps.a, p.A, p.lda) || !map_b(&maps.b, p.B, p.ldb) ||
        !map_a(&two.a2, p.A2 ? p.A2 : p.A, p.A2 ? p.lda2 : p.lda) ||
        !map_b(&two.b2, p.B2 ? p.B2 : p.B, p.B2 ? p.ldb2 : p.ldb))
        return GEMM_ERR_CUDA;
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    fill_trans(a, p, dev);
    const int64_t k_blocks = ceil_div(p.K, tcg::skinny_kstage());
    a.num_m_blocks = 1;
    a.num_n_blocks = static_cast<int32_t>(plan.tiles);
    a.num_k_blocks = static_cast<int32_t>(p.B2 ? 2 * k_blocks : k_blocks);
    a.num_tiles = static_cast<int32_t>(plan.tiles);
    a.sk_tiles = static_cast<int32_t>(plan.tiles);  // every tile shared block by block
    a.group_m = 1;
    a.splits = plan.splits;
    a.k2_block = p.B2 ? static_cast<int32_t>(k_blocks) : INT_MAX;
    if (plan.splits > 1) {
        Workspace w;
        const size_t bytes = static_cast<size_t>(plan.tiles) * plan.splits * 128 * mp * sizeof(float);
        const gemm_status st =
            get_workspace(dev->index, p.stream, bytes, static_cast<size_t>(plan.tiles), &w);
        if (st != GEMM_OK)
            return st;
        a.workspace = w.partials;
        a.counters = w.counters;
    }
    const cudaError_t e = tcg::launch_skinny_trans(plan.bm, maps, two, a, plan.grid, p.stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// The second kernel of a product in parts (parts 0: there is none).
struct AddParts {
    const float *W = nullptr;
    int64_t ldw = 0, part_rows = 0, second = 0;  // second: rows before the second stacked source's
    int parts = 0;
};

// Whether the product of this plan goes through a buffer of parts.
bool in_parts(const gemm_plan &plan) { return plan.kernel != 2 && plan.splits > 1; }

// Add the parts of the product p.
gemm_status add_parts(const TransProblem &p, const AddParts &add)
{
    if (add.parts == 0)
        return GEMM_OK;
    const bool c_used = p.C != nullptr && p.beta != 0.0f;
    for (int i = 0; i < (p.D2 ? 2 : 1); ++i)
        if (tcg::launch_add_parts(add.W + i * add.second * add.ldw, add.ldw, add.part_rows, add.parts,
                                  c_used ? p.C : nullptr, p.ldc, i == 0 ? p.D : p.D2, i == 0 ? p.ldd : p.ldd2,
                                  p.out, p.alpha, p.beta, static_cast<int32_t>(p.M),
                                  static_cast<int32_t>(p.N), p.stream) != cudaSuccess)
            return GEMM_ERR_CUDA;
    return GEMM_OK;
}

// Launch the product (arguments already checked; M, N > 0).  In parts, *add says
// what add_parts has to add.
gemm_status run_trans(const TransProblem &p, gemm_plan plan, const DeviceInfo *dev, AddParts *add)
{
    const bool c_used = p.C != nullptr && p.beta != 0.0f;
    const int stored = (p.ta ? 1 : 0) | (p.tb ? 2 : 0);
    if (plan.kernel == 2)
        return run_trans_skinny(p, plan, dev);
    const int parts = plan.splits;
    const bool pair = plan.kernel != 1;
    const int nsub = plan.kernel == 4 ? 2 : 1;
    const int bn = pair ? 256 : plan.bn;
    int grid = plan.grid;
    if (pair) {
        const int resident = tcg::tile_max_clusters(256, true, nsub, 1);
        if (resident <= 0)
            return GEMM_ERR_CUDA;
        grid = grid < 2 * resident ? grid : 2 * resident;
    }
    GemmMaps maps;
    TileMapsTwo two;
    std::memset(&maps, 0, sizeof(maps));
    std::memset(&two, 0, sizeof(two));
    const CUtensorMapDataType t = ab_type(p.bf16);
    const uint32_t b_rows = static_cast<uint32_t>(pair ? bn / 2 : bn);
    // K-major: boxes of 64 K x the tile's rows; stored the other way: 64 columns x 64 K
    auto map_a = [&](CUtensorMap *m, const void *A, int64_t lda) {
        return p.ta ? encode_2d(m, t, A, p.M, p.K, lda * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                    : encode_2d(m, t, A, p.K, p.M, lda * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto map_b = [&](CUtensorMap *m, const void *B, int64_t ldb) {
        return p.tb ? encode_2d(m, t, B, p.N, p.K, ldb * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                    : encode_2d(m, t, B, p.K, p.N, ldb * 2, 64, b_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (p.K > 0 && (!map_a(&maps.a, p.A, p.lda) || !map_b(&maps.b, p.B, p.ldb) ||
                    (p.A2 && !map_a(&two.a2, p.A2, p.lda2)) || (p.B2 && !map_b(&two.b2, p.B2, p.ldb2))))
        return GEMM_ERR_CUDA;
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    fill_trans(a, p, dev);
    const int64_t m_blocks = ceil_div(p.M, plan.bm), k_blocks = ceil_div(p.K, 64);
    const bool more_k = p.B2 != nullptr, more_m = p.D2 != nullptr;
    if (parts > 1) {
        // every part's tiles, one part's block rows after the other, into a float32
        // workspace of whole tiles' rows; C, alpha and D's type come with the adding
        const int64_t part_m = more_m ? 2 * m_blocks : m_blocks;
        const int64_t ldw = ceil_div(p.N, 4) * 4, rows = parts * part_m * plan.bm;
        void *w = nullptr;
        const gemm_status st = get_dequant_buffer(dev->index, p.stream, p.parts_use,
                                                  static_cast<size_t>(rows) * ldw * sizeof(float), &w);
        if (st != GEMM_OK)
            return st;
        a.M = static_cast<int32_t>(rows);
        a.alpha = 1.0f;
        a.has_c = 0;
        a.D = w;
        a.ldd = ldw;
        a.out_kind = GEMM_OUT_F32;
        a.part_m = static_cast<int32_t>(part_m);
        a.num_m_blocks = static_cast<int32_t>(parts * part_m);
        a.num_n_blocks = static_cast<int32_t>(ceil_div(p.N, bn));
        a.num_k_blocks = static_cast<int32_t>(ceil_div(more_k ? 2 * k_blocks : k_blocks, parts));
        a.num_tiles = a.num_m_blocks * a.num_n_blocks;
        a.k2_block = more_k ? static_cast<int32_t>(k_blocks) : INT_MAX;
        a.m2_block = more_m ? static_cast<int32_t>(m_blocks) : INT_MAX;
        a.group_m = a.num_m_blocks < kGroupM ? a.num_m_blocks : kGroupM;
        a.splits = 1;
        a.d_tma = 1;
        a.co_tail = p.co_tail ? 1 : 0;
        // (the pitch is whole 16 bytes: a row's padding is written too)
        if (!encode_out(&maps.d, w, GEMM_OUT_F32, rows, ldw, ldw))
            return GEMM_ERR_CUDA;
        a.N = static_cast<int32_t>(ldw);
        add->W = static_cast<const float *>(w);
        add->ldw = ldw;
        add->part_rows = part_m * plan.bm;
        add->second = m_blocks * plan.bm;
        add->parts = parts;
        const cudaError_t e = tcg::launch_tile_major(stored, bn, pair, 1, maps, two, a, grid, p.stream);
        return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    }
    a.num_m_blocks = static_cast<int32_t>(more_m ? 2 * m_blocks : m_blocks);
    a.num_n_blocks = static_cast<int32_t>(ceil_div(p.N, bn * nsub));
    a.num_k_blocks = static_cast<int32_t>(more_k ? 2 * k_blocks : k_blocks);
    a.num_tiles = a.num_m_blocks * a.num_n_blocks;
    a.k2_block = more_k ? static_cast<int32_t>(k_blocks) : INT_MAX;
    a.m2_block = more_m ? static_cast<int32_t>(m_blocks) : INT_MAX;
    a.group_m = a.num_m_blocks < kGroupM ? a.num_m_blocks : kGroupM;
    a.splits = 1;
    a.c_tma = c_used && aligned16(p.C) && (p.ldc * 4) % 16 == 0 ? 1 : 0;
    a.d_tma =
        out_tma(p.D, p.ldd, p.out, p.N) && (!more_m || out_tma(p.D2, p.ldd2, p.out, p.N)) ? 1 : 0;
    a.D2 = p.D2;
    a.ldd2 = p.ldd2;
    a.co_tail = p.co_tail ? 1 : 0;
    a.d_wide = a.d_tma && !c_used && p.out != GEMM_OUT_F32 ? 1 : 0;
    const uint32_t d_cols = a.d_wide ? 64 : 32;
    if ((a.c_tma && !encode_2d(&maps.c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.C, p.N, p.M, p.ldc * 4, 32, 32,
                               CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (a.d_tma && !encode_out(&maps.d, p.D, p.out, p.M, p.N, p.ldd, d_cols)) ||
        (a.d_tma && more_m && !encode_out(&two.d2, p.D2, p.out, p.M, p.N, p.ldd2, d_cols)))
        return GEMM_ERR_CUDA;
    const cudaError_t e = tcg::launch_tile_major(stored, bn, pair, nsub, maps, two, a, grid, p.stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status check_trans(const TransProblem &p)
{
    if (p.M < 0 || p.N < 0 || p.K < 0 || !out_ok(p.out))
        return GEMM_ERR_INVALID_ARG;
    if (p.M > kMaxDim || p.N > kMaxDim || p.K > kMaxDim)
        return GEMM_ERR_UNSUPPORTED;
    if (p.M == 0 || p.N == 0)
        return GEMM_OK;
    const bool c_used = p.C != nullptr && p.beta != 0.0f;
    const Mat a{p.A, p.lda, p.ta ? p.K : p.M, p.ta ? p.M : p.K, 2, true};
    const Mat b{p.B, p.ldb, p.tb ? p.K : p.N, p.tb ? p.N : p.K, 2, true};
    const Mat c{p.C, p.ldc, c_used ? p.M : 0, p.N, 4, false};
    const Mat d{p.D, p.ldd, p.M, p.N, out_size(p.out), false};
    gemm_status st = check_mats({a, b, c, d});
    if (st != GEMM_OK)
        return st;
    if (any_overlap({span_of(d)}, {span_of(a), span_of(b)}))
        return GEMM_ERR_ALIAS;
    const bool in_place = c_used && static_cast<const void *>(p.C) == p.D && p.out == GEMM_OUT_F32 &&
                          p.ldc == p.ldd;
    if (c_used && !in_place && any_overlap({span_of(d)}, {span_of(c)}))
        return GEMM_ERR_ALIAS;
    return GEMM_OK;
}

}  // namespace

gemm_plan gated_plan(int64_t M, int64_t N, int64_t K, bool keep, int sm_count)
{
    gemm_plan p;
    std::memset(&p, 0, sizeof(p));
    if (M == 0 || N == 0)
        return p;
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    // M <= 64 rows: as the plain form decides between the two kernels, for the
    // 2 N rows of both weight matrices (the skinny kernel keeps no products)
    const bool skinny_ok = M <= 64 && K > 0 && !keep;
    if (skinny_ok && (fk == 2 || (fk != 1 && fk != 3 && skinny_wins(M, 2 * N, K)))) {
        set_skinny_plan(p, M, 128 * ceil_div(N, 64), K, sm_count, false);
        return p;
    }
    if (fk == 1 || (fk == 3 && K > 0)) {
        set_gated_tile_plan(p, fk, fbn, M, N, sm_count);
        return p;
    }
    // waves of CTAs (pairs) x accumulator width plus a fixed cost per tile, pairs
    // at 0.8 (each SM moves 2/3 of the operand bytes; 128 columns / pairs, 2973 x 1184 x
    // 1073: 3 waves 22.9 us, 2 waves 19.4; 777 x 2743 x 1000: 2 waves 16.5, 2 18.8);
    // short sums on single CTAs, whose tiles end without the pair's hand-over
    // (single / pair, 4096 x 14336, bf16: K = 128 63 / 76 us, 512 85 / 90, 1024 150 / 132)
    int kernel = 1, bn = 256;
    double best = -1.0;
    for (int w : {256, 128, 64}) {
        const int64_t tiles = ceil_div(M, 128) * ceil_div(N, w / 2);
        const double cost = static_cast<double>(ceil_div(tiles, sm_count) * (w + 32));
        if (best < 0 || cost < best) {
            best = cost;
            bn = w;
        }
    }
    const int pairs = sm_count / 2;
    if (K >= 768 && pairs > 0) {
        const int64_t tiles = ceil_div(M, 256) * ceil_div(N, 128);
        if (0.8 * static_cast<double>(ceil_div(tiles, pairs) * (256 + 32)) <= best) {
            kernel = 3;
            bn = 256;
        }
    }
    set_gated_tile_plan(p, kernel, bn, M, N, sm_count);
    return p;
}

gemm_plan gated_e2m1_plan(int64_t M, int64_t N, int64_t K, int sm_count)
{
    gemm_plan p;
    std::memset(&p, 0, sizeof(p));
    if (M == 0 || N == 0)
        return p;
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    // M <= 64: the skinny kernel, except for short sums, over one wave of tiles at that,
    // where its join of the parts costs more than the sum (skinny / tile: 8 x 934 x 384
    // 7.4 / 5.4 us, 16 x 5632 x 2048 9.7 / 6.8, 52 x 3012 x 3488 11.1 / 9.3, 2 x 12529 x 64
    // 7.9 / 6.7; 32 x 8192 x 1024 5.8 / 6.1, 16 x 2048 x 2048 6.8 / 7.1, 8 x 14336 x 512
    // 6.1 / 7.5)
    const bool one_wave = ceil_div(N, 64) <= sm_count;
    if (M <= 64 && K > 256 && fk != 11 && !(one_wave && K < (M > 16 || N >= 4096 ? 4096 : 2048))) {
        set_e2m1_skinny_plan(p, M, ceil_div(N, 64), K, sm_count);
        return p;
    }
    // 256 columns: half as much of A is read, and a wave of tiles takes about 1.6 times
    // as long (128 / 256 columns: 2048 x 4096 x 4096 7 / 4 waves 47 / 33 us, 1024 x 14336 x
    // 1024 12 / 6 26 / 23, 200 x 14336 x 4096 3 / 2 22.9 / 22.5, 512 x 4096 x 1024 2 / 1 7.6 /
    // 7.6, 300 x 1000 x 4096 1 / 1 9.8 / 12.4), but for the shortest sums (4096 x 14336 x 512
    // 48 / 24 67 / 72, 1763 x 7578 x 288 11 / 6 18.7 / 21.3)
    const int64_t w128 = ceil_div(ceil_div(M, 128) * ceil_div(N, 64), sm_count);
    const int64_t w256 = ceil_div(ceil_div(M, 128) * ceil_div(N, 128), sm_count);
    const int bn = fk == 11 ? fbn : (K > 512 && 3 * w256 <= 2 * w128 ? 256 : 128);
    p.kernel = 11;
    p.bm = 128;
    p.bn = bn;
    p.stages = tcg::tile_gated_mx_stages(bn);
    p.tiles = ceil_div(M, 128) * ceil_div(N, bn / 2);
    p.splits = 1;
    p.grid = static_cast<int32_t>(p.tiles < sm_count ? p.tiles : sm_count);
    return p;
}

// m_sources, k_sources: sources stacked along M (their block rows count as one
// problem's) and along K (one longer sum); stored: bit 0 A K x M, bit 1 B K x N.
gemm_plan trans_plan(int64_t M, int64_t N, int64_t K, int m_sources, int k_sources, int stored, int sm_count)
{
    gemm_plan p;
    std::memset(&p, 0, sizeof(p));
    if (M == 0 || N == 0)
        return p;
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    // few rows of A: the skinny kernel, where it shares a long sum over the SMs and B
    // is long enough to stream; a sum in parts has less to join (skinny / parts, 16 and 64
    // rows, bf16: 2816 x 1024 9.3 / 8.7 and 11.6 / 8.5 us, 16384 x 512 17.1 / 11.6 and 23.3 /
    // 11.8, 5632 x 2048 12.1 / 11.8 and 14.9 / 12.0; 4096 x 4096 11.9 / 14.7 and 14.1 / 13.3,
    // 14336 x 4096 24.0 / 29.4 and 27.2 / 30.8)
    const bool skinny_ok = M <= 64 && K > 0 && stored == 2 && m_sources == 1;
    const bool streams = k_sources * K <= INT64_MAX / N && k_sources * K * N > 12 << 20;
    if (skinny_ok && (fk == 2 || (fk != 1 && fk != 3 && fk != 4 && streams && skinny_wins(M, N, k_sources * K)))) {
        set_skinny_plan(p, M, N, k_sources * ceil_div(K, tcg::skinny_kstage()) * tcg::skinny_kstage(),
                        sm_count, false);
        return p;
    }
    Form forms[kMaxForms];
    const int n = trans_forms(M, N, K, m_sources, k_sources, stored, sm_count, forms);
    Form best = forms[0];
    for (int i = 1; i < n; ++i)
        if (form_ns(forms[i], sm_count) <= form_ns(best, sm_count))
            best = forms[i];
    if (fk == 1 || ((fk == 3 || fk == 4) && K > 0)) {
        best = Form{fk, fbn, 1, 0, 0, 0, 0};
        best.tiles = m_sources * ceil_div(M, fk == 1 ? 128 : 256) * ceil_div(N, fbn);
    }
    set_form_plan(p, best, M, N, sm_count);
    return p;
}

namespace {

// The plans of a product and of one that starts on the SMs it leaves (both tile
// kernels with static schedules): either the second also takes the first one's SMs, and
// its last CTAs start once those are done, or it keeps to the rest.  (All gradients,
// bf16, the second product spread over every SM by its own best form / planned together:
// 1000 x 1367 x 1000 30.9 / 26.0 us, 2048 x 2816 x 1024 71.6 / 41.7, 3000 x 700 x 700
// 30.9 / 25.3, 8192 x 5632 x 2048 512 / 525.)
void plan_side_by_side(const TransProblem &a, const TransProblem &b, int sm_count, gemm_plan *plan_a,
                       gemm_plan *plan_b)
{
    Form fa[kMaxForms], fb[kMaxForms];
    const int na = trans_forms(a.M, a.N, a.K, 1, 2, 2, sm_count, fa);
    const int nb = trans_forms(b.M, b.N, b.K, 2, 1, 3, sm_count, fb);
    int64_t best = INT64_MAX;
    int best_a = 0, best_b = 0;
    int64_t best_sms = sm_count;
    for (int i = 0; i < na; ++i) {
        const int64_t ns = form_ns(fa[i], sm_count), cl = fa[i].kernel == 1 ? 1 : 2;
        const int64_t used = cl * fa[i].tiles < sm_count ? cl * fa[i].tiles : sm_count;
        for (int j = 0; j < nb; ++j) {
            const int64_t after = ns + form_ns(fb[j], sm_count);
            const int64_t beside = form_ns(fb[j], sm_count - used);
            const int64_t both = beside > ns ? beside : ns;
            if (both < best || after < best) {
                best = both <= after ? both : after;
                best_a = i;
                best_b = j;
                best_sms = both <= after ? sm_count - used : sm_count;
            }
        }
    }
    std::memset(plan_a, 0, sizeof(*plan_a));
    std::memset(plan_b, 0, sizeof(*plan_b));
    set_form_plan(*plan_a, fa[best_a], a.M, a.N, sm_count);
    set_form_plan(*plan_b, fb[best_b], b.M, b.N, best_sms);
}

}  // namespace

gemm_plan plan_of_trans(const TransProblem &p, const DeviceInfo *dev)
{
    const int stored = (p.ta ? 1 : 0) | (p.tb ? 2 : 0);
    return trans_plan(p.M, p.N, p.K, p.D2 ? 2 : 1, p.B2 ? 2 : 1, stored, dev->sm_count);
}

}  // namespace host
}  // namespace tcg

using namespace tcg::host;

extern "C" {

gemm_status gemm_gated(int64_t M, int64_t N, int64_t K, int dtype_is_bf16, const void *A, int64_t lda,
                       const void *Bg, int64_t ldbg, const void *Bu, int64_t ldbu, void *G, int64_t ldg,
                       void *U, int64_t ldu, void *D, int64_t ldd, int out, int act, void *stream)
{
    if (dtype_is_bf16 != 0 && dtype_is_bf16 != 1)
        return GEMM_ERR_INVALID_ARG;
    GatedProblem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.bf16 = dtype_is_bf16 == 1;
    p.A = A;
    p.lda = lda;
    p.Bg = Bg;
    p.ldbg = ldbg;
    p.Bu = Bu;
    p.ldbu = ldbu;
    p.G = G;
    p.ldg = ldg;
    p.U = U;
    p.ldu = ldu;
    p.D = D;
    p.ldd = ldd;
    p.out = out;
    p.act = act;
    p.stream = static_cast<cudaStream_t>(stream);
    return run_gated(p);
}

gemm_status gemm_gated_e2m1(int64_t M, int64_t N, int64_t K, const uint8_t *Aq, int64_t ldaq,
                            const uint8_t *As, int64_t ldas, const uint8_t *Bgq, int64_t ldbgq,
                            const uint8_t *Bgs, int64_t ldbgs, const uint8_t *Buq, int64_t ldbuq,
                            const uint8_t *Bus, int64_t ldbus, void *D, int64_t ldd, int out, int act,
                            void *stream)
{
    GatedProblem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.fp4 = true;
    p.A = Aq;
    p.lda = ldaq;
    p.As = As;
    p.ldas = ldas;
    p.Bg = Bgq;
    p.ldbg = ldbgq;
    p.Bgs = Bgs;
    p.ldbgs = ldbgs;
    p.Bu = Buq;
    p.ldbu = ldbuq;
    p.Bus = Bus;
    p.ldbus = ldbus;
    p.D = D;
    p.ldd = ldd;
    p.out = out;
    p.act = act;
    p.stream = static_cast<cudaStream_t>(stream);
    return run_gated(p);
}

gemm_status gemm_trans(int64_t M, int64_t N, int64_t K, int dtype_is_bf16, int trans_a, const void *A,
                       int64_t lda, int trans_b, const void *B, int64_t ldb, const float *C, int64_t ldc,
                       void *D, int64_t ldd, int out, float alpha, float beta, void *stream)
{
    if ((dtype_is_bf16 != 0 && dtype_is_bf16 != 1) || (trans_a != 0 && trans_a != 1) ||
        (trans_b != 0 && trans_b != 1))
        return GEMM_ERR_INVALID_ARG;
    if (trans_a == 0 && trans_b == 0) {
        const Problem q{M, N, K, dtype_is_bf16 == 1, A, M, lda, nullptr, B, ldb, C, ldc, D, ldd,
                        out, alpha, beta, false, static_cast<cudaStream_t>(stream)};
        return run(q);
    }
    TransProblem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.bf16 = dtype_is_bf16 == 1;
    p.ta = trans_a == 1;
    p.tb = trans_b == 1;
    p.A = A;
    p.lda = lda;
    p.B = B;
    p.ldb = ldb;
    p.C = C;
    p.ldc = ldc;
    p.D = D;
    p.ldd = ldd;
    p.out = out;
    p.alpha = alpha;
    p.beta = beta;
    p.stream = static_cast<cudaStream_t>(stream);
    gemm_status st = check_trans(p);
    if (st != GEMM_OK || M == 0 || N == 0)
        return st;
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const gemm_plan plan = plan_of_trans(p, dev);
    std::unique_lock<std::mutex> hold;
    if (in_parts(plan))
        hold = std::unique_lock<std::mutex>(buffer_mutex(dev->index, p.stream));
    AddParts add;
    if ((st = run_trans(p, plan, dev, &add)) != GEMM_OK)
        return st;
    return add_parts(p, add);
}

gemm_status gemm_gated_backward(int64_t M, int64_t N, int64_t K, int dtype_is_bf16, const void *dD,
                                int64_t lddd, const void *G, int64_t ldg, const void *U, int64_t ldu,
                                const void *A, int64_t lda, const void *Bg, int64_t ldbg, const void *Bu,
                                int64_t ldbu, void *dG, int64_t lddg, void *dU, int64_t lddu, void *dA,
                                int64_t ldda, void *dBg, int64_t lddbg, void *dBu, int64_t lddbu, int out,
                                int act, void *stream)
{
    if ((dtype_is_bf16 != 0 && dtype_is_bf16 != 1) || M < 0 || N < 0 || K < 0 || !out_ok(out) || !act_ok(act))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return GEMM_ERR_UNSUPPORTED;
    // which gradients are asked for (an empty one needs no pointer)
    const bool want_a = dA != nullptr && M > 0 && K > 0;
    const bool want_b = (dBg != nullptr || dBu != nullptr) && N > 0 && K > 0;
    const int es = out_size(out);
    const Mat dd{dD, lddd, M, N, 2, false}, g{G, ldg, M, N, 2, false}, u{U, ldu, M, N, 2, false};
    const Mat dg{dG, lddg, M, N, 2, true}, du{dU, lddu, M, N, 2, true};
    const Mat a{A, lda, want_b ? M : 0, K, 2, true};
    const Mat bg{Bg, ldbg, want_a ? N : 0, K, 2, true}, bu{Bu, ldbu, want_a ? N : 0, K, 2, true};
    const Mat da{dA, ldda, want_a ? M : 0, K, es, false};
    const Mat dbg{dBg, lddbg, want_b ? N : 0, K, es, false}, dbu{dBu, lddbu, want_b ? N : 0, K, es, false};
    gemm_status st = check_mats({dd, g, u, dg, du, a, bg, bu, da, dbg, dbu});
    if (st != GEMM_OK)
        return st;
    // dG may take G's place and dU U's, exactly
    const Span sg = dG == G && lddg == ldg ? Span{nullptr, 0} : span_of(g);
    const Span su = dU == U && lddu == ldu ? Span{nullptr, 0} : span_of(u);
    if (any_overlap({span_of(dg), span_of(du), span_of(da), span_of(dbg), span_of(dbu)},
                    {span_of(dd), span_of(a), span_of(bg), span_of(bu)}) ||
        any_overlap({span_of(dg)}, {sg, span_of(u)}) || any_overlap({span_of(du)}, {span_of(g), su}) ||
        any_overlap({span_of(da)}, {span_of(g), span_of(u)}) ||
        any_overlap({span_of(dbg)}, {span_of(g), span_of(u)}) ||
        any_overlap({span_of(dbu)}, {span_of(g), span_of(u)}))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype_is_bf16 == 1;
    if (M > 0 && N > 0 &&
        tcg::launch_gated_slope(dD, lddd, G, ldg, U, ldu, dG, lddg, dU, lddu, static_cast<int32_t>(M),
                                static_cast<int32_t>(N), bf16, act, cs) != cudaSuccess)
        return GEMM_ERR_CUDA;
    TransProblem pa{}, pb{};
    AddParts add_a, add_b;
    if (want_a) {
        // dA = [dG dU] [Bg; Bu]: one sum over 2 N, Bg and Bu read as stored (K columns contiguous)
        pa.M = M;
        pa.N = K;
        pa.K = N;
        pa.bf16 = bf16;
        pa.tb = true;
        pa.A = dG;
        pa.lda = lddg;
        pa.B = Bg;
        pa.ldb = ldbg;
        pa.A2 = dU;
        pa.lda2 = lddu;
        pa.B2 = Bu;
        pa.ldb2 = ldbu;
        pa.D = dA;
        pa.ldd = ldda;
        pa.out = out;
        pa.alpha = 1.0f;
        pa.stream = cs;
    }
    if (want_b) {
        // [dBg; dBu] = [dG dU]^T A: both gradients' tiles in one launch, which fills the
        // SMs as dA's tiles run out (both only need dG and dU: dA's kernel let this
        // one start once it had passed its own wait for them)
        pb.co_tail = want_a;
        pb.parts_use = kBufParts + 1;
        pb.M = N;
        pb.N = K;
        pb.K = M;
        pb.bf16 = bf16;
        pb.ta = true;
        pb.tb = true;
        pb.A = dG;
        pb.lda = lddg;
        pb.A2 = dU;
        pb.lda2 = lddu;
        pb.B = A;
        pb.ldb = lda;
        pb.D = dBg;
        pb.ldd = lddbg;
        pb.D2 = dBu;
        pb.ldd2 = lddbu;
        pb.out = out;
        pb.alpha = 1.0f;
        pb.stream = cs;
    }
    gemm_plan plan_a{}, plan_b{};
    if (want_a)
        plan_a = plan_of_trans(pa, dev);
    if (want_b)
        plan_b = plan_of_trans(pb, dev);
    int fk = 0, fbn = 0;
    forced_tile(&fk, &fbn);
    if (want_a && want_b && plan_a.kernel != 2 && M > 0 && N > 0 && fk == 0)
        plan_side_by_side(pa, pb, dev->sm_count, &plan_a, &plan_b);
    std::unique_lock<std::mutex> hold;
    if (in_parts(plan_a) || in_parts(plan_b))
        hold = std::unique_lock<std::mutex>(buffer_mutex(dev->index, cs));
    if ((want_a && (st = run_trans(pa, plan_a, dev, &add_a)) != GEMM_OK) ||
        (want_b && (st = run_trans(pb, plan_b, dev, &add_b)) != GEMM_OK))
        return st;
    // (sums in parts are added last, so that the products run side by side)
    if ((st = add_parts(pa, add_a)) != GEMM_OK || (st = add_parts(pb, add_b)) != GEMM_OK)
        return st;
    return GEMM_OK;
}

gemm_status gemm_quantize_e2m1(int64_t M, int64_t K, int type, const void *X, int64_t ldx, uint8_t *Q,
                               int64_t ldq, uint8_t *S, int64_t lds, void *Y, int64_t ldy, void *stream)
{
    if (M < 0 || K < 0 || !out_ok(type))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || K > kMaxDim || K % 32 != 0)
        return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || K == 0)
        return GEMM_OK;
    const int es = out_size(type);
    const Mat x{X, ldx, M, K, es, false}, q{Q, ldq, M, K / 2, 1, true}, s{S, lds, K / 32, M, 1, false},
        y{Y, ldy, Y ? M : 0, K, es, false};
    gemm_status st = check_mats({x, q, s, y});
    if (st != GEMM_OK)
        return st;
    // Y may take X's place, exactly
    const Span sy = Y == X && ldy == ldx ? Span{nullptr, 0} : span_of(y);
    if (any_overlap({span_of(q), span_of(s), sy}, {span_of(x)}) ||
        any_overlap({span_of(q), span_of(s)}, {span_of(y)}))
        return GEMM_ERR_ALIAS;
    DeviceInfo *dev = nullptr;
    if ((st = device_info(&dev)) != GEMM_OK)
        return st;
    const cudaError_t e =
        tcg::launch_quantize_e2m1(X, ldx, type, Q, ldq, S, lds, Y, ldy, static_cast<int32_t>(M),
                                  static_cast<int32_t>(K), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // extern "C"
