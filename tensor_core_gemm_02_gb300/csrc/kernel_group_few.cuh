// kernel_group_few.cuh -- products over groups of few rows (decoding): the weights stream.
//
// D[i] = alpha A[i] B_g^T with a handful of rows in each group is bound by reading every used
// B_g once.  As in kernel_skinny.cuh the operands change places: 128 rows of B_g are the
// MMA's M side and MP <= 64 rows of A its N side (rows past the group's are other groups' or
// zero, multiplied and never stored), so a stage is 32 KB of weights and 256 MP bytes of A.
// A tile is 128 columns of D by MP rows of a group; its tiles come from the offsets as in
// kernel_group.cuh.
//
// Split: CS CTAs of a cluster share each tile's sum, CTA c the c-th part of its K blocks, where
// there are fewer tiles than SMs and the sums are long.  Each CTA ends with the sums of its part
// for 128 columns x MP rows, keeps those of its own MP / CS rows and writes the others into the
// peer's shared memory; each then adds the parts in order and stores its rows: no workspace, no
// atomics, the same bits every time.
//
// Float32 results: the accumulators, which drop what does not fit them, are emptied every eight stages
// (512 of K each) into float32 registers, which round to nearest; while one tile buffer is read the MMAs go
// on in the other.  (Positive operands, relative error, one accumulator / emptied: K of 14336 4.6e-5 / 3.0e-6,
// 57344 1.9e-4 / 3.1e-6.)  For results of 16 bits one accumulator takes an issuer's whole share.
//
// Bound by HBM: 8 groups of 4 rows, 14336 x 4096 bf16 141 to 143 us (6.6 TB/s; float32 143 to 144), two of one
// row 40 to 43 (5.4 to 5.8 TB/s; the tile kernel 83); 2 of 64 groups, 2816 x 1024 7.1 us (launch, offsets,
// first loads, epilogue).  More rows, bf16: 48 a group of 8 x 14336 x 4096 146 against the tile kernel's 152, 64 148
// against 151, 100 of 8 x 2816 x 1024 17.6 against 14.8, hence the change at 48.
//
//   warp 0     producer: per stage two K blocks of B (boxes of 64 x 128, or stored K x N two
//              boxes of 64 x 64) and of A (a box of MP rows, or MP / 4 tile::gather4)
//   warps 1-2  MMA issuers, one for each of a stage's K blocks, into accumulators of their own
//              (one thread issues an MMA every ~117 cycles: 16 KB of B a K block would stop at
//              35 bytes a clock and SM)
//   warps 3-6  epilogue: lanes walk along N, whole lines of D
#pragma once

#include "kernel_group.cuh"

namespace tcg {

template <int MP_, int CS_>
struct FewCfg {
    static constexpr int MP = MP_, CS = CS_, BN = 128, KBOX = 2;
    static constexpr uint32_t B_BYTES = BN * 128u * KBOX, A_BYTES = MP * 128u * KBOX;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = MP == 16 ? 6 : (MP == 32 ? 5 : 4);
    static constexpr int CHUNK = 8;  // stages, a K block each an issuer, between roundings of float32 results
    static constexpr uint32_t OFF_B = 0, OFF_A = STAGES * B_BYTES;
    // sums from the peer: two tiles' in turn, MP / CS rows of 128 floats
    static constexpr uint32_t RED_BYTES = CS > 1 ? MP / CS * BN * 4u : 0u;
    static constexpr uint32_t OFF_RED = STAGES * STAGE_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_RED + 2 * RED_BYTES;
    static constexpr uint32_t NUM_BARS = 2 * STAGES + 4 + 16;
    static constexpr uint32_t SMEM_ALLOC = OFF_BAR + NUM_BARS * 8 + 16 + 1024;
    static constexpr int THREADS = 32 * 7;
    static constexpr uint32_t TMEM_COLS = MP == 16 ? 64 : (MP == 32 ? 128 : 256);  // 2 tiles x 2 issuers x MP
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(CS == 1 || CS == 2, "one or two parts");
};

template <int MP, int CS, bool MAJB>
__global__ void __launch_bounds__(FewCfg<MP, CS>::THREADS, 1)
    group_few_kernel(const __grid_constant__ GroupMaps maps, const GroupArgs args)
{
    using Cfg = FewCfg<MP, CS>;
    constexpr int STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x / 32u, 0);
    const uint32_t lane = threadIdx.x % 32u;
    const uint32_t bar0 = base + Cfg::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    // the peer's sums for tile buffer b, lane quarter q: written / read (the latter arrives at
    // the writer)
    auto redf_bar = [&](int b, uint32_t q) { return bar0 + 8u * (2 * STAGES + 4 + 4 * b + q); };
    auto rede_bar = [&](int b, uint32_t q) { return bar0 + 8u * (2 * STAGES + 12 + 4 * b + q); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bar0 - raw) + 8 * Cfg::NUM_BARS);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    const uint32_t rank = CS > 1 ? cluster_ctarank() : 0u;
    const int32_t set = static_cast<int32_t>(blockIdx.x) / CS, sets = static_cast<int32_t>(gridDim.x) / CS;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 2);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 2);
            mbar_init(acce_bar(b), 4);
            for (uint32_t q = 0; q < 4u; ++q) {
                mbar_init(redf_bar(b, q), 1);
                mbar_init(rede_bar(b, q), 1);
            }
        }
        *abort_flag = 0u;
        fence_mbar_init();
        fence_proxy_async_smem();
        if (args.loads) {
            tma_prefetch_desc(&maps.a);
            tma_prefetch_desc(&maps.b);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    GroupRows<MP> gr;
    gr.init(args.offsets, args.groups, args.rows, lane);
    tc_fence_before_sync();
    if (CS > 1)
        cluster_sync_all();
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    if (threadIdx.x == 0) {
        grid_launch_dependents();
        if (!gr.ok && blockIdx.x == 0)
            record_error(args.status, kStatusIndex, 0);
    }
    const int32_t num_tiles = gr.total * args.num_n_blocks;
    // this CTA's stages of every tile
    const int32_t all = (args.K + 127) / 128;
    const int32_t st0 = static_cast<int32_t>(static_cast<int64_t>(all) * rank / CS);
    const int32_t nst = static_cast<int32_t>(static_cast<int64_t>(all) * (rank + 1) / CS) - st0;  // (K > 0, CS = 2: long)
    // stages that an accumulator takes
    const int32_t fill = args.out_kind == kOutF32 ? Cfg::CHUNK : nst;

    // (whole warp) a tile's first row, the end of its group's and its first column
    int32_t g = 0, row0 = 0, end = 0, n0 = 0;
    auto locate = [&](int32_t t) {
        gr.find(t / args.num_n_blocks, lane);
        const int32_t r = t - gr.base_last * args.num_n_blocks;
        g = gr.g_last;
        // (the row blocks of a group one after the other: its weights come from L2 then)
        row0 = gr.lo_last + r % gr.blocks_last * MP;
        end = gr.hi_last;
        n0 = r / gr.blocks_last * Cfg::BN;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int s = 0;
        uint32_t ph = 0;
        int pending = 0;
        bool first = true, alive = true;
        for (int32_t t = set; t < num_tiles && alive; t += sets) {
            locate(t);
            int32_t rows[4] = {0, 0, 0, 0};
            const bool gather_lane = lane < MP / 4;
            if (args.gather && gather_lane) {
                int32_t v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int32_t m = row0 + 4 * static_cast<int32_t>(lane) + r;
                    v[r] = m < end ? __ldcg(args.idx + m) : 0;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (v[r] < 0 || v[r] >= args.table_rows)
                        record_error(args.status, kStatusIndex, 0);
                    else
                        rows[r] = v[r];
                }
            }
            for (int32_t i = 0; i < nst; ++i) {
                if (!warp_wait_bounded<true>(empty_bar(s), ph ^ 1u, abort_flag, args.status, args.timeout_ns,
                                             kWhereProducerEmpty)) {
                    alive = false;
                    break;
                }
                const uint32_t sb = base + Cfg::OFF_B + s * Cfg::B_BYTES, sa = base + Cfg::OFF_A + s * Cfg::A_BYTES;
                if (lane == 0)
                    mbar_arrive_expect_tx(full_bar(s), Cfg::STAGE_BYTES + (first ? args.extra_tx : 0u));
                first = false;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < Cfg::KBOX; ++j) {
                    const int32_t k = (st0 + i) * 128 + 64 * j;
                    if (lane == 0) {
                        if constexpr (MAJB) {
                            tma_load_3d(sb + 16384u * j, &maps.b, full_bar(s), n0, k, g);
                            tma_load_3d(sb + 16384u * j + 8192u, &maps.b, full_bar(s), n0 + 64, k, g);
                        } else {
                            tma_load_3d(sb + 16384u * j, &maps.b, full_bar(s), k, n0, g);
                        }
                    }
                    const uint32_t to = sa + MP * 128u * j;
                    if (args.gather) {
                        if (gather_lane)
                            tma_gather4(to + lane * 512u, &maps.a, full_bar(s), k, rows[0], rows[1], rows[2], rows[3]);
                    } else if (lane == 0) {
                        tma_load_2d(to, &maps.a, full_bar(s), k, row0);
                    }
                }
                pending = min(pending + 1, STAGES);
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!alive) {
            int ds = s;
            uint32_t dph = ph;
            for (int i = 0; i < pending; ++i) {
                if (--ds < 0) {
                    ds = STAGES - 1;
                    dph ^= 1u;
                }
                wait_drain(full_bar(ds), dph, 10000000ull);
            }
        }
    } else if (warp <= 2) {
        // ------------------------------------------------------------ MMA issuers
        if (lane == 0) {
            const uint32_t e = warp - 1u;
            const uint32_t idesc = idesc_f16_f32acc(args.ab_bf16 != 0, 128, MP, MAJB, false);
            int s = 0, ab = 0;
            uint32_t ph = 0, aph = 0;
            bool alive = true;
            for (int32_t t = set; t < num_tiles && alive; t += sets) {
                for (int32_t i0 = 0; i0 < nst && alive; i0 += fill) {
                    if (!wait_bounded<true>(acce_bar(ab), aph ^ 1u, abort_flag, args.status, args.timeout_ns,
                                            kWhereMmaAccEmpty)) {
                        alive = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((2 * ab + e) * MP);
                    const int32_t here = min(fill, nst - i0);
                    for (int32_t i = 0; i < here; ++i) {
                        if (!wait_bounded(full_bar(s), ph, abort_flag, args.status, args.timeout_ns, kWhereMmaFull)) {
                            alive = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t sb = base + Cfg::OFF_B + s * Cfg::B_BYTES + 16384u * e;
                        const uint32_t sa = base + Cfg::OFF_A + s * Cfg::A_BYTES + MP * 128u * e;
                        const uint64_t wd = MAJB ? sdesc_mn_sw128(sb) : sdesc_k_sw128(sb);
                        const uint64_t xd = sdesc_k_sw128(sa);
                        constexpr uint32_t kStepW = MAJB ? 128u : 2u;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_f16(d_tmem, wd + kStepW * k, xd + 2u * k, idesc, (i | k) != 0 ? 1u : 0u);
                        tc_commit(empty_bar(s));
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!alive)
                        break;
                    tc_commit(accf_bar(ab));
                    if (++ab == 2) {
                        ab = 0;
                        aph ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const uint32_t q = warp & 3u;
        constexpr int kMine = MP / CS;  // rows this CTA finishes
        int ab = 0, rb = 0;  // accumulators; the peer's sums
        uint32_t aph = 0, use = 0;  // use: times both buffers of the peer's sums have been used before
        bool alive = true;
        for (int32_t t = set; t < num_tiles; t += sets) {
            locate(t);
            const int32_t n = n0 + 32 * static_cast<int32_t>(q) + static_cast<int32_t>(lane);
            int32_t row_idx[(kMine + 31) / 32];  // (loaded while the tile's MMAs run)
#pragma unroll
            for (int j0 = 0; j0 < kMine; j0 += 32) {
                const int32_t m = row0 + static_cast<int32_t>(rank) * kMine + j0 + static_cast<int32_t>(lane);
                row_idx[j0 / 32] =
                    args.idx && static_cast<int32_t>(lane) + j0 < kMine && m < end ? __ldcg(args.idx + m) : 0;
            }
            // v: the sums of this CTA's rows, both issuers'; w: of the peer's
            float v[kMine], w[CS > 1 ? kMine : 1];
            const int mine0 = static_cast<int>(rank) * kMine;
            const auto take = [&](auto more) {
                constexpr bool kMore = decltype(more)::value;
                tc_fence_after_sync();
                const uint32_t acc = tmem_base + ((32u * q) << 16) + static_cast<uint32_t>(2 * ab * MP);
                // 8 rows' from row j
                auto take8 = [&](int j, float *to) {
                    uint32_t a[8], b[8];
                    tc_ld_32x32b_x8(acc + static_cast<uint32_t>(j), a);
                    tc_ld_32x32b_x8(acc + static_cast<uint32_t>(MP + j), b);
                    tc_wait_ld8(a);
                    tc_wait_ld8(b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = __fadd_rn(__uint_as_float(a[i]), __uint_as_float(b[i]));
                        to[i] = kMore ? __fadd_rn(to[i], x) : x;
                    }
                };
#pragma unroll
                for (int j = 0; j < kMine; j += 8) {
                    take8(mine0 + j, v + j);
                    if constexpr (CS > 1)
                        take8(static_cast<int>(rank ^ 1u) * kMine + j, w + j);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(acce_bar(ab));
                if (++ab == 2) {
                    ab = 0;
                    aph ^= 1u;
                }
            };
            alive = warp_wait_bounded<true>(accf_bar(ab), aph, abort_flag, args.status, args.timeout_ns,
                                            kWhereEpiAccFull);
            if (!alive)
                break;
            take(Bool<false>{});
            for (int32_t i = fill; i < nst; i += fill) {
                // (inline, or the call would save the sums' registers)
                alive = warp_wait_bounded_inline(accf_bar(ab), aph, abort_flag, args.status, args.timeout_ns,
                                                 kWhereEpiAccFull);
                if (!alive)
                    break;
                take(Bool<true>{});
            }
            if (!alive)
                break;
            // (a bad index makes its row zero: bit j, row j of this CTA's)
            uint64_t bad = 0;
            if (args.idx) {
#pragma unroll
                for (int j0 = 0; j0 < kMine; j0 += 32) {
                    const int32_t r = row_idx[j0 / 32];
                    bad |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, r < 0 || r >= args.table_rows)) << j0;
                }
            }
            if constexpr (CS > 1) {
                const uint32_t peer = rank ^ 1u;
                // the peer has read the buffer's last sums
                if (use > 0 && !warp_wait_cluster(rede_bar(rb, q), (use - 1u) & 1u, abort_flag, args.status,
                                                  args.timeout_ns, kWhereEpiC))
                    break;
                const uint32_t to = mapa_shared(base + Cfg::OFF_RED + rb * Cfg::RED_BYTES + (32u * q + lane) * 4u, peer);
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    st_shared_cluster_u32(to + static_cast<uint32_t>(j) * 512u, __float_as_uint(w[j]));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(redf_bar(rb, q), peer));
                if (!warp_wait_cluster(redf_bar(rb, q), use & 1u, abort_flag, args.status, args.timeout_ns, kWhereEpiC))
                    break;
                const uint32_t from = base + Cfg::OFF_RED + rb * Cfg::RED_BYTES + (32u * q + lane) * 4u;
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    v[j] = __fadd_rn(v[j], __uint_as_float(ld_shared_u32(from + static_cast<uint32_t>(j) * 512u)));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(rede_bar(rb, q), peer));
                if (++rb == 2) {
                    rb = 0;
                    ++use;
                }
            }
            if (n < args.N) {
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int32_t row = row0 + mine0 + j;
                    if (row < end) {
                        const float x = (bad >> j) & 1u ? 0.f : mul_rn(args.alpha, v[j]);
                        const int64_t o = static_cast<int64_t>(row) * args.ldd + n;
                        if (args.out_kind == kOutF32)
                            static_cast<float *>(args.D)[o] = x;
                        else
                            static_cast<uint16_t *>(args.D)[o] =
                                args.out_kind == kOutBF16 ? f32_to_bf16_rn(x) : f32_to_f16_rn(x);
                    }
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before_sync();
    if (CS > 1)
        cluster_sync_all();  // the peer may write into this CTA's shared memory until here
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace tcg
