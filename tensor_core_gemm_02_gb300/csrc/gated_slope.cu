// gated_slope.cu -- the elementwise part of the gated form's backward pass:
//     dG = dD * U * act'(G),   dU = dD * act(G)
// in float32 from 16-bit matrices, rounded once to the operand type (dG and dU
// are operands of the products that follow, and the tensor cores take 16-bit
// operands; both are also the caller's outputs).
//
// Bound by memory: 6 bytes read and 4 written per element.  A thread takes
// eight columns of one row (three 16-byte loads, two 16-byte stores), blocks
// are wide along the columns; rows whose base or pitch is not 16-byte aligned,
// and the columns past the last multiple of eight, go element by element.
// Measured: 8192 x 14336 171 us (6.9 TB/s, the rate of a plain copy); gelu, with the
// longest arithmetic, 195.
#include <cuda_runtime.h>

#include "act.cuh"
#include "common.cuh"
#include "launch.h"

namespace tcg {

namespace {

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t h)
{
    if (BF16)
        return __uint_as_float(h << 16);
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<unsigned short>(h)));
    return f;
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

template <int ACT>
__device__ __forceinline__ void slope_one(float d, float g, float u, float &dg, float &du)
{
    float a, s;
    act_value_slope<ACT>(g, a, s);
    dg = d * u * s;
    du = d * a;
}

template <bool BF16, int ACT, bool VEC>
__global__ void __launch_bounds__(256)
    gated_slope_kernel(const unsigned short *dD, int64_t lddd, const unsigned short *G, int64_t ldg,
                       const unsigned short *U, int64_t ldu, unsigned short *dG, int64_t lddg,
                       unsigned short *dU, int64_t lddu, int32_t M, int32_t N)
{
    grid_dependency_wait();
    if (threadIdx.x == 0)
        grid_launch_dependents();
    const int64_t col = 8 * (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x);
    if (col >= N)
        return;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y; row < M;
         row += static_cast<int64_t>(gridDim.y) * blockDim.y) {
        const unsigned short *pd = dD + row * lddd + col, *pg = G + row * ldg + col, *pu = U + row * ldu + col;
        unsigned short *qg = dG + row * lddg + col, *qu = dU + row * lddu + col;
        if (VEC && col + 8 <= N) {
            const uint4 xd = __ldcs(reinterpret_cast<const uint4 *>(pd));
            const uint4 xg = __ldcs(reinterpret_cast<const uint4 *>(pg));
            const uint4 xu = __ldcs(reinterpret_cast<const uint4 *>(pu));
            const uint32_t d[4] = {xd.x, xd.y, xd.z, xd.w}, g[4] = {xg.x, xg.y, xg.z, xg.w};
            const uint32_t u[4] = {xu.x, xu.y, xu.z, xu.w};
            uint32_t og[4], ou[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float dg0, du0, dg1, du1;
                slope_one<ACT>(widen<BF16>(d[i] & 0xFFFFu), widen<BF16>(g[i] & 0xFFFFu),
                               widen<BF16>(u[i] & 0xFFFFu), dg0, du0);
                slope_one<ACT>(widen<BF16>(d[i] >> 16), widen<BF16>(g[i] >> 16), widen<BF16>(u[i] >> 16),
                               dg1, du1);
                og[i] = narrow2<BF16>(dg0, dg1);
                ou[i] = narrow2<BF16>(du0, du1);
            }
            *reinterpret_cast<uint4 *>(qg) = make_uint4(og[0], og[1], og[2], og[3]);
            *reinterpret_cast<uint4 *>(qu) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        } else {
            // (all loads before the first store: one round trip, not one per element)
            const int n = N - col < 8 ? static_cast<int>(N - col) : 8;
            unsigned short d[8], g[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = i < n;
                d[i] = in ? pd[i] : 0;
                g[i] = in ? pg[i] : 0;
                u[i] = in ? pu[i] : 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < n) {
                    float dg, du;
                    slope_one<ACT>(widen<BF16>(d[i]), widen<BF16>(g[i]), widen<BF16>(u[i]), dg, du);
                    qg[i] = BF16 ? f32_to_bf16_rn(dg) : f32_to_f16_rn(dg);
                    qu[i] = BF16 ? f32_to_bf16_rn(du) : f32_to_f16_rn(du);
                }
            }
        }
    }
}

template <bool BF16, int ACT>
cudaError_t launch_slope_act(bool vec, const cudaLaunchConfig_t &cfg, const void *dD, int64_t lddd,
                             const void *G, int64_t ldg, const void *U, int64_t ldu, void *dG,
                             int64_t lddg, void *dU, int64_t lddu, int32_t M, int32_t N)
{
    auto kfn = vec ? gated_slope_kernel<BF16, ACT, true> : gated_slope_kernel<BF16, ACT, false>;
    using T = unsigned short;
    return cudaLaunchKernelEx(&cfg, kfn, static_cast<const T *>(dD), lddd, static_cast<const T *>(G), ldg,
                              static_cast<const T *>(U), ldu, static_cast<T *>(dG), lddg,
                              static_cast<T *>(dU), lddu, M, N);
}

template <bool BF16, typename... Args>
cudaError_t launch_slope_type(int32_t act, Args... args)
{
    switch (act) {
    case kActSilu: return launch_slope_act<BF16, kActSilu>(args...);
    case kActGelu: return launch_slope_act<BF16, kActGelu>(args...);
    case kActGeluTanh: return launch_slope_act<BF16, kActGeluTanh>(args...);
    case kActRelu: return launch_slope_act<BF16, kActRelu>(args...);
    case kActSigmoid: return launch_slope_act<BF16, kActSigmoid>(args...);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_gated_slope(const void *dD, int64_t lddd, const void *G, int64_t ldg,
                               const void *U, int64_t ldu, void *dG, int64_t lddg, void *dU,
                               int64_t lddu, int32_t M, int32_t N, bool bf16, int32_t act,
                               cudaStream_t stream)
{
    auto aligned = [](const void *p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
    };
    const bool vec = aligned(dD, lddd) && aligned(G, ldg) && aligned(U, ldu) && aligned(dG, lddg) &&
                     aligned(dU, lddu);
    const int64_t chunks = (static_cast<int64_t>(N) + 7) / 8;
    unsigned tx = 8;
    while (tx < 256 && tx < chunks)
        tx *= 2;
    const unsigned ty = 256 / tx;
    const int64_t gy = (static_cast<int64_t>(M) + ty - 1) / ty;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((chunks + tx - 1) / tx),
                       static_cast<unsigned>(gy < 65535 ? gy : 65535), 1);
    cfg.blockDim = dim3(tx, ty, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? launch_slope_type<true>(act, vec, cfg, dD, lddd, G, ldg, U, ldu, dG, lddg, dU, lddu, M, N)
                : launch_slope_type<false>(act, vec, cfg, dD, lddd, G, ldg, U, ldu, dG, lddg, dU, lddu, M, N);
}

}  // namespace tcg
