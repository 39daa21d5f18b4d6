// add_parts.cu -- the end of a product whose sum was cut into parts: add each
// element's parts in order, then the epilogue fma.rn(alpha, sum, beta C).
//
// Bound by memory (the parts are at most a few per element, in L2 as a rule).  A
// thread takes four columns of one row; all parts' loads go out before the
// first add waits (unrolled by four).  Order of the parts, so the result is the same
// on every call.  Measured, product and adding together (uncut before): 512 x 512 x 8192
// 14 us (36), 300 x 300 x 4000 10 (21).
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"

namespace tcg {

namespace {

template <int OUT>
__global__ void __launch_bounds__(256)
    add_parts_kernel(const float *W, int64_t ldw, int64_t part_rows, int32_t parts, const float *C,
                     int64_t ldc, void *D, int64_t ldd, float alpha, float beta, int32_t M, int32_t N,
                     bool d_vec)
{
    grid_dependency_wait();
    if (threadIdx.x == 0)
        grid_launch_dependents();
    const int64_t col = 4 * (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x);
    if (col >= N)
        return;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y; row < M;
         row += static_cast<int64_t>(gridDim.y) * blockDim.y) {
        const float *w = W + row * ldw + col;  // (ldw is a multiple of four)
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int32_t p = 0; p < parts; ++p) {
            const float4 x = __ldcs(reinterpret_cast<const float4 *>(w + p * part_rows * ldw));
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        }
        const int n = N - col < 4 ? static_cast<int>(N - col) : 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = C != nullptr && i < n ? fma_rn(alpha, v[i], mul_rn(beta, C[row * ldc + col + i]))
                                         : mul_rn(alpha, v[i]);
        if (OUT == kOutF32) {
            float *d = static_cast<float *>(D) + row * ldd + col;
            if (d_vec && n == 4) {
                *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                for (int i = 0; i < n; ++i)
                    d[i] = v[i];
            }
        } else {
            unsigned short *d = static_cast<unsigned short *>(D) + row * ldd + col;
            const uint32_t lo = OUT == kOutBF16 ? pack_bf16x2(v[0], v[1]) : pack_f16x2(v[0], v[1]);
            const uint32_t hi = OUT == kOutBF16 ? pack_bf16x2(v[2], v[3]) : pack_f16x2(v[2], v[3]);
            if (d_vec && n == 4) {
                *reinterpret_cast<uint2 *>(d) = make_uint2(lo, hi);
            } else {
                const unsigned short h[4] = {
                    static_cast<unsigned short>(lo), static_cast<unsigned short>(lo >> 16),
                    static_cast<unsigned short>(hi), static_cast<unsigned short>(hi >> 16)};
                for (int i = 0; i < n; ++i)
                    d[i] = h[i];
            }
        }
    }
}

}  // namespace

cudaError_t launch_add_parts(const float *W, int64_t ldw, int64_t part_rows, int32_t parts, const float *C,
                             int64_t ldc, void *D, int64_t ldd, int out, float alpha, float beta, int32_t M,
                             int32_t N, cudaStream_t stream)
{
    const int64_t es = out == kOutF32 ? 4 : 2;
    const bool d_vec = (reinterpret_cast<uintptr_t>(D) % static_cast<uintptr_t>(4 * es)) == 0 && ldd % 4 == 0;
    const int64_t quads = (static_cast<int64_t>(N) + 3) / 4;
    unsigned tx = 16;
    while (tx < 256 && tx < quads)
        tx *= 2;
    const unsigned ty = 256 / tx;
    const int64_t gy = (static_cast<int64_t>(M) + ty - 1) / ty;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((quads + tx - 1) / tx),
                       static_cast<unsigned>(gy < 65535 ? gy : 65535), 1);
    cfg.blockDim = dim3(tx, ty, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kfn = out == kOutF32 ? add_parts_kernel<kOutF32>
                              : (out == kOutBF16 ? add_parts_kernel<kOutBF16> : add_parts_kernel<kOutF16>);
    return cudaLaunchKernelEx(&cfg, kfn, W, ldw, part_rows, parts, C, ldc, D, ldd, alpha, beta, M, N, d_vec);
}

}  // namespace tcg
