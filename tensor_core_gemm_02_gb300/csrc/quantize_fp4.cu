// quantize_fp4.cu -- rows of 32-element blocks to FP4 E2M1 codes with UE8M0
// block scales, as gemm_e2m1 and gemm_gated_e2m1 take them.
//
// Per block, with m = max |x|: the scale byte is s = max(0, floor(log2 m) + 125),
// that is the power of two 2^(s - 127) that puts m's leading bit on E2M1's
// largest exponent (2); the exponent field of m's float32 pattern minus 2 is
// s.  An element is x 2^(127 - s) -- exact, a power of two -- rounded to the
// nearest E2M1 value, ties to the even code, magnitudes above 6 to 6.  A block
// of zeros has s = 0; a block that holds an infinity or a NaN has s = 255 (NaN)
// and zero codes.
//
// Bound by memory: per element its own size read and 17/32 byte written (plus
// its size again where the values are wanted too).  A warp reads 256
// consecutive elements of a row, eight per lane, so loads and code stores are
// whole lines, and a block is four neighbouring lanes (two shuffles for its
// maximum).  The scales are stored one row per 32-element block, so a thread
// block covers 32 rows: their scale bytes meet in shared memory and leave as
// 32-byte runs, whole sectors.  All loads of a warp's rows go out first.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"

namespace tcg {

namespace {

constexpr int kQRows = 32;   // rows per thread block
constexpr int kQCols = 256;  // columns per thread block
constexpr int kQWarps = 8;
constexpr int kQSteps = kQRows / kQWarps;  // rows per warp

// Eight floats (scaled) -> eight E2M1 codes, element i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8_from_f32(const float (&v)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// The value of code c (bit 3 the sign): exponent field e, mantissa bit m.
__device__ __forceinline__ float e2m1_value(uint32_t c)
{
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float v = e == 0 ? 0.5f * static_cast<float>(m)
                           : __uint_as_float(((e + 126u) << 23) | (m << 22));
    return (c & 8u) != 0 ? -v : v;
}

template <typename T>
struct Elem;  // eight elements of a row: load, store, one at a time or whole

template <>
struct Elem<float> {
    template <bool VEC>
    static __device__ __forceinline__ void load(const float *p, float (&v)[8])
    {
        if (VEC) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = p[i];
        }
    }
    template <bool VEC>
    static __device__ __forceinline__ void store(float *p, const float (&v)[8])
    {
        if (VEC) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = v[i];
        }
    }
};

// 16-bit elements by their bits; BF16 says which type they are
template <bool BF16>
struct Half {
    unsigned short bits;
};

template <bool BF16>
struct Elem<Half<BF16>> {
    static __device__ __forceinline__ float widen(uint32_t h)
    {
        if (BF16)
            return __uint_as_float(h << 16);
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<unsigned short>(h)));
        return f;
    }
    template <bool VEC>
    static __device__ __forceinline__ void load(const Half<BF16> *p, float (&v)[8])
    {
        if (VEC) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = widen(w[i] & 0xFFFFu);
                v[2 * i + 1] = widen(w[i] >> 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = widen(p[i].bits);
        }
    }
    template <bool VEC>
    static __device__ __forceinline__ void store(Half<BF16> *p, const float (&v)[8])
    {
        if (VEC) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = BF16 ? pack_bf16x2(v[2 * i], v[2 * i + 1]) : pack_f16x2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i].bits = BF16 ? f32_to_bf16_rn(v[i]) : f32_to_f16_rn(v[i]);
        }
    }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kQWarps)
    quantize_e2m1_kernel(const T *X, int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *S, int64_t lds,
                         T *Y, int64_t ldy, int32_t M, int32_t K, int64_t tiles, int32_t col_tiles)
{
    __shared__ __align__(16) uint8_t sc[kQCols / 32][kQRows];
    grid_dependency_wait();
    if (threadIdx.x == 0)
        grid_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x / 32u), lane = static_cast<int>(threadIdx.x % 32u);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row0 = t / col_tiles * kQRows;
        const int64_t col = t % col_tiles * kQCols + 8 * lane;
        const bool have = col < K;  // (K is a multiple of 32: all eight or none, a quad alike)
        float v[kQSteps][8];
#pragma unroll
        for (int i = 0; i < kQSteps; ++i) {
            const int64_t row = row0 + warp + kQWarps * i;
            if (have && row < M)
                Elem<T>::template load<VEC>(X + row * ldx + col, v[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kQSteps; ++i) {
            const int64_t row = row0 + warp + kQWarps * i;
            // max |x| by its bits: infinities and NaNs come out on top
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const bool nan = top >= 0x7F800000u;
            const uint32_t e = top >> 23;
            const uint32_t s = nan ? 255u : (e > 2u ? e - 2u : 0u);
            const float inv = nan ? 0.f : __uint_as_float((254u - s) << 23);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = nan ? 0.f : v[i][j] * inv;
            const uint32_t w = e2m1x8_from_f32(y);
            if (have && row < M) {
                *reinterpret_cast<uint32_t *>(Q + row * ldq + col / 2) = w;
                if (Y != nullptr) {
                    const float f = nan ? __uint_as_float(0x7FC00000u)
                                        : __uint_as_float(s == 0 ? 0x00400000u : s << 23);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j] = e2m1_value((w >> (4 * j)) & 15u) * f;
                    Elem<T>::template store<VEC>(Y + row * ldy + col, y);
                }
            }
            if (lane % 4 == 0)
                sc[lane / 4][warp + kQWarps * i] = static_cast<uint8_t>(s);
        }
        __syncthreads();
        // scale row b of the tile: 32 bytes, four per thread
        if (threadIdx.x < kQCols / 32 * kQRows / 4) {
            const int b = static_cast<int>(threadIdx.x) / (kQRows / 4);
            const int r = static_cast<int>(threadIdx.x) % (kQRows / 4) * 4;
            const int64_t kb = t % col_tiles * (kQCols / 32) + b;
            if (kb < K / 32) {
                uint8_t *dst = S + kb * lds + row0 + r;
                if (row0 + r + 4 <= M && (reinterpret_cast<uintptr_t>(dst) & 3u) == 0) {
                    *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(&sc[b][r]);
                } else {
                    for (int j = 0; j < 4 && row0 + r + j < M; ++j)
                        dst[j] = sc[b][r + j];
                }
            }
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_quantize_type(const void *X, int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *S,
                                 int64_t lds, void *Y, int64_t ldy, int32_t M, int32_t K,
                                 cudaStream_t stream)
{
    const int64_t per16 = 16 / static_cast<int64_t>(sizeof(T));
    const bool vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && ldx % per16 == 0 &&
                     (Y == nullptr || ((reinterpret_cast<uintptr_t>(Y) & 15u) == 0 && ldy % per16 == 0));
    const int32_t col_tiles = static_cast<int32_t>((static_cast<int64_t>(K) + kQCols - 1) / kQCols);
    const int64_t tiles = (static_cast<int64_t>(M) + kQRows - 1) / kQRows * col_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < (int64_t(1) << 30) ? tiles : (int64_t(1) << 30)), 1, 1);
    cfg.blockDim = dim3(32 * kQWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kfn = vec ? quantize_e2m1_kernel<T, true> : quantize_e2m1_kernel<T, false>;
    return cudaLaunchKernelEx(&cfg, kfn, static_cast<const T *>(X), ldx, Q, ldq, S, lds,
                              static_cast<T *>(Y), ldy, M, K, tiles, col_tiles);
}

}  // namespace

cudaError_t launch_quantize_e2m1(const void *X, int64_t ldx, int type, uint8_t *Q, int64_t ldq,
                                 uint8_t *S, int64_t lds, void *Y, int64_t ldy, int32_t M, int32_t K,
                                 cudaStream_t stream)
{
    switch (type) {
    case kOutF32: return launch_quantize_type<float>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    case kOutBF16: return launch_quantize_type<Half<true>>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    case kOutF16: return launch_quantize_type<Half<false>>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
