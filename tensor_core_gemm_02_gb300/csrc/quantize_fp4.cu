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
// Measured: 8192 x 14336 bf16 with the values 86 us (6.2 TB/s), without them 57 (5.2
// TB/s); float32 145 us (6.9 TB/s) and 82; 16 x 4096 2 us.  (One element a lane: 129.)
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp4.cuh"
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

// Two E2M1 codes (a byte: the lower nibble first) -> two f16, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(r)
        : "r"(byte));
    return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float f16_to_f32(uint32_t h)
{
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<unsigned short>(h)));
    return f;
}

// Eight elements of a row, as loaded, for each element type: load and store (VEC:
// in 16-byte pieces), the largest magnitude among the block's four lanes as
// float32 bits, the codes for a scale s, and the values of codes.  16-bit
// elements stay packed in pairs as far as that goes: with every element widened
// to float32 and decoded by itself the instructions, not memory, set the
// time (8192 x 14336 bf16 with values: 129 us, 0.60 of the measured copy rate).
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

struct ElemF32 {
    using T = float;
    float v[8];
    template <bool VEC>
    __device__ __forceinline__ void load(const float *p)
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
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.f;
    }
    template <bool VEC>
    __device__ __forceinline__ void store(float *p) const
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
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        return quad_max(m);
    }
    __device__ __forceinline__ uint32_t codes(uint32_t s) const
    {
        const float inv = __uint_as_float((254u - s) << 23);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = v[i] * inv;
        return e2m1x8_from_f32(y);
    }
    __device__ __forceinline__ void values(uint32_t w, uint32_t s)
    {
        const float f = __uint_as_float(s == 255u ? 0x7FC00000u : (s == 0u ? 0x00400000u : s << 23));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = e2m1x2_to_f16x2(w >> (8 * i));
            v[2 * i] = f16_to_f32(h & 0xFFFFu) * f;
            v[2 * i + 1] = f16_to_f32(h >> 16) * f;
        }
    }
};

template <bool BF16>
struct Elem16 {
    using T = unsigned short;
    uint32_t w[4];  // element 2 i in the lower half of w[i]
    template <bool VEC>
    __device__ __forceinline__ void load(const unsigned short *p)
    {
        if (VEC) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = p[2 * i] | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
        }
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    template <bool VEC>
    __device__ __forceinline__ void store(unsigned short *p) const
    {
        if (VEC) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] = static_cast<unsigned short>(w[i]);
                p[2 * i + 1] = static_cast<unsigned short>(w[i] >> 16);
            }
        }
    }
    // magnitudes without their signs order like their bits, infinities and NaNs on top
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                               max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        m = quad_max(max(m & 0xFFFFu, m >> 16));
        return BF16 ? m << 16 : __float_as_uint(f16_to_f32(m));
    }
    __device__ __forceinline__ uint32_t codes(uint32_t s) const
    {
        float y[8];
        if (BF16) {
            // the power of two is applied in pairs: exact, but for results below bf16's
            // range, whose code is 0 either way (their sign stays)
            const uint32_t h = (254u - s) << 7, inv = h | (h << 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p;
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(w[i]), "r"(inv));
                y[2 * i] = __uint_as_float(p << 16);
                y[2 * i + 1] = __uint_as_float(p & 0xFFFF0000u);
            }
        } else {
            const float inv = __uint_as_float((254u - s) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = f16_to_f32(w[i] & 0xFFFFu) * inv;
                y[2 * i + 1] = f16_to_f32(w[i] >> 16) * inv;
            }
        }
        return e2m1x8_from_f32(y);
    }
    __device__ __forceinline__ void values(uint32_t c, uint32_t s)
    {
        if (BF16) {
            e2m1x8_to_bf16(c, ue8m0_to_bf16x2(s), w);
        } else {
            // finite f16 blocks have s - 127 in [-26, 13]: below 2^-14 as a product of two
            const int t = static_cast<int>(s) - 127;
            const int a = t < -14 ? -14 : t;
            uint32_t fa = static_cast<uint32_t>(a + 15) << 10, fb = static_cast<uint32_t>(t - a + 15) << 10;
            if (s == 255u)
                fa = 0x7E00u, fb = 0x3C00u;
            if (s == 0u)
                fa = fb = 0x3C00u;  // (a block of zeros)
            fa |= fa << 16;
            fb |= fb << 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h = e2m1x2_to_f16x2(c >> (8 * i));
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(fa));
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(fb));
                w[i] = h;
            }
        }
    }
};

template <typename E, bool VEC>
__global__ void __launch_bounds__(32 * kQWarps)
    quantize_e2m1_kernel(const typename E::T *X, int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *S,
                         int64_t lds, typename E::T *Y, int64_t ldy, int32_t M, int32_t K, int64_t tiles,
                         int32_t col_tiles)
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
        E v[kQSteps];
#pragma unroll
        for (int i = 0; i < kQSteps; ++i) {
            const int64_t row = row0 + warp + kQWarps * i;
            if (have && row < M)
                v[i].template load<VEC>(X + row * ldx + col);
            else
                v[i].clear();
        }
#pragma unroll
        for (int i = 0; i < kQSteps; ++i) {
            const int64_t row = row0 + warp + kQWarps * i;
            const uint32_t top = v[i].top();
            const bool nan = top >= 0x7F800000u;
            const uint32_t e = top >> 23;
            const uint32_t s = e > 2u ? e - 2u : 0u;
            const uint32_t w = nan ? 0u : v[i].codes(s);
            if (have && row < M) {
                *reinterpret_cast<uint32_t *>(Q + row * ldq + col / 2) = w;
                if (Y != nullptr) {
                    v[i].values(w, nan ? 255u : s);
                    v[i].template store<VEC>(Y + row * ldy + col);
                }
            }
            if (lane % 4 == 0)
                sc[lane / 4][warp + kQWarps * i] = static_cast<uint8_t>(nan ? 255u : s);
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

template <typename E>
cudaError_t launch_quantize_type(const void *X, int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *S,
                                 int64_t lds, void *Y, int64_t ldy, int32_t M, int32_t K,
                                 cudaStream_t stream)
{
    using T = typename E::T;
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
    auto kfn = vec ? quantize_e2m1_kernel<E, true> : quantize_e2m1_kernel<E, false>;
    return cudaLaunchKernelEx(&cfg, kfn, static_cast<const T *>(X), ldx, Q, ldq, S, lds,
                              static_cast<T *>(Y), ldy, M, K, tiles, col_tiles);
}

}  // namespace

cudaError_t launch_quantize_e2m1(const void *X, int64_t ldx, int type, uint8_t *Q, int64_t ldq,
                                 uint8_t *S, int64_t lds, void *Y, int64_t ldy, int32_t M, int32_t K,
                                 cudaStream_t stream)
{
    switch (type) {
    case kOutF32: return launch_quantize_type<ElemF32>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    case kOutBF16: return launch_quantize_type<Elem16<true>>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    case kOutF16: return launch_quantize_type<Elem16<false>>(X, ldx, Q, ldq, S, lds, Y, ldy, M, K, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tcg
