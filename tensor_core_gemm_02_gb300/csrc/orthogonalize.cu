// orthogonalize.cu -- the elementwise ends of gemm_orthogonalize: the matrices' norms, and
// the normalised matrices as two float16 parts.
//
// Both are bound by memory: the first reads X, the second reads it again (mostly from L2
// where the stack is small) and writes 4 bytes an element (4096 x 14336 bf16: 23 us, 5.1 TB/s,
// and 52, 6.8 TB/s).  A thread block takes a part of a
// matrix's rows; its sum of squares is float32 (each thread's over its own elements, then
// the block's by shuffles), the parts of a matrix are added in order by every block of the
// second kernel: no atomics, the same bits every time.
//
// The normalised matrix is scaled by a power of two before it is rounded to float16: X / |X|
// has elements down to 1 / |X|, and float16 keeps its 11 bits only above 2^-14.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_group.h"

namespace tcg {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 1024;

// W elements of a row from element `at` of X on (those below n), as float32: eight at once where
// rows are whole 16 bytes apart, or two.
template <int TYPE, int W>
__device__ __forceinline__ void load_piece(const void *X, int64_t at, int32_t n, float (&v)[W])
{
    if (TYPE == kOutF32) {
        const float *p = static_cast<const float *>(X) + at;
        if (W == 8 && n >= 8) {
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(p));
            const float4 b = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2 % W] = a.z, v[3 % W] = a.w;
            v[4 % W] = b.x, v[5 % W] = b.y, v[6 % W] = b.z, v[7 % W] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[i] = i < n ? __ldcg(p + i) : 0.f;
        }
    } else {
        const unsigned short *p = static_cast<const unsigned short *>(X) + at;
        uint32_t w[4] = {0, 0, 0, 0};
        if (W == 8 && n >= 8) {
            const uint4 a = __ldcg(reinterpret_cast<const uint4 *>(p));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i < n)
                    w[i / 2] |= static_cast<uint32_t>(__ldcg(p + i)) << (16 * (i & 1));
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const unsigned short h = static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1)));
            v[i] = TYPE == kOutBF16 ? cvt_bf16_f32(h) : cvt_f16_f32(h);
        }
    }
}

// The pieces of a row that a thread takes, one every `step`, as row and piece of it
// (one division at the start: 64-bit ones for every piece cost more than the memory).
struct Walk {
    int64_t row, d_row;
    int32_t at, d_at, per_row;
    __device__ __forceinline__ Walk(int64_t first, int64_t step, int32_t per)
        : row(first / per), d_row(step / per), at(static_cast<int32_t>(first % per)),
          d_at(static_cast<int32_t>(step % per)), per_row(per)
    {
    }
    __device__ __forceinline__ void next()
    {
        row += d_row;
        at += d_at;
        if (at >= per_row) {
            at -= per_row;
            ++row;
        }
    }
};

__device__ __forceinline__ float block_sum(float x)
{
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    if (threadIdx.x % 32 == 0)
        part[threadIdx.x / 32] = x;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 32; ++i)
        s += part[i];
    return s;
}

// (In pieces of eight rows that are not 16 bytes apart would ask for every 32-byte sector up to
// eight times: 8 x 1000 x 1367, the whole of gemm_orthogonalize, float16 535 -> 523 us, float32 922
// -> 895 with pieces of two.)
template <int TYPE, int W>
__global__ void __launch_bounds__(kThreads)
    square_sums_kernel(const void *X, int64_t ldx, int64_t stride_x, int32_t M, int32_t N, float *partial)
{
    const int32_t parts = static_cast<int32_t>(gridDim.x), g = static_cast<int32_t>(blockIdx.y);
    const int32_t per_row = (N + W - 1) / W;
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kAhead = W == 8 ? 4 : 8;  // pieces in flight
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    Walk w(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, static_cast<int64_t>(parts) * kThreads, per_row);
    while (w.row < M) {
        float v[kAhead][W];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            load_piece<TYPE, W>(X, g * stride_x + w.row * ldx + W * w.at, w.row < M ? N - W * w.at : 0, v[j]);
            w.next();
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e)
                sum[j % 4] = fmaf(v[j][e], v[j][e], sum[j % 4]);
    }
    const float s = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (threadIdx.x == 0)
        partial[static_cast<int64_t>(g) * parts + blockIdx.x] = s;
}

template <int TYPE, int W>
__global__ void __launch_bounds__(kThreads)
    normalize_kernel(const void *X, int64_t ldx, int64_t stride_x, int32_t M, int32_t N, const float *partial,
                     int32_t parts, float scale, float eps, uint16_t *Xs, int64_t lds, int64_t stride_s, int64_t lo)
{
    const int32_t g = static_cast<int32_t>(blockIdx.y);
    constexpr int kAhead = W == 8 ? 4 : 8;  // pieces in flight
    const int32_t per_row = (N + 7) / 8 * (8 / W);  // (rows of Xs are whole 16 bytes: the last pieces fill the padding)
    grid_dependency_wait();
    grid_launch_dependents();
    float sum = 0.f;
    for (int32_t i = static_cast<int32_t>(threadIdx.x); i < parts; i += kThreads)
        sum += __ldcg(partial + static_cast<int64_t>(g) * parts + i);
    const float f = norm_factor(scale, block_sum(sum), eps);
    Walk w(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, static_cast<int64_t>(gridDim.x) * kThreads,
           per_row);
    while (w.row < M) {
        float v[kAhead][W];
        int64_t to[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const bool there = w.row < M;
            load_piece<TYPE, W>(X, g * stride_x + w.row * ldx + W * w.at, there ? N - W * w.at : 0, v[j]);
            to[j] = there ? w.row * lds + W * w.at : -1;
            w.next();
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (to[j] < 0)
                break;
            uint32_t hi[W / 2], low[W / 2];
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const float x0 = v[j][2 * e] * f, x1 = v[j][2 * e + 1] * f;
                hi[e] = pack_f16x2(x0, x1);
                low[e] = pack_f16x2(x0 - cvt_f16_f32(static_cast<unsigned short>(hi[e])),
                                    x1 - cvt_f16_f32(static_cast<unsigned short>(hi[e] >> 16)));
            }
            uint16_t *p = Xs + g * stride_s + to[j];
            if constexpr (W == 8) {
                *reinterpret_cast<uint4 *>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(p + lo) = make_uint4(low[0], low[1], low[2], low[3]);
            } else {
                *reinterpret_cast<uint32_t *>(p) = hi[0];
                *reinterpret_cast<uint32_t *>(p + lo) = low[0];
            }
        }
    }
}

// One 32 x 32 block on or below the diagonal: the parts' sums in order, written here and, transposed,
// above the diagonal.
__global__ void __launch_bounds__(kThreads)
    join_parts_kernel(const float *Q, int64_t ldq, int64_t stride_q, int32_t parts, int32_t s, uint16_t *P,
                      int64_t ldp, int64_t stride_p, int64_t lo)
{
    __shared__ float sum[32][33];
    const int32_t t = static_cast<int32_t>(blockIdx.x);
    int32_t bi = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
    while (bi * (bi + 1) / 2 > t)
        --bi;
    while ((bi + 1) * (bi + 2) / 2 <= t)
        ++bi;
    const int32_t r0 = 32 * bi, c0 = 32 * (t - bi * (bi + 1) / 2), g = static_cast<int32_t>(blockIdx.y);
    const int32_t lane = static_cast<int32_t>(threadIdx.x) % 32, warp = static_cast<int32_t>(threadIdx.x) / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const float *q = Q + static_cast<int64_t>(g) * parts * stride_q;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int32_t k = 0; k < parts; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t r = r0 + warp + 8 * j, c = c0 + lane;
            if (r < s && c < s)
                v[j] += __ldcg(q + k * stride_q + r * ldq + c);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sum[warp + 8 * j][lane] = v[j];
    __syncthreads();
    uint16_t *p = P + g * stride_p;
    for (int32_t i = static_cast<int32_t>(threadIdx.x); i < 32 * 16; i += kThreads) {
        const int32_t a = i / 16, b = i % 16 * 2;  // row and first column of a pair
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m == 1 && r0 == c0)
                break;
            // (a diagonal block's elements above the diagonal are those below it)
            const bool f0 = m == 1 || (r0 == c0 && b > a), f1 = m == 1 || (r0 == c0 && b + 1 > a);
            const float x0 = f0 ? sum[b][a] : sum[a][b], x1 = f1 ? sum[b + 1][a] : sum[a][b + 1];
            const int32_t row = (m ? c0 : r0) + a, col = (m ? r0 : c0) + b;
            if (row >= s || col >= s)
                continue;
            const uint32_t hi = pack_f16x2(x0, x1);  // (an odd s: the second one is padding)
            uint16_t *to = p + row * ldp + col;
            *reinterpret_cast<uint32_t *>(to) = hi;
            if (lo)
                *reinterpret_cast<uint32_t *>(to + lo) =
                    pack_f16x2(x0 - cvt_f16_f32(static_cast<unsigned short>(hi)),
                               x1 - cvt_f16_f32(static_cast<unsigned short>(hi >> 16)));
        }
    }
}

bool vec_ok(const void *X, int64_t ldx, int64_t stride_x, int type)
{
    const int64_t es = type == kOutF32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx * es % 16 == 0 && stride_x * es % 16 == 0;
}

template <class... P, class... A>
cudaError_t launch(void (*kfn)(P...), dim3 grid, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kfn, static_cast<P>(args)...);
}

unsigned blocks_for(int64_t M, int64_t N, int64_t per_thread)
{
    const int64_t pieces = (N + 7) / 8 * M;
    const int64_t b = (pieces + kThreads * per_thread - 1) / (kThreads * per_thread);
    return static_cast<unsigned>(b < 1 ? 1 : (b > 2048 ? 2048 : b));
}

}  // namespace

int orthogonalize_parts(int64_t M, int64_t N)
{
    const unsigned b = blocks_for(M, N, 4);
    return static_cast<int>(b < kMaxParts ? b : kMaxParts);
}

cudaError_t launch_square_sums(const void *X, int64_t ldx, int64_t stride_x, int type, int32_t M, int32_t N,
                               int32_t count, float *partial, int parts, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(parts), static_cast<unsigned>(count));
    auto go = [&](auto k) { return launch(k, grid, stream, X, ldx, stride_x, M, N, partial); };
    const bool vec = vec_ok(X, ldx, stride_x, type);
    if (type == kOutF32)
        return vec ? go(square_sums_kernel<kOutF32, 8>) : go(square_sums_kernel<kOutF32, 2>);
    if (type == kOutBF16)
        return vec ? go(square_sums_kernel<kOutBF16, 8>) : go(square_sums_kernel<kOutBF16, 2>);
    return vec ? go(square_sums_kernel<kOutF16, 8>) : go(square_sums_kernel<kOutF16, 2>);
}

cudaError_t launch_normalize(const void *X, int64_t ldx, int64_t stride_x, int type, int32_t M, int32_t N,
                             int32_t count, const float *partial, int parts, float scale, float eps,
                             uint16_t *Xs, int64_t lds, int64_t stride_s, int64_t lo, cudaStream_t stream)
{
    const dim3 grid(blocks_for(M, N, 4), static_cast<unsigned>(count));
    auto go = [&](auto k) {
        return launch(k, grid, stream, X, ldx, stride_x, M, N, partial, parts, scale, eps, Xs, lds, stride_s, lo);
    };
    const bool vec = vec_ok(X, ldx, stride_x, type);
    if (type == kOutF32)
        return vec ? go(normalize_kernel<kOutF32, 8>) : go(normalize_kernel<kOutF32, 2>);
    if (type == kOutBF16)
        return vec ? go(normalize_kernel<kOutBF16, 8>) : go(normalize_kernel<kOutBF16, 2>);
    return vec ? go(normalize_kernel<kOutF16, 8>) : go(normalize_kernel<kOutF16, 2>);
}

cudaError_t launch_join_parts(const float *Q, int64_t ldq, int64_t stride_q, int32_t parts, int32_t s, int32_t count,
                              uint16_t *P, int64_t ldp, int64_t stride_p, int64_t lo, cudaStream_t stream)
{
    const unsigned nb = (static_cast<unsigned>(s) + 31) / 32;
    return launch(join_parts_kernel, dim3(nb * (nb + 1) / 2, static_cast<unsigned>(count)), stream, Q, ldq, stride_q,
                  parts, s, P, ldp, stride_p, lo);
}

}  // namespace tcg
