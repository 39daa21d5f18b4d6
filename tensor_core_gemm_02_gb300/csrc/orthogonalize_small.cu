// orthogonalize_small.cu -- gemm_orthogonalize for small matrices: all steps in one launch.
//
// The tile kernels take three launches a step, about 5 us each however little there is to do.  Here
// a matrix is one thread block's, or a cluster's of eight with an eighth of its longer side each,
// and stays in shared memory in float32 from the norm to the last step.  With X as s x l, s <= l (a
// tall matrix is read and written transposed), a step is
//   P = X X^T   each block over its own columns; the blocks' sums are added in order, an eighth of P
//               by each block, which hands its part to all;
//   Q = b P + c P P   by every block for itself;
//   X <- a X + Q X    each block its own columns.
// Products are float32 FMAs: a thread has four rows times four rows (or four columns), 64 FMAs for
// eight 16-byte loads of shared memory, about half of the SMs' rate.  Where s x s leaves threads
// over, groups of threads share the sums, and their parts are added in order: no atomics, the
// same bits every time.  Rows T apart are a thread's, T = s / 4, and pitches are odd multiples of 16
// bytes, so that the loads of a warp meet no bank twice.
//
// Bound by latency: 38 x 24 in five steps 19 us; 4096 x 16, on eight blocks, 38, 6.5 a step, of which the
// FMAs take 2.7 and the exchange 2.  (With 64 x 64 products a step takes 12 us and more, and the tile
// kernels' launches are no slower.)
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_group.h"

namespace tcg {

namespace {

constexpr int kThreads = 256;
constexpr int kClusterMost = 8;

__device__ __forceinline__ float load_element(const void *X, int64_t at, int type)
{
    if (type == kOutF32)
        return __ldcg(static_cast<const float *>(X) + at);
    const unsigned short h = __ldcg(static_cast<const unsigned short *>(X) + at);
    return type == kOutBF16 ? cvt_bf16_f32(h) : cvt_f16_f32(h);
}

__device__ __forceinline__ void store_element(void *Y, int64_t at, int type, float v)
{
    if (type == kOutF32)
        static_cast<float *>(Y)[at] = v;
    else
        static_cast<uint16_t *>(Y)[at] = type == kOutBF16 ? f32_to_bf16_rn(v) : f32_to_f16_rn(v);
}

__device__ __forceinline__ float dot4(const float4 &x, const float4 &y, float sum)
{
    return fmaf(x.w, y.w, fmaf(x.z, y.z, fmaf(x.y, y.y, fmaf(x.x, y.x, sum))));
}

// parts[g][i][j] = group g's part of sum over k < 4 k4 of A[i][k] A[j][k], for i, j < 4 T; returns the groups
__device__ __forceinline__ int32_t products(const float *A, int32_t pitch, int32_t T, int32_t k4, float *parts)
{
    const int32_t tiles = T * T, groups = kThreads / tiles, s4 = 4 * T;
    const int32_t tile = static_cast<int32_t>(threadIdx.x) % tiles, g = static_cast<int32_t>(threadIdx.x) / tiles;
    const int32_t ti = tile / T, tj = tile % T;
    if (g < groups) {
        float acc[4][4] = {};
        const float *x = A + ti * pitch, *y = A + tj * pitch;
        for (int32_t k = g; k < k4; k += groups) {
            float4 p[4], q[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = *reinterpret_cast<const float4 *>(x + r * T * pitch + 4 * k);
                q[r] = *reinterpret_cast<const float4 *>(y + r * T * pitch + 4 * k);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] = dot4(p[r], q[c], acc[r][c]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                parts[(g * s4 + ti + T * r) * s4 + tj + T * c] = acc[r][c];
    }
    __syncthreads();
    return groups;
}

__global__ void __launch_bounds__(kThreads, 1) orthogonalize_small_kernel(const SmallArgs a)
{
    extern __shared__ float4 smem4[];
    __shared__ float warp_sum[kThreads / 32], totals[kClusterMost];
    const int32_t tid = static_cast<int32_t>(threadIdx.x);
    const int32_t C = a.cluster, rank = C > 1 ? static_cast<int32_t>(cluster_ctarank()) : 0;
    const int32_t g = static_cast<int32_t>(blockIdx.x) / C;
    const int32_t T = (a.s + 3) / 4, s4 = 4 * T, px = a.px, ps = a.ps;
    float *x = reinterpret_cast<float *>(smem4), *y = x + s4 * px;
    float *own = y + s4 * px, *P = own + s4 * ps, *Q = P + s4 * ps, *parts = Q + s4 * ps;
    const int32_t k0 = rank * a.lc, cols = max(0, min(a.lc, a.l - k0)), lc4 = (a.lc + 3) / 4;

    for (int32_t i = tid; i < s4 * px / 4; i += kThreads)  // (rows and columns that only fill up)
        reinterpret_cast<float4 *>(x)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    // element (i, k) of X is X[i][k], or X[k][i] of a tall matrix; neighbours in memory by neighbours
    const int32_t in_row = a.tall ? a.s : cols, n_rows = a.tall ? cols : a.s;
    float sum = 0.f;
    for (int32_t e = tid; e < in_row * n_rows; e += kThreads) {
        const int32_t r = e / in_row, c = e - r * in_row;
        const float v = load_element(a.X, g * a.stride_x + (a.tall ? (k0 + r) * a.ldx + c : r * a.ldx + k0 + c), a.type);
        x[a.tall ? c * px + r : r * px + c] = v;
        sum = fmaf(v, v, sum);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (tid % 32 == 0)
        warp_sum[tid / 32] = sum;
    if (C > 1)
        cluster_sync_all();  // (every block runs: its shared memory may be written)
    else
        __syncthreads();
    if (tid < C) {
        float t = 0.f;
        for (int i = 0; i < kThreads / 32; ++i)
            t += warp_sum[i];
        if (C > 1)
            st_shared_cluster_u32(mapa_shared(smem_u32(totals + rank), static_cast<uint32_t>(tid)), __float_as_uint(t));
        else
            totals[0] = t;
    }
    if (C > 1)
        cluster_sync_all();
    else
        __syncthreads();
    float total = 0.f;
    for (int32_t c = 0; c < C; ++c)
        total += totals[c];
    const float f = norm_factor(1.0f, total, a.eps);
    for (int32_t i = tid; i < s4 * px; i += kThreads)
        x[i] *= f;
    __syncthreads();

    for (int32_t step = 0; step < a.steps; ++step) {
        int32_t groups = products(x, px, T, lc4, parts);
        float *to = C > 1 ? own : P;
        for (int32_t e = tid; e < s4 * s4; e += kThreads) {
            float v = 0.f;
            for (int32_t k = 0; k < groups; ++k)
                v += parts[k * s4 * s4 + e];
            const int32_t i = e / s4;
            to[i * ps + e - i * s4] = v;
        }
        if (C > 1) {
            cluster_sync_all();
            for (int32_t e = tid + kThreads * rank; e < s4 * ps; e += kThreads * C) {
                float v[kClusterMost];
#pragma unroll
                for (uint32_t c = 0; c < kClusterMost; ++c)
                    v[c] = __uint_as_float(ld_shared_cluster_u32(mapa_shared(smem_u32(own + e), c)));
                float t = 0.f;
#pragma unroll
                for (int c = 0; c < kClusterMost; ++c)
                    t += v[c];
#pragma unroll
                for (uint32_t c = 0; c < kClusterMost; ++c)
                    st_shared_cluster_u32(mapa_shared(smem_u32(P + e), c), __float_as_uint(t));
            }
            cluster_sync_all();
        } else {
            __syncthreads();
        }
        groups = products(P, ps, T, T, parts);
        for (int32_t e = tid; e < s4 * s4; e += kThreads) {
            float v = 0.f;
            for (int32_t k = 0; k < groups; ++k)
                v += parts[k * s4 * s4 + e];
            const int32_t i = e / s4, at = i * ps + e - i * s4;
            Q[at] = fmaf(a.b, P[at], a.c * v);
        }
        __syncthreads();
        for (int32_t e = tid; e < T * lc4; e += kThreads) {
            const int32_t ti = e / lc4, k = e - ti * lc4;
            float4 acc[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int32_t j = 0; j < s4; j += 4) {
                float4 u[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    u[c] = *reinterpret_cast<const float4 *>(x + (j + c) * px + 4 * k);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 w = *reinterpret_cast<const float4 *>(Q + (ti + T * r) * ps + j);
                    const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        acc[r].x = fmaf(ws[c], u[c].x, acc[r].x);
                        acc[r].y = fmaf(ws[c], u[c].y, acc[r].y);
                        acc[r].z = fmaf(ws[c], u[c].z, acc[r].z);
                        acc[r].w = fmaf(ws[c], u[c].w, acc[r].w);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int32_t at = (ti + T * r) * px + 4 * k;
                const float4 old = *reinterpret_cast<const float4 *>(x + at);
                *reinterpret_cast<float4 *>(y + at) =
                    make_float4(fmaf(a.a, old.x, acc[r].x), fmaf(a.a, old.y, acc[r].y), fmaf(a.a, old.z, acc[r].z),
                                fmaf(a.a, old.w, acc[r].w));
            }
        }
        __syncthreads();
        float *t = x;
        x = y;
        y = t;
    }
    for (int32_t e = tid; e < in_row * n_rows; e += kThreads) {
        const int32_t r = e / in_row, c = e - r * in_row;
        store_element(a.Y, g * a.stride_y + (a.tall ? (k0 + r) * a.ldy + c : r * a.ldy + k0 + c), a.out,
                      x[a.tall ? c * px + r : r * px + c]);
    }
}

// a pitch of at least n floats: an odd number of 16-byte pieces
int64_t odd_pitch(int64_t n) { return 4 * ((n + 3) / 4 | 1); }

}  // namespace

size_t orthogonalize_small_shared(int64_t s, int64_t l, int cluster)
{
    const int64_t s4 = (s + 3) / 4 * 4, lc = (l + cluster - 1) / cluster;
    return static_cast<size_t>(2 * s4 * odd_pitch(lc) + 3 * s4 * odd_pitch(s4) + 16 * kThreads) * sizeof(float);
}

cudaError_t launch_orthogonalize_small(SmallArgs a, int64_t count, cudaStream_t stream)
{
    a.lc = (a.l + a.cluster - 1) / a.cluster;
    a.px = static_cast<int32_t>(odd_pitch(a.lc));
    a.ps = static_cast<int32_t>(odd_pitch((a.s + 3) / 4 * 4));
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(orthogonalize_small_kernel),
                                     static_cast<uint32_t>(kSmallShared), done);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(count * a.cluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = orthogonalize_small_shared(a.s, a.l, a.cluster);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TCG_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, orthogonalize_small_kernel, a);
}

}  // namespace tcg
