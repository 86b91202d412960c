// linear_i8.cu -- rows of 8-bit codes times 8-bit weights on CUDA cores (dspark_linear_i8, DSPARK_PATH_CUDA_CORE):
//   out[out_row[t]][n] = (sum_k x[t][k] w[n][k]) * x_scale[t] * w_scale[n] + bias[n]
// 64 x 64 output tiles, K in slices of 64 staged in shared memory as words of four codes, dot products of four
// codes an instruction into 32-bit integers: the sums are exact. Any K, strides and alignment.
#include "common.cuh"
#include "internal.h"
#include "linear.cuh"

namespace dspark {

namespace {

constexpr int kTile = 64, kSlice = 16;   // rows and channels of a tile, words of four codes a slice

// words [kSlice] of four codes of one row from code k0 on; zeros past K
__device__ __forceinline__ int word_at(const int8_t* row, int k, int K, bool aligned)
{
    if (k >= K) return 0;
    if (aligned && k + 4 <= K) return *reinterpret_cast<const int*>(row + k);
    uint32_t w = 0;
    for (int i = 0; i < 4 && k + i < K; ++i) w |= (uint32_t)(uint8_t)row[k + i] << (8 * i);
    return (int)w;
}

template <typename T>
__global__ void __launch_bounds__(256) linear_simt_kernel(LinearParams p)
{
    __shared__ int xs[kSlice][kTile + 1], ws[kSlice][kTile + 1];
    pdl_enter();
    const int live = linear_rows(p, blockIdx.x == 0 && threadIdx.x == 0);
    const int channels = (p.N + kTile - 1) / kTile;
    const long long t0 = (long long)(blockIdx.x / channels) * kTile;
    if (t0 >= live) return;
    const int n0 = (int)(blockIdx.x % channels) * kTile;
    const bool ax = ((reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)p.x_rs) & 3) == 0;
    const bool aw = ((reinterpret_cast<uintptr_t>(p.w) | (uintptr_t)p.w_rs) & 3) == 0;
    const int ti = threadIdx.x / 16, ni = threadIdx.x % 16;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 4 * kSlice) {
        for (int i = threadIdx.x; i < kSlice * kTile; i += 256) {
            const int k = i % kSlice, row = i / kSlice;
            xs[k][row] = t0 + row < live ? word_at(p.x + (t0 + row) * p.x_rs, k0 + 4 * k, p.K, ax) : 0;
            ws[k][row] = n0 + row < p.N ? word_at(p.w + (long long)(n0 + row) * p.w_rs, k0 + 4 * k, p.K, aw) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSlice; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = __dp4a(xs[k][ti + 16 * u], ws[k][ni + 16 * v], acc[u][v]);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long t = t0 + ti + 16 * u;
        if (t >= live) continue;
        const long long row = linear_place(p, (int)t);
        if (row < 0) continue;
        const float xsc = p.x_scale[t];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = n0 + ni + 16 * v;
            if (n < p.N)
                static_cast<T*>(p.out)[row * p.o_rs + n] = linear_out<T>((float)acc[u][v], xsc, p.w_scale[n], p.bias ? p.bias[n] : 0.f);
        }
    }
}

}  // namespace

cudaError_t launch_linear_simt(const LinearParams& p, cudaStream_t s)
{
    const long long tiles = (long long)cdiv(p.N, kTile) * cdiv(p.T, kTile);
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles);
    const cudaError_t e = p.dtype == DSPARK_BF16 ? launch_pdl(linear_simt_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, p)
                                                 : launch_pdl(linear_simt_kernel<float>, grid, dim3(256), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
