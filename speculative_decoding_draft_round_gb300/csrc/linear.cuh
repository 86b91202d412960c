// linear.cuh -- what the 8-bit products' kernels share: how many rows live, where a row goes, its last step.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace dspark {

__device__ __forceinline__ int linear_rows(const LinearParams& p, bool report)
{
    if (!p.n_rows) return p.T;
    const int n = *p.n_rows;
    if (n >= 0 && n <= p.T) return n;
    if (report) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    return n < 0 ? 0 : p.T;
}

// The row of out that row t goes to, -1 for none.
__device__ __forceinline__ long long linear_place(const LinearParams& p, int t)
{
    if (!p.out_row) return t;
    const int r = p.out_row[t];
    if (r < p.out_rows) return r < 0 ? -1 : r;
    raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    return -1;
}

template <typename T>
__device__ __forceinline__ T linear_out(float sum, float x_scale, float w_scale, float bias);
template <>
__device__ __forceinline__ float linear_out<float>(float sum, float x_scale, float w_scale, float bias)
{
    return fmaf(sum * x_scale, w_scale, bias);
}
template <>
__device__ __forceinline__ __nv_bfloat16 linear_out<__nv_bfloat16>(float sum, float x_scale, float w_scale, float bias)
{
    return __float2bfloat16_rn(fmaf(sum * x_scale, w_scale, bias));
}

}  // namespace dspark
