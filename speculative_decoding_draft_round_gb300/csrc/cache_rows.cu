// cache_rows.cu -- key and value rows into the 4-bit cache (dspark_cache_append) and back out as
// values (dspark_cache_read). Layout and rounding in dspark.h.
//
// A thread takes 8 channels of a row: one 32-bit word of codes. The 4 threads of a group of 32
// channels find its largest magnitude with two shuffles. Both kernels move each byte once.
#include "cache.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kRowsThreads = 256;
constexpr int kVec = 8;   // channels a thread

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, bool aligned, float (&x)[kVec])
{
    if (aligned) {
        // plain loads, not the read-only path: the rows may come from the kernel just waited for
        alignas(16) uint32_t u[kVec * sizeof(T) / 4];
#pragma unroll
        for (int i = 0; i < (int)(kVec * sizeof(T) / 16); ++i)
            reinterpret_cast<uint4*>(u)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (sizeof(T) == 4)
                x[i] = __uint_as_float(u[i % (kVec * sizeof(T) / 4)]);
            else
                x[i] = __uint_as_float(i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = to_f32<T>(p[i]);
    }
}

__device__ __forceinline__ void store_vec(float* p, const float (&x)[kVec])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[kVec])
{
    uint4 v;
    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = v;
}

// x / s rounded to the nearest integer, ties to even, in -7 .. 7 (s > 0). The remainder x - c s of the
// guess c is one rounding of an exact difference, so its comparison with s / 2 decides exactly.
__device__ __forceinline__ int nearest_code(float x, float s, float inv)
{
    float c = fminf(fmaxf(rintf(x * inv), -8.f), 8.f);
    const float r = fmaf(-c, s, x), h = 0.5f * s;
    const bool odd = ((int)c & 1) != 0;
    if (r > h || (r == h && odd)) c += 1.f;
    else if (r < -h || (r == -h && odd)) c -= 1.f;
    return (int)fminf(fmaxf(c, -7.f), 7.f);
}

// Flat index = ((token * 2 + (0 = K, 1 = V)) * Hkv + head) * (D / 8) + vec: a warp's threads read
// consecutive channels; the 4 threads of a group are 4 aligned lanes.
struct RowAt {
    int t, half, h, vec;
};

__device__ __forceinline__ RowAt row_at(long long i, int Hkv, int vecs)
{
    RowAt a;
    a.vec = (int)(i % vecs);
    const long long row = i / vecs;
    a.h = (int)(row % Hkv);
    const long long th = row / Hkv;
    a.half = (int)(th & 1);
    a.t = (int)(th >> 1);
    return a;
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) cache_append_kernel(CacheRowsParams p, int aligned)
{
    pdl_enter();
    const int vecs = p.c.D / kVec, groups = p.c.D / kCacheGroup;
    const long long n = (long long)p.T * 2 * p.c.Hkv * vecs;
    const long long i = (long long)blockIdx.x * kRowsThreads + threadIdx.x;
    const bool in = i < n;
    const RowAt a = row_at(in ? i : n - 1, p.c.Hkv, vecs);
    int page = 0, slot = 0;
    const bool live = in && cache_slot(p.c, p.request[a.t], p.position[a.t], p.status, page, slot);
    float x[kVec] = {};
    if (live) {
        const T* src = a.half == 0 ? static_cast<const T*>(p.k) + a.t * p.k_ts + a.h * p.k_hs
                                   : static_cast<const T*>(p.v) + a.t * p.v_ts + a.h * p.v_hs;
        load_vec<T>(src + a.vec * kVec, aligned, x);
    }
    float top = 0.f;
    bool odd_input = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float m = fabsf(x[j]);
        if (m <= FLT_MAX) {
            top = fmaxf(top, m);
        } else {   // an infinity takes the largest code, NaN the code of 0
            odd_input = true;
            x[j] = x[j] != x[j] ? 0.f : copysignf(FLT_MAX, x[j]);
        }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!live) return;
    if (odd_input) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
    const float s8 = __bfloat162float(__float2bfloat16_rn(top * (1.f / 7.f)));
    const __half sh = __float2half_rn(fminf(s8, kCacheMaxScale));
    const float s = __half2float(sh);
    uint32_t word = 0x88888888u;   // the code of 0
    if (s > 0.f) {
        const float inv = 1.f / s;
        word = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) word |= (uint32_t)(nearest_code(x[j], s, inv) + 8) << (4 * j);
    }
    const CacheBlock b = cache_block(p.c.page_size, p.c.D);
    uint8_t* blk = cache_page_block(p.c, page, a.h, b.bytes);
    const uint32_t codes = a.half == 0 ? 0u : b.v_codes;
    *reinterpret_cast<uint32_t*>(blk + codes + (uint32_t)slot * (p.c.D / 2) + a.vec * 4) = word;
    if (a.vec % 4 == 0) {
        const int g = a.vec / 4;
        const uint32_t at = a.half == 0 ? b.k_scales + (uint32_t)(slot * groups + g) * 2u
                                        : b.v_scales + v_scale_at(slot, g, groups);
        *reinterpret_cast<__half*>(blk + at) = sh;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) cache_read_kernel(CacheRowsParams p)
{
    pdl_enter();
    const int vecs = p.c.D / kVec, groups = p.c.D / kCacheGroup;
    const long long n = (long long)p.T * 2 * p.c.Hkv * vecs;
    const long long i = (long long)blockIdx.x * kRowsThreads + threadIdx.x;
    if (i >= n) return;
    const RowAt a = row_at(i, p.c.Hkv, vecs);
    int page = 0, slot = 0;
    float x[kVec] = {};
    if (cache_slot(p.c, p.request[a.t], p.position[a.t], p.status, page, slot)) {
        const CacheBlock b = cache_block(p.c.page_size, p.c.D);
        const uint8_t* blk = cache_page_block(p.c, page, a.h, b.bytes);
        const int g = a.vec / 4;
        const uint32_t codes = a.half == 0 ? 0u : b.v_codes;
        const uint32_t at = a.half == 0 ? b.k_scales + (uint32_t)(slot * groups + g) * 2u
                                        : b.v_scales + v_scale_at(slot, g, groups);
        const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + codes + (uint32_t)slot * (p.c.D / 2) + a.vec * 4);
        const float s = __half2float(*reinterpret_cast<const __half*>(blk + at));
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[j] = (float)((int)((word >> (4 * j)) & 15u) - 8) * s;
    }
    T* dst = static_cast<T*>(a.half == 0 ? p.k_out : p.v_out) + ((size_t)a.t * p.c.Hkv + a.h) * p.c.D + a.vec * kVec;
    store_vec(dst, x);
}

template <typename T>
bool rows_aligned(const CacheRowsParams& p)
{
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v);
    const int64_t strides = p.k_ts | p.k_hs | p.v_ts | p.v_hs;
    return base % 16 == 0 && (strides * (int64_t)sizeof(T)) % 16 == 0;
}

long long rows_grid(const CacheRowsParams& p)
{
    const long long n = (long long)p.T * 2 * p.c.Hkv * (p.c.D / kVec);
    return (n + kRowsThreads - 1) / kRowsThreads;
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsParams& p, cudaStream_t s)
{
    const dim3 grid((unsigned)rows_grid(p));
    const cudaError_t e =
        p.dtype == DSPARK_BF16
            ? launch_pdl(cache_append_kernel<__nv_bfloat16>, grid, dim3(kRowsThreads), 0, s, p,
                         (int)rows_aligned<__nv_bfloat16>(p))
            : launch_pdl(cache_append_kernel<float>, grid, dim3(kRowsThreads), 0, s, p, (int)rows_aligned<float>(p));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheRowsParams& p, cudaStream_t s)
{
    const dim3 grid((unsigned)rows_grid(p));
    const cudaError_t e = p.dtype == DSPARK_BF16
                              ? launch_pdl(cache_read_kernel<__nv_bfloat16>, grid, dim3(kRowsThreads), 0, s, p)
                              : launch_pdl(cache_read_kernel<float>, grid, dim3(kRowsThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
