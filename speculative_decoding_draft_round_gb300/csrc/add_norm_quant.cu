// add_norm_quant.cu -- a layer's residual sum, the norm of its rows and their 8-bit codes, one pass over the rows
// (dspark_add_norm_quant).
//
//   s = rn(x + residual),  p = s * gain,  y = p / sqrt(sum s^2 / N + eps),
//   scale = max|y| / 127,  code = rint(127 p / max|p|): the norm cancels from the code.
//
// Codes are exact. In fp32 the quotient 127 p / max|p| carries four roundings, 127 * 4 * 2^-24 < 2^-14 in all, so its
// nearest whole number is the exact one's unless it lies within 2^-14 of a half. Those few are settled
// from the exact products s * gain (48 bits) and the exact largest of them (fp32 head and remainder). Rows whose
// products or squares leave fp32's range, and those with a NaN or an infinity, are done in 64 bits altogether.
//
// The bytes bound it: a row is read once into registers (above 12288 wide part of it goes through local memory) and every
// output leaves from there. Measured, in bf16 with a residual: 32749 rows of 5120 to values (1341 MB) 235 us, 201 at the
// copy's rate; to codes 2176 rows of 4096 16 us in a row (inputs in the L2), 9 at the copy's rate, where instructions (some
// 40 an element) and the two barriers a row count, and 16 rows 3 us. A warp a row up to 1024 wide; above, two or three
// pieces of 8 a thread (four took 26 us for those 2176 rows: fewer warps wait for the barriers).
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kNormMaxN = 32768;
constexpr float kNearHalf = 0.5f - 0x1.0p-14f;

template <typename T>
__device__ __forceinline__ float rounded(float x);   // to T and back
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

template <typename T>
__device__ __forceinline__ T narrowed(float x);
template <>
__device__ __forceinline__ float narrowed<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrowed<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 8 elements of a row in 16-byte pieces
template <typename T>
struct Piece {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];   // y or sum may lie there
    }
    __device__ __forceinline__ void store(T* p) const
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const;
    __device__ __forceinline__ void set(const float (&f)[8]);
};
template <>
__device__ __forceinline__ void Piece<__nv_bfloat16>::get(float (&f)[8]) const
{
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void Piece<__nv_bfloat16>::set(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void Piece<float>::get(float (&f)[8]) const
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(u[i].x);
        f[4 * i + 1] = __uint_as_float(u[i].y);
        f[4 * i + 2] = __uint_as_float(u[i].z);
        f[4 * i + 3] = __uint_as_float(u[i].w);
    }
}
template <>
__device__ __forceinline__ void Piece<float>::set(const float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
        u[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
}

__device__ __forceinline__ int live_rows(const int32_t* n_rows, int T, int* status, bool report)
{
    if (!n_rows) return T;
    const int n = *n_rows;
    if (n >= 0 && n <= T) return n;
    if (report) raise_status(status, DSPARK_ERR_DEVICE_INPUT);
    return n < 0 ? 0 : T;
}

// A row's statistics. m: bits of max|s * gain| in fp32 (above 0x7F800000: a NaN), lo: the largest remainder of the
// products that have it, as bits that compare as whole numbers.
struct RowStats {
    float sum;
    uint32_t m;
};

__device__ __forceinline__ int ordered(float x)
{
    const int b = __float_as_int(x);
    return b >= 0 ? b : b ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int b) { return __int_as_float(b >= 0 ? b : b ^ 0x7FFFFFFF); }

// What the product s * g leaves beyond its fp32 rounding, where that is the row's largest
__device__ __forceinline__ int remainder_at(float s, float g, uint32_t m, int lo)
{
    const float h = __fmul_rn(s, g), rest = __fmaf_rn(s, g, -h);
    return (__float_as_uint(h) & 0x7FFFFFFFu) == m ? max(lo, ordered(h < 0.f ? -rest : rest)) : lo;
}

// The rows' threads: a warp, or a whole CTA of NT. Every reduction takes fresh words of shared memory, so that one
// barrier is enough for each; they come in this order.
template <int NT>
struct Team {
    static constexpr int kWarps = NT / 32;
    float* sums;       // [kWarps]
    uint32_t* tops;    // [kWarps]
    int* lo;           // [1]
    double* wide;      // [2][kWarps]

    __device__ __forceinline__ RowStats stats(float sum, uint32_t m) const
    {
        sum = warp_sum(sum);
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (kWarps > 1) {
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            if (lane == 0) {
                sums[warp] = sum;
                tops[warp] = m;
                if (warp == 0) *lo = INT32_MIN;
            }
            __syncthreads();
            sum = 0.f;
            m = 0u;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                sum += sums[w];
                m = max(m, tops[w]);
            }
        }
        return RowStats{sum, m};
    }
    // the largest of what the threads that hold the row's largest product found
    __device__ __forceinline__ float largest(bool holds, int x) const
    {
        if constexpr (kWarps == 1) {
            x = __reduce_max_sync(0xffffffffu, holds ? x : INT32_MIN);
        } else {
            if (holds) atomicMax(lo, x);
            __syncthreads();
            x = *lo;
        }
        return from_ordered(x);
    }
    // sum of a, largest of b
    __device__ __noinline__ void in_64(double& a, double& b) const
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b = fmax(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        if constexpr (kWarps > 1) {
            if ((threadIdx.x & 31) == 0) {
                wide[threadIdx.x >> 5] = a;
                wide[kWarps + (threadIdx.x >> 5)] = b;
            }
            __syncthreads();
            a = b = 0.0;
            for (int w = 0; w < kWarps; ++w) {
                a += wide[w];
                b = fmax(b, wide[kWarps + w]);
            }
        }
    }
};

__device__ __forceinline__ double product(float s, float g) { return (double)s * (double)g; }

// NaN counts as infinity
__device__ __forceinline__ double larger(double top, double h)
{
    return h <= top ? top : h < (double)INFINITY ? h : (double)INFINITY;
}

// 127 p has up to 55 bits and the division rounds, so the quotient tells k only; whether the code is k or k + 1 tells the
// sign of 254 |p| - (2 k + 1) top = (256 |p| - (2 k + 1) top) - 2 |p|. Next to k + 1/2 the bracket is near 2 |p| and, as |p|
// and top have 48 bits and top / |p| is at most 254, a whole number of at most 50 bits: the fused multiply-add is exact.
__device__ __noinline__ int code_in_64(float s, float g, double top)
{
    const double p = fabs(product(s, g)), k = floor(p * 127.0 / top), d = __fma_rn(-(2.0 * k + 1.0), top, 256.0 * p) - 2.0 * p;
    const int q = (int)k, n = q + (d > 0.0 || (d == 0.0 && (q & 1)) ? 1 : 0);   // a tie goes to the even one
    return product(s, g) < 0.0 ? -n : n;
}

// Whether a row's fp32 statistics can be used: what is formed from them neither overflows nor loses bits below the
// normal range.
__device__ __forceinline__ bool in_range(const RowStats& st, int N)
{
    const float m = __uint_as_float(st.m);
    return st.m < 0x7F800000u && m >= 1e-30f && m <= 1e30f && st.sum <= 1e30f && st.sum >= 1e-25f * (float)N;
}

// What the row's elements are turned with.
struct RowScales {
    float inv, scale, per;   // y = p * inv, the codes' scale, code = p * per
    float m, lo;             // max|p|: its fp32 rounding and what that leaves (rows whose statistics are in range)
    double top;              // max|p| (the others)
};

// The code of a quotient f near a half, k + 1/2: the sign of 254 |p| - (2 k + 1) max|p|, whose heads are near enough to
// leave each other exactly and whose remainders are exact. 64 bits only where that is next to nothing: on this chip a
// division in 64 bits by a warp takes as long as its whole row (2176 rows of 4096 29 us with one for every such code).
// Each rounding is spelt out: a product that the compiler fused with the difference would be exact there, and its
// remainder counted twice.
__device__ __noinline__ int settled(float s, float g, float f, const RowScales& r)
{
    const float h = __fmul_rn(s, g), rest = __fmaf_rn(s, g, -h), k = floorf(fabsf(f)), o = 2.f * k + 1.f;
    const float a = __fmul_rn(254.f, fabsf(h)), b = __fmul_rn(o, r.m);
    const float heads = __fsub_rn(__fmaf_rn(254.f, fabsf(h), -a), __fmaf_rn(o, r.m, -b));
    const float rests = __fsub_rn(__fmul_rn(254.f, h < 0.f ? -rest : rest), __fmul_rn(o, r.lo));
    const float d = __fadd_rn(__fsub_rn(a, b), __fadd_rn(heads, rests));
    // heads alone (no gain): d has the sign of the difference itself, and is 0 for a tie, which goes to the even code
    const bool exact = rest == 0.f && r.lo == 0.f;
    if (fabsf(d) <= 0x1.0p-34f * r.m && !exact) return code_in_64(s, g, (double)r.m + (double)r.lo);
    const int q = (int)k + (d > 0.f || (d == 0.f && ((int)k & 1)) ? 1 : 0);
    return f < 0.f ? -q : q;
}

template <int NT>
__device__ __forceinline__ void finish(const NormParams& p, const RowStats& st, RowScales& k)
{
    const float m = __uint_as_float(st.m);
    k.inv = p.norm ? 1.f / sqrtf(st.sum / (float)p.N + p.eps) : 1.f;
    const float top = m * k.inv;
    k.scale = top <= FLT_MAX ? top / 127.f : m * (k.inv / 127.f);   // the largest |y| may be past fp32's end and this not
    k.per = 127.f / m;
    k.m = m;
    k.lo = 0.f;
}

// CTAs an SM that the registers have to leave room for: the branches in 64 bits, which hardly any row takes, would cost
// one otherwise (32749 rows of 5120 in bf16 309 us instead of 236).
template <typename T, int NT, int V>
constexpr int kCtas = NT == 32    ? (V == 1 ? 4 : V < 4 ? 3 : 2)
                      : NT == 128 ? 7
                      : NT == 256 ? 3
                      : NT == 512 && V == 2 && sizeof(T) == 2 ? 2 : 1;

// N a multiple of 8, rows and outputs on 16-byte (codes on 8-byte) boundaries: V pieces of 8 elements a thread, kept in
// registers. NT = 32: a row is a warp, eight to a CTA.
template <typename T, int NT, int V>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT, kCtas<T, NT, V>) norm_vec_kernel(NormParams p)
{
    constexpr int kRows = NT == 32 ? 8 : 1, kWarps = NT / 32;
    __shared__ float s_sums[kWarps];
    __shared__ uint32_t s_tops[kWarps];
    __shared__ int s_lo;
    __shared__ double s_wide[2 * kWarps];
    const Team<NT> team{s_sums, s_tops, &s_lo, s_wide};
    pdl_enter();
    const int t = blockIdx.x * kRows + (kRows > 1 ? (int)(threadIdx.x >> 5) : 0);
    const int tid = kRows > 1 ? threadIdx.x & 31 : threadIdx.x;
    if (t >= live_rows(p.n_rows, p.T, p.status, blockIdx.x == 0 && threadIdx.x == 0)) return;
    const T* x = static_cast<const T*>(p.x) + t * p.x_rs;
    const T* r = static_cast<const T*>(p.residual) + t * p.r_rs;
    const int pieces = p.N / 8;
    Piece<T> a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = min(i * NT + tid, pieces - 1);   // past the end: the last piece again, left out below
        a[i].load(x + c * 8);
        if (p.residual) b[i].load(r + c * 8);
    }
    float s[V][8], sum = 0.f;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * NT + tid;
        a[i].get(s[i]);
        if (p.residual) {
            float f[8];
            b[i].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = rounded<T>(s[i][e] + f[e]);
            if (p.sum && c < pieces) {
                a[i].set(s[i]);
                a[i].store(static_cast<T*>(p.sum) + t * p.s_rs + c * 8);
            }
        }
        float g[8];
        if (p.gain) load8(p.gain + min(c, pieces - 1) * 8, g);
        if (c < pieces) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum = fmaf(s[i][e], s[i][e], sum);
                m = max(m, __float_as_uint(p.gain ? s[i][e] * g[e] : s[i][e]) & 0x7FFFFFFFu);
            }
        }
    }
    const RowStats st = team.stats(sum, m);
    RowScales k;
    bool wide = !in_range(st, p.N), bad = false;
    if (!wide) {
        finish<NT>(p, st, k);
        if (p.codes && p.gain) {
            int lo = INT32_MIN;
            if (m == st.m) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = i * NT + tid;
                    if (c >= pieces) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) lo = remainder_at(s[i][e], p.gain[c * 8 + e], st.m, lo);
                }
            }
            k.lo = team.largest(m == st.m, lo);
        }
    } else {
        double ss = 0.0, top = 0.0;
        for (int i = 0; i < V; ++i) {
            const int c = i * NT + tid;
            if (c >= pieces) continue;
            for (int e = 0; e < 8; ++e) {
                ss += (double)s[i][e] * s[i][e];
                top = larger(top, fabs(product(s[i][e], p.gain ? p.gain[c * 8 + e] : 1.f)));
            }
        }
        team.in_64(ss, top);
        const double inv = p.norm ? 1.0 / sqrt(ss / p.N + (double)p.eps) : 1.0;
        bad = !(top < INFINITY) || !(ss < INFINITY);
        k.top = top;
        k.inv = (float)inv;
        k.scale = bad ? NAN : top > 0.0 ? (float)(top * inv / 127.0) : 0.f;
        if (bad && tid == 0) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
        if (p.y) {
            // the norm may bring back what a product alone would lose
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * NT + tid;
                if (c >= pieces) continue;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = (float)(top > 0.0 || bad ? product(s[i][e], p.gain ? p.gain[c * 8 + e] : 1.f) * inv : 0.0);
                a[i].set(y);
                a[i].store(static_cast<T*>(p.y) + t * p.y_rs + c * 8);
            }
        }
    }
    if (p.codes && tid == 0) p.scale[t] = k.scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * NT + tid;
        if (c >= pieces) continue;
        float g[8];
        if (p.gain) load8(p.gain + c * 8, g);
        if (p.y && !wide) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (p.gain ? s[i][e] * g[e] : s[i][e]) * k.inv;
            a[i].set(y);
            a[i].store(static_cast<T*>(p.y) + t * p.y_rs + c * 8);
        }
        if (p.codes) {
            int q[8];
            if (!wide) {
                // 1.5 * 2^23 added: the sum's low bits are the nearest whole number
                float f[8], off = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] = (p.gain ? s[i][e] * g[e] : s[i][e]) * k.per;
                    const float n = f[e] + 12582912.f;
                    q[e] = __float_as_int(n);
                    off = fmaxf(off, fabsf(f[e] - (n - 12582912.f)));
                }
                if (off > kNearHalf) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (fabsf(f[e] - ((f[e] + 12582912.f) - 12582912.f)) > kNearHalf)
                            q[e] = settled(s[i][e], p.gain ? g[e] : 1.f, f[e], k);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = bad || k.top == 0.0 ? 0 : code_in_64(s[i][e], p.gain ? g[e] : 1.f, k.top);
            }
            uint2 w;
            w.x = (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | q[3] << 24;
            w.y = (q[4] & 255) | (q[5] & 255) << 8 | (q[6] & 255) << 16 | q[7] << 24;
            *reinterpret_cast<uint2*>(p.codes + t * p.c_rs + c * 8) = w;
        }
    }
}

// Any width up to kNormMaxN, any alignment: the row of s in shared memory.
constexpr int kAnyThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(NormParams p)
{
    constexpr int NT = kAnyThreads, kWarps = NT / 32;
    extern __shared__ float row[];
    __shared__ float s_sums[kWarps];
    __shared__ uint32_t s_tops[kWarps];
    __shared__ int s_lo;
    __shared__ double s_wide[2 * kWarps];
    const Team<NT> team{s_sums, s_tops, &s_lo, s_wide};
    pdl_enter();
    const int t = blockIdx.x, tid = threadIdx.x;
    if (t >= live_rows(p.n_rows, p.T, p.status, t == 0 && tid == 0)) return;
    const T* x = static_cast<const T*>(p.x) + t * p.x_rs;
    const T* r = static_cast<const T*>(p.residual) + t * p.r_rs;
    auto gain = [&](int c) { return p.gain ? __ldg(p.gain + c) : 1.f; };
    float sum = 0.f;
    uint32_t m = 0u;
#pragma unroll 4
    for (int c = tid; c < p.N; c += NT) {
        float s = to_f32<T>(x[c]);
        if (p.residual) {
            s = rounded<T>(s + to_f32<T>(r[c]));
            if (p.sum) static_cast<T*>(p.sum)[t * p.s_rs + c] = narrowed<T>(s);
        }
        row[c] = s;                       // read again by this thread only
        sum = fmaf(s, s, sum);
        m = max(m, __float_as_uint(s * gain(c)) & 0x7FFFFFFFu);
    }
    const RowStats st = team.stats(sum, m);
    RowScales k;
    bool wide = !in_range(st, p.N), bad = false;
    if (!wide) {
        finish<NT>(p, st, k);
        if (p.codes && p.gain) {
            int lo = INT32_MIN;
            if (m == st.m)
                for (int c = tid; c < p.N; c += NT) lo = remainder_at(row[c], gain(c), st.m, lo);
            k.lo = team.largest(m == st.m, lo);
        }
        for (int c = tid; c < p.N; c += NT) {
            const float g = gain(c), h = row[c] * g;
            if (p.y) static_cast<T*>(p.y)[t * p.y_rs + c] = narrowed<T>(h * k.inv);
            if (p.codes) {
                const float f = h * k.per, n = rintf(f);
                p.codes[t * p.c_rs + c] = (int8_t)(fabsf(f - n) > kNearHalf ? settled(row[c], g, f, k) : (int)n);
            }
        }
    } else {
        double ss = 0.0, top = 0.0;
        for (int c = tid; c < p.N; c += NT) {
            ss += (double)row[c] * row[c];
            top = larger(top, fabs(product(row[c], gain(c))));
        }
        team.in_64(ss, top);
        const double inv = p.norm ? 1.0 / sqrt(ss / p.N + (double)p.eps) : 1.0;
        bad = !(top < INFINITY) || !(ss < INFINITY);
        k.scale = bad ? NAN : top > 0.0 ? (float)(top * inv / 127.0) : 0.f;
        if (bad && tid == 0) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
        for (int c = tid; c < p.N; c += NT) {
            if (p.y)
                static_cast<T*>(p.y)[t * p.y_rs + c] =
                    narrowed<T>((float)(top > 0.0 || bad ? product(row[c], gain(c)) * inv : 0.0));
            if (p.codes) p.codes[t * p.c_rs + c] = (int8_t)(bad || top == 0.0 ? 0 : code_in_64(row[c], gain(c), top));
        }
    }
    if (p.codes && tid == 0) p.scale[t] = k.scale;
}

bool on(const void* p, int64_t stride_bytes, size_t bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride_bytes % (int64_t)bytes == 0;
}

bool vec_rows(const NormParams& p)
{
    const int64_t size = p.dtype == DSPARK_BF16 ? 2 : 4;
    return p.N % 8 == 0 && on(p.x, p.x_rs * size, 16) && (!p.residual || on(p.residual, p.r_rs * size, 16)) &&
           (!p.sum || on(p.sum, p.s_rs * size, 16)) && (!p.y || on(p.y, p.y_rs * size, 16)) &&
           (!p.codes || on(p.codes, p.c_rs, 8)) && on(p.gain, 0, 16);
}

// kFrom .. kTo: the pieces a thread that the widths left to NT threads need
template <typename T, int NT, int kFrom, int kTo>
cudaError_t launch_vec(const NormParams& p, cudaStream_t s)
{
    if constexpr (kFrom < kTo)
        if (cdiv(p.N / 8, NT) > kFrom) return launch_vec<T, NT, kFrom + 1, kTo>(p, s);
    constexpr int kRows = NT == 32 ? 8 : 1;
    return launch_pdl(norm_vec_kernel<T, NT, kFrom>, dim3(cdiv(p.T, kRows)), dim3(NT == 32 ? 256 : NT), 0, s, p);
}

template <typename T>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s)
{
    if (vec_rows(p)) {
        // a warp while a row fits one; wider ones two pieces a thread, or three where two would idle many threads
        if (p.N <= 1024) return launch_vec<T, 32, 1, 4>(p, s);
        if (p.N <= 2048) return launch_vec<T, 128, 2, 2>(p, s);
        if (p.N <= 6144) return launch_vec<T, 256, 2, 3>(p, s);
        if (p.N <= 12288) return launch_vec<T, 512, 2, 3>(p, s);
        return launch_vec<T, 1024, 2, 4>(p, s);
    }
    static std::atomic<uint64_t> admitted{0};
    const cudaError_t e = admit_smem(norm_any_kernel<T>, kNormMaxN * sizeof(float), admitted);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_any_kernel<T>, dim3(p.T), dim3(kAnyThreads), p.N * sizeof(float), s, p);
}

}  // namespace

cudaError_t launch_add_norm_quant(const NormParams& p, cudaStream_t s)
{
    const cudaError_t e = p.dtype == DSPARK_BF16 ? launch_norm<__nv_bfloat16>(p, s) : launch_norm<float>(p, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
