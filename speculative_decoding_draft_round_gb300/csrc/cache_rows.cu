// cache_rows.cu -- key and value rows into the 4-bit cache (dspark_cache_append) and back out as
// values (dspark_cache_read). Layout and rounding in dspark.h.
//
// A thread takes 8 channels of a row: one 32-bit word of codes. The 4 threads of a group of 32
// channels find its largest magnitude with two shuffles. Both kernels move each byte once.
//
// Bound: the bytes, 2 us for 2176 tokens of 8 heads of 128 in bf16 and 12.7 us for 16384, but a code costs more than its
// two bytes: 7.3 and 37 us for the append (65 us while its indices took divisions and a border's codes a loop), 4.9 and
// 22 us for reading back. 50000 tokens of 4 heads of 64 in fp32: 31 and 31 us of 34 for both.
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

// The 8 codes of v in a word: v / s rounded to the nearest integer, ties to even, in -7 .. 7 (s > 0), plus 8.
//
// Adding 1.5 2^23 + 8 rounds v / s to an integer, whose 4 bits are then the number's lowest. The
// product with about 1 / s may fall on the wrong side of a border. The remainder x - c s is one rounding of an exact
// difference, so one that is not below s / 2 shows that, or a tie: these rare pieces (a tie needs few bits in v) are
// looked at again.
constexpr float kRound = 12582912.f + 8.f;

// v may pass 7 s by less than half a step, unless the scale is one that fp16 holds badly: the caller holds it to 7 s then.
__device__ __forceinline__ uint32_t code_word(const float (&v)[kVec], float s)
{
    const float inv = __fdividef(1.f, s), h = 0.5f * s;
    uint32_t word = 0;
    bool settle = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float t = fmaf(v[j], inv, kRound);
        settle |= fabsf(fmaf(kRound - t, s, v[j])) >= h;
        word |= (__float_as_uint(t) & 15u) << (4 * j);
    }
    if (settle) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const uint32_t code = (word >> (4 * j)) & 15u;
            const float r = fmaf(8.f - (float)code, s, v[j]), off = fabsf(r);
            if (off > h || (off == h && (code & 1u))) word += (r > 0.f ? 1u : ~0u) << (4 * j);
        }
    }
    return word;
}

// A CTA takes `tokens` consecutive tokens. Their pages and slots are looked up once, then thread after thread
// takes a piece of 8 channels: piece = ((token * 2 + (0 = K, 1 = V)) * Hkv + head) * (D / 8) + vec, so that a
// warp's threads read consecutive channels and the 4 threads of a group are 4 aligned lanes.
constexpr int kMaxTokens = 64;

struct RowAt {
    int t, half, h, vec;
};

// Quotients by a multiplication: magic = ceil(2^32 / d), off by less than d in the product, is exact while the number
// times d stays below 2^32. Pieces of a CTA: fewer than 8 kRowsThreads, or those of one token.
struct RowMagic {
    uint32_t each, vecs;
};

__device__ __forceinline__ RowAt row_at(uint32_t i, uint32_t each, int Hkv, uint32_t vecs, RowMagic magic)
{
    RowAt a;
    a.t = (int)__umulhi(i, magic.each);
    const uint32_t in = i - a.t * each;
    const int row = (int)__umulhi(in, magic.vecs);
    a.vec = (int)(in - row * vecs);
    a.half = row >= Hkv;
    a.h = row - a.half * Hkv;
    return a;
}

__device__ __forceinline__ void look_up(const CacheRowsParams& p, int first, int count, int2* s_at)
{
    if ((int)threadIdx.x < count) {
        int page = -1, slot = 0;
        const int t = first + threadIdx.x;
        if (!cache_slot(p.c, p.request[t], p.position[t], p.status, page, slot)) page = -1;
        s_at[threadIdx.x] = make_int2(page, slot);
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) cache_append_kernel(CacheRowsParams p, int aligned, int tokens, RowMagic magic)
{
    pdl_enter();
    __shared__ int2 s_at[kMaxTokens];
    const uint32_t vecs = p.c.D / kVec, groups = p.c.D / kCacheGroup, each = 2 * p.c.Hkv * vecs;
    const int first = blockIdx.x * tokens, count = min(tokens, p.T - first);
    look_up(p, first, count, s_at);
    const uint32_t n = count * each;   // a multiple of 8: the 4 lanes of a group stay together
    const CacheBlock b = cache_block(p.c.page_size, p.c.D);
    for (uint32_t i = threadIdx.x; i < (n + 31) / 32 * 32; i += kRowsThreads) {
        const RowAt a = row_at(min(i, n - 1), each, p.c.Hkv, vecs, magic);
        const int2 at = s_at[a.t];
        const bool live = i < n && at.x >= 0;
        float x[kVec] = {};
        if (live) {
            const int64_t t = first + a.t;
            const T* src = a.half == 0 ? static_cast<const T*>(p.k) + t * p.k_ts + a.h * p.k_hs
                                       : static_cast<const T*>(p.v) + t * p.v_ts + a.h * p.v_hs;
            load_vec<T>(src + a.vec * kVec, aligned, x);
        }
        uint32_t most = 0;   // magnitudes order like their bits
#pragma unroll
        for (int j = 0; j < kVec; ++j) most = max(most, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        float top = __uint_as_float(most);
        const bool odd_input = most >= 0x7F800000u;
        if (odd_input) {   // an infinity takes the largest code, NaN the code of 0
            top = 0.f;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (fabsf(x[j]) <= FLT_MAX) top = fmaxf(top, fabsf(x[j]));
                else x[j] = x[j] != x[j] ? 0.f : copysignf(FLT_MAX, x[j]);
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (!live) continue;
        if (odd_input) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
        const float s8 = __bfloat162float(__float2bfloat16_rn(top * (1.f / 7.f)));
        const __half sh = __float2half_rn(fminf(s8, kCacheMaxScale));
        const float s = __half2float(sh);
        if (odd_input || s < 0x1p-13f || s >= kCacheMaxScale) {   // few bits of the scale are left, or it is the largest
            const float hold = 7.f * s;
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] = fminf(fmaxf(x[j], -hold), hold);
        }
        const uint32_t word = s > 0.f ? code_word(x, s) : 0x88888888u;   // the code of 0
        uint8_t* blk = cache_page_block(p.c, at.x, a.h, b.bytes);
        const uint32_t codes = a.half == 0 ? 0u : b.v_codes;
        *reinterpret_cast<uint32_t*>(blk + codes + (uint32_t)at.y * (p.c.D / 2) + a.vec * 4) = word;
        if (a.vec % 4 == 0) {
            const int g = a.vec / 4;
            const uint32_t to = a.half == 0 ? b.k_scales + (uint32_t)(at.y * groups + g) * 2u
                                            : b.v_scales + v_scale_at(at.y, g, groups);
            *reinterpret_cast<__half*>(blk + to) = sh;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) cache_read_kernel(CacheRowsParams p, int tokens, RowMagic magic)
{
    pdl_enter();
    __shared__ int2 s_at[kMaxTokens];
    const uint32_t vecs = p.c.D / kVec, groups = p.c.D / kCacheGroup, each = 2 * p.c.Hkv * vecs;
    const int first = blockIdx.x * tokens, count = min(tokens, p.T - first);
    look_up(p, first, count, s_at);
    const uint32_t n = count * each;
    const CacheBlock b = cache_block(p.c.page_size, p.c.D);
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < n; i += kRowsThreads) {
        const RowAt a = row_at(i, each, p.c.Hkv, vecs, magic);
        const int2 at = s_at[a.t];
        float x[kVec] = {};
        if (at.x >= 0) {
            const uint8_t* blk = cache_page_block(p.c, at.x, a.h, b.bytes);
            const int g = a.vec / 4;
            const uint32_t codes = a.half == 0 ? 0u : b.v_codes;
            const uint32_t from = a.half == 0 ? b.k_scales + (uint32_t)(at.y * groups + g) * 2u
                                              : b.v_scales + v_scale_at(at.y, g, groups);
            const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + codes + (uint32_t)at.y * (p.c.D / 2) + a.vec * 4);
            const float s = __half2float(*reinterpret_cast<const __half*>(blk + from));
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] = (float)((int)((word >> (4 * j)) & 15u) - 8) * s;
        }
        T* dst = static_cast<T*>(a.half == 0 ? p.k_out : p.v_out) + ((size_t)(first + a.t) * p.c.Hkv + a.h) * p.c.D + a.vec * kVec;
        store_vec(dst, x);
    }
}

template <typename T>
bool rows_aligned(const CacheRowsParams& p)
{
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v);
    const int64_t strides = p.k_ts | p.k_hs | p.v_ts | p.v_hs;
    return base % 16 == 0 && (strides * (int64_t)sizeof(T)) % 16 == 0;
}

RowMagic rows_magic(const CacheRowsParams& p)
{
    auto of = [](uint64_t d) { return (uint32_t)(((1ull << 32) + d - 1) / d); };
    const int vecs = p.c.D / kVec;
    return RowMagic{of(2ull * p.c.Hkv * vecs), of(vecs)};
}

// Tokens of a CTA: pieces for eight rounds of its threads, fewer where that leaves SMs without work
int rows_tokens(const CacheRowsParams& p)
{
    const int each = 2 * p.c.Hkv * (p.c.D / kVec);
    int tokens = 8 * kRowsThreads / each;
    const long long fair = ((long long)p.T + 8ll * num_sms() - 1) / (8ll * num_sms());
    if (tokens > fair) tokens = (int)fair;
    return tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsParams& p, cudaStream_t s)
{
    const int tokens = rows_tokens(p);
    const RowMagic magic = rows_magic(p);
    const dim3 grid(cdiv(p.T, tokens)), block(kRowsThreads);
    const cudaError_t e =
        p.dtype == DSPARK_BF16
            ? launch_pdl(cache_append_kernel<__nv_bfloat16>, grid, block, 0, s, p, (int)rows_aligned<__nv_bfloat16>(p), tokens, magic)
            : launch_pdl(cache_append_kernel<float>, grid, block, 0, s, p, (int)rows_aligned<float>(p), tokens, magic);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheRowsParams& p, cudaStream_t s)
{
    const int tokens = rows_tokens(p);
    const RowMagic magic = rows_magic(p);
    const dim3 grid(cdiv(p.T, tokens)), block(kRowsThreads);
    const cudaError_t e = p.dtype == DSPARK_BF16 ? launch_pdl(cache_read_kernel<__nv_bfloat16>, grid, block, 0, s, p, tokens, magic)
                                                 : launch_pdl(cache_read_kernel<float>, grid, block, 0, s, p, tokens, magic);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
