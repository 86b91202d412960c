// cache.cuh -- the paged cache of 4-bit keys and values (layout in dspark.h): where a token's rows
// are, and how codes become values.
#pragma once

#include <cuda_fp16.h>
#include <float.h>

#include "common.cuh"

namespace dspark {

constexpr int kCacheGroup = 32;            // channels that share a scale
constexpr int kScaleTokens = 16;           // tokens of one run of V scales
constexpr float kCacheMaxScale = 9344.f;   // 8 significant bits, and 7 * 9344 is finite in fp16

// byte offsets of the parts of one head's block of n tokens
struct CacheBlock {
    uint32_t v_codes, k_scales, v_scales, bytes;
};

__host__ __device__ inline CacheBlock cache_block(int n, int D)
{
    const uint32_t codes = (uint32_t)n * (D / 2), scales = (uint32_t)n * (D / 16);
    return CacheBlock{codes, 2 * codes, 2 * codes + scales, 2 * (codes + scales)};
}

// byte offset, inside the V scales, of token `slot`'s scale of group g
__device__ __forceinline__ uint32_t v_scale_at(int slot, int g, int groups)
{
    return (uint32_t)(((slot / kScaleTokens) * groups + g) * kScaleTokens + slot % kScaleTokens) * 2u;
}

// Pages a multiple of 16 tokens: the page of token `at` is (at / 16) / (page / 16), with the quotient by a
// multiplication: magic = ceil(2^32 / (page / 16)), 0 for pages of 16. Exact below 2^31 tokens (the error of
// the magic number, below page / 16 <= 16, times at / 16 < 2^27 stays below 2^32).
inline int page_magic(int page_size)
{
    const unsigned d = (unsigned)page_size / 16;
    return d == 1 ? 0 : (int)(unsigned)(((1ull << 32) + d - 1) / d);
}

__device__ __forceinline__ int page_of(int at, int magic)
{
    const uint32_t n = (uint32_t)at >> 4;
    return (int)(magic == 0 ? n : __umulhi(n, (uint32_t)magic));
}

// The block of head h in `page`
__device__ __forceinline__ uint8_t* cache_page_block(const dspark_cache& c, int page, int h, uint32_t block_bytes)
{
    return static_cast<uint8_t*>(c.pages) + ((size_t)page * c.Hkv + h) * block_bytes;
}

// The page and slot of a flat token; false for padding (request < 0) and, recorded, for what is out
// of range.
__device__ __forceinline__ bool cache_slot(const dspark_cache& c, int request, int position, int* status, int& page,
                                           int& slot)
{
    if (request < 0) return false;
    bool ok = request < c.R;
    int at = 0;
    if (ok) {
        const int ctx = c.ctx_len[request];
        // table_width * page_size is below 2^31 (checked on the host)
        ok = ctx >= 0 && position >= 0 && (long long)ctx + position < (long long)c.table_width * c.page_size;
        if (ok) at = ctx + position;
    }
    if (ok) {
        page = c.table[(size_t)request * c.table_width + at / c.page_size];
        slot = at % c.page_size;
        ok = page >= 0 && page < c.n_pages;
    }
    if (!ok) raise_status(status, DSPARK_ERR_DEVICE_INPUT);
    return ok;
}

}  // namespace dspark
