// cache_attend.cu -- attention of the flat verify batch over the 4-bit cache (dspark_cache_attend):
// the CUDA-core kernel, fp32 throughout, for every head width.
//
//   z_i = scale q . k_i over the visible keys i, out = sum exp(z_i) v_i / sum exp(z_i)
//
// in one pass over the keys: each warp keeps a running maximum m (in log2 units), the sum l of
// 2^(z - m) and the weighted sum o, and rescales l and o when m grows; the warps' states join at the
// end. A CTA takes one flat row and one key / value head: its G query heads, four at a time, share
// each key's codes. A warp takes 32 keys at a time: a lane forms the products of one key, then the
// lanes share the channels of the value rows.
//
// Instructions bound it (2 D fp32 products a row and key, and the codes turned again for every four heads of a query):
// 1.1 ms for 128 single rows of 32 heads over up to 4096 tokens (0.05 ms of bytes), 6.7 ms for 17 rows a request. It
// serves the head widths that the matrix kernels do not, and is what they are checked against.
#include "attend_plan.cuh"
#include "cache.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kWarps = 8;
constexpr int kRows = 4;      // query heads that share a pass over the keys
constexpr int kMaxE = 8;      // channels of a value row a lane holds (D <= 256)

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) cache_attend_simt_kernel(AttendParams p)
{
    pdl_enter();
    __shared__ float s_q[kRows][256];
    __shared__ float s_o[kWarps][kRows][256];
    __shared__ float2 s_ml[kWarps][kRows];
    __shared__ int s_bad[kRows];
    const int D = p.c.D, groups = D / kCacheGroup, P = p.c.page_size;
    const int t = blockIdx.x, kvh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CacheBlock cb = cache_block(P, D);
    // the request of row t: the last r with offsets[r] <= t
    int lo = 0, hi = p.c.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int r = lo, first = p.offsets[r], last = p.offsets[r + 1];
    const int ctx = p.c.ctx_len[r];
    bool live = t >= first && t < last && first >= 0;
    if (live && (last > p.T || last - first > p.max_q || ctx < 0)) {
        raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        live = ctx >= 0 && t - first < p.max_q;
    }
    if (t == 0 && kvh == 0)   // decreasing offsets: once a call
        for (int i = threadIdx.x; i < p.c.R; i += kWarps * 32)
            if (p.offsets[i + 1] < p.offsets[i] || p.offsets[i] < 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    const long long here = live ? (long long)ctx + (t - first) : -1;   // this row's position
    const long long cap = (long long)p.c.table_width * P;
    if (here >= cap) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    const int n_keys = (int)min(here + 1, cap);
    // the keys from `from` on and those below the sinks
    const int from = p.window > 0 ? (int)max(0ll, min(here - p.window + 1, cap)) : 0;
    const int sinks = p.window > 0 ? min(p.sinks, from) : 0;
    const int span = live ? sinks + max(0, n_keys - from) : 0;   // key u: u for u < sinks, else from + u - sinks
    for (int g0 = 0; g0 < p.G; g0 += kRows) {
        const int rows = min(kRows, p.G - g0);
        __syncthreads();
        if (threadIdx.x < kRows) s_bad[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * D; i += kWarps * 32) {
            const int row = i / D, c = i % D;
            float x = 0.f;
            if (live && row < rows)
                x = to_f32<T>(static_cast<const T*>(p.q)[t * p.q_ts + (int64_t)(kvh * p.G + g0 + row) * p.q_hs + c]);
            if (!(fabsf(x) <= FLT_MAX)) s_bad[row] = 1;
            s_q[row][c] = x * (p.scale * kLog2e);
        }
        __syncthreads();
        float m[kRows], l[kRows], o[kRows][kMaxE];
#pragma unroll
        for (int row = 0; row < kRows; ++row) {
            m[row] = -INFINITY;
            l[row] = 0.f;
#pragma unroll
            for (int e = 0; e < kMaxE; ++e) o[row][e] = 0.f;
        }
        for (uint32_t u0 = warp * 32; u0 < (uint32_t)span; u0 += kWarps * 32) {   // may pass what an int holds
            // products of key u0 + lane
            const uint32_t u = u0 + lane;
            const uint8_t* blk = nullptr;
            int slot = 0;
            if (u < (uint32_t)span) {
                const int key = (int)u < sinks ? (int)u : from + (int)u - sinks;
                const int page = p.c.table[(size_t)r * p.c.table_width + key / P];
                slot = key % P;
                if (page >= 0 && page < p.c.n_pages) blk = cache_page_block(p.c, page, kvh, cb.bytes);
                else raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
            }
            float z[kRows];
#pragma unroll
            for (int row = 0; row < kRows; ++row) z[row] = blk ? 0.f : -INFINITY;
            if (blk) {
                const uint32_t* words = reinterpret_cast<const uint32_t*>(blk + (uint32_t)slot * (D / 2));
                const __half* scales = reinterpret_cast<const __half*>(blk + cb.k_scales) + slot * groups;
                for (int g = 0; g < groups; ++g) {
                    float part[kRows] = {};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t word = words[g * 4 + w];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float k = (float)((int)((word >> (4 * j)) & 15u) - 8);
#pragma unroll
                            for (int row = 0; row < kRows; ++row)
                                part[row] = fmaf(s_q[row][g * 32 + w * 8 + j], k, part[row]);
                        }
                    }
                    const float s = __half2float(scales[g]);
#pragma unroll
                    for (int row = 0; row < kRows; ++row) z[row] = fmaf(part[row], s, z[row]);
                }
            }
            float w[kRows];
#pragma unroll
            for (int row = 0; row < kRows; ++row) {
                const float top = fmaxf(m[row], warp_max(z[row]));
                const float base = top == -INFINITY ? 0.f : top;   // no key so far: the weights stay 0
                const float keep = exp2f(m[row] - base);
                w[row] = exp2f(z[row] - base);
                l[row] = l[row] * keep + w[row];
                m[row] = top;
#pragma unroll
                for (int e = 0; e < kMaxE; ++e) o[row][e] *= keep;
            }
            // value rows: lane holds channels e * 32 + lane, group e
            const unsigned seen = __ballot_sync(0xffffffffu, blk != nullptr);
            for (int v = 0; v < 32; ++v) {
                if (!((seen >> v) & 1u)) continue;
                const uint8_t* b = reinterpret_cast<const uint8_t*>(
                    __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(blk), v));
                const int sl = __shfl_sync(0xffffffffu, slot, v);
                float wv[kRows];
#pragma unroll
                for (int row = 0; row < kRows; ++row) wv[row] = __shfl_sync(0xffffffffu, w[row], v);
#pragma unroll
                for (int e = 0; e < kMaxE; ++e) {
                    if (e < groups) {
                        const uint32_t byte = b[cb.v_codes + (uint32_t)sl * (D / 2) + e * 16 + lane / 2];
                        const float s = __half2float(
                            *reinterpret_cast<const __half*>(b + cb.v_scales + v_scale_at(sl, e, groups)));
                        const float x = (float)((int)((byte >> (4 * (lane & 1))) & 15u) - 8) * s;
#pragma unroll
                        for (int row = 0; row < kRows; ++row) o[row][e] = fmaf(wv[row], x, o[row][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int row = 0; row < kRows; ++row) {
            const float sum = warp_sum(l[row]);
            if (lane == 0) s_ml[warp][row] = make_float2(m[row], sum);
#pragma unroll
            for (int e = 0; e < kMaxE; ++e)
                if (e < groups) s_o[warp][row][e * 32 + lane] = o[row][e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
            const int row = i / D, c = i % D;
            float top = -INFINITY;
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
            float sum = 0.f, acc = 0.f;
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_ml[w][row].x == -INFINITY ? 0.f : exp2f(s_ml[w][row].x - top);
                sum = fmaf(f, s_ml[w][row].y, sum);
                acc = fmaf(f, s_o[w][row][c], acc);
            }
            const bool none = top == -INFINITY;
            const float bad = s_bad[row] ? NAN : 0.f;
            const size_t at = (size_t)t * p.Hq + kvh * p.G + g0 + row;
            store1(static_cast<T*>(p.out) + at * D + c, (none ? 0.f : acc / sum) + bad);
            if (c == 0 && p.lse) p.lse[at] = (none ? -INFINITY : (top + log2f(sum)) * kLn2) + bad;
            if (c == 0 && s_bad[row]) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
        }
    }
}

}  // namespace

cudaError_t launch_cache_attend_simt(const AttendParams& p, cudaStream_t s)
{
    const dim3 grid(p.T, p.c.Hkv), block(kWarps * 32);
    const cudaError_t e = p.dtype == DSPARK_BF16
                              ? launch_pdl(cache_attend_simt_kernel<__nv_bfloat16>, grid, block, 0, s, p)
                              : launch_pdl(cache_attend_simt_kernel<float>, grid, block, 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
