// qk_norm_rope.cu -- norms of the queries and keys by head and their rotation by position, one pass
// over the rows (dspark_qk_norm_rope).
//
//   y = x / sqrt(sum x^2 / D + eps) * gain;  pair i turns by phi_i = 2 pi frac(freq[i] position).
//
// The turn per position is a 64-bit fraction, so freq * position modulo 2^64 is the exact fraction of
// a turn: no angle is ever large, and sincospif sees arguments in [-1, 1). A CTA takes one token: the
// sines and cosines of its rot / 2 pairs are formed once and serve every head of q and k.
#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 1024;

// cos and sin of pair i at `pos`
__device__ __forceinline__ float2 turn(uint64_t freq, long long pos)
{
    const uint64_t f = freq * (uint64_t)pos;               // fraction of a turn, units of 2^-64
    const float half_turns = (float)(int32_t)(f >> 32) * 0x1.0p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c, s);
}

// The absolute position of token t; false for padding
__device__ __forceinline__ bool token_position(const RopeParams& p, int t, long long& pos)
{
    pos = p.position[t];
    if (p.request) {
        const int r = p.request[t];
        if (r < 0) return false;
        if (r >= p.R) {
            raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
            return false;
        }
        if (p.ctx_len) pos += p.ctx_len[r];
    }
    return true;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Any even D up to 1024, any strides and alignment: one warp per head, the head's row in registers
// one element per lane and step, read again for the pair's other element.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(RopeParams p)
{
    pdl_enter();
    __shared__ float2 s_cs[kRopeMaxD / 2];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long pos = 0;
    const bool live = token_position(p, t, pos);
    const int half = p.rot / 2;
    if (live)
        for (int i = threadIdx.x; i < half; i += kRopeThreads) s_cs[i] = turn(p.freq[i], pos);
    __syncthreads();
    for (int hh = warp; hh < p.Hq + p.Hkv; hh += kRopeThreads / 32) {
        const bool is_q = hh < p.Hq;
        const int h = is_q ? hh : hh - p.Hq;
        const T* x = is_q ? static_cast<const T*>(p.q) + t * p.q_ts + h * p.q_hs
                          : static_cast<const T*>(p.k) + t * p.k_ts + h * p.k_hs;
        T* y = is_q ? static_cast<T*>(p.q_out) + ((size_t)t * p.Hq + h) * p.D
                    : static_cast<T*>(p.k_out) + ((size_t)t * p.Hkv + h) * p.D;
        const float* gain = is_q ? p.q_gain : p.k_gain;
        if (!live) {
            for (int c = lane; c < p.D; c += 32) y[c] = from_f32<T>(0.f);
            continue;
        }
        float inv = 1.f;
        if (p.norm) {
            float sum = 0.f;
            for (int c = lane; c < p.D; c += 32) {
                const float v = to_f32<T>(x[c]);
                sum = fmaf(v, v, sum);
            }
            inv = 1.f / sqrtf(warp_sum(sum) / (float)p.D + p.eps);
        }
        auto value = [&](int c) { return to_f32<T>(x[c]) * inv * (gain ? gain[c] : 1.f); };
        for (int i = lane; i < half; i += 32) {
            const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? 2 * i + 1 : i + half;
            const float ya = value(a), yb = value(b);
            const float2 cs = s_cs[i];
            y[a] = from_f32<T>(ya * cs.x - yb * cs.y);
            y[b] = from_f32<T>(ya * cs.y + yb * cs.x);
        }
        for (int c = p.rot + lane; c < p.D; c += 32) y[c] = from_f32<T>(value(c));
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t s)
{
    const cudaError_t e = p.dtype == DSPARK_BF16
                              ? launch_pdl(rope_any_kernel<__nv_bfloat16>, dim3(p.T), dim3(kRopeThreads), 0, s, p)
                              : launch_pdl(rope_any_kernel<float>, dim3(p.T), dim3(kRopeThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
