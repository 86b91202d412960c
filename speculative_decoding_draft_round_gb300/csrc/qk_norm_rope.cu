// qk_norm_rope.cu -- norms of the queries and keys by head and their rotation by position, one pass
// over the rows (dspark_qk_norm_rope).
//
//   y = x / sqrt(sum x^2 / D + eps) * gain;  pair i turns by phi_i = 2 pi frac(freq[i] position).
//
// The turn per position is a 64-bit fraction, so freq * position modulo 2^64 is the exact fraction of
// a turn: no angle is ever large, and sincospif sees arguments in [-1, 1). The sines and cosines of a
// token's rot / 2 pairs are formed once for many heads.
//
// The bytes bound it: each row read once and written once. rope_vec_kernel keeps 16-byte pieces in registers
// between the norm's sum and the rotation, with several heads' loads in flight; rope_any_kernel takes the
// shapes that the pieces do not fit. The first takes rsqrtf (2 units in the last place: listed fp32 rows are off by
// 7.8e-8 of their size against 64 bits, by 7.0e-8 in plain fp32), the second divides by a root. Measured: 32749 tokens
// of 40 heads of 128 in bf16 (671 MB) 114 us, 99 us at the copy's rate (148 us while a condition around each load made
// it wait for the one before); 2176 such tokens 13 us of 6.6, where the chain position, context, sines, rows is what is
// left; 16384 with half-split pairs 67 us of 49, the shuffles that bring a pair's other half.
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

// ------------------------------------------------------------------ 8 channels a lane
//
// D a multiple of 8 up to 256, rot of 16 (of 2 when interleaved), 16-byte aligned rows: a head is LPH lanes (D / 8
// rounded up to a power of two), a warp takes 32 / LPH heads at a time, kUnroll such loads in flight, and `share` warps
// share a token (one where there are tokens enough: the sines serve all its heads then).
template <typename T>
struct Vec {
    uint32_t u[2 * sizeof(T)];   // 8 elements
};

template <typename T>
__device__ __forceinline__ Vec<T> load_row(const T* p)
{
    Vec<T> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        v.u[4 * i] = x.x;
        v.u[4 * i + 1] = x.y;
        v.u[4 * i + 2] = x.z;
        v.u[4 * i + 3] = x.w;
    }
    return v;
}

// elements 2 i and 2 i + 1
template <typename T>
__device__ __forceinline__ uint64_t pair(const Vec<T>& v, int i)
{
    if (sizeof(T) == 4) return pack2(__uint_as_float(v.u[(2 * i) % (2 * sizeof(T))]), __uint_as_float(v.u[(2 * i + 1) % (2 * sizeof(T))]));
    return pack2(__uint_as_float(v.u[i % 4] << 16), __uint_as_float(v.u[i % 4] & 0xFFFF0000u));
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&y)[8])
{
    uint32_t u[2 * sizeof(T)];
#pragma unroll
    for (int i = 0; i < 8 / (4 / (int)sizeof(T)); ++i) {
        if (sizeof(T) == 4) {
            u[i % (2 * sizeof(T))] = __float_as_uint(y[i]);
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[(2 * i) % 8], y[(2 * i + 1) % 8]);
            u[i % (2 * sizeof(T))] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
}

// 24 warps an SM in CTAs of four: 16384 tokens with half-split pairs 67 us, 80 with the 16 warps that unbounded registers
// leave; in CTAs of eight 69
constexpr int kVecWarps = 4, kVecCtas = 6;

// Which channels pair: half-split, neighbours, and neighbours with a rot that is no multiple of 8, so that a lane holds
// pairs that are turned and pairs that are not. (With that test for all neighbours 32749 tokens took 1 us more.)
enum Pairs { kHalves, kNeighbours, kMixed };

template <typename T, int LPH, Pairs kPairs>
__global__ void __launch_bounds__(kVecWarps * 32, kVecCtas) rope_vec_kernel(RopeParams p, int share)
{
    constexpr bool kInter = kPairs != kHalves;
    constexpr int kHeads = 32 / LPH;                      // heads of a warp's step
    constexpr int kUnroll = sizeof(T) == 4 ? 2 : 4;
    pdl_enter();
    __shared__ float2 s_cs[kVecWarps][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * (kVecWarps / share) + warp / share, part = warp % share;
    if (t >= p.T) return;
    const int l = lane % LPH, sub = lane / LPH, c0 = l * 8;
    const bool on = c0 < p.D;
    // Loads without a condition (lanes and heads past the ends repeat the last), the first under way before the position.
    Vec<T> v[kUnroll];
    auto load = [&](int is_k, int h0) {
        const T* x0 = static_cast<const T*>(is_k ? p.k : p.q) + (int64_t)t * (is_k ? p.k_ts : p.q_ts) + (on ? c0 : p.D - 8);
        const int64_t hs = is_k ? p.k_hs : p.q_hs;
        const int last = (is_k ? p.Hkv : p.Hq) - 1;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) v[k] = load_row<T>(x0 + min(h0 + k * share * kHeads + sub, last) * hs);
    };
    load(0, part * kHeads);
    long long pos = 0;
    if (!token_position(p, t, pos)) {   // padding
        const float zero[8] = {};
        for (int h = part * kHeads + sub; h < p.Hq + p.Hkv; h += share * kHeads)
            if (on)
                store_row<T>(h < p.Hq ? static_cast<T*>(p.q_out) + ((size_t)t * p.Hq + h) * p.D + c0
                                      : static_cast<T*>(p.k_out) + ((size_t)t * p.Hkv + h - p.Hq) * p.D + c0, zero);
        return;
    }
    const int half = p.rot / 2;
    for (int i = lane; i < half; i += 32) s_cs[warp][i] = turn(p.freq[i], pos);
    __syncwarp();
    // what each of the lane's channels takes of itself and of its pair's other channel
    const int step = half / 8;                            // lanes between the channels of a pair
    const bool turned = c0 < p.rot, second = !kInter && l >= step;
    const int mate = kInter || !turned ? lane : lane + (second ? -step : step);
    const int mate_c0 = (mate % LPH) * 8;
    float own[8], other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = c0 + i;
        const float2 cs = c < p.rot ? s_cs[warp][kInter ? c / 2 : c - (second ? half : 0)] : make_float2(1.f, 0.f);
        own[i] = cs.x;
        other[i] = (kInter ? (i & 1) != 0 : second) ? cs.y : -cs.y;
    }
    const float per = 1.f / (float)p.D;
#pragma unroll 1
    for (int is_k = 0; is_k < 2; ++is_k) {
        const int heads = is_k ? p.Hkv : p.Hq;
        T* y0 = static_cast<T*>(is_k ? p.k_out : p.q_out) + (size_t)t * heads * p.D + c0;
        const float* gain = is_k ? p.k_gain : p.q_gain;
        uint64_t a[4], b[4];                              // the factors above times the gains
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u[2], v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 2 * i + e;
                u[e] = own[c] * (gain && on ? gain[c0 + c] : 1.f);
                v[e] = other[c] * (gain && on ? gain[kInter ? c0 + (c ^ 1) : min(mate_c0 + c, p.D - 1)] : 1.f);
            }
            a[i] = pack2(u[0], u[1]);
            b[i] = pack2(v[0], v[1]);
        }
#pragma unroll 1
        for (int h0 = part * kHeads; h0 < heads; h0 += share * kHeads * kUnroll) {
            if (is_k || h0 > part * kHeads) load(is_k, h0);
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int h = h0 + k * share * kHeads + sub;
                uint64_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = pair(v[k], i);
                float inv = 1.f;
                if (p.norm) {
                    uint64_t two = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) two = fma2(x[i], x[i], two);
                    float sum, more;
                    unpack2(two, sum, more);
                    sum = on ? sum + more : 0.f;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    inv = rsqrtf(fmaf(sum, per, p.eps));
                }
                const uint64_t inv2 = pack2(inv, inv);
                Vec<T> w = v[k];
                if (!kInter) {
#pragma unroll
                    for (int i = 0; i < 2 * (int)sizeof(T); ++i) w.u[i] = __shfl_sync(0xffffffffu, v[k].u[i], mate);
                }
                float y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t o;
                    if (kInter) {
                        float lo, hi;
                        unpack2(x[i], lo, hi);
                        o = pack2(hi, lo);
                    } else {
                        o = pair(w, i);
                    }
                    // channels that are not turned leave the others' alone: 0 times an infinity would be NaN
                    uint64_t r = mul2(x[i], a[i]);
                    if (kPairs == kMixed ? c0 + 2 * i < p.rot : turned) r = fma2(o, b[i], r);
                    unpack2(mul2(r, inv2), y[2 * i], y[2 * i + 1]);
                }
                if (on && h < heads) store_row<T>(y0 + (size_t)h * p.D, y);
            }
        }
    }
}

template <typename T>
bool vec_fits(const RopeParams& p)
{
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                           reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out);
    const int64_t strides = p.q_ts | p.q_hs | p.k_ts | p.k_hs;
    return p.D % 8 == 0 && p.D <= 256 && (p.interleaved || p.rot % 16 == 0) && base % 16 == 0 &&
           (strides * (int64_t)sizeof(T)) % 16 == 0;
}

template <typename T, Pairs kPairs>
cudaError_t launch_lanes(const RopeParams& p, cudaStream_t s)
{
    const int lph = p.D <= 32 ? 4 : p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    // Warps that share a token: as many as give each SM some 16 warps, and each warp a head. Each forms the token's sines:
    // 2176 tokens take 13 us with one or two warps a token, 19 with four.
    int share = 1;
    while (share < kVecWarps && (long long)p.T * share < 16ll * num_sms() && share * (32 / lph) < p.Hq) share *= 2;
    const dim3 grid(cdiv(p.T, kVecWarps / share)), block(kVecWarps * 32);
    switch (lph) {
    case 4: return launch_pdl(rope_vec_kernel<T, 4, kPairs>, grid, block, 0, s, p, share);
    case 8: return launch_pdl(rope_vec_kernel<T, 8, kPairs>, grid, block, 0, s, p, share);
    case 16: return launch_pdl(rope_vec_kernel<T, 16, kPairs>, grid, block, 0, s, p, share);
    default: return launch_pdl(rope_vec_kernel<T, 32, kPairs>, grid, block, 0, s, p, share);
    }
}

template <typename T>
cudaError_t launch_vec(const RopeParams& p, cudaStream_t s)
{
    if (!p.interleaved) return launch_lanes<T, kHalves>(p, s);
    return p.rot % 8 == 0 ? launch_lanes<T, kNeighbours>(p, s) : launch_lanes<T, kMixed>(p, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t s)
{
    const bool bf = p.dtype == DSPARK_BF16;
    if (bf ? vec_fits<__nv_bfloat16>(p) : vec_fits<float>(p)) {
        const cudaError_t v = bf ? launch_vec<__nv_bfloat16>(p, s) : launch_vec<float>(p, s);
        return v != cudaSuccess ? v : cudaGetLastError();
    }
    const cudaError_t e = bf
                              ? launch_pdl(rope_any_kernel<__nv_bfloat16>, dim3(p.T), dim3(kRopeThreads), 0, s, p)
                              : launch_pdl(rope_any_kernel<float>, dim3(p.T), dim3(kRopeThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
