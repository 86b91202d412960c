// logits.cu -- penalties for tokens seen, biases and grammar masks on rows of logits (dspark_adjust_logits), and the
// table of what each request has seen (dspark_seen_add).
//
// A request's rows share its row of the table and its biases: a CTA takes stretches of the vocabulary of one request, lists
// the ids of a stretch that something bears on, runs the rows past as they are, and goes through the list afterwards, a
// thread an id and row. (Adjusted in the threads that load them, those ids held up whole warps: 128 x 17 x 151936 in bf16
// took 236 us, 167 to 177 now, of 111 at the copy's rate; 28 warps an SM wait for loads. In place it takes 157 us: the time is
// less the rows' than that of the CTAs with long lists, for text's ids crowd at the vocabulary's low end.) In place, only 16-byte pieces that a
// mask changes and listed ids are written, and pieces that a mask hides whole are written without being read.
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

// ------------------------------------------------------------------ the table

constexpr int kSeenThreads = 256;
constexpr int kSeenStretch = 8192;       // ids whose new counts a CTA holds: 32 KB
constexpr int kSeenMarks = 32768;        // ids whose marks it holds, a bit each: 4 KB (with stretches of 8192 the
                                         // prompts below took 20 us, each one's pass over the tokens most of it)

__device__ __forceinline__ int seen_tokens(const SeenParams& p, int r, bool report)
{
    if (!p.n) return p.W;
    const int n = p.n[r];
    if (n >= 0 && n <= p.W) return n;
    if (report) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    return n < 0 ? 0 : p.W;
}

// one more token, at most 32767 counted
__device__ __forceinline__ void count_one(int16_t* at)
{
    unsigned short* w = reinterpret_cast<unsigned short*>(at);
    unsigned short old = *reinterpret_cast<volatile unsigned short*>(w);
    while ((old & 0x7FFF) != 0x7FFF) {   // a try fails only where another token got through
        const unsigned short was = atomicCAS(w, old, (unsigned short)(old + 1));
        if (was == old) return;
        old = was;
    }
}

__device__ __forceinline__ void mark_one(int16_t* at)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    atomicOr(reinterpret_cast<unsigned*>(a & ~uintptr_t(3)), a & 2 ? 0x80000000u : 0x8000u);
}

// grid (stretches of the vocabulary, requests). 128 fresh rows of 151936 with prompts of up to 4096 tokens take 8 us, the 39 MB
// 6 of them. A fresh row is written whole, each CTA the stretch whose tokens it has
// counted in shared memory; otherwise the CTAs of a request share its tokens, and each goes into the row by an atomic.
__global__ void __launch_bounds__(kSeenThreads) seen_add_kernel(SeenParams p)
{
    __shared__ int s_new[kSeenStretch];
    pdl_enter();
    const int r = blockIdx.y, tid = threadIdx.x;
    const int n = seen_tokens(p, r, blockIdx.x == 0 && tid == 0);
    const int32_t* tokens = p.tokens + r * p.tokens_rs;
    int16_t* row = p.seen + r * p.seen_rs;
    const int all = n + (p.extra ? 1 : 0);
    auto token = [&](int i) { return i < n ? tokens[i] : p.extra[r]; };
    if (!p.fresh || !p.fresh[r]) {
        for (int i = blockIdx.x * kSeenThreads + tid; i < all; i += gridDim.x * kSeenThreads) {
            const int v = token(i);
            if (v < 0 || v >= p.V) {
                raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
                continue;
            }
            if (p.prompt) mark_one(row + v);
            else count_one(row + v);
        }
        return;
    }
    const int stretch = p.prompt ? kSeenMarks : kSeenStretch, v0 = blockIdx.x * stretch;
    for (int i = tid; i < (p.prompt ? kSeenMarks / 32 : kSeenStretch); i += kSeenThreads) s_new[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < all; i += kSeenThreads) {
        const int v = token(i), d = v - v0;
        if ((unsigned)d < (unsigned)stretch && v < p.V) {
            if (p.prompt) atomicOr(&s_new[d >> 5], 1 << (d & 31));
            else atomicAdd(&s_new[d], 1);
        } else if (blockIdx.x == 0 && (unsigned)v >= (unsigned)p.V) {
            raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        }
    }
    __syncthreads();
    const int words = min(stretch, ((p.V + 7) & ~7) - v0);   // a row's own words: what lies behind them is another's
    for (int i = tid * 8; i < words; i += kSeenThreads * 8) {
        uint32_t w[4];
        const uint32_t marks = p.prompt ? (uint32_t)s_new[i >> 5] >> (i & 31) : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (p.prompt)
                w[j] = ((marks >> (2 * j)) & 1u) << 15 | ((marks >> (2 * j + 1)) & 1u) << 31;
            else
                w[j] = (uint32_t)min(s_new[i + 2 * j], 32767) | (uint32_t)min(s_new[i + 2 * j + 1], 32767) << 16;
        }
        *reinterpret_cast<uint4*>(row + v0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ the logits

constexpr int kAdjThreads = 256;
constexpr int kAdjEach = 8;                              // ids a thread
constexpr int kAdjStretch = kAdjThreads * kAdjEach;      // ids a CTA
constexpr int kAdjRows = 4;                              // rows whose loads are in flight together
constexpr int kAdjMaxS = DSPARK_MAX_GAMMA + 1;

template <typename T>
struct Logits8 {
    uint32_t u[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ float logit(const Logits8<T>& x, int e);
template <>
__device__ __forceinline__ float logit<float>(const Logits8<float>& x, int e) { return __uint_as_float(x.u[e]); }
template <>
__device__ __forceinline__ float logit<__nv_bfloat16>(const Logits8<__nv_bfloat16>& x, int e)
{
    return __uint_as_float(e & 1 ? x.u[e / 2] & 0xFFFF0000u : x.u[e / 2] << 16);
}
template <typename T>
__device__ __forceinline__ void set_logit(Logits8<T>& x, int e, float z);
template <>
__device__ __forceinline__ void set_logit<float>(Logits8<float>& x, int e, float z) { x.u[e] = __float_as_uint(z); }
template <>
__device__ __forceinline__ void set_logit<__nv_bfloat16>(Logits8<__nv_bfloat16>& x, int e, float z)
{
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(z));
    x.u[e / 2] = e & 1 ? (x.u[e / 2] & 0xFFFFu) | h << 16 : (x.u[e / 2] & 0xFFFF0000u) | h;
}

// kVec: a thread's ids are 8 neighbours, loaded 16 bytes at a time; else every 256th, one at a time.
template <typename T, bool kVec>
__device__ __forceinline__ int id_of(int v0, int e)
{
    return kVec ? v0 + threadIdx.x * kAdjEach + e : v0 + e * kAdjThreads + threadIdx.x;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load_logits(Logits8<T>& x, const T* row, int v0, int V)
{
    if constexpr (kVec) {
        const uint4* src = reinterpret_cast<const uint4*>(row + v0 + threadIdx.x * kAdjEach);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 q = src[i];
            x.u[4 * i] = q.x;
            x.u[4 * i + 1] = q.y;
            x.u[4 * i + 2] = q.z;
            x.u[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kAdjEach; ++e) {
            const int v = id_of<T, kVec>(v0, e);
            set_logit<T>(x, e, v < V ? to_f32<T>(row[v]) : 0.f);
        }
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_logits(const Logits8<T>& x, T* row, int v0, int V)
{
    if constexpr (kVec) {
        uint4* dst = reinterpret_cast<uint4*>(row + v0 + threadIdx.x * kAdjEach);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            dst[i] = make_uint4(x.u[4 * i], x.u[4 * i + 1], x.u[4 * i + 2], x.u[4 * i + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < kAdjEach; ++e) {
            const int v = id_of<T, kVec>(v0, e);
            if (v >= V) continue;
            if constexpr (sizeof(T) == 4) row[v] = __uint_as_float(x.u[e]);
            else row[v] = __ushort_as_bfloat16((unsigned short)(x.u[e / 2] >> (16 * (e & 1))));
        }
    }
}

// -infinity where the bit is 0
template <typename T>
__device__ __forceinline__ void hide(Logits8<T>& x, unsigned allowed);
template <>
__device__ __forceinline__ void hide<float>(Logits8<float>& x, unsigned allowed)
{
#pragma unroll
    for (int e = 0; e < kAdjEach; ++e)
        if (!((allowed >> e) & 1u)) x.u[e] = 0xFF800000u;
}
template <>
__device__ __forceinline__ void hide<__nv_bfloat16>(Logits8<__nv_bfloat16>& x, unsigned allowed)
{
#pragma unroll
    for (int i = 0; i < kAdjEach / 2; ++i) {
        const uint32_t keep = ((allowed >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((allowed >> (2 * i)) & 2u ? 0xFFFF0000u : 0u);
        x.u[i] = (x.u[i] & keep) | (0xFF80FF80u & ~keep);
    }
}

template <typename T>
__device__ __forceinline__ T narrowed(float x);
template <>
__device__ __forceinline__ float narrowed<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrowed<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// An id that something bears on: the times it has been put out before the rows, bit 30 if it is known, its biases
struct Touched {
    int id;
    int known;
    float bias;
};

// grid (stretches, requests). Plain loads all over: the kernel before this one may write the table (dspark_seen_add), the
// masks or the logits while this one's first CTAs already stand, which loads through the read-only path do not allow for.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(AdjustParams p)
{
    __shared__ int s_token[kAdjMaxS];        // what row j has before it, one more each row; -1: none
    __shared__ int s_mask[kAdjMaxS];
    __shared__ int s_bias_id[kAdjThreads];
    __shared__ float s_bias[kAdjThreads];
    __shared__ Touched s_list[kAdjStretch];
    __shared__ int s_touched;
    pdl_enter();
    const int r = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    int keep = p.keep ? p.keep[r] : p.S - 1;
    if (keep < 0 || keep >= p.S) {
        if (first && tid == 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        keep = keep < 0 ? 0 : p.S - 1;
    }
    const int rows = keep + 1;
    if (tid < rows) {
        int v = -1, m = -1;
        if (p.tokens && tid > 0) {
            v = p.tokens[(size_t)r * (p.S - 1) + tid - 1];
            if (v >= p.V) {
                if (first) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
                v = -1;
            }
        }
        if (p.mask) {
            m = p.mask_row ? p.mask_row[(size_t)r * p.S + tid] : r * p.S + tid;
            if (m >= p.n_masks) {
                if (first) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
                m = -1;
            }
        }
        s_token[tid] = v;
        s_mask[tid] = m;
    }
    auto factor = [&](const float* f, float none, bool above) {
        if (!f) return none;
        const float x = f[r];
        if (fabsf(x) <= FLT_MAX && (!above || x > 0.f)) return x;
        if (first && tid == 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        return none;
    };
    const float rep = factor(p.repetition, 1.f, true), pres = factor(p.presence, 0.f, false),
                freq = factor(p.frequency, 0.f, false);
    const bool penal = rep != 1.f || pres != 0.f || freq != 0.f;
    int b0 = 0, b1 = 0;
    if (p.bias_offsets) {
        b0 = p.bias_offsets[r];
        b1 = p.bias_offsets[r + 1];
        if (b0 < 0 || b1 < b0 || b1 > p.n_bias) {
            if (first && tid == 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
            b0 = b1 = 0;
        }
    }
    // the entries of the biases, 256 at a time; all there is for most requests
    auto fetch = [&](int b) {
        const int i = b + tid;
        if (i >= b1) return;
        const int v = p.bias_token[i];
        if (first && (v < 0 || v >= p.V)) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        s_bias_id[tid] = v < 0 || v >= p.V ? -1 : v;
        s_bias[tid] = p.bias_value[i];
    };
    fetch(b0);
    __syncthreads();
    const bool in_place = p.out == p.logits;
    const size_t base = (size_t)r * p.S * p.V;
    const T* src = static_cast<const T*>(p.logits) + base;
    T* dst = static_cast<T*>(p.out) + base;
    for (int v0 = blockIdx.x * kAdjStretch; v0 < p.V; v0 += gridDim.x * kAdjStretch) {
        // what this thread's ids have been, and what they are given
        int count[kAdjEach];
        float bias[kAdjEach] = {};
        unsigned known = 0u, biased = 0u;                    // bits by id
#pragma unroll
        for (int e = 0; e < kAdjEach; ++e) count[e] = 0;
        if (p.seen && penal) {
            const int16_t* row = p.seen + r * p.seen_rs;
            if constexpr (kVec) {
                const int v = v0 + tid * kAdjEach;
                if (v < p.V) {
                    const uint4 q = *reinterpret_cast<const uint4*>(row + v);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < kAdjEach; ++e) {
                        const uint32_t c = (w[e / 2] >> (16 * (e & 1))) & 0xFFFFu;
                        count[e] = c & 0x7FFF;
                        known |= (c != 0u ? 1u : 0u) << e;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < kAdjEach; ++e) {
                    const int v = id_of<T, kVec>(v0, e);
                    const uint32_t c = v < p.V ? (uint16_t)row[v] : 0u;
                    count[e] = c & 0x7FFF;
                    known |= (c != 0u ? 1u : 0u) << e;
                }
            }
        }
        for (int b = b0; b < b1; b += kAdjThreads) {
            if (b1 - b0 > kAdjThreads) {   // more than one load of them: again for each stretch
                __syncthreads();
                fetch(b);
                __syncthreads();
            }
            const int n = min(b1 - b, kAdjThreads);
            for (int k = 0; k < n; ++k) {
                const int d = s_bias_id[k] - v0;
                if ((unsigned)d >= (unsigned)kAdjStretch || s_bias_id[k] < 0) continue;
                const int owner = kVec ? d / kAdjEach : d % kAdjThreads, slot = kVec ? d % kAdjEach : d / kAdjThreads;
                if (owner == tid) {
                    const float x = s_bias[k];
#pragma unroll
                    for (int e = 0; e < kAdjEach; ++e)
                        if (e == slot) bias[e] += x;
                    biased |= 1u << slot;
                }
            }
        }
        // the ids that something bears on, into a list: few, and in no thread's way while the rows pass
        if (tid == 0) s_touched = 0;
        __syncthreads();
        unsigned touch = known | biased;
        if (penal)
            for (int j = 1; j < rows; ++j) {
                const int d = s_token[j] - v0;
                if (s_token[j] < 0 || (unsigned)d >= (unsigned)kAdjStretch) continue;
                if ((kVec ? d / kAdjEach : d % kAdjThreads) == tid) touch |= 1u << (kVec ? d % kAdjEach : d / kAdjThreads);
            }
        if (touch) {
            int at = atomicAdd(&s_touched, __popc(touch));
#pragma unroll
            for (int e = 0; e < kAdjEach; ++e)
                if ((touch >> e) & 1u)
                    s_list[at++] = Touched{id_of<T, kVec>(v0, e), count[e] | (int)((known >> e) & 1u) << 30, bias[e]};
        }
        // the rows as they are, less what masks hide
        const bool inside = kVec ? v0 + tid * kAdjEach < p.V : v0 + tid < p.V;
        for (int j0 = 0; inside && j0 < rows; j0 += kAdjRows) {
            Logits8<T> x[kAdjRows];
            unsigned allowed[kAdjRows];
#pragma unroll
            for (int u = 0; u < kAdjRows; ++u) {
                const int j = j0 + u, m = j < rows ? s_mask[j] : -1;
                allowed[u] = 0xFFu;
                if (m >= 0) {
                    const uint32_t* bits = p.mask + m * p.mask_rs;
                    if constexpr (kVec) {
                        allowed[u] = reinterpret_cast<const uint8_t*>(bits)[(v0 + tid * kAdjEach) / 8];
                    } else {
                        allowed[u] = 0u;
#pragma unroll
                        for (int e = 0; e < kAdjEach; ++e) {
                            const int v = id_of<T, kVec>(v0, e);
                            if (v < p.V) allowed[u] |= ((bits[v / 32] >> (v % 32)) & 1u) << e;
                        }
                    }
                }
                if (j < rows && allowed[u] != 0u && (!in_place || allowed[u] != 0xFFu))
                    load_logits<T, kVec>(x[u], src + (size_t)j * p.V, v0, p.V);
            }
#pragma unroll
            for (int u = 0; u < kAdjRows; ++u) {
                if (j0 + u >= rows) continue;
                if (allowed[u] != 0xFFu) hide<T>(x[u], allowed[u]);
                if (!in_place || allowed[u] != 0xFFu) store_logits<T, kVec>(x[u], dst + (size_t)(j0 + u) * p.V, v0, p.V);
            }
        }
        // and the list, a thread an id and row, over what was stored
        __syncthreads();
        const int pairs = s_touched * rows;
        for (int i = tid; i < pairs; i += kAdjThreads) {
            const int j = i % rows;
            const Touched w = s_list[i / rows];
            const int m = s_mask[j];
            if (m >= 0 && !((p.mask[m * p.mask_rs + w.id / 32] >> (w.id % 32)) & 1u)) continue;
            int n = w.known & 0x3FFFFFFF;
            if (penal)
                for (int k = 1; k <= j; ++k) n += s_token[k] == w.id;
            const size_t at = (size_t)j * p.V + w.id;
            float z = to_f32<T>(src[at]);
            if (w.known >> 30 || n > 0) {
                z = z > 0.f ? __fdiv_rn(z, rep) : z * rep;
                z = fmaf(-freq, (float)n, z);
                if (n > 0) z -= pres;
            }
            dst[at] = narrowed<T>(z + w.bias);
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_adjust(const AdjustParams& p, cudaStream_t s)
{
    // CTAs of a request take its stretches in turn; some 24 an SM keep the requests' unequal rows level
    const int stretches = cdiv(p.V, kAdjStretch), most = cdiv(24 * num_sms(), p.R);
    const dim3 grid(stretches < most ? stretches : most, p.R);
    const uintptr_t where = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.out);
    // rows of whole 16-byte pieces
    if (p.V % 8 == 0 && where % 16 == 0) return launch_pdl(adjust_kernel<T, true>, grid, dim3(kAdjThreads), 0, s, p);
    return launch_pdl(adjust_kernel<T, false>, grid, dim3(kAdjThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_seen_add(const SeenParams& p, cudaStream_t s)
{
    const dim3 grid(cdiv(p.V, p.prompt ? kSeenMarks : kSeenStretch), p.R);
    const cudaError_t e = launch_pdl(seen_add_kernel, grid, dim3(kSeenThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_adjust_logits(const AdjustParams& p, cudaStream_t s)
{
    const cudaError_t e = p.dtype == DSPARK_BF16 ? launch_adjust<__nv_bfloat16>(p, s) : launch_adjust<float>(p, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
