// cache_attend_mma.cu -- attention of the flat verify batch over the 4-bit cache with the codes turned
// into matrix fragments in registers (dspark_cache_attend, D = 64 or 128, few rows a request).
//
//   out = sum_i 2^(t_i - m) v_i / sum_i 2^(t_i - m),  t_i = log2(e) scale q . k_i, in one pass over the keys.
//
// What bounds it: a cached token is 9 D / 8 bytes a head, and its 2 D codes have to become fp16 before a
// product. A warp therefore turns codes into the B fragments of m16n8k16 products in registers, with no
// step through shared memory in fp16, and uses each for all rows of the block: the G heads of all the
// request's queries (MT tiles of 16 rows).
//  - The order of the channels inside q . k is free, so a lane takes the consecutive bytes of one key
//    that make one load, and q's fragments are laid out to match. A lane's channels lie in one group: one
//    scale a key. For the values the two tokens that share a register are joined by a byte permutation
//    before their nibbles are taken apart.
//  - (u - 8) s is exact in fp16 (the cache's scales have 8 bits), q is scaled by a power of two into
//    fp16's range, exactly for bf16; so the scores carry fp32 rounding only. fp32 rows enter as two fp16 terms, and
//    their weights too.
//  - m only has to be near the maximum: it is raised when a score passes it by 2^5, the weights have a
//    factor 2^10, so that they stay below fp16's largest number and small ones above its smallest.
// The keys of all (request, head, row block) items form one line of 64-token tiles, cut into equal runs,
// one a CTA, whatever the lengths are. A run that ends inside an item leaves a part (sum, maximum,
// unnormalised rows) in the workspace, and a second small kernel joins the parts in order. Tiles come by
// bulk copies into a ring of stages, issued by a warp of its own; warp w of the four others takes tokens
// 16 w .. 16 w + 15 of each tile, and their states join through shared memory at an item's end.
#include "attend_plan.cuh"
#include "cache.cuh"
#include "internal.h"
#include "tma.cuh"

namespace dspark {

namespace {

constexpr int kStages = 4;
constexpr int kWarps = 4;                       // consumer warps, one slice of 16 tokens each
constexpr int kThreads = (kWarps + 1) * 32;     // and the warp that issues the copies
constexpr float kShift = 10.f;                  // weights are 2^(t - m + kShift) <= 2^15
constexpr float kSlack = 5.f;                   // m is raised when a score passes it by this
constexpr unsigned long long kDrainNs = 4000000000ull;

template <int D>
struct Tile {
    static constexpr uint32_t v_codes = kTile * D / 2;
    static constexpr uint32_t k_scales = kTile * D;
    static constexpr uint32_t v_scales = k_scales + kTile * D / 16;
    static constexpr uint32_t bytes = v_scales + kTile * D / 16;
};

__device__ __forceinline__ bool a_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                       unsigned long long limit_ns)
{
    if (*abort) return false;
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            raise_status(status, DSPARK_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

__device__ __noinline__ void a_drain(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kDrainNs) {
    }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// The 8 codes of a word times the scale pair s: h[j] = nibbles j and j + 4. 0x6400 | u is 1024 + u in fp16
// and 0x6400 | 16 u is 1024 + 16 u; the differences and products are exact.
__device__ __forceinline__ void dequant(uint32_t w, __half2 s, uint32_t (&h)[4])
{
    const __half2 off = __half2half2(__ushort_as_half(0x6408));      // 1032
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));
    const __half2 m72 = __half2half2(__ushort_as_half(0xD480));      // -72
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo = (w & 0x000F000Fu) | 0x64006400u, hi = (w & 0x00F000F0u) | 0x64006400u;
        h[2 * k] = as_u32(__hmul2(__hsub2(as_half2(lo), off), s));
        h[2 * k + 1] = as_u32(__hmul2(__hfma2(as_half2(hi), sixteenth, m72), s));
        w >>= 8;
    }
}

__device__ __forceinline__ uint32_t pack(float a, float b) { return as_u32(__floats2half2_rn(a, b)); }

// the rounding error of pack(a, b), packed
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi)
{
    const float2 h = __half22float2(as_half2(hi));
    return pack(a - h.x, b - h.y);
}

__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8])
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

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2)
    cache_attend_mma_kernel(AttendParams p, AttendScratch ws, unsigned long long wait_ns)
{
    constexpr bool kSplit = sizeof(T) == 4;   // fp32 rows: two fp16 terms
    constexpr int MB = 16 * MT;               // rows of a block
    constexpr int KS = D / 16;                // products a key tile
    constexpr int NT = D / 8;                 // channel tiles
    constexpr int CH = D / 4;                 // channels of a lane
    constexpr int W = D / 32;                 // words of a key a lane holds
    using L = Tile<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* s_red = reinterpret_cast<float*>(smem + kStages * L::bytes);         // [kWarps][MB][D]
    int* s_pre = reinterpret_cast<int*>(s_red + kWarps * MB * D);               // [R + 1]
    __shared__ uint64_t s_bar[2 * kStages];
    __shared__ uint32_t s_valid[kStages];
    __shared__ float2 s_ml[kWarps][MB];
    __shared__ float s_sum[MB], s_top[MB];
    __shared__ int s_scan[kThreads / 32 + 1];
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_addr(smem), bar0 = smem_addr(s_bar);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    pdl_wait();
    pdl_trigger();
    // ---------------- the line of tiles and this CTA's run of it
    const int total = plan_line<kThreads>(p, MB, s_pre, s_scan, blockIdx.x == 0);
    const int per = (total + gridDim.x - 1) / gridDim.x;
    const int begin = (int)min((long long)blockIdx.x * per, (long long)total);
    const int end = min(begin + per, total);
    volatile int* abort = &s_abort;

    if (warp == kWarps) {
        // ---------------- producer: lane (part, run of slices in one page) issues one copy
        const int P = p.c.page_size;
        const int run = P % 64 == 0 ? 4 : P % 32 == 0 ? 2 : 1;
        const int runs = kTile / 16 / run;
        const int part = lane & 3, sl = (lane >> 2) * run;
        const CacheBlock cb = cache_block(P, D);
        int at = begin, count = 0;
        ItemWalk it;
        it.start(s_pre, p.c.R, begin);
        while (at < end && !*abort) {
            it.settle(p, MB, s_pre, at);
            const int u1 = min(it.span.tiles, it.u + (end - at));
            for (int u = it.u; u < u1 && !*abort; ++u, ++count) {
                const int st = count % kStages;
                const int key0 = it.span.key0(u) + sl * 16;
                const uint8_t* src = nullptr;
                uint32_t bytes = 0, dst = 0;
                if (lane < 4 * runs && key0 < it.span.keys) {
                    const int page = p.c.table[(size_t)it.r * p.c.table_width + key0 / P];
                    if (page >= 0 && page < p.c.n_pages) {
                        const uint32_t slot = key0 % P;
                        src = cache_page_block(p.c, page, it.head(), cb.bytes);
                        const uint32_t row = part < 2 ? D / 2 : D / 16;   // bytes a token
                        const uint32_t from = part == 0 ? 0u : part == 1 ? cb.v_codes : part == 2 ? cb.k_scales : cb.v_scales;
                        const uint32_t to = part == 0 ? 0u : part == 1 ? L::v_codes : part == 2 ? L::k_scales : L::v_scales;
                        src += from + slot * row;
                        bytes = run * 16 * row;
                        dst = sbase + st * L::bytes + to + sl * 16 * row;
                    } else {
                        raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
                    }
                }
                const uint32_t have = __ballot_sync(0xffffffffu, bytes != 0 && part == 0);
                uint32_t sum = bytes;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                bool ok = true;
                if (count >= kStages) ok = a_wait(empty(st), ((count / kStages) - 1) & 1u, abort, p.status, wait_ns);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane == 0) {
                    s_valid[st] = have;
                    if (sum) mbar_expect_tx(full(st), sum);
                    else mbar_arrive(full(st));
                }
                __syncwarp();
                if (bytes) bulk_load(dst, src, bytes, full(st));
            }
            at += u1 - it.u;
        }
        // after an abort the copies in flight land before the CTA leaves
        if (*abort && lane == 0)
            for (int c = max(0, count - kStages); c < count; ++c) a_drain(full(c % kStages), (c / kStages) & 1u);
    } else {
        // ---------------- consumers
        const int g = lane >> 2, i = lane & 3;
        int at = begin, count = 0;
        ItemWalk it;
        it.start(s_pre, p.c.R, begin);
        const int run = p.c.page_size % 64 == 0 ? 4 : p.c.page_size % 32 == 0 ? 2 : 1;
        const float to_log2 = p.scale * kLog2e;
        while (at < end) {
            it.settle(p, MB, s_pre, at);
            const int u0 = it.u, u1 = min(it.span.tiles, u0 + (end - at));
            const int h = it.head(), row0 = it.block() * MB, n_rows = it.span.n_q * p.G;
            // q's fragments: lane (g, i) holds channels CH i .. of rows g and g + 8 of each row tile
            uint32_t qa[MT][KS][4], qb[kSplit ? MT : 1][kSplit ? KS : 1][4];
            float fac[MT][2];
            int pos[MT][2];
            bool bad[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = row0 + mt * 16 + hf * 8 + g;
                    const bool real = row < n_rows;
                    const int j = min(row, n_rows - 1) / p.G, hd = h * p.G + min(row, n_rows - 1) % p.G;
                    pos[mt][hf] = it.span.ctx + j;
                    const T* src = static_cast<const T*>(p.q) + (int64_t)(it.span.first + j) * p.q_ts + hd * p.q_hs + i * CH;
                    float x[CH];
                    if (p.q_aligned) {
#pragma unroll
                        for (int c = 0; c < CH * (int)sizeof(T) / 16; ++c) {
                            const uint4 v = reinterpret_cast<const uint4*>(src)[c];
                            const uint32_t uu[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (kSplit) {
                                    x[(c * 4 + e) % CH] = __uint_as_float(uu[e]);
                                } else {
                                    x[(c * 8 + 2 * e) % CH] = __uint_as_float(uu[e] << 16);
                                    x[(c * 8 + 2 * e + 1) % CH] = __uint_as_float(uu[e] & 0xFFFF0000u);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; ++c) x[c] = to_f32<T>(src[c]);
                    }
                    float top = 0.f;
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        top = fmaxf(top, fabsf(x[c]));
                        odd |= !(fabsf(x[c]) <= FLT_MAX);
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const unsigned odds = __ballot_sync(0xffffffffu, odd);
                    bad[mt][hf] = real && ((odds >> (lane & 28)) & 15u) != 0;
                    // the row's largest element to 2^12 .. 2^13
                    const int ex = (int)(__float_as_uint(top) >> 23);
                    const float up = __uint_as_float((uint32_t)min(266 - ex, 254) << 23);
                    fac[mt][hf] = fmaxf(to_log2 / up, 1e-37f);   // 0 times a masked score would be NaN
                    const float keep = real && !bad[mt][hf] ? 1.f : 0.f;
#pragma unroll
                    for (int c = 0; c < CH; ++c) x[c] = keep != 0.f ? x[c] * up : 0.f;
                    // word w of the lane's channels gives products 2 w and 2 w + 1
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int c = (ks / 2) * 8 + (ks % 2) * 2;
                        qa[mt][ks][hf] = pack(x[c], x[c + 4]);
                        qa[mt][ks][2 + hf] = pack(x[c + 1], x[c + 5]);
                        if (kSplit) {
                            qb[kSplit ? mt : 0][kSplit ? ks : 0][hf] = pack_rest(x[c], x[c + 4], qa[mt][ks][hf]);
                            qb[kSplit ? mt : 0][kSplit ? ks : 0][2 + hf] = pack_rest(x[c + 1], x[c + 5], qa[mt][ks][2 + hf]);
                        }
                    }
                    if (bad[mt][hf] && i == 0) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
                }
            const int pos_lo = it.span.ctx + row0 / p.G;                                    // of the block's rows
            const int pos_hi = it.span.ctx + min(row0 + MB - 1, n_rows - 1) / p.G;
            float o[MT][NT][4], top[MT][2], sum[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
                top[mt][0] = top[mt][1] = -INFINITY;
                sum[mt][0] = sum[mt][1] = 0.f;
            }
            for (int u = u0; u < u1; ++u, ++count) {
                const int st = count % kStages;
                const int key0 = it.span.key0(u) + warp * 16;
                const bool ok = a_wait(full(st), (count / kStages) & 1u, abort, p.status, wait_ns);
                const uint8_t* tile = smem + st * L::bytes;
                bool work = __all_sync(0xffffffffu, ok) && key0 <= pos_hi && key0 < it.span.keys &&
                            ((s_valid[st] >> (4 * (warp / run))) & 1u);
                if (p.window > 0) work = work && ((long long)key0 + 15 > (long long)pos_lo - p.window || key0 < p.sinks);
                if (work) {
                    // ---------------- scores of 16 keys
                    float s[MT][2][4];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int tok = warp * 16 + nt * 8 + g;
                        const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + i * (D / 8));
                        uint32_t w[W];
                        if (W == 4) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(src);
                        else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(src);
                        const __half2 sc = __half2half2(
                            *reinterpret_cast<const __half*>(tile + L::k_scales + (tok * (D / 32) + i * D / 128) * 2));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
                        for (int x = 0; x < W; ++x) {
                            uint32_t b[4];
                            dequant(w[x], sc, b);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma16816(s[mt][nt], qa[mt][2 * x], b[0], b[1]);
                                mma16816(s[mt][nt], qa[mt][2 * x + 1], b[2], b[3]);
                                if (kSplit) {
                                    mma16816(s[mt][nt], qb[kSplit ? mt : 0][kSplit ? 2 * x : 0], b[0], b[1]);
                                    mma16816(s[mt][nt], qb[kSplit ? mt : 0][kSplit ? 2 * x + 1 : 0], b[2], b[3]);
                                }
                            }
                        }
                    }
                    // ---------------- mask; weights 2^(t - m + kShift)
                    const bool edge = key0 + 15 > pos_lo || key0 + 15 >= it.span.keys ||
                                      (p.window > 0 && (long long)key0 <= (long long)pos_hi - p.window);
                    if (edge) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int key = key0 + nt * 8 + 2 * i + (e & 1), at_ = pos[mt][e >> 1];
                                    bool see = key <= at_ && key < it.span.keys;
                                    if (p.window > 0)
                                        see = see && ((long long)key > (long long)at_ - p.window || key < p.sinks);
                                    if (!see) s[mt][nt][e] = -INFINITY;
                                }
                    }
                    uint32_t pa[MT][4], pb[kSplit ? MT : 1][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        float mx[2];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            mx[hf] = fac[mt][hf] * fmaxf(fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]),
                                                         fmaxf(s[mt][1][2 * hf], s[mt][1][2 * hf + 1]));
                        const bool raise = mx[0] > top[mt][0] + kSlack || mx[1] > top[mt][1] + kSlack;
                        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                float m = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                                m = fmaxf(m, top[mt][hf]);
                                const float keep = m == top[mt][hf] ? 1.f : ex2(top[mt][hf] - m);
                                top[mt][hf] = m;
                                sum[mt][hf] *= keep;
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    o[mt][n][2 * hf] *= keep;
                                    o[mt][n][2 * hf + 1] *= keep;
                                }
                            }
                        }
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float base = top[mt][hf] == -INFINITY ? 0.f : kShift - top[mt][hf];
                            float e[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                e[x] = ex2(fmaf(s[mt][x >> 1][2 * hf + (x & 1)], fac[mt][hf], base));
                            sum[mt][hf] += (e[0] + e[1]) + (e[2] + e[3]);
                            pa[mt][hf] = pack(e[0], e[1]);
                            pa[mt][2 + hf] = pack(e[2], e[3]);
                            if (kSplit) {
                                pb[kSplit ? mt : 0][hf] = pack_rest(e[0], e[1], pa[mt][hf]);
                                pb[kSplit ? mt : 0][2 + hf] = pack_rest(e[2], e[3], pa[mt][2 + hf]);
                            }
                        }
                    }
                    // ---------------- values: tokens 2 i, 2 i + 1 and 8 above; lanes of odd i take the odd token
                    // first, so that the four i of a load touch different halves of 128 bytes
                    const uint32_t sel_lo = (i & 1) ? 0x1054u : 0x5410u, sel_hi = (i & 1) ? 0x3276u : 0x7632u;
                    uint32_t va[2][W / 2], vb[2][W / 2];
                    __half2 vs[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int t0 = warp * 16 + k * 8 + 2 * i;
                        const uint32_t* a = reinterpret_cast<const uint32_t*>(tile + L::v_codes + (t0 + (i & 1)) * (D / 2) + g * (D / 16));
                        const uint32_t* b = reinterpret_cast<const uint32_t*>(tile + L::v_codes + (t0 + 1 - (i & 1)) * (D / 2) + g * (D / 16));
                        if (W == 4) {
                            *reinterpret_cast<uint2*>(va[k]) = *reinterpret_cast<const uint2*>(a);
                            *reinterpret_cast<uint2*>(vb[k]) = *reinterpret_cast<const uint2*>(b);
                        } else {
                            va[k][0] = *a;
                            vb[k][0] = *b;
                        }
                        const uint32_t two = *reinterpret_cast<const uint32_t*>(
                            tile + L::v_scales + ((warp * (D / 32) + g * D / 256) * 16 + k * 8 + 2 * i) * 2);
                        uint32_t keep = two;
                        if (edge) {   // what no token wrote may be anything: its scale becomes 0
                            const int k0 = key0 + k * 8 + 2 * i;
                            if (k0 >= it.span.keys) keep = 0;
                            else if (k0 + 1 >= it.span.keys) keep &= 0xFFFFu;
                        }
                        vs[k] = as_half2(keep);
                    }
#pragma unroll
                    for (int x = 0; x < W / 2; ++x)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t b0[4], b1[4];
                            const uint32_t sel = z == 0 ? sel_lo : sel_hi;
                            dequant(__byte_perm(va[0][x], vb[0][x], sel), vs[0], b0);
                            dequant(__byte_perm(va[1][x], vb[1][x], sel), vs[1], b1);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) {
                                    mma16816(o[mt][x * 8 + z * 4 + e], pa[mt], b0[e], b1[e]);
                                    if (kSplit) mma16816(o[mt][x * 8 + z * 4 + e], pb[kSplit ? mt : 0], b0[e], b1[e]);
                                }
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
            }
            // ---------------- the four warps' states join
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float x = sum[mt][hf];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (bad[mt][hf]) x = NAN;
                    if (i == 0) s_ml[warp][mt * 16 + hf * 8 + g] = make_float2(top[mt][hf], x);
                }
            bar_consumers();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = mt * 16 + hf * 8 + g;
                    float m = -INFINITY, l = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w][row].x);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        l = fmaf(s_ml[w][row].x == -INFINITY ? 0.f : ex2(s_ml[w][row].x - m), s_ml[w][row].y, l);
                    const float f = top[mt][hf] == -INFINITY ? 0.f : ex2(top[mt][hf] - m);
                    if (warp == 0 && i == 0) {
                        s_top[row] = m;
                        s_sum[row] = l;
                    }
                    // [row][channel / 4 of the lane][lane i][4]: stores of a quad are neighbours
                    float* dst = s_red + ((size_t)warp * MB + row) * D;
#pragma unroll
                    for (int qd = 0; qd < CH / 4; ++qd) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = qd * 4 + e;
                            x[e] = o[mt][c % NT][2 * hf + c / NT] * f;
                        }
                        *reinterpret_cast<float4*>(dst + (qd * 4 + i) * 4) = make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
            bar_consumers();
            const bool whole = u0 == 0 && u1 == it.span.tiles;
            const int slot = at == begin ? 0 : 1;   // a run's first item, or its last
            float* part = ws.rows + ((size_t)blockIdx.x * 2 + slot) * MB * D;
            for (int x = tid; x < MB * D / 8; x += kWarps * 32) {
                const int row = x / (D / 8), c8 = x % (D / 8);            // channels 8 c8 ..
                const int ii = c8 / (CH / 8), q0 = (c8 % (CH / 8)) * 2;   // lane and its float4s
                float v[8] = {};
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 y = *reinterpret_cast<const float4*>(
                            s_red + ((size_t)w * MB + row) * D + ((q0 + k) * 4 + ii) * 4);
                        v[4 * k] += y.x;
                        v[4 * k + 1] += y.y;
                        v[4 * k + 2] += y.z;
                        v[4 * k + 3] += y.w;
                    }
                const float m = s_top[row], l = s_sum[row];
                if (!whole) {
                    store8<float>(part + row * D + c8 * 8, v);
                    if (c8 == 0) ws.ml[((size_t)blockIdx.x * 2 + slot) * MB + row] = make_float2(m, l);
                } else if (row0 + row < n_rows) {
                    const int rr = row0 + row;
                    const size_t dst = (size_t)(it.span.first + rr / p.G) * p.Hq + h * p.G + rr % p.G;
                    // no visible key: zeros; a row that is not finite: NaN
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= inv;
                    store8<T>(static_cast<T*>(p.out) + dst * D + c8 * 8, v);
                    if (c8 == 0 && p.lse) p.lse[dst] = l == 0.f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
                }
            }
            // an item that starts here and goes on: its parts are joined by the next kernel
            if (tid == 0 && u0 == 0 && u1 < it.span.tiles) {
                const int parts = (at + it.span.tiles - 1) / per - (int)blockIdx.x + 1;
                ws.todo[blockIdx.x] = make_int4(it.r, it.q, parts, slot);
            }
            at += u1 - u0;
            // no item of this run goes on past it
            if (at >= end && tid == 0 && !(u0 == 0 && u1 < it.span.tiles)) ws.todo[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        if (begin >= end && tid == 0) ws.todo[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
}

template <typename T, int D, int MT>
cudaError_t launch_mma(const AttendParams& p, AttendScratch ws, int runs, cudaStream_t s)
{
    constexpr int MB = 16 * MT;
    const size_t smem = kStages * Tile<D>::bytes + sizeof(float) * kWarps * MB * D + sizeof(int) * (p.c.R + 1);
    cudaError_t e = cudaFuncSetAttribute(cache_attend_mma_kernel<T, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attend_mma_kernel<T, D, MT>, dim3(runs), dim3(kThreads), smem, s, p, ws, wait_limit_ns());
}

// Joins the parts of the item that started in run blockIdx.x and went on, one row a warp; and zeros the
// rows of the batch that no request has.
template <typename T, int D, int MB>
__global__ void __launch_bounds__(128) cache_merge_kernel(AttendParams p, AttendScratch ws)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 todo = ws.todo[blockIdx.x];
    const int row = blockIdx.y * 4 + warp;
    if (todo.x >= 0) {
        const RequestSpan sp = request_span(p, todo.x, MB, false);
        const int nmb = sp.blocks, h = todo.y / nmb, rr = (todo.y % nmb) * MB + row;
        if (rr < sp.n_q * p.G) {
            // part 0 in this run's slot, the others first in the following runs
            auto at = [&](int k) { return k == 0 ? (size_t)blockIdx.x * 2 + todo.w : (size_t)(blockIdx.x + k) * 2; };
            float m = -INFINITY;
            for (int k = lane; k < todo.z; k += 32) m = fmaxf(m, ws.ml[at(k) * MB + row].x);
            m = warp_max(m);
            const float base = m == -INFINITY ? 0.f : m;
            float l = 0.f, v[D / 32] = {};
            for (int k = 0; k < todo.z; ++k) {
                const float2 ml = ws.ml[at(k) * MB + row];
                const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - base);
                l = fmaf(f, ml.y, l);   // NaN of a row that is not finite stays
                const float* src = ws.rows + (at(k) * MB + row) * D + lane * (D / 32);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) v[c] = fmaf(f, src[c], v[c]);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t dst = (size_t)(sp.first + rr / p.G) * p.Hq + h * p.G + rr % p.G;
            T* out = static_cast<T*>(p.out) + dst * D + lane * (D / 32);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) store1(out + c, v[c] * inv);
            if (lane == 0 && p.lse) p.lse[dst] = l == 0.f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
        }
    }
    zero_rows<T>(p, D, (blockIdx.y * gridDim.x + blockIdx.x) * 128 + threadIdx.x, gridDim.x * gridDim.y * 128);
}

template <typename T, int D>
cudaError_t launch_merge(const AttendParams& p, AttendScratch ws, int MB, int runs, cudaStream_t s)
{
    const dim3 grid(runs, MB / 4);
    return MB == 16 ? launch_pdl(cache_merge_kernel<T, D, 16>, grid, dim3(128), 0, s, p, ws)
                    : launch_pdl(cache_merge_kernel<T, D, 32>, grid, dim3(128), 0, s, p, ws);
}

template <typename T>
bool q_aligned(const AttendParams& p)
{
    return reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && ((p.q_ts | p.q_hs) * (int64_t)sizeof(T)) % 16 == 0;
}

}  // namespace

// Rows of a block: 32 share the codes' conversion where a request has more than 16 (bf16; two fp16 terms
// of 32 rows do not fit a thread's registers).
int attend_block_rows(const AttendParams& p)
{
    return p.dtype == DSPARK_BF16 && (long long)p.max_q * p.G > 16 ? 32 : 16;
}

int attend_runs(const AttendParams& p) { return num_sms() * (attend_block_rows(p) == 16 ? 3 : 2); }

bool attend_mma_supported(const AttendParams& p)
{
    if (p.c.D != 64 && p.c.D != 128) return false;
    // tiles and rows are counted in 32 bits
    const int MB = attend_block_rows(p);
    const long long rows = (long long)p.max_q * p.G;
    const long long tiles = cdiv((long long)p.c.table_width * p.c.page_size, kTile) + 1;
    return rows < (1ll << 30) && (double)p.c.R * p.c.Hkv * (double)(rows / MB + 1) * (double)tiles < 2147483647.0;
}

size_t attend_mma_scratch(const AttendParams& p, AttendScratch* ws, void* base)
{
    const int MB = attend_block_rows(p), runs = attend_runs(p);
    size_t o = 0;
    const size_t rows = o;
    o = align_up(o + sizeof(float) * (size_t)runs * 2 * MB * p.c.D, 256);
    const size_t ml = o;
    o = align_up(o + sizeof(float2) * (size_t)runs * 2 * MB, 256);
    const size_t todo = o;
    o = align_up(o + sizeof(int4) * (size_t)runs, 256);
    if (ws) {
        char* b = static_cast<char*>(base);
        ws->rows = reinterpret_cast<float*>(b + rows);
        ws->ml = reinterpret_cast<float2*>(b + ml);
        ws->todo = reinterpret_cast<int4*>(b + todo);
    }
    return o;
}

cudaError_t launch_cache_attend_mma(const AttendParams& p0, const AttendScratch& ws, cudaStream_t s)
{
    AttendParams p = p0;
    const bool bf = p.dtype == DSPARK_BF16;
    p.q_aligned = bf ? q_aligned<__nv_bfloat16>(p) : q_aligned<float>(p);
    const int runs = attend_runs(p), MB = attend_block_rows(p);
    cudaError_t e;
    if (p.c.D == 64)
        e = !bf        ? launch_mma<float, 64, 1>(p, ws, runs, s)
            : MB == 16 ? launch_mma<__nv_bfloat16, 64, 1>(p, ws, runs, s)
                       : launch_mma<__nv_bfloat16, 64, 2>(p, ws, runs, s);
    else
        e = !bf        ? launch_mma<float, 128, 1>(p, ws, runs, s)
            : MB == 16 ? launch_mma<__nv_bfloat16, 128, 1>(p, ws, runs, s)
                       : launch_mma<__nv_bfloat16, 128, 2>(p, ws, runs, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_merge(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    const int runs = attend_runs(p), MB = attend_block_rows(p);
    const bool bf = p.dtype == DSPARK_BF16;
    const cudaError_t e = p.c.D == 64 ? (bf ? launch_merge<__nv_bfloat16, 64>(p, ws, MB, runs, s)
                                            : launch_merge<float, 64>(p, ws, MB, runs, s))
                                      : (bf ? launch_merge<__nv_bfloat16, 128>(p, ws, MB, runs, s)
                                            : launch_merge<float, 128>(p, ws, MB, runs, s));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
