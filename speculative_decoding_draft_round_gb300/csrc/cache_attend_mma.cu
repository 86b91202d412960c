// cache_attend_mma.cu -- attention of the flat verify batch over the 4-bit cache with the codes turned
// into matrix fragments in registers (dspark_cache_attend, D = 64 or 128, few rows a request).
//
//   out = sum_i 2^(t_i - m) v_i / sum_i 2^(t_i - m),  t_i = log2(e) scale q . k_i, in one pass over the keys.
//
// What bounds it: a cached token is 9 D / 8 bytes a head, and its 2 D codes have to become fp16 before a
// product. A warp therefore turns codes into the A fragments of m16n8k16 products in registers, with no
// step through shared memory in fp16: 16 keys (then 16 channels of the values) by the block's rows, which
// are the G heads of the request's queries, 8 at a time (NB column tiles). So few rows waste little.
//  - The order of the channels inside q . k is free, so a lane takes the consecutive bytes of one key
//    that make one load, and q's fragments are laid out to match. A lane's channels lie in one group: one
//    scale a key. For the values the two tokens that share a register are joined by a byte permutation
//    before their nibbles are taken apart; the weights turn by movmatrix.
//  - (u - 8) s is exact in fp16 (the cache's scales have 8 bits), q is scaled by a power of two into
//    fp16's range, exactly for bf16; so the scores carry fp32 rounding only. fp32 rows enter as two fp16 terms, and
//    their weights too.
//  - m only has to be near the maximum: it is raised when a score passes it by 2^5, the weights have a
//    factor 2^10, so that they stay below fp16's largest number and small ones above its smallest.
// The keys of all (request, head, row block) items form one line of 32-token tiles, cut into equal runs,
// one a warp, whatever the lengths are. A warp works alone: it copies its tiles into stages of its own by
// 16-byte asynchronous copies, stages - 1 tiles ahead, and no barrier joins it to others (bulk copies of the
// tile's four parts cost more: their operands are uniform, a divergent loop of about 60 instructions a tile). A run that ends inside an item
// leaves a part (maximum, sum, unnormalised rows) in the workspace, and a second small kernel joins the
// parts in order.
//
// Measured, with the joining kernel: 128 single rows of 32 heads (8 key heads of 128) over up to 4096 tokens 84 us, of
// 50 us for the bytes; two rows over up to 131072 tokens 49 of 21 us; 9 rows in a window of 1024 keys after up to 16384
// 46 of 12 us. The kernel alone issues in 62% of the cycles at 54% of the memory's rate (single rows): what a key costs
// is its 2 D codes to fp16 and its share of the products' set-up, some 420 instructions for 16 tokens.
#include "attend_convert.cuh"
#include "attend_plan.cuh"
#include "cache.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kTile = 32;                       // tokens of a tile
constexpr int kWarps = 4;                       // of a CTA, each with a run of its own
constexpr int kThreads = kWarps * 32;
constexpr int kBatch = 16;                      // tiles whose places the lanes look up at once

template <int D>
struct Tile {
    static constexpr uint32_t v_codes = kTile * D / 2;
    static constexpr uint32_t k_scales = kTile * D;
    static constexpr uint32_t v_scales = k_scales + kTile * D / 16;
    static constexpr uint32_t bytes = v_scales + kTile * D / 16;
};

// Variants: CTAs on an SM. Registers count for more than warps: two column tiles with three CTAs (168 registers, 224
// bytes of spills) took 58 us for a window of 512 keys and 16 rows a request, with two 47; one column tile of bf16 took
// 86 us with four for the decode batch (128 x up to 4096 tokens), 84 with three, 92 with two. More stages than three:
// no gain.
template <int NB>
constexpr int kCtas = NB == 1 ? 3 : 2;
constexpr int kStages = 3;   // tiles a warp has in flight

__device__ __forceinline__ uint32_t shared_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes; zeros where there is nothing to copy
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the 8 x 8 matrix of 16-bit elements whose row g lanes (g, i) hold, two a lane, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// the rounding error of pack(a, b), packed
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi)
{
    const float2 h = __half22float2(as_half2(hi));
    return pack(a - h.x, b - h.y);
}

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

// What lane 2 j + half of a warp knows of tile j of a batch: the block that holds its 16 tokens of that
// half, the slot of the first, and whether they are there: not beyond the keys, nor in a page out of range.
struct Place {
    const uint8_t* block;
    uint32_t slot;
    bool there;
};

template <typename T, int D, int NB>
__global__ void __launch_bounds__(kThreads, kCtas<NB>)
    cache_attend_mma_kernel(AttendParams p, AttendScratch ws)
{
    constexpr bool kSplit = sizeof(T) == 4;   // fp32 rows: two fp16 terms
    constexpr int kMB = 8 * NB;               // rows of a block
    constexpr int KS = D / 16;                // products of 16 channels
    constexpr int MT = D / 16;                // tiles of 16 value channels
    constexpr int CH = D / 4;                 // q's channels of a lane
    constexpr int CV = D / 8;                 // value channels of a lane
    constexpr int W = D / 32;                 // words of a key a lane holds
    using L = Tile<D>;
    extern __shared__ __align__(128) uint8_t smem[];                     // [kWarps][kStages] tiles, [R + 1] ints
    int* s_pre = reinterpret_cast<int*>(smem + kWarps * kStages * L::bytes);
    __shared__ long long s_scan[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, i = lane & 3;
    uint8_t* const stages = smem + warp * kStages * L::bytes;
    const uint32_t sbase = shared_addr(stages);
    pdl_wait();
    pdl_trigger();
    // ---------------- the line of tiles and this warp's run of it
    const int total = plan_line<kThreads, kTile>(p, kMB, s_pre, s_scan, blockIdx.x == 0);
    const int runs = gridDim.x * kWarps, run_id = blockIdx.x * kWarps + warp;
    const int per = (int)(((long long)total + runs - 1) / runs);
    const int begin = (int)min((long long)run_id * per, (long long)total);
    const int end = (int)min((long long)begin + per, (long long)total);
    if (begin >= end) {
        if (lane == 0) ws.todo[run_id].parts = 0;
        return;
    }
    const CacheBlock cb = cache_block(p.c.page_size, D);
    // Where the tiles from `at` on are: one lane looks up each half tile, kBatch tiles at a time.
    auto look_up = [&](int at) {
        Place w{static_cast<const uint8_t*>(p.c.pages), 0, false};
        const int tile = at + (lane >> 1);
        if (tile < end) {
            ItemWalk<kTile> it;
            it.start(s_pre, p.c.R, tile);
            it.settle(p, kMB, s_pre, tile);
            const int key0 = it.span.key0(it.u) + (lane & 1) * 16;
            if (key0 < it.span.keys) {
                const int at_page = page_of(key0, p.page_magic);
                const int page = p.c.table[(size_t)it.r * p.c.table_width + at_page];
                if (page >= 0 && page < p.c.n_pages) {
                    w.block = cache_page_block(p.c, page, it.head(), cb.bytes);
                    w.slot = key0 - at_page * p.c.page_size;
                    w.there = true;
                } else {
                    raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
                }
            }
        }
        return w;
    };
    // Tile n of the run into its stage. Chunks of 512 bytes, 16 a lane: those of the K and V codes, and one of
    // the scales, whose lanes are (part, half, 16 bytes).
    constexpr int kChunks = kTile * D / 2 / 512, kScaleLanes = D / 16;
    const int sc_half = (lane / kScaleLanes) & 1;
    const bool sc_v = lane >= 2 * kScaleLanes;
    const uint32_t sc_from = (sc_v ? cb.v_scales : cb.k_scales) + (lane % kScaleLanes) * 16;
    const uint32_t sc_to = (sc_v ? L::v_scales : L::k_scales) + (lane % (2 * kScaleLanes)) * 16;
    auto issue = [&](int n, uint32_t dst, const Place& w, uint32_t have) {
        const uint8_t* blk[2];
        uint32_t slot[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int from = 2 * (n % kBatch) + hf;
            blk[hf] = reinterpret_cast<const uint8_t*>(
                (uintptr_t)__shfl_sync(0xffffffffu, (unsigned long long)(uintptr_t)w.block, from));
            slot[hf] = __shfl_sync(0xffffffffu, w.slot, from);
        }
        dst += sbase;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int hf = c / (kChunks / 2);
            const uint8_t* src = blk[hf] + slot[hf] * (D / 2) + (c % (kChunks / 2)) * 512 + lane * 16;
            const bool in = (have >> hf) & 1u;
            copy16(dst + c * 512 + lane * 16, src, in);
            copy16(dst + L::v_codes + c * 512 + lane * 16, src + cb.v_codes, in);
        }
        if (lane < 4 * kScaleLanes)
            copy16(dst + sc_to, (sc_half ? blk[1] : blk[0]) + sc_from + (sc_half ? slot[1] : slot[0]) * (D / 16),
                   (have >> sc_half) & 1u);
    };
    Place place = look_up(begin);
    uint32_t there[2];                     // by batch parity: which half tiles hold keys
    there[0] = __ballot_sync(0xffffffffu, place.there);
    there[1] = 0;
    const int n_tiles = end - begin;
#pragma unroll 1
    for (int n = 0; n < kStages - 1; ++n) {   // at most kBatch - 1
        if (n < n_tiles) issue(n, n * L::bytes, place, there[0] >> (2 * n));
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    const float to_log2 = p.scale * kLog2e;
    const DequantConst dq = dequant_const();
    int at = begin, count = 0;
    uint32_t st = 0;                       // the stage of tile `count`, in bytes
    ItemWalk<kTile> it;
    it.start(s_pre, p.c.R, begin);
    AttendTodo todo = {};
#pragma unroll 1
    while (at < end) {
        it.settle(p, kMB, s_pre, at);
        const int u0 = it.u, u1 = min(it.span.tiles, u0 + (end - at));
        const int h = it.head(), row0 = it.block() * kMB, n_rows = it.span.n_q * p.G;
        // q's fragments: lane (g, i) holds channels CH i .. of row g of each column tile
        uint32_t qa[NB][KS][2], qb[kSplit ? NB : 1][kSplit ? KS : 1][2];
        float fac[NB][2];     // of the rows 2 i and 2 i + 1, whose scores this lane gets
        bool bad[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int row = row0 + nb * 8 + g;
            const bool real = row < n_rows;
            const int j = min(row, n_rows - 1) / p.G, hd = h * p.G + min(row, n_rows - 1) % p.G;
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
            const unsigned odds = __ballot_sync(0xffffffffu, odd && real);
            const bool mine = ((odds >> (lane & 28)) & 15u) != 0;
            const float up = row_up((int)(__float_as_uint(top) >> 23)), f = row_factor(to_log2, up);
            const bool keep = real && !mine;
#pragma unroll
            for (int c = 0; c < CH; ++c) x[c] = keep ? x[c] * up : 0.f;
            // word w of the lane's channels gives products 2 w and 2 w + 1
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int c = (ks / 2) * 8 + (ks % 2) * 2;
                qa[nb][ks][0] = pack(x[c], x[c + 4]);
                qa[nb][ks][1] = pack(x[c + 1], x[c + 5]);
                if (kSplit) {
                    qb[kSplit ? nb : 0][kSplit ? ks : 0][0] = pack_rest(x[c], x[c + 4], qa[nb][ks][0]);
                    qb[kSplit ? nb : 0][kSplit ? ks : 0][1] = pack_rest(x[c + 1], x[c + 5], qa[nb][ks][1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                fac[nb][e] = __shfl_sync(0xffffffffu, f, (2 * i + e) * 4);
                bad[nb][e] = ((odds >> ((2 * i + e) * 4)) & 15u) != 0;
            }
            if (mine && i == 0) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
        }
        const int pos_lo = it.span.ctx + row0 / p.G;                                    // of the block's rows
        const int pos_hi = it.span.ctx + min(row0 + kMB - 1, n_rows - 1) / p.G;
        // tiles from in_lo to in_hi are seen by every row to their ends
        const int in_hi = min(pos_lo, it.span.keys - 1) - (kTile - 1);
        const int in_lo = p.window > 0 ? (int)max(0ll, (long long)pos_hi - p.window + 1) : 0;
        float o[NB][MT][4], top[NB][2], sum[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][m][e] = 0.f;
            top[nb][0] = top[nb][1] = -INFINITY;
            sum[nb][0] = sum[nb][1] = 0.f;
        }
#pragma unroll 1
        for (int u = u0; u < u1; ++u, ++count) {
            const uint8_t* tile = stages + st;
            const int key0 = it.span.key0(u);
            const uint32_t have = (((count / kBatch) & 1 ? there[1] : there[0]) >> (2 * (count % kBatch))) & 3u;
            {
                // the tile kStages - 1 further on into the stage that the last iteration left
                const int next = count + kStages - 1;
                if (next < n_tiles) {
                    if (next % kBatch == 0) {
                        place = look_up(begin + next);
                        const uint32_t b = __ballot_sync(0xffffffffu, place.there);
                        if ((next / kBatch) & 1) there[1] = b;
                        else there[0] = b;
                    }
                    issue(next, st == 0 ? (kStages - 1) * L::bytes : st - L::bytes, place,
                          ((next / kBatch) & 1 ? there[1] : there[0]) >> (2 * (next % kBatch)));
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                __syncwarp();
            }
            if (have != 0) {
                // ---------------- scores of 32 keys: lane (g, i) gets keys g, g + 8 of each 16 by rows 2 i, 2 i + 1
                float s[2][NB][4];
#pragma unroll
                for (int sl = 0; sl < 2; ++sl) {
                    uint32_t w[2][W];
                    __half2 sc[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int tok = sl * 16 + k * 8 + g;
                        const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + i * (D / 8));
                        if (W == 4) *reinterpret_cast<uint4*>(w[k]) = *reinterpret_cast<const uint4*>(src);
                        else *reinterpret_cast<uint2*>(w[k]) = *reinterpret_cast<const uint2*>(src);
                        sc[k] = __half2half2(
                            *reinterpret_cast<const __half*>(tile + L::k_scales + (tok * (D / 32) + i * D / 128) * 2));
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[sl][nb][e] = 0.f;
#pragma unroll
                    for (int x = 0; x < W; ++x) {
                        uint32_t a[4], b[4];
                        dequant(w[0][x], sc[0], dq, a);
                        dequant(w[1][x], sc[1], dq, b);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                mma16816(s[sl][nb], a[2 * k], b[2 * k], a[2 * k + 1], b[2 * k + 1], qa[nb][2 * x + k][0],
                                         qa[nb][2 * x + k][1]);
                                if (kSplit)
                                    mma16816(s[sl][nb], a[2 * k], b[2 * k], a[2 * k + 1], b[2 * k + 1],
                                             qb[kSplit ? nb : 0][kSplit ? 2 * x + k : 0][0],
                                             qb[kSplit ? nb : 0][kSplit ? 2 * x + k : 0][1]);
                            }
                        }
                    }
                }
                // ---------------- mask; weights 2^(t - m + kShift)
                const bool edge = key0 > in_hi || key0 < in_lo || have != 3u;
                if (edge) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int r2 = 0; r2 < 2; ++r2) {
                            const int own = it.span.ctx + min(row0 + nb * 8 + 2 * i + r2, n_rows - 1) / p.G;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int key = key0 + k * 8 + g;
                                bool see = key <= own && key < it.span.keys && ((have >> (k >> 1)) & 1u);
                                if (p.window > 0)
                                    see = see && ((long long)key > (long long)own - p.window || key < p.sinks);
                                if (!see) s[k >> 1][nb][2 * (k & 1) + r2] = -INFINITY;
                            }
                        }
                }
                uint32_t pa[2][NB][2], pb[2][NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float mx[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mx[e] = fac[nb][e] * fmaxf(fmaxf(s[0][nb][e], s[0][nb][2 + e]), fmaxf(s[1][nb][e], s[1][nb][2 + e]));
                    if (__any_sync(0xffffffffu, mx[0] > top[nb][0] + kSlack || mx[1] > top[nb][1] + kSlack)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            m = fmaxf(m, top[nb][e]);
                            const float keep = m == top[nb][e] ? 1.f : ex2(top[nb][e] - m);
                            top[nb][e] = m;
                            sum[nb][e] *= keep;
#pragma unroll
                            for (int n = 0; n < MT; ++n) {
                                o[nb][n][e] *= keep;
                                o[nb][n][2 + e] *= keep;
                            }
                        }
                    }
                    const float base0 = top[nb][0] == -INFINITY ? 0.f : kShift - top[nb][0];
                    const float base1 = top[nb][1] == -INFINITY ? 0.f : kShift - top[nb][1];
#pragma unroll
                    for (int sl = 0; sl < 2; ++sl)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float e0 = ex2(fmaf(s[sl][nb][2 * k], fac[nb][0], base0));
                            const float e1 = ex2(fmaf(s[sl][nb][2 * k + 1], fac[nb][1], base1));
                            sum[nb][0] += e0;
                            sum[nb][1] += e1;
                            const uint32_t hi = pack(e0, e1);
                            pa[sl][nb][k] = transpose8(hi);   // row g, tokens 2 i and 2 i + 1 of 8
                            if (kSplit) pb[sl][nb][k] = transpose8(pack_rest(e0, e1, hi));
                        }
                }
                // ---------------- values: tokens 2 i, 2 i + 1 and 8 above; lanes of odd i take the odd token
                // first, so that the four i of a load touch both halves of 128 bytes
                const uint32_t sel_lo = (i & 1) ? 0x1054u : 0x5410u, sel_hi = (i & 1) ? 0x3276u : 0x7632u;
#pragma unroll
                for (int sl = 0; sl < 2; ++sl) {
                    uint32_t va[2][W / 2], vb[2][W / 2];
                    __half2 vs[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int t0 = sl * 16 + k * 8 + 2 * i;
                        const uint8_t* v = tile + L::v_codes + g * (D / 16);
                        const uint32_t* a = reinterpret_cast<const uint32_t*>(v + (t0 + (i & 1)) * (D / 2));
                        const uint32_t* b = reinterpret_cast<const uint32_t*>(v + (t0 + 1 - (i & 1)) * (D / 2));
                        if (W == 4) {
                            *reinterpret_cast<uint2*>(va[k]) = *reinterpret_cast<const uint2*>(a);
                            *reinterpret_cast<uint2*>(vb[k]) = *reinterpret_cast<const uint2*>(b);
                        } else {
                            va[k][0] = *a;
                            vb[k][0] = *b;
                        }
                        uint32_t two = *reinterpret_cast<const uint32_t*>(
                            tile + L::v_scales + ((sl * (D / 32) + g * D / 256) * 16 + k * 8 + 2 * i) * 2);
                        if (edge) {   // what no token wrote may be anything: its scale becomes 0
                            const int k0 = key0 + t0;
                            if (k0 >= it.span.keys || !((have >> sl) & 1u)) two = 0;
                            else if (k0 + 1 >= it.span.keys) two &= 0xFFFFu;
                        }
                        vs[k] = as_half2(two);
                    }
#pragma unroll
                    for (int x = 0; x < W / 2; ++x)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t b0[4], b1[4];
                            const uint32_t sel = z == 0 ? sel_lo : sel_hi;
                            dequant(__byte_perm(va[0][x], vb[0][x], sel), vs[0], dq, b0);
                            dequant(__byte_perm(va[1][x], vb[1][x], sel), vs[1], dq, b1);
                            // tile m has channels CV g + 2 m in rows g and CV g + 2 m + 1 in rows g + 8
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    float(&acc)[4] = o[nb][x * 4 + z * 2 + e];
                                    mma16816(acc, b0[2 * e], b0[2 * e + 1], b1[2 * e], b1[2 * e + 1], pa[sl][nb][0],
                                             pa[sl][nb][1]);
                                    if (kSplit)
                                        mma16816(acc, b0[2 * e], b0[2 * e + 1], b1[2 * e], b1[2 * e + 1], pb[sl][nb][0],
                                                 pb[sl][nb][1]);
                                }
                        }
                }
            }
            st = st == (kStages - 1) * L::bytes ? 0 : st + L::bytes;
            __syncwarp();
        }
        // ---------------- the item's end in this run
        const bool whole = u0 == 0 && u1 == it.span.tiles;
        const int slot = at == begin ? 0 : 1;   // a run's first item, or its last
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[nb][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
                if (bad[nb][e]) l = NAN;
                // lane (g, i): channels CV g .. of row 2 i + e
                const int row = nb * 8 + 2 * i + e, rr = row0 + row;
                if (rr >= n_rows) continue;
                if (!whole) {
                    const size_t part_row = ((size_t)run_id * 2 + slot) * kMB + row;
                    float* dst = ws.rows + part_row * D + g * CV;
#pragma unroll
                    for (int c = 0; c < CV; c += 4)
                        *reinterpret_cast<float4*>(dst + c) = make_float4(o[nb][c / 2][e], o[nb][c / 2][2 + e],
                                                                         o[nb][c / 2 + 1][e], o[nb][c / 2 + 1][2 + e]);
                    if (g == 0) ws.ml[part_row] = make_float2(top[nb][e], l);
                } else {
                    const size_t dst = (size_t)(it.span.first + rr / p.G) * p.Hq + h * p.G + rr % p.G;
                    // no visible key: zeros; a row that is not finite: NaN
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int c = 0; c < CV; c += 8) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = o[nb][(c + k) / 2][2 * (k & 1) + e] * inv;
                        store8<T>(static_cast<T*>(p.out) + dst * D + g * CV + c, v);
                    }
                    if (g == 0 && p.lse) p.lse[dst] = l == 0.f ? -INFINITY : (top[nb][e] + log2f(l) - kShift) * kLn2;
                }
            }
        // an item that starts here and goes on: the next kernel joins its parts
        if (u0 == 0 && u1 < it.span.tiles) {
            todo.parts = (at + it.span.tiles - 1) / per - run_id + 1;
            todo.slot = slot;
            todo.first = it.span.first;
            todo.head = h;
            todo.row0 = row0;
            todo.rows = min(kMB, n_rows - row0);
        }
        at += u1 - u0;
    }
    if (lane == 0) ws.todo[run_id] = todo;
}

// Joins the parts of the items that started in the runs of one CTA and went on: a warp takes one run's item,
// or, where an item has many parts, the whole CTA one row after the other. Loads of several parts are in
// flight at once: two dependent loads, of the run's note and of the parts, are what this costs. Also zeros the rows of the batch
// that no request has.
constexpr int kMergeMany = 8;   // parts of an item from which on the CTA shares it

template <int E>
__device__ __forceinline__ void load_part(const float* src, float (&v)[E])
{
    static_assert(E == 2 || E == 4, "one load");
    if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x, v[1] = x.y;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_merge_kernel(AttendParams p, AttendScratch ws)
{
    pdl_enter();
    __shared__ float2 s_ml[kWarps];
    __shared__ float s_o[kWarps][D];
    constexpr int E = D / 32, kAhead = kMergeMany;   // parts whose loads are under way
    const int kMB = ws.block_rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    struct Sum {
        float m, l, v[E];
    };
    auto combine = [&](Sum& s, float m, float l, const float (&v)[E]) {
        const float top = fmaxf(s.m, m), base = top == -INFINITY ? 0.f : top;
        const float f = ex2(s.m - base), h = ex2(m - base);
        s.m = top;
        s.l = s.l * f + l * h;   // NaN of a row that is not finite stays
#pragma unroll
        for (int c = 0; c < E; ++c) s.v[c] = s.v[c] * f + v[c] * h;
    };
    // part 0 is in its run's slot, the others first in the runs that follow
    auto add = [&](const AttendTodo& todo, int run, int row, int k0, int step) {
        Sum s = {};
        s.m = -INFINITY;
        for (int k = k0; k < todo.parts; k += step * kAhead) {
            float2 ml[kAhead];
            float v[kAhead][E];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {   // loads without a condition, or each would wait for the one before
                const int kk = min(k + x * step, todo.parts - 1);
                const size_t a = ((size_t)(run + kk) * 2 + (kk == 0 ? todo.slot : 0)) * kMB + row;
                ml[x] = ws.ml[a];
                load_part<E>(ws.rows + a * D + lane * E, v[x]);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x)
                if (k + x * step < todo.parts) combine(s, ml[x].x, ml[x].y, v[x]);
        }
        return s;
    };
    auto write = [&](const AttendTodo& todo, int row, const Sum& s) {
        const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
        const int rr = todo.row0 + row;
        const size_t dst = (size_t)(todo.first + rr / p.G) * p.Hq + todo.head * p.G + rr % p.G;
        T* out = static_cast<T*>(p.out) + dst * D + lane * E;
#pragma unroll
        for (int c = 0; c < E; ++c) store1(out + c, s.v[c] * inv);
        if (lane == 0 && p.lse) p.lse[dst] = s.l == 0.f ? -INFINITY : (s.m + log2f(s.l) - kShift) * kLn2;
    };
    AttendTodo own = {};
    if ((int)blockIdx.x * kWarps + warp < ws.runs) own = ws.todo[blockIdx.x * kWarps + warp];
    if (own.parts > 0 && own.parts < kMergeMany)
        for (int row = blockIdx.y; row < own.rows; row += gridDim.y)
            write(own, row, add(own, blockIdx.x * kWarps + warp, row, 0, 1));
    const int many = __syncthreads_or(own.parts >= kMergeMany);
    if (many) {
        for (int w = 0; w < kWarps; ++w) {
            const int run = blockIdx.x * kWarps + w;
            if (run >= ws.runs) break;
            const AttendTodo todo = ws.todo[run];
            if (todo.parts < kMergeMany) continue;
            for (int row = blockIdx.y; row < todo.rows; row += gridDim.y) {
                Sum s = add(todo, run, row, warp, kWarps);
                __syncthreads();
                if (lane == 0) s_ml[warp] = make_float2(s.m, s.l);
#pragma unroll
                for (int c = 0; c < E; ++c) s_o[warp][lane * E + c] = s.v[c];
                __syncthreads();
                if (warp != 0) continue;
                for (int x = 1; x < kWarps; ++x) {
                    float v[E];
#pragma unroll
                    for (int c = 0; c < E; ++c) v[c] = s_o[x][lane * E + c];
                    combine(s, s_ml[x].x, s_ml[x].y, v);
                }
                write(todo, row, s);
            }
        }
    }
    zero_rows<T>(p, D, (blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x, gridDim.x * gridDim.y * kThreads);
}

// Rows of a block: 8 where no request has more, else 16
int block_rows(const AttendParams& p) { return (long long)p.max_q * p.G <= 8 ? 8 : 16; }

int grid_ctas(const AttendParams& p)
{
    return num_sms() * (block_rows(p) == 8 ? kCtas<1> : kCtas<2>);
}

template <typename T, int D, int NB>
cudaError_t launch_rows(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    auto smem = [](int R) { return kWarps * kStages * Tile<D>::bytes + sizeof(int) * (R + 1); };
    static std::atomic<uint64_t> admitted{0};
    const cudaError_t e = admit_smem(cache_attend_mma_kernel<T, D, NB>, smem(DSPARK_MAX_SLOTS), admitted);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attend_mma_kernel<T, D, NB>, dim3(grid_ctas(p)), dim3(kThreads), smem(p.c.R), s, p, ws);
}

template <typename T, int D>
cudaError_t launch_mma(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    return block_rows(p) == 8 ? launch_rows<T, D, 1>(p, ws, s) : launch_rows<T, D, 2>(p, ws, s);
}

template <typename T, int D>
cudaError_t launch_merge(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    const long long most = (long long)p.max_q * p.G < ws.block_rows ? (long long)p.max_q * p.G : ws.block_rows;
    return launch_pdl(cache_merge_kernel<T, D>, dim3(cdiv(ws.runs, kWarps), (unsigned)(most < 32 ? most : 32)), dim3(kThreads), 0,
                      s, p, ws);
}

template <typename T>
bool q_aligned(const AttendParams& p)
{
    return reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && ((p.q_ts | p.q_hs) * (int64_t)sizeof(T)) % 16 == 0;
}

}  // namespace

bool attend_mma_supported(const AttendParams& p)
{
    if (p.c.D != 64 && p.c.D != 128) return false;
    return tiles_fit(p, block_rows(p), kTile);
}

size_t attend_scratch(const AttendParams& p, AttendScratch* ws, void* base)
{
    const bool tc = attend_tc_supported(p);
    const int MB = tc ? attend_tc_block_rows() : block_rows(p);
    const size_t runs = tc ? num_sms() : (size_t)grid_ctas(p) * kWarps;
    size_t o = 0;
    const size_t rows = o;
    o = align_up(o + sizeof(float) * runs * 2 * MB * p.c.D, 256);
    const size_t ml = o;
    o = align_up(o + sizeof(float2) * runs * 2 * MB, 256);
    const size_t todo = o;
    o = align_up(o + sizeof(AttendTodo) * runs, 256);
    if (ws) {
        char* b = static_cast<char*>(base);
        ws->rows = reinterpret_cast<float*>(b + rows);
        ws->ml = reinterpret_cast<float2*>(b + ml);
        ws->todo = reinterpret_cast<AttendTodo*>(b + todo);
        ws->runs = (int)runs;
        ws->block_rows = MB;
    }
    return o;
}

cudaError_t launch_cache_attend(const AttendParams& p0, const AttendScratch& ws, cudaStream_t s)
{
    AttendParams p = p0;
    const bool bf = p.dtype == DSPARK_BF16;
    p.q_aligned = bf ? q_aligned<__nv_bfloat16>(p) : q_aligned<float>(p);
    if (attend_tc_supported(p)) return launch_cache_attend_tc(p, ws, s);
    const cudaError_t e =
        p.c.D == 64 ? (bf ? launch_mma<__nv_bfloat16, 64>(p, ws, s) : launch_mma<float, 64>(p, ws, s))
                    : (bf ? launch_mma<__nv_bfloat16, 128>(p, ws, s) : launch_mma<float, 128>(p, ws, s));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_merge(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    const bool bf = p.dtype == DSPARK_BF16;
    const cudaError_t e =
        p.c.D == 64 ? (bf ? launch_merge<__nv_bfloat16, 64>(p, ws, s) : launch_merge<float, 64>(p, ws, s))
                    : (bf ? launch_merge<__nv_bfloat16, 128>(p, ws, s) : launch_merge<float, 128>(p, ws, s));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
