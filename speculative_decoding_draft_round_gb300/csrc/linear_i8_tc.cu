// linear_i8_tc.cu -- rows of 8-bit codes times 8-bit weights on the fifth-generation tensor cores (dspark_linear_i8):
//   out[out_row[t]][n] = (sum_k x[t][k] w[n][k]) * x_scale[t] * w_scale[n] + bias[n]
//
// This chip's rate for 8-bit integers is a small part of its 16-bit one, and a code is exact in fp16: the products run as
// kind::f16. A product of codes is a whole number of at most 2^14, so fp32 sums lose nothing below 2^24.
//
// Weights are the M side. They arrive as bytes, which is all the memory traffic there is for few rows, are widened in
// registers and written to tensor memory, where the MMA reads them: through shared memory pass one byte in and one byte
// out a weight instead of six. The rows x, widened once a call by linear_layout_kernel (they are read by every tile of
// channels), are the N side, K-major in shared memory. Two CTAs share an MMA (cta_group::2): 128 channels each, and each
// holds half of the tile's rows of x, so that a CTA reads 16 KB of weights and at most 24 KB of x for 2 x 128 x 192 x 128
// products.
//   kind::f16 widening: byte ^ 0x80 put under the exponent of 1024 is 1024 + (w + 128) in fp16, less 1152 is w.
//
// Warps: 0 copies (TMA ring of 128-wide steps of K), 1 issues MMAs (first CTA of a pair), 2-9 widen (a quarter of the
// lanes and half of the step each, into a slot of tensor memory), 10-13 take finished sums out (one of two accumulators).
// Tiles that would leave SMs idle are split along K over the pairs of a cluster, which add up their sums through
// distributed shared memory in a fixed order.
// Measured, layout included, rows x K x channels, calls from Python in a row (replayed from a graph): 6007 x 8192 x 8192
// 482 to 497 us (474) of 416 at the library's bf16 rate, 2176 x 4096 x 6144 92 to 94 us (91) of 57, 128 x 4096 x 151936
// 139 us (130) of 99, 16 x 4096 x 6144 16.5 to 17.5 us (14.5, two launches). A tile's way out costs much: four full tiles a
// pair (1536 x K x 9728) take 70 us at K = 1024, 78 at 2048, 91 at 4096, 142 at 8192. For few rows a step takes 900 cycles
// from copy to release where its MMAs are 512, at any number of slots and widening warps, with x shared between pairs or
// not; which limit that is has not been found.
// The kernel is launched without programmatic dependence. A first form that had it, that asked for tensor memory before
// it knew that the other CTA of the pair had begun, and whose second CTA did not wait for the last arrivals, came to a
// stop in calls made back to back; which of the three it was is not known. Now a pair asks for tensor memory when both
// CTAs stand, and leaves when every arrival at its barriers has been made.
// Waits at barriers in shared memory are bounded by the global timer; one that runs out records DSPARK_ERR_TIMEOUT, the
// CTAs stop issuing, let copies and MMAs land, free their tensor memory and return. Not bounded are the waits inside
// tcgen05.alloc and the barriers of a cluster, where a pair's CTAs wait for each other only.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "linear.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace dspark {

namespace {

constexpr int kChannels = 128;                        // of a CTA: the lanes of tensor memory
constexpr int kMostRows = 192;                        // rows of x of a tile
constexpr int kStep = 128;                            // K of a stage
constexpr uint32_t kWBytes = kChannels * kStep;       // 16 KB of weights
constexpr uint32_t kRingBytes = 200 << 10;
constexpr int kMostStages = 10;
constexpr int kMostSplit = 4;                         // pairs of a cluster
constexpr int kThreads = 14 * 32;
constexpr int kWideners = 8, kFirstWidener = 2, kFirstOut = 10;
// Two accumulators of a column a row first, then slots for a step's widened weights: two, or four where there is room.
constexpr uint32_t kTmemCols = 512, kSlotCols = kStep / 2;
constexpr int kMostSlots = 4;
constexpr unsigned long long kDrainNs = 4000000000ull;   // own copies and MMAs land long before

// Barriers, from the ring's end on
enum Bar { kFull = 0, kDone = kMostStages, kReady = 2 * kMostStages, kSumFull = kReady + kMostSlots, kSumEmpty = kSumFull + 2,
           kFin = kSumEmpty + 2, kBars = kFin + 1 };
constexpr uint32_t kMiscBytes = kBars * 8 + 8 + 4 * kMostRows * 8;
constexpr uint32_t kSmem = kRingBytes + 1024 + kMiscBytes;
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
static_assert(2 * kMostRows + 2 * kSlotCols <= kTmemCols && 2 * 128 + 4 * kSlotCols <= kTmemCols, "tensor memory");

struct LinearPlan {
    int rows;        // of x a tile, a multiple of 32
    int stages;
    int slots;       // of widened weights
    int split;       // pairs along K
    int band;        // tiles of rows that share a pass over the channels
    int x_pitch;     // halves
    unsigned long long wait_ns;
};

// ------------------------------------------------------------------ layouts

constexpr int kLayoutThreads = 256;

__device__ __forceinline__ uint32_t half_of(int code) { return __half_as_ushort(__int2half_rn(code)); }

// rows [rows][K] of bytes, any alignment, to rows of 16-byte pitch; a thread moves 16 bytes
__device__ __forceinline__ void pad_bytes(const int8_t* src, int64_t rs, int K, int8_t* dst, int64_t pitch, long long i)
{
    const int each = (int)(pitch / 16);
    const long long row = i / each;
    const int c = (int)(i % each) * 16;
    const int8_t* s = src + row * rs + c;
    const int n = min(16, K - c);
    uint32_t w[4];
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(s) & 3);
    const uint32_t* a = reinterpret_cast<const uint32_t*>(s - off);
    // words that hold at least one byte of the row
    uint32_t q[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) q[j] = 4 * j < n + (int)off ? a[j] : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = __funnelshift_r(q[j], q[j + 1], 8 * off);
        const int left = n - 4 * j;
        if (left < 4) w[j] &= left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    }
    *reinterpret_cast<uint4*>(dst + row * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The first x_blocks CTAs widen x to fp16, the others lay the weights out on 16-byte boundaries.
__global__ void __launch_bounds__(kLayoutThreads)
    linear_layout_kernel(LinearParams p, __half* x16, int x_pitch, int8_t* w16, int64_t w_pitch, unsigned x_blocks)
{
    pdl_enter();
    if (blockIdx.x >= x_blocks) {
        const long long i = (long long)(blockIdx.x - x_blocks) * kLayoutThreads + threadIdx.x;
        if (i < p.N * (w_pitch / 16)) pad_bytes(p.w, p.w_rs, p.K, w16, w_pitch, i);
        return;
    }
    const int live = linear_rows(p, blockIdx.x == 0 && threadIdx.x == 0);
    const long long i = (long long)blockIdx.x * kLayoutThreads + threadIdx.x;
    const int each = x_pitch / 8;
    const long long row = i / each;
    if (row >= live) return;
    const int c = (int)(i % each) * 8;
    const int8_t* s = p.x + row * p.x_rs + c;
    int v[8];
    if (((reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)p.x_rs) & 7) == 0 && c + 8 <= p.K) {
        const int2 q = *reinterpret_cast<const int2*>(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (int8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < p.K ? s[e] : 0;
    }
    uint4 o;
    o.x = half_of(v[0]) | half_of(v[1]) << 16;
    o.y = half_of(v[2]) | half_of(v[3]) << 16;
    o.z = half_of(v[4]) | half_of(v[5]) << 16;
    o.w = half_of(v[6]) | half_of(v[7]) << 16;
    *reinterpret_cast<uint4*>(x16 + row * x_pitch + c) = o;
}

// ------------------------------------------------------------------ pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

// What the arrival tells of is in tensor memory and ordered by the tcgen05 fences (or is a copy's, which the copy engine's
// barrier ordered): it needs no release of this thread's other writes to the cluster.
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same in two halves, without an order of anything written
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

constexpr unsigned long long kShortNs = 1000000;

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                       unsigned long long limit_ns)
{
    // a try may suspend the warp for a time of its own, so under a short limit tries do not suspend
    const unsigned long long t0 = globaltimer();
    while (!(limit_ns < kShortNs ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
        if (*abort) return false;
        if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            raise_status(status, DSPARK_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

struct Waits {
    volatile int* abort;
    int* status;
    unsigned long long limit_ns;
    __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity) const
    {
        // one try that may suspend the warp before the timer is looked at, which takes longer than most waits
        return mbar_test_wait(bar, parity) || (limit_ns >= kShortNs && mbar_try_wait(bar, parity)) ||
               wait_slow(bar, parity, abort, status, limit_ns);
    }
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
};

__device__ __noinline__ void drain(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kDrainNs) {
    }
}

__device__ __forceinline__ void pair_alloc(uint32_t* slot)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_dealloc(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemCols) : "memory");
}

// Four K steps of 16, 256 channels of both CTAs' tensor memory times the rows in both CTAs' shared memory; a converged
// warp of the first CTA, one elected lane issues
__device__ __forceinline__ void pair_mma4(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

// arrive on a barrier of both CTAs when every MMA issued so far is done
__device__ __forceinline__ void pair_commit(uint32_t bar, uint16_t both)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(both)
        : "memory");
}

__device__ __forceinline__ uint4 load16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float load_at(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// four codes as fp16, two words
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// ------------------------------------------------------------------ tiles

struct Tile {
    int n0, t0, rows, cols;   // first channel and row, live rows, columns of the MMA (rows rounded up to 32)
};

struct Tiles {
    int live, blocks, runs, rows, band;   // rows of x, tiles along the channels and along the rows
    __device__ __forceinline__ Tiles(const LinearParams& p, const LinearPlan& g, int live_)
        : live(live_), blocks((p.N + 2 * kChannels - 1) / (2 * kChannels)), runs((live_ + g.rows - 1) / g.rows), rows(g.rows),
          band(g.band) {}
    __device__ __forceinline__ long long count() const { return (long long)blocks * runs; }
    __device__ __forceinline__ Tile at(long long i) const
    {
        const long long per = (long long)band * blocks;
        const int b = (int)(i / per);
        const int in = (int)(i % per), width = min(band, runs - b * band);
        Tile t;
        t.n0 = in / width * 2 * kChannels;
        t.t0 = (b * band + in % width) * rows;
        t.rows = min(rows, live - t.t0);
        t.cols = (t.rows + 31) & ~31;
        return t;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(LinearParams p, LinearPlan g, const __grid_constant__ CUtensorMap wmap,
                     const __grid_constant__ CUtensorMap xmap)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring = smem_addr(smem), bars = ring + kRingBytes;
    auto bar = [&](int i) { return bars + 8u * i; };
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kRingBytes + 8 * kBars);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    float* s_scale = reinterpret_cast<float*>(s_tmem + 2);             // [4][kMostRows] of a tile's rows, each warp its own
    int* s_place = reinterpret_cast<int*>(s_scale + 4 * kMostRows);    // where they go

    cluster_arrive();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), half = rank & 1u, first = rank & ~1u;
    const uint16_t both = (uint16_t)(3u << first);
    if (tid == 0) {
        for (int i = 0; i < kMostStages; ++i) {
            mbar_init(bar(kFull + i), 1);
            mbar_init(bar(kDone + i), 1);
        }
        for (int i = 0; i < kMostSlots; ++i) mbar_init(bar(kReady + i), 2 * kWideners);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kSumFull + i), 1);
            mbar_init(bar(kSumEmpty + i), 2 * 4);
        }
        mbar_init(bar(kFin), 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    __syncwarp();
    cluster_wait();                      // the pair's other CTA stands: the allocation is one of both
    if (warp == 1) pair_alloc(s_tmem);
    tc5::fence_before();
    __syncthreads();
    cluster_sync();
    tc5::fence_after();
    const uint32_t tmem = *s_tmem;

    const Waits wait{s_abort, p.status, g.wait_ns};
    const Tiles tiles(p, g, linear_rows(p, false));
    const long long count = tiles.count();
    const uint32_t cluster_size = 2u * g.split;
    const long long tile0 = blockIdx.x / cluster_size, hop = gridDim.x / cluster_size;
    const int all = (p.K + kStep - 1) / kStep;
    const int k_lo = (int)((long long)all * (rank >> 1) / g.split), k_hi = (int)((long long)all * ((rank >> 1) + 1) / g.split);
    const uint32_t box = (uint32_t)g.rows / 2 * 128;       // bytes of 64 channels of K of this CTA's rows of x
    const uint32_t stage_bytes = kWBytes + 2 * box;
    const uint32_t w_slots = tmem + 2 * g.rows;

    if (warp == 0) {
        // ---------------- copies
        if (lane == 0) {
            const uint64_t pol_w = tiles.runs > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
            const uint64_t pol_x = l2_policy_evict_last();
            int st = 0, issued = 0;
            uint32_t phase = 1;                            // of the stage's release: passes at once the first time round
            bool ok = true;
            for (long long i = tile0; i < count && ok; i += hop) {
                const Tile t = tiles.at(i);
                const int row0 = t.t0 + (int)half * (t.cols / 2);
                for (int k = k_lo; k < k_hi; ++k) {
                    if (issued >= g.stages && !wait.one(bar(kDone + st), phase)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = ring + st * stage_bytes, full = bar(kFull + st);
                    mbar_expect_tx(full, stage_bytes);
                    tma_load_2d(dst, &wmap, k * kStep, t.n0 + (int)half * kChannels, full, pol_w);
                    tma_load_2d(dst + kWBytes, &xmap, k * kStep, row0, full, pol_x);
                    tma_load_2d(dst + kWBytes + box, &xmap, k * kStep + 64, row0, full, pol_x);
                    issued = min(issued + 1, g.stages);
                    if (++st == g.stages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
            }
            // copies still in flight land before the CTA leaves (also where only a later wait of another warp runs out)
            for (int back = issued; back > 0; --back) {
                const int s = (st - back + g.stages) % g.stages;
                // the phase that the stage's last copy ends
                drain(bar(kFull + s), s < st ? phase ^ 1u : phase);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMAs, by the first CTA of a pair
        if (half == 0) {
            int st = 0, it = 0, slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long i = tile0; i < count && ok; i += hop, ++it) {
                const Tile t = tiles.at(i);
                const int b = it & 1;
                if (it >= 2 && !wait.warp(bar(kSumEmpty + b), ((it >> 1) - 1) & 1u)) break;
                tc5::fence_after();
                const uint32_t idesc = (1u << 4) | ((uint32_t)(t.cols >> 3) << 17) | ((2u * kChannels >> 4) << 24);
                const uint32_t d = tmem + b * g.rows;
                for (int k = k_lo; k < k_hi; ++k) {
                    if (!wait.warp(bar(kReady + slot), phase)) {
                        ok = false;
                        break;
                    }
                    tc5::fence_after();
                    const uint32_t x = ring + st * stage_bytes + kWBytes, w = w_slots + slot * kSlotCols;
                    pair_mma4(d, w, tc5::desc_sw128(x), idesc, k != k_lo);
                    pair_mma4(d, w + 32, tc5::desc_sw128(x + box), idesc, 1u);
                    pair_commit(bar(kDone + st), both);
                    if (++st == g.stages) st = 0;
                    if (++slot == g.slots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) pair_commit(bar(kSumFull + b), both);
            }
            pair_commit(bar(kFin), both);
        }
    } else if (warp < kFirstOut) {
        // ---------------- widening: lane 32 (warp % 4) + lane, half `part` of the step
        const int part = (warp - kFirstWidener) >> 2;
        const uint32_t row = (uint32_t)(warp & 3) * 32 + lane;
        const uint32_t lanes = w_slots + ((uint32_t)((warp & 3) * 32) << 16) + part * 32;
        const uint32_t ready = at_rank(bar(kReady), first);
        int st = 0, n = 0, slot = 0, back = 0;             // back: the stage of the step that had the slot before
        uint32_t phase = 0, back_phase = 0;
        bool ok = true;
        for (long long i = tile0; i < count && ok; i += hop) {
            for (int k = k_lo; k < k_hi; ++k, ++n) {
                if (!wait.warp(bar(kFull + st), phase)) {
                    ok = false;
                    break;
                }
                uint32_t v[2][16];
                const uint32_t src = ring + st * stage_bytes + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 q = load16(src + (((uint32_t)(4 * part + c) ^ (row & 7u)) << 4));
                    uint32_t* o = &v[c >> 1][8 * (c & 1)];
                    widen4(q.x, o[0], o[1]);
                    widen4(q.y, o[2], o[3]);
                    widen4(q.z, o[4], o[5]);
                    widen4(q.w, o[6], o[7]);
                }
                if (n >= g.slots) {
                    // that step's MMAs have read the slot
                    if (!wait.warp(bar(kDone + back), back_phase)) {
                        ok = false;
                        break;
                    }
                    tc5::fence_after();
                    if (++back == g.stages) {
                        back = 0;
                        back_phase ^= 1u;
                    }
                }
                tc5::st16(lanes + slot * kSlotCols, v[0]);
                tc5::st16(lanes + slot * kSlotCols + 16, v[1]);
                tc5::wait_st();
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(ready + 8u * slot);
                if (++slot == g.slots) slot = 0;
                if (++st == g.stages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        }
        // the last steps' releases too have arrived before the CTA leaves
        for (int left = min(n, g.slots); left > 0 && ok; --left) {
            ok = wait.warp(bar(kDone + back), back_phase);
            if (++back == g.stages) {
                back = 0;
                back_phase ^= 1u;
            }
        }
    } else {
        // ---------------- sums out
        const int q = warp & 3;
        const uint32_t sums = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t empty = at_rank(bar(kSumEmpty), first);
        int it = 0;
        for (long long i = tile0; i < count; i += hop, ++it) {
            const Tile t = tiles.at(i);
            const int b = it & 1, n = t.n0 + (int)half * kChannels + q * 32 + lane;
            float* scale = s_scale + q * kMostRows;
            int* place = s_place + q * kMostRows;
            if (g.split == 1)
                for (int c = lane; c < t.rows; c += 32) {
                    scale[c] = p.x_scale[t.t0 + c];
                    place[c] = (int)linear_place(p, t.t0 + c);
                }
            const float ws = n < p.N ? p.w_scale[n] : 0.f, bias = n < p.N && p.bias ? p.bias[n] : 0.f;
            __syncwarp();
            if (!wait.warp(bar(kSumFull + b), (it >> 1) & 1u)) break;
            tc5::fence_after();
            for (int c0 = 0; c0 < t.cols; c0 += 32) {
                uint32_t v[32];
                tc5::ld32(sums + b * g.rows + c0, v);
                if (g.split > 1) {
                    // the ring is free: every copy has landed and every MMA is done
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        reinterpret_cast<uint32_t*>(smem)[(c0 + j) * kChannels + q * 32 + lane] = v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int c = c0 + j;
                        if (c < t.rows && n < p.N && place[c] >= 0)
                            static_cast<T*>(p.out)[place[c] * p.o_rs + n] = linear_out<T>(__uint_as_float(v[j]), scale[c], ws, bias);
                    }
                }
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(empty + 8u * b);
        }
    }
    __syncthreads();
    if (warp == 1) {
        // every MMA issued is done, and its arrivals here have been made, before the CTAs leave (also after an abort)
        drain(bar(kFin), 0u);
        __syncwarp();
    }
    cluster_sync();
    if (g.split > 1 && tile0 < count) {
        // the pairs' sums: each adds up its share of the rows, in the order of the pairs
        const Tile t = tiles.at(tile0);
        const int pair = (int)(rank >> 1), c_lo = t.rows * pair / g.split, c_hi = t.rows * (pair + 1) / g.split;
        const int ch = tid & 127, n = t.n0 + (int)half * kChannels + ch;
        if (tid < 3 * 128 && n < p.N) {
            const float ws = p.w_scale[n], bias = p.bias ? p.bias[n] : 0.f;
            for (int c = c_lo + (tid >> 7); c < c_hi; c += 3) {
                const uint32_t mine = ring + (uint32_t)(c * kChannels + ch) * 4;
                float sum = 0.f;
                for (int s = 0; s < g.split; ++s) sum += load_at(at_rank(mine, 2 * s + half));
                const long long row = linear_place(p, t.t0 + c);
                if (row >= 0) static_cast<T*>(p.out)[row * p.o_rs + n] = linear_out<T>(sum, p.x_scale[t.t0 + c], ws, bias);
            }
        }
        cluster_sync();
    }
    if (warp == 1) {
        tc5::fence_after();
        pair_dealloc(tmem);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        (void)cudaGetLastError();
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch,
            uint32_t box_cols, uint32_t box_rows)
{
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
    return encode_fn()(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool weights_fit(const LinearParams& p)
{
    return reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && p.w_rs % 16 == 0 && p.w_rs >= p.K;
}

size_t x_pitch(const LinearParams& p) { return align_up((size_t)p.K, 8); }
size_t x_bytes(const LinearParams& p) { return align_up((size_t)p.T * x_pitch(p) * 2, 256); }
size_t w_pitch(const LinearParams& p) { return align_up((size_t)p.K, 16); }

template <typename T>
cudaError_t configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int pairs, unsigned clusters, cudaStream_t s)
{
    static std::atomic<uint64_t> admitted{0};
    const cudaError_t e = admit_smem(linear_tc_kernel<T>, kSmem, admitted);
    if (e != cudaSuccess) return e;
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3(clusters * 2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * pairs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaSuccess;
}

// Clusters of `pairs` pairs that the device holds at a time
template <typename T>
cudaError_t clusters_held(int pairs, int* n)
{
    static std::atomic<int> held[64][kMostSplit + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>& h = held[dev & 63][pairs];
    *n = dev < 64 ? h.load(std::memory_order_acquire) : 0;
    if (*n > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    e = configure<T>(cfg, attr, pairs, 1, nullptr);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(n, linear_tc_kernel<T>, &cfg);
    if (e == cudaSuccess && *n < 1) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess && dev < 64) h.store(*n, std::memory_order_release);
    return e;
}

template <typename T>
cudaError_t launch_tc(const LinearParams& p, void* ws, cudaStream_t s)
{
    LinearPlan g;
    g.wait_ns = wait_limit_ns();
    g.x_pitch = (int)x_pitch(p);
    g.rows = p.T >= kMostRows ? kMostRows : (int)align_up((size_t)p.T, 32);
    g.stages = (int)(kRingBytes / (kWBytes + (uint32_t)g.rows * 128));
    if (g.stages > kMostStages) g.stages = kMostStages;
    g.slots = g.rows > 128 ? 2 : kMostSlots;
    // a band's rows of x stay in the L2 while the weights pass
    const long long row_bytes = (long long)g.rows * g.x_pitch * 2;
    g.band = (int)(row_bytes > (32ll << 20) ? 1 : row_bytes < (32ll << 10) ? 1024 : (32ll << 20) / row_bytes);
    const long long tiles = (long long)cdiv(p.N, 2 * kChannels) * cdiv(p.T, g.rows);
    const int steps = cdiv(p.K, kStep);
    int held = 0;
    cudaError_t e = cudaSuccess;
    for (g.split = kMostSplit; g.split > 1; --g.split) {
        if (steps < 2 * g.split) continue;
        e = clusters_held<T>(g.split, &held);
        if (e != cudaSuccess) return e;
        if (tiles <= held) break;
    }
    if (g.split == 1) {
        e = clusters_held<T>(1, &held);
        if (e != cudaSuccess) return e;
    }
    const unsigned clusters = (unsigned)(tiles < held ? tiles : held);

    __half* x16 = static_cast<__half*>(ws);
    int8_t* w16 = static_cast<int8_t*>(ws) + x_bytes(p);
    const bool fit = weights_fit(p);
    CUtensorMap wmap, xmap;
    if (!encode(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, fit ? p.w : w16, p.K, p.N, fit ? p.w_rs : w_pitch(p), kStep, kChannels) ||
        !encode(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x16, p.K, p.T, (uint64_t)g.x_pitch * 2, 64, g.rows / 2))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    e = configure<T>(cfg, attr, g.split, clusters, s);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, linear_tc_kernel<T>, p, g, wmap, xmap);
    return e;
}

}  // namespace

bool linear_tc_supported(const LinearParams& p)
{
    // blocks of the layouts and bytes of a row of x in a grid and a pitch
    return encode_fn() != nullptr && (long long)p.T * x_pitch(p) / 8 / kLayoutThreads < (1ll << 30) &&
           (long long)p.N * w_pitch(p) / 16 / kLayoutThreads < (1ll << 30);
}

size_t linear_tc_scratch(const LinearParams& p)
{
    return x_bytes(p) + (weights_fit(p) ? 0 : (size_t)p.N * w_pitch(p));
}

cudaError_t launch_linear_layout(const LinearParams& p, void* ws, cudaStream_t s)
{
    const unsigned xb = (unsigned)cdiv((long long)p.T * x_pitch(p) / 8, kLayoutThreads);
    const unsigned wb = weights_fit(p) ? 0u : (unsigned)cdiv((long long)p.N * w_pitch(p) / 16, kLayoutThreads);
    __half* x16 = static_cast<__half*>(ws);
    const cudaError_t e = launch_pdl(linear_layout_kernel, dim3(xb + wb), dim3(kLayoutThreads), 0, s, p, x16, (int)x_pitch(p),
                                     static_cast<int8_t*>(ws) + x_bytes(p), (int64_t)w_pitch(p), xb);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_linear_tc(const LinearParams& p, void* ws, cudaStream_t s)
{
    const cudaError_t e = p.dtype == DSPARK_BF16 ? launch_tc<__nv_bfloat16>(p, ws, s) : launch_tc<float>(p, ws, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
