// cache_attend_tc.cu -- attention of the flat batch over the 4-bit cache on the fifth-generation tensor
// cores (dspark_cache_attend, bf16, D = 64 or 128, where requests have many rows).
//
//   out = sum_i 2^(t_i - m) v_i / sum_i 2^(t_i - m),  t_i = log2(e) scale q . k_i, in one pass over the keys.
//
// An item is 128 rows (query heads of consecutive queries) of one request and key / value head, a tile 128
// tokens. The items' tiles form one line that is cut into equal runs, one a CTA and SM, whatever the lengths
// are; a block's tiles are those its own rows reach. Per tile, by warp:
//   12 - 19 turn codes into fp16 (exact: scales have 8 bits) in shared memory, 16 bytes of them at a time, as they lie
//           in the cache: rows of tokens with the 128-byte swizzle, K-major for the keys and not for the values. The
//           next tile's codes are loaded before.
//   0       issues S = Q K^T (128 x 128 x D, operands in shared memory), a tile ahead.
//   1       issues O += P V (128 x D x 128, P in tensor memory).
//   4 - 11  one row a thread, even and odd items apart, so that one's end is under the other's tiles: the maximum,
//           weights 2^(t - m + 10) as fp16 into the tensor memory that S had, their sum. m only has to be near the
//           maximum: O is rescaled when a score passes m by 2^5.
//   2, 3, 20, 21  rows of q of the next item, scaled by a power of two into fp16's range, exactly, into shared memory.
// All waits are bounded by the global timer; one that runs out records DSPARK_ERR_TIMEOUT and ends the CTA's
// loops, its MMAs land, and tensor memory is freed.
//
// Bound: prompts need 4 D flops for each row and key, 59 us at the tensor cores' rate for 2 x 2048 rows of 32 heads after
// 650 tokens on average, and take 212; after 2000 tokens 108, and take 270 to 300. Few rows need the cache's bytes once,
// 54 us for 128 requests of up to 17 rows and 4096 tokens, and take 231 (28% tensor, 48% of the issue slots). A tile of
// few rows takes about 2700 cycles, whatever the rows are: one group's weights take 2100 to 2400 of them (four loads of
// tensor memory for the maximum, four for the weights, 330 cycles each, twice as long for the first because the loop's
// instructions have to come back), then its products and the next S follow in 300. Items of few tiles add the way of the
// next item's q rows (7000 cycles after its buffer is free, two buffers). Tried and slower: sixteen converting warps (64
// registers a thread), weights in one pass from scores kept apart from them, two threads a row (265 and 242 us: the fixed
// parts do not halve), the two groups on alternate tiles of an item (297 and 259 us: with both at work the conversion takes
// 2800 cycles a tile, and one O has to be read out between items), prefetches by the converting warps themselves, bulk
// prefetches (3 ms: they hold up the shared-memory fences), values transposed on their way into shared memory (276 us).
#include <algorithm>

#include "attend_convert.cuh"
#include "attend_plan.cuh"
#include "cache.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace dspark {

namespace {

constexpr int kTile = 128;                     // tokens
constexpr int kMB = 128;                       // rows of a block
constexpr int kThreads = 736;
constexpr int kWarpS = 0, kWarpPv = 1, kWarpSoft = 4, kWarpConv = 12, kWarpQ2 = 20, kWarpAhead = 22;
constexpr int kAhead = 4;    // tiles whose codes are under way
constexpr int kQWarps = 4;   // warps 2, 3 and kWarpQ2 on
constexpr unsigned long long kDrainNs = 4000000000ull;
// S of even tiles at 0, of odd tiles at 128; O of even items at 256, of odd items at 384
// (O's columns in the order of converted codes: channels 0 4 1 5 2 6 3 7 of every 8)
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
// instruction descriptors, kind::f16: D fp32, A and B fp16, M = 128; K-major but for V, whose channels are contiguous
constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kMB >> 4) << 24);
template <int D>
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kMB >> 4) << 24);

// ------------------------------------------------------------------ the line of tiles

struct Request {
    int first, n_q, ctx, keys, n_rows, blocks;
};

__device__ __forceinline__ Request request_of(const AttendParams& p, int r, bool report)
{
    const RequestSpan<kTile> s = request_span<kTile>(p, r, kMB, report);
    return Request{s.first, s.n_q, s.ctx, s.keys, s.n_q * p.G, s.blocks};
}

// The tiles of one block: those of the sinks, then those from its first query's window to its last query's
// own key (one range when they touch).
struct BlockTiles {
    int tiles, sink_tiles, lo_tile;
    __device__ __forceinline__ int key0(int u) const { return (u < sink_tiles ? u : lo_tile + u - sink_tiles) * kTile; }
};

__device__ __forceinline__ BlockTiles block_tiles(const AttendParams& p, const Request& q, int b)
{
    const int j0 = b * kMB / p.G, j1 = min((b + 1) * kMB - 1, q.n_rows - 1) / p.G;
    const int keys = (int)min((long long)q.keys, (long long)q.ctx + j1 + 1);
    BlockTiles t;
    const int all = tiles_of(keys, kTile);
    t.sink_tiles = t.lo_tile = 0;
    t.tiles = all;
    if (p.window > 0) {
        const int from = (int)max(0ll, (long long)q.ctx + j0 - p.window + 1);
        const int sink_tiles = (int)(((long long)min(p.sinks, from) + kTile - 1) / kTile), lo = from / kTile;
        if (sink_tiles < lo) {
            t.sink_tiles = sink_tiles;
            t.lo_tile = lo;
            t.tiles = sink_tiles + max(0, all - lo);
        }
    }
    t.tiles = max(t.tiles, 1);
    return t;
}

// Tiles of one head of request q; by a whole warp, or by one thread.
template <bool kWarpWide>
__device__ __forceinline__ int head_tiles(const AttendParams& p, const Request& q)
{
    int sum = 0;
    for (int b = kWarpWide ? (threadIdx.x & 31) : 0; b < q.blocks; b += kWarpWide ? 32 : 1) sum += block_tiles(p, q, b).tiles;
    return kWarpWide ? __reduce_add_sync(0xffffffffu, sum) : sum;
}

// pre[r] = tiles before request r's; the total is returned. All threads of the CTA.
__device__ __forceinline__ int plan(const AttendParams& p, int* pre, long long* scan, bool report)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = p.c.R;
    if (R <= 64) {   // few requests, perhaps of many blocks: a warp each
        for (int r = warp; r < R; r += kThreads / 32) {
            const int n = head_tiles<true>(p, request_of(p, r, report && lane == 0)) * p.c.Hkv;
            if (lane == 0) pre[r + 1] = n;
        }
    } else {
        for (int r = tid; r < R; r += kThreads) pre[r + 1] = head_tiles<false>(p, request_of(p, r, report)) * p.c.Hkv;
    }
    __syncthreads();
    const int each = (R + kThreads - 1) / kThreads, r0 = min(tid * each, R), r1 = min(r0 + each, R);
    long long sum = 0;
    for (int r = r0; r < r1; ++r) sum += pre[r + 1];
    return sum_line<kThreads>(p, r0, r1, sum, pre, scan, report);
}

// Items of a run one after the other: request r, head h, block b, from tile u on. Warp-wide; not inlined,
// since the four roles' code has to stay in the instruction cache.
struct Walk {
    int r = 0, h = 0, b = 0, u = 0;
    Request q;
    BlockTiles t;
    __device__ __noinline__ void start(const AttendParams& p, const int* pre, int at)
    {
        int lo = 0, hi = p.c.R;   // the request with pre[r] <= at < pre[r + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= at) lo = mid;
            else hi = mid;
        }
        r = lo;
        q = request_of(p, r, false);
        const int per_head = (pre[r + 1] - pre[r]) / p.c.Hkv;
        h = (at - pre[r]) / per_head;
        int rem = (at - pre[r]) % per_head;
        for (int b0 = 0; b0 < q.blocks; b0 += 32) {
            const int lane = threadIdx.x & 31;
            const int n = b0 + lane < q.blocks ? block_tiles(p, q, b0 + lane).tiles : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, rem < inc);
            if (past) {
                const int k = __ffs(past) - 1;
                b = b0 + k;
                u = rem - __shfl_sync(0xffffffffu, inc - n, k);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, inc, 31);
        }
        t = block_tiles(p, q, b);
    }
    __device__ __noinline__ void advance(const AttendParams& p, const int* pre)
    {
        u = 0;
        if (++b == q.blocks) {
            b = 0;
            if (++h == p.c.Hkv) {
                h = 0;
                do ++r;
                while (r + 1 < p.c.R && pre[r + 1] == pre[r]);
                q = request_of(p, r, false);
            }
        }
        t = block_tiles(p, q, b);
    }
};

// ------------------------------------------------------------------ waits

// A waiting warp is suspended by its try for up to kNap and then looks at the timer and the abort flag. The time of a
// try is a hint that a suspension may pass, so under a limit below kNap tries do not suspend.
constexpr uint32_t kNapNs = 100000;

__device__ __forceinline__ bool try_for(uint32_t bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                       unsigned long long limit_ns)
{
    const unsigned long long t0 = globaltimer();
    while (!(limit_ns < kNapNs ? mbar_test_wait(bar, parity) : try_for(bar, parity, kNapNs))) {
        if (*abort) return false;
        if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            raise_status(status, DSPARK_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same for a count in shared memory that another warp raises to `least`. Inline: called, it cost the verify batch 3 us.
__device__ __forceinline__ bool wait_count(const volatile int* count, int least, volatile int* abort, int* status,
                                           unsigned long long limit_ns)
{
    bool ok = true;
    const unsigned long long t0 = globaltimer();
    while (ok && *count < least) {
        if (*abort) ok = false;
        if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            raise_status(status, DSPARK_ERR_TIMEOUT);
            ok = false;
        }
        __nanosleep(100);
    }
    return ok;
}

// Warp-wide: true where every lane saw the phase end.
struct Waits {
    volatile int* abort;
    int* status;
    unsigned long long limit_ns;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        const bool ok = mbar_test_wait(bar, parity) || wait_slow(bar, parity, abort, status, limit_ns);
        return __all_sync(0xffffffffu, ok);
    }
    __device__ __forceinline__ bool reaches(const volatile int* count, int least) const
    {
        return __all_sync(0xffffffffu, wait_count(count, least, abort, status, limit_ns));
    }
};

__device__ __noinline__ void drain(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kDrainNs) {
    }
}

__device__ __forceinline__ void store16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 load16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Query and head in the group of the rows of a block. The quotients by G of numbers below 2048 come by a
// multiplication: g_magic = ceil(2^32 / G), off by less than G <= 1024, is exact there.
struct RowMap {
    int j0, g0, G;
    uint32_t magic;
    __device__ __forceinline__ RowMap(int row0, int G_, uint32_t m) : j0(row0 / G_), g0(row0 % G_), G(G_), magic(m) {}
    __device__ __forceinline__ void at(int row, int& j, int& g) const
    {
        const int x = g0 + row, q = magic == 0 ? x : (int)__umulhi((uint32_t)x, magic);
        j = j0 + q;
        g = x - q * G;
    }
};

// 8 channels of a row of q off 16-byte boundaries
__device__ __forceinline__ uint4 load_halves(const __nv_bfloat16* src)
{
    const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// Barriers, pairs by the parity of the tile (Q: of the item) first. A waiter is never two phases behind: each
// phase needs an arrival that the waiter, or one that waits for it, makes after it saw the phase before.
enum Bar {
    kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kQFull = 8,
    kFree = 10,     // an item's products are done and its rows are out of q's buffer
    kSFull = 12, kPFull = 14,
    kPvDone = 16,   // O += P V of a tile has landed
    kODone = 18,    // that of an item's last tile in this run; by the item's parity, as the next three
    kOFree = 20,    // the item's rows are out of O
    kBegun = 22,    // the item's first S is issued
    kFin = 24,
    kRun = 26,      // where a tile's codes are is in s_run
    kBars = 34
};

// Where 16 tokens of a tile lie: their first key's codes, from there on to its scale, and how many hold something.
struct Run {
    const uint8_t* codes;
    int scales, left;
};

// The codes of a tile that one converting thread takes, of keys and of values: 32 channels of one token for every
// 64 channels of a head, with their scales.
template <int D>
struct Raw {
    uint4 k[D / 64], v[D / 64];
    uint16_t ks[D / 64], vs[D / 64];
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attend_tc_kernel(AttendParams p, AttendScratch ws, unsigned long long wait_ns)
{
    constexpr uint32_t kOperand = 128 * D * 2;   // bytes of Q, K or V of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t q_buf = smem_addr(smem), k_buf = q_buf + 2 * kOperand, v_buf = q_buf + 4 * kOperand;
    int* s_pre = reinterpret_cast<int*>(smem + 6 * kOperand);
    __shared__ uint64_t s_bar[kBars];
    __shared__ float s_fac[2][kMB];
    __shared__ __align__(8) uint8_t s_valid[4][8];   // of tile n & 3: which runs of 16 tokens hold keys
    __shared__ long long s_scan[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ __align__(16) Run s_run[8][8];       // of tile n & 7, by converting warp
    __shared__ int s_done;                           // tiles whose keys the first converting warp is through with
    __shared__ AttendTodo s_todo[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar0 = smem_addr(s_bar);
    auto bar = [&](int k) { return bar0 + 8u * k; };
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(kKFull + b), 8);
            mbar_init(bar(kVFull + b), 8);
            mbar_init(bar(kKEmpty + b), 1);
            mbar_init(bar(kVEmpty + b), 1);
            mbar_init(bar(kQFull + b), kQWarps);
            mbar_init(bar(kFree + b), 4);
            mbar_init(bar(kSFull + b), 2);    // its MMAs, and the issuing thread for what it saw (s_valid)
            mbar_init(bar(kPFull + b), 4);
            mbar_init(bar(kPvDone + b), 1);
            mbar_init(bar(kFin + b), 1);
            mbar_init(bar(kODone + b), 1);
            mbar_init(bar(kOFree + b), 4);
            mbar_init(bar(kBegun + b), 1);
        }
        s_abort = 0;
        s_done = 0;
        for (int b = 0; b < 8; ++b) mbar_init(bar(kRun + b), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == kWarpPv) tc5::alloc(&s_tmem, kTmemCols);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();
    const int total = plan(p, s_pre, s_scan, blockIdx.x == 0);
    const int per = (int)(((long long)total + gridDim.x - 1) / gridDim.x);
    const int begin = (int)min((long long)blockIdx.x * per, (long long)total);
    const int end = (int)min((long long)begin + per, (long long)total);
    const Waits wait{&s_abort, p.status, wait_ns};
    AttendTodo todo = {};

    if (begin < end && warp == kWarpS) {
        // ---------------- S = Q K^T
        Walk w;
        w.start(p, s_pre, begin);
        const uint64_t q_desc = tc5::desc_sw128(q_buf), k_desc = tc5::desc_sw128(k_buf);
        bool ok = true;
        int n = 0;
        for (int at = begin, item = 0; at < end && ok; ++item) {
            const int tiles = min(w.t.tiles - w.u, end - at);
            ok = wait(bar(kQFull + (item & 1)), (item >> 1) & 1u);
            for (int u = 0; u < tiles && ok; ++u, ++n) {
                const int b = n & 1;
                if (!wait(bar(kKFull + b), (n >> 1) & 1u)) ok = false;
                if (ok && n >= 2 && !wait(bar(kPvDone + b), ((n >> 1) - 1) & 1u)) ok = false;   // S replaces its weights
                if (!ok) break;
                tc5::fence_after();
                // the start address of a descriptor counts 16 bytes: 16 K elements on are 2
                const uint64_t qd = q_desc + (uint64_t)((item & 1) * (kOperand >> 4)), kd = k_desc + (uint64_t)(b * (kOperand >> 4));
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tc5::mma_ss4_warp<2, 2>(tmem + b * 128, qd + c * (16384 / 16), kd + c * (16384 / 16), kIdescS, c);
                tc5::commit_warp(bar(kSFull + b));
                tc5::commit_warp(bar(kKEmpty + b));
                if (lane == 0) {
                    mbar_arrive(bar(kSFull + b));
                    if (u == 0) mbar_arrive(bar(kBegun + (item & 1)));
                }
                __syncwarp();
            }
            at += tiles;
            if (at < end) w.advance(p, s_pre);
        }
        // every MMA issued above lands before tensor memory is freed
        tc5::commit_warp(bar(kFin));
        drain(bar(kFin), 0u);
        __syncwarp();
    } else if (begin < end && warp == kWarpPv) {
        // ---------------- O (+)= P V
        Walk w;
        w.start(p, s_pre, begin);
        const uint64_t v_desc = tc5::desc_sw128_mn(v_buf, 16384);
        bool ok = true;
        int n = 0;
        for (int at = begin, item = 0; at < end && ok; ++item) {
            const int tiles = min(w.t.tiles - w.u, end - at);
            for (int u = 0; u < tiles && ok; ++u, ++n) {
                const int b = n & 1;
                if (!wait(bar(kVFull + b), (n >> 1) & 1u) || !wait(bar(kPFull + b), (n >> 1) & 1u)) ok = false;
                if (ok && u == 0 && item >= 2 && !wait(bar(kOFree + (item & 1)), ((item >> 1) - 1) & 1u)) ok = false;
                if (!ok) break;
                tc5::fence_after();
                const uint64_t vd = v_desc + (uint64_t)(b * (kOperand >> 4));   // 16 tokens on are 16 rows of 128 bytes
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tc5::mma_ts4_warp<2048 / 16>(tmem + kTmemO + (item & 1) * 128, tmem + b * 128 + c * 32,
                                                 vd + c * (8192 / 16), kIdescO<D>, c > 0 || u > 0);
                tc5::commit_warp(bar(kPvDone + b));
                tc5::commit_warp(bar(kVEmpty + b));
                if (u + 1 == tiles) tc5::commit_warp(bar(kODone + (item & 1)));
            }
            at += tiles;
            if (at < end) w.advance(p, s_pre);
        }
        tc5::commit_warp(bar(kFin + 1));
        drain(bar(kFin + 1), 0u);
        __syncwarp();
    } else if (begin < end && (warp == 2 || warp == 3 || warp == kWarpQ2 || warp == kWarpQ2 + 1)) {
        // ---------------- rows of q, one item ahead
        Walk w;
        w.start(p, s_pre, begin);
        const float to_log2 = p.scale * kLog2e;
        constexpr int kLanes = D / 8, kRows = 32 / kLanes;   // a row of D channels is D / 8 lanes
        constexpr int kFlight = 8;                           // loads in flight
        const int c = lane % kLanes, sub = (warp < 4 ? warp - 2 : warp - kWarpQ2 + 2) * kRows + lane / kLanes;
        bool ok = true;
        for (int at = begin, item = 0; at < end && ok; ++item) {
            const int tiles = min(w.t.tiles - w.u, end - at), b = item & 1;
            const RowMap map(w.b * kMB, p.G, p.g_magic);
            const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)w.q.first * p.q_ts +
                                      (int64_t)w.h * p.G * p.q_hs + c * 8;
            const int left = min(kMB, w.q.n_rows - w.b * kMB);
#pragma unroll 1
            for (int r = sub; r < kMB && ok; r += kFlight * kQWarps * kRows) {
                uint4 v[kFlight];
                if (p.q_aligned) {   // one test for all: a test each would make the loads wait for one another
#pragma unroll
                    for (int e = 0; e < kFlight; ++e) {
                        const int row = r + e * kQWarps * kRows;
                        int j, g;
                        map.at(min(row, left - 1), j, g);
                        v[e] = *reinterpret_cast<const uint4*>(q0 + (int64_t)j * p.q_ts + (int64_t)g * p.q_hs);
                    }
                } else {
#pragma unroll 1
                    for (int e = 0; e < kFlight; ++e) {
                        const int row = r + e * kQWarps * kRows;
                        int j, g;
                        map.at(min(row, left - 1), j, g);
                        const uint4 y = load_halves(q0 + (int64_t)j * p.q_ts + (int64_t)g * p.q_hs);
#pragma unroll
                        for (int k = 0; k < kFlight; ++k)
                            if (k == e) v[k] = y;
                    }
                }
                // the buffer is free when the rows of the item two before are out of it; the first loads are under way
                if (r == sub && item >= 2) ok = wait(bar(kFree + b), ((item >> 1) - 1) & 1u);
                if (!ok) break;
                // magnitudes of bf16 order like their bits, two at a time; the rows' shuffles side by side
                uint32_t two[kFlight];
#pragma unroll
                for (int e = 0; e < kFlight; ++e)
                    two[e] = __vmaxu2(__vmaxu2(v[e].x & 0x7FFF7FFFu, v[e].y & 0x7FFF7FFFu),
                                      __vmaxu2(v[e].z & 0x7FFF7FFFu, v[e].w & 0x7FFF7FFFu));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int e = 0; e < kFlight; ++e) two[e] = __vmaxu2(two[e], __shfl_xor_sync(0xffffffffu, two[e], o));
#pragma unroll
                for (int e = 0; e < kFlight; ++e) {
                    const int row = r + e * kQWarps * kRows;
                    const uint32_t x[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
                    const uint32_t top = max(two[e] & 0xFFFFu, two[e] >> 16);
                    const bool bad = top >= 0x7F80u;   // an infinity or NaN
                    const float up = row_up((int)(top >> 7));
                    if (c == 0) {
                        if (bad && row < left) raise_status(p.status, DSPARK_ERR_NONFINITE_INPUT);
                        // a row that is not finite has the factor NaN and so weights, sum and result; rows past
                        // the request's repeat its last one and are not written
                        s_fac[b][row] = bad ? NAN : row_factor(to_log2, up);
                    }
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = __uint_as_float(x[k] << 16) * up;
                        f[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u) * up;
                    }
                    // in the order of converted codes: channels 0 4 1 5 2 6 3 7
                    store16(q_buf + b * kOperand + (c / 8) * 16384 + row * 128 + (((c % 8) ^ (row & 7)) * 16), pack(f[0], f[4]),
                            pack(f[1], f[5]), pack(f[2], f[6]), pack(f[3], f[7]));
                }
            }
            if (!ok) break;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQFull + b));
            at += tiles;
            if (at < end) w.advance(p, s_pre);
        }
    } else if (begin < end && warp == kWarpAhead) {
        // ---------------- where the codes of the tiles to come are, and they themselves into the L2 cache: what the
        // converting warps have under way, 18 KB an SM, the memory's latency alone would keep below 2.5 TB/s
        Walk w;
        w.start(p, s_pre, begin);
        const CacheBlock cb = cache_block(p.c.page_size, D);
        const int slice = lane >> 2, sub = lane & 3;   // 16 tokens, and part of their lines
        const int tiles = end - begin, magic = p.page_magic, P = p.c.page_size;
        BlockTiles it = w.t;   // in registers: the walk's memory is swept out of the L1 cache by the codes
        int u = w.u, keys = w.q.keys, h = w.h, key, page;
        const int32_t* row = p.c.table + (size_t)w.r * p.c.table_width;
        auto look_up = [&]() {
            key = it.key0(u) + slice * 16;
            page = key < keys ? row[page_of(key, magic)] : -1;
        };
        look_up();
#pragma unroll 1
        for (int n = 0; n < tiles; ++n) {
            // An entry is free when tile n - 8 is: the first warp is past the keys of tile n - 5, the others past those
            // of tile n - 7, or it would have waited for them.
            if (!wait.reaches(&s_done, n - kAhead)) break;
            __threadfence_block();
            const int left = keys - key, slot = key - page_of(key, magic) * P;
            const bool in = page >= 0 && page < p.c.n_pages;
            if (left > 0 && !in && sub == 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
            const uint8_t* blk = cache_page_block(p.c, in ? page : 0, h, cb.bytes);
            if (sub == 0)
                s_run[n & 7][slice] = Run{blk + slot * (D / 2), (int)cb.k_scales + slot * (D / 16) - slot * (D / 2), in ? left : 0};
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kRun + (n & 7)));
            if (in) {
                const uint8_t* k = blk + slot * (D / 2) + sub * 128;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    prefetch_l2(k + c * 512);
                    prefetch_l2(k + cb.v_codes + c * 512);
                }
                if (sub < 2) prefetch_l2(blk + (sub ? cb.v_scales : cb.k_scales) + slot * (D / 16));
            }
            if (n + 1 < tiles) {
                if (++u == it.tiles) {
                    w.advance(p, s_pre);
                    u = 0;
                    it = w.t;
                    keys = w.q.keys;
                    h = w.h;
                    row = p.c.table + (size_t)w.r * p.c.table_width;
                }
                look_up();
            }
        }
    } else if (begin < end && warp >= kWarpConv) {
        // ---------------- codes to fp16
        // A warp has 16 tokens, all in one page; 16 bytes of codes and a scale are 32 channels and become 4 units of
        // 16 bytes. D = 128: lane / 4 is one of 8 tokens, twice; 64: lane / 2 one of the 16. Loads are contiguous. Of
        // the 8 lanes that store at a time those of one token have two pairs with the same banks, so that one pair
        // takes its units in another order (flip), and the two tokens are ones whose orders do not meet either.
        constexpr int kUnits = D / 64, kQ = D / 32;
        const int cw = warp - kWarpConv, qc = lane % kQ, l4 = lane / kQ;
        const int tok = D == 128 ? (l4 & 4) | (0x9C >> (2 * (l4 & 3)) & 3) : l4;   // 0 3 1 2 4 7 5 6
        const bool flip = D == 128 && qc >= 2;
        const uint32_t own = (D == 128 ? (qc >> 1) * 16384 : 0) + (cw * 16 + tok) * 128 + (((((qc & 1) * 4) ^ (tok & 7)) * 16) ^ (flip ? 16u : 0u));
        const CacheBlock cb = cache_block(p.c.page_size, D);
        const uint32_t to_scale = tok * (D / 16) + qc * 2, to_v_scale = cb.v_scales - cb.k_scales + qc * 32 + tok * 2;
        const uint32_t to_code = tok * (D / 2) + qc * 16;
        const DequantConst dq = dequant_const();
        Raw<D> x;
        Run run;
        // Loads without a condition, from page 0 where there is none: what is merged into their registers after them
        // would wait for them.
        auto load_k = [&](int n) {
            run = s_run[n & 7][cw];
            const uint8_t* from = run.codes + to_code;
            const uint8_t* scale = run.codes + run.scales + to_scale;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                x.k[i] = *reinterpret_cast<const uint4*>(from + i * (8 * D / 2));
                x.ks[i] = *reinterpret_cast<const uint16_t*>(scale + i * (8 * D / 16));
            }
        };
        auto load_v = [&]() {
            const uint8_t* from = run.codes + cb.v_codes + to_code;
            const uint8_t* scale = run.codes + run.scales + to_v_scale;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                x.v[i] = *reinterpret_cast<const uint4*>(from + i * (8 * D / 2));
                x.vs[i] = *reinterpret_cast<const uint16_t*>(scale + i * 16);
            }
        };
        // what no token wrote may be anything: its scale becomes 0
        auto put = [&](uint32_t dst, const uint4 (&codes)[D / 64], const uint16_t (&scale)[D / 64], int n_in) {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const uint32_t sc = i * 8 + tok < n_in ? scale[i] : 0u;
                const __half2 s2 = as_half2(sc | (sc << 16));
                const uint32_t c4[4] = {flip ? codes[i].y : codes[i].x, flip ? codes[i].x : codes[i].y,
                                        flip ? codes[i].w : codes[i].z, flip ? codes[i].z : codes[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t h[4];
                    dequant(c4[c], s2, dq, h);
                    store16((dst + own + i * 1024) ^ (c * 16), h[0], h[1], h[2], h[3]);
                }
            }
            fence_proxy_async();
            __syncwarp();
        };
        const int tiles = end - begin;
        if (wait(bar(kRun), 0u)) {
            load_k(0);
            load_v();
#pragma unroll 1
            for (int n = 0; n < tiles; ++n) {
                // The registers that a conversion frees take the next tile's codes at once: their way is as long as
                // the other conversion and the waits. (A second set that is copied at the loop's end stops there for
                // the loads instead.)
                const int b = n & 1, n_in = run.left, next = min(n + 1, tiles - 1);
                if (n >= 2 && !wait(bar(kKEmpty + b), ((n >> 1) - 1) & 1u)) break;
                put(k_buf + b * kOperand, x.k, x.ks, n_in);
                if (lane == 0) {
                    s_valid[n & 3][cw] = n_in > 0;
                    mbar_arrive(bar(kKFull + b));
                    if (cw == 0) {
                        __threadfence_block();
                        *(volatile int*)&s_done = n + 1;
                    }
                }
                if (!wait(bar(kRun + (next & 7)), (next >> 3) & 1u)) break;
                load_k(next);
                if (n >= 2 && !wait(bar(kVEmpty + b), ((n >> 1) - 1) & 1u)) break;
                put(v_buf + b * kOperand, x.v, x.vs, n_in);
                if (lane == 0) mbar_arrive(bar(kVFull + b));
                load_v();
            }
        }
    } else if (begin < end && warp >= kWarpSoft) {
        // ---------------- weights: one row a thread
        const int grp = (warp - kWarpSoft) >> 2, quarter = (warp - kWarpSoft) & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16), o_at = lanes + kTmemO + grp * 128;
        Walk w;
        w.start(p, s_pre, begin);
        bool ok = true;
        int n = 0;
        for (int at = begin, item = 0; at < end; ++item) {
            const int u0 = w.u, u1 = min(w.t.tiles, u0 + (end - at));
            const int row0 = w.b * kMB, rr = row0 + row;
            if ((item & 1) != grp) {   // the other group's
                n += u1 - u0;
                at += u1 - u0;
                if (at < end) w.advance(p, s_pre);
                continue;
            }
            const bool any = row0 + quarter * 32 < w.q.n_rows;   // the warp has rows of the item
            // the factors are there; and with the item's first S issued the barriers of S are at its tiles
            ok = wait(bar(kQFull + grp), (item >> 1) & 1u) && wait(bar(kBegun + grp), (item >> 1) & 1u);
            if (!ok) break;
            const float fac = s_fac[item & 1][row];
            const uint64_t fac2 = pack2(fac, fac);
            // keys this row sees: from lo (and below the sinks) to hi
            const int own = w.q.ctx + min(rr, w.q.n_rows - 1) / p.G;
            const int hi = min(own, w.q.keys - 1);
            const int lo = p.window > 0 ? (int)max(0ll, (long long)own - p.window + 1) : 0;
            // tiles from in_lo to in_hi are seen by every row to their ends
            const int pos_lo = w.q.ctx + row0 / p.G, pos_hi = w.q.ctx + min(row0 + kMB - 1, w.q.n_rows - 1) / p.G;
            const int in_hi = min(pos_lo, w.q.keys - 1) - (kTile - 1);
            const int in_lo = p.window > 0 ? (int)max(0ll, (long long)pos_hi - p.window + 1) : 0;
            const BlockTiles it = w.t;   // in registers: the walk's memory is swept out of the L1 cache by the codes
            float top = -INFINITY, sum = 0.f;
            for (int u = u0; u < u1; ++u, ++n) {
                const int b = n & 1, key0 = it.key0(u);
                ok = wait(bar(kSFull + b), (n >> 1) & 1u);
                if (!ok) break;
                if (any) {
                    tc5::fence_after();
                    const uint32_t s_at = lanes + b * 128;
                    const unsigned long long valid = *reinterpret_cast<const unsigned long long*>(s_valid[n & 3]);
                    const bool edge = key0 > in_hi || key0 < in_lo || valid != 0x0101010101010101ull;
                    auto seen = [&](int c) {   // bit j: key key0 + 32 c + j is visible
                        const int base = key0 + c * 32;
                        const uint32_t v = ((valid >> (16 * c)) & 1u ? 0xFFFFu : 0u) |
                                           ((valid >> (16 * c + 8)) & 1u ? 0xFFFF0000u : 0u);
                        return below(hi + 1 - base) & (~below(lo - base) | below(p.window > 0 ? p.sinks - base : 0)) & v;
                    };
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // four chains
                    uint32_t x[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tc5::ld32(s_at + c * 32, x);
                        if (edge) {   // hidden scores become -infinity, there too
                            const uint32_t see = seen(c);
                            uint32_t y[16];
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    y[j] = x[hf * 16 + j] = (see >> (hf * 16 + j)) & 1u ? x[hf * 16 + j] : 0xFF800000u;
                                tc5::st16(s_at + c * 32 + hf * 16, y);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(x[j]));
                    }
                    if (edge) tc5::wait_st();
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fac;
                    if (u == u0) {
                        top = mx == mx ? mx : -INFINITY;   // NaN: a row that is not finite
                    } else if (__any_sync(0xffffffffu, mx > top + kSlack)) {
                        const float m = fmaxf(mx, top);
                        const float keep = m == top ? 1.f : ex2(top - m);
                        top = m;
                        sum *= keep;
                        ok = wait(bar(kPvDone + (b ^ 1)), ((n - 1) >> 1) & 1u);
                        if (!ok) break;
                        tc5::fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            tc5::ld16(o_at + c * 16, y);
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * keep);
                            tc5::st16(o_at + c * 16, y);
                        }
                    }
                    const float base = top == -INFINITY ? 0.f : kShift - top;
                    const uint64_t base2 = pack2(base, base);
                    uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tc5::ld32(s_at + c * 32, x);
                        uint32_t y[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float t0, t1;
                            unpack2(fma2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), fac2, base2), t0, t1);
                            const float e0 = ex2(t0), e1 = ex2(t1);
                            sum2[j & 1] = add2(sum2[j & 1], pack2(e0, e1));
                            y[j] = pack(e0, e1);
                        }
                        tc5::st16(s_at + c * 16, y);   // over scores that this thread has read
                    }
                    tc5::wait_st();
                    tc5::fence_before();
                    float s0, s1;
                    unpack2(add2(sum2[0], sum2[1]), s0, s1);
                    sum += s0 + s1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + b));
            }
            if (!ok) break;
            // ---------------- the item's end in this run
            const bool whole = u0 == 0 && u1 == w.t.tiles;
            const int slot = at == begin ? 0 : 1;   // a run's first item, or its last
            // warps without rows wait too: their arrivals below must not count for the item before
            ok = wait(bar(kODone + grp), (item >> 1) & 1u);
            if (!ok) break;
            if (any) {
                tc5::fence_after();
                const bool real = rr < w.q.n_rows;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                if (whole) {
                    // rows as bf16 into q's buffer, whose products are done, each row's 16-byte units turned by
                    // the row, and out from there in whole pieces
                    const uint32_t stage = q_buf + grp * kOperand + (uint32_t)quarter * 32 * (D * 2);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t x[32];
                        tc5::ld32(o_at + c * 32, x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {   // channels 2 e and 2 e + 1
                                const int at = 8 * k + (e & 1) * 4 + (e >> 1);
                                const __nv_bfloat162 v =
                                    __floats2bfloat162_rn(__uint_as_float(x[at]) * inv, __uint_as_float(x[at + 2]) * inv);
                                y[e] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                            store16(stage + lane * (D * 2) + (((c * 4 + k) ^ (lane & 7)) * 16), y[0], y[1], y[2], y[3]);
                        }
                    }
                    tc5::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kOFree + grp));
                    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
                    const RowMap map(row0, p.G, p.g_magic);
                    const int c = lane % kLanes, left = min(32, w.q.n_rows - row0 - quarter * 32);
                    __nv_bfloat16* o0 = static_cast<__nv_bfloat16*>(p.out) + ((size_t)w.q.first * p.Hq + w.h * p.G) * D + c * 8;
#pragma unroll 4
                    for (int r = lane / kLanes; r < left; r += kRows) {
                        int j, g;
                        map.at(quarter * 32 + r, j, g);
                        *reinterpret_cast<uint4*>(o0 + ((size_t)j * p.Hq + g) * D) = load16(stage + r * (D * 2) + ((c ^ (r & 7)) * 16));
                    }
                    if (real && p.lse) {
                        p.lse[(size_t)(w.q.first + rr / p.G) * p.Hq + w.h * p.G + rr % p.G] =
                            sum == 0.f ? -INFINITY : (top + log2f(sum) - kShift) * kLn2;
                    }
                    __syncwarp();
                } else {
                    const size_t part = ((size_t)blockIdx.x * 2 + slot) * kMB + row;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t x[32];
                        tc5::ld32(o_at + c * 32, x);
                        if (real) {
                            uint4* o = reinterpret_cast<uint4*>(ws.rows + part * D + c * 32);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int at = (k / 2) * 8 + k % 2;
                                o[k] = make_uint4(x[at], x[at + 2], x[at + 4], x[at + 6]);
                            }
                        }
                        __syncwarp();
                    }
                    if (real) ws.ml[part] = make_float2(top, sum);
                    tc5::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kOFree + grp));
                }
            } else if (lane == 0) {
                mbar_arrive(bar(kOFree + grp));
            }
            if (lane == 0) mbar_arrive(bar(kFree + grp));
            // an item that starts here and goes on: the next kernel joins its parts
            if (u0 == 0 && u1 < w.t.tiles) {
                todo.parts = (at + w.t.tiles - 1) / per - (int)blockIdx.x + 1;
                todo.slot = slot;
                todo.first = w.q.first;
                todo.head = w.h;
                todo.row0 = row0;
                todo.rows = min(kMB, w.q.n_rows - row0);
            }
            at += u1 - u0;
            if (at < end) w.advance(p, s_pre);
        }
        if (!ok) todo.parts = 0;
    }
    if (warp == kWarpSoft || warp == kWarpSoft + 4) {
        // the group that had the run's last item has the note
        if (lane == 0) s_todo[(warp - kWarpSoft) >> 2] = todo;
    }
    tc5::fence_before();
    __syncthreads();
    if (tid == 0) ws.todo[blockIdx.x] = s_abort ? AttendTodo{} : s_todo[s_todo[1].parts > 0];
    if (warp == kWarpPv) {
        tc5::fence_after();
        tc5::dealloc(tmem, kTmemCols);
    }
}

constexpr size_t kStatic = 4096;   // more than the kernel's fixed shared memory
constexpr size_t kMostSmem = 227 * 1024 - kStatic;

template <int D>
size_t tc_smem(int R) { return 6 * 128 * D * 2 + sizeof(int) * (R + 1) + 1024; }

template <int D>
cudaError_t launch_tc(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    static std::atomic<uint64_t> admitted{0};
    const cudaError_t e = admit_smem(cache_attend_tc_kernel<D>, kMostSmem, admitted);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attend_tc_kernel<D>, dim3(ws.runs), dim3(kThreads), tc_smem<D>(p.c.R), s, p, ws,
                      wait_limit_ns());
}

}  // namespace

bool attend_tc_supported(const AttendParams& p)
{
    if (p.dtype != DSPARK_BF16 || (p.c.D != 64 && p.c.D != 128)) return false;
    // A tile costs the same here for 1 row and for 128, and an item as much again as some tiles; the warp kernel's tiles
    // cost by blocks of 16 rows, its items little. 128 requests of up to 4096 tokens, 4 query heads a key head: 36 rows
    // 232 us here and 198 there, 48 rows 234 and 231, 64 rows 234 and 283, 128 rows 245 and 469; 8 requests of up to
    // 8192: 48 rows 47 and 46, 64 rows 48 and 58. Where a row reaches few keys the warp kernel holds out longer: 32
    // requests of up to 2048 tokens, 48 rows 61 and 52, 68 rows 62 and 58, 128 rows 68 and 85; a window of 512 keys, 48
    // rows 75 and 50, 68 rows 78 and 59, 128 rows 84 and 94. The lengths are on the device, so what a row can reach goes by
    // the table's width: requests far shorter than their tables take this kernel where the other would be quicker.
    const long long rows = (long long)p.max_q * p.G, room = (long long)p.c.table_width * p.c.page_size;
    const long long reach = p.window > 0 ? std::min(room, (long long)p.window + p.sinks) : room;
    if (rows <= (reach <= 18 * kTile ? 80 : 48)) return false;
    if ((p.c.D == 64 ? tc_smem<64>(p.c.R) : tc_smem<128>(p.c.R)) > kMostSmem) return false;
    return tiles_fit(p, kMB, kTile);
}

int attend_tc_block_rows() { return kMB; }

cudaError_t launch_cache_attend_tc(const AttendParams& p, const AttendScratch& ws, cudaStream_t s)
{
    const cudaError_t e = p.c.D == 64 ? launch_tc<64>(p, ws, s) : launch_tc<128>(p, ws, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
