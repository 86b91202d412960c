// attend_plan.cuh -- how the matrix kernels of dspark_cache_attend lay the keys of all requests, heads and
// row blocks out as one line of tiles of TILE tokens, from the lengths on the device.
#pragma once

#include "cache.cuh"
#include "internal.h"

namespace dspark {

// Tiles are counted in 32 bits, with room for what a run looks ahead.
constexpr long long kMostTiles = (1ll << 31) - 65536;

// Whether they suffice for T rows of which a request has at most max_q, in blocks of MB, and tiles of `tile` tokens: a
// request's blocks are those of its rows and one more. Offsets that count rows twice may ask for more than this says;
// the plan looks again.
inline bool tiles_fit(const AttendParams& p, int MB, int tile)
{
    const long long rows = (long long)(p.max_q < p.T ? p.max_q : p.T) * p.G, all = (long long)p.T * p.G / MB + p.c.R;
    const long long each = p.c.R * (rows / MB + 1), blocks = each < all ? each : all;
    const long long tiles = ((long long)p.c.table_width * p.c.page_size + tile - 1) / tile + 1;
    return rows < (1ll << 30) && (double)blocks * p.c.Hkv * (double)tiles < (double)kMostTiles;
}

// Tiles of `keys` tokens, which may be as many as an int counts
__device__ __forceinline__ int tiles_of(int keys, int tile) { return (int)(((uint32_t)keys + tile - 1) / tile); }

// The item that a run starts and does not end: its rows, and how many runs have parts of it (0: none).
struct __align__(16) AttendTodo {
    int parts, slot;               // and the run's slot that holds the first
    int first, head, row0, rows;   // flat row of the request, key / value head, first row and rows of the block
    int pad[2];
};

// What a run leaves of items that other runs share.
struct AttendScratch {
    float* rows;    // [runs][2][block rows][D] weighted sums
    float2* ml;     // [runs][2][block rows] maximum (log2 units) and sum of the weights
    AttendTodo* todo;   // [runs]
    int runs, block_rows;
};

// A request's rows and the tiles its queries reach: the tiles of the sinks, then those from the first
// query's window on (one range when they touch).
template <int TILE>
struct RequestSpan {
    int first, n_q, ctx, keys, tiles, sink_tiles, lo_tile, blocks;
    __device__ __forceinline__ int key0(int u) const
    {
        return (u < sink_tiles ? u : lo_tile + u - sink_tiles) * TILE;
    }
};

template <int TILE>
__device__ __forceinline__ RequestSpan<TILE> request_span(const AttendParams& p, int r, int MB, bool report)
{
    RequestSpan<TILE> s;
    const int a = p.offsets[r], b = p.offsets[r + 1], ctx = p.c.ctx_len[r];
    const int last = min(b, p.T);
    bool odd = a < 0 || b < a || b > p.T || ctx < 0;
    s.first = a;
    s.n_q = a < 0 || ctx < 0 ? 0 : max(0, last - a);
    if (s.n_q > p.max_q) {
        odd = true;
        s.n_q = p.max_q;
    }
    s.ctx = ctx;
    const int cap = p.c.table_width * p.c.page_size;
    long long keys = (long long)ctx + s.n_q;
    if (s.n_q > 0 && keys > cap) {
        odd = true;
        keys = cap;
    }
    if (odd && report) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
    s.keys = s.n_q > 0 ? (int)keys : 0;
    const int all = tiles_of(s.keys, TILE);
    s.sink_tiles = s.lo_tile = 0;
    s.tiles = all;
    if (p.window > 0 && s.n_q > 0) {
        const int from = (int)max(0ll, (long long)ctx - p.window + 1);
        const int sink_tiles = (int)(((long long)min(p.sinks, from) + TILE - 1) / TILE), lo = from / TILE;
        if (sink_tiles < lo) {
            s.sink_tiles = sink_tiles;
            s.lo_tile = lo;
            s.tiles = sink_tiles + max(0, all - lo);
        }
    }
    s.tiles = max(s.tiles, 1);
    s.blocks = (int)(((long long)s.n_q * p.G + MB - 1) / MB);
    return s;
}

// The sum over all NT threads of `sum` in `total`, and what the threads before this one have of it. scan has NT / 32
// entries.
template <int NT>
__device__ __forceinline__ long long scan_tiles(long long sum, long long* scan, long long& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long long before = inc - sum;
    total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    return before;
}

// pre[r + 1] holds request r's tiles; r0 .. r1 are the thread's own requests, with `sum` tiles; pre[r] becomes the tiles
// before request r's. Returns the total, 0 where it is more than 32 bits count (offsets that repeat rows): no row is
// computed then.
template <int NT>
__device__ __forceinline__ int sum_line(const AttendParams& p, int r0, int r1, long long sum, int* pre, long long* scan,
                                        bool report)
{
    long long total, before = scan_tiles<NT>(sum, scan, total);
    if (total > kMostTiles) {
        if (report && threadIdx.x == 0) raise_status(p.status, DSPARK_ERR_DEVICE_INPUT);
        total = 0;
    }
    if (threadIdx.x == 0) pre[0] = 0;
    for (int r = r0; r < r1; ++r) {
        before += pre[r + 1];
        pre[r + 1] = (int)before;
    }
    __syncthreads();
    return (int)total;
}

// pre[r] = tiles before request r's; returns the total. Called by all NT threads of the CTA. pre has R + 1 entries, scan
// NT / 32.
template <int NT, int TILE>
__device__ __forceinline__ int plan_line(const AttendParams& p, int MB, int* pre, long long* scan, bool report)
{
    const int R = p.c.R, each = (R + NT - 1) / NT, r0 = min((int)threadIdx.x * each, R), r1 = min(r0 + each, R);
    long long sum = 0;
    for (int r = r0; r < r1; ++r) {
        const RequestSpan<TILE> s = request_span<TILE>(p, r, MB, report);
        const int n = s.tiles * s.blocks * p.c.Hkv;   // one request's: checked on the host
        pre[r + 1] = n;
        sum += n;
    }
    return sum_line<NT>(p, r0, r1, sum, pre, scan, report);
}

// The item a tile of the line belongs to: request r, item q (head, row block) and tile u of the item.
template <int TILE>
struct ItemWalk {
    int r, q, u;
    RequestSpan<TILE> span;
    __device__ __forceinline__ void start(const int* pre, int R, int at)
    {
        int lo = 0, hi = R;   // the request with pre[r] <= at < pre[r + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= at) lo = mid;
            else hi = mid;
        }
        r = lo - 1;
    }
    __device__ __forceinline__ void settle(const AttendParams& p, int MB, const int* pre, int at)
    {
        if (r < 0 || at >= pre[r + 1]) {
            do ++r;
            while (at >= pre[r + 1]);
            span = request_span<TILE>(p, r, MB, false);
        }
        q = (at - pre[r]) / span.tiles;
        u = (at - pre[r]) % span.tiles;
    }
    __device__ __forceinline__ int head() const { return q / span.blocks; }
    __device__ __forceinline__ int block() const { return q % span.blocks; }
};

template <typename T>
__device__ __forceinline__ void store1(T* p, float x);
template <>
__device__ __forceinline__ void store1<float>(float* p, float x) { *p = x; }
template <>
__device__ __forceinline__ void store1<__nv_bfloat16>(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The rows of the batch before the first request's and after the last's: out = 0, lse = -inf. Thread
// `index` of `threads`.
template <typename T>
__device__ __forceinline__ void zero_rows(const AttendParams& p, int D, int index, int threads)
{
    const int lo = min(max(p.offsets[0], 0), p.T), hi = max(lo, min(p.offsets[p.c.R], p.T));
    const long long vecs = (long long)p.Hq * D * sizeof(T) / 16, rows = lo + (p.T - hi);
    for (long long x = index; x < rows * vecs; x += threads) {
        const long long k = x / vecs, t = k < lo ? k : hi + (k - lo);
        reinterpret_cast<uint4*>(p.out)[t * vecs + x % vecs] = make_uint4(0, 0, 0, 0);
    }
    if (p.lse)
        for (long long x = index; x < rows * p.Hq; x += threads) {
            const long long k = x / p.Hq, t = k < lo ? k : hi + (k - lo);
            p.lse[t * p.Hq + x % p.Hq] = -INFINITY;
        }
}

}  // namespace dspark
