// api.cu -- the C ABI of libdspark (include/dspark.h): argument validation,
// workspace layout and the launch sequence of each call. Every step of the
// round runs in this library's kernels; nothing here computes on the host.
#include <float.h>
#include <stdio.h>
#include <string.h>

#include <atomic>

#include "attend_plan.cuh"
#include "cache.cuh"
#include "common.cuh"
#include "internal.h"

using namespace dspark;

namespace {

// ------------------------------------------------------------ launch accounting

std::atomic<unsigned long long> g_launches{0};

constexpr unsigned long long kDefaultWaitNs = 4000000000ull;   // 4 s
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};

struct KernelTimer {
    int kernel = -1;
    dspark_event_pair* events = nullptr;
    int capacity = 0;
    int32_t* count = nullptr;
} g_timer;

bool timing(int kernel) { return g_timer.kernel == kernel && g_timer.count && *g_timer.count < g_timer.capacity; }

const char* kernel_name(int kernel)
{
    static const char* names[] = {"draft_setup", "draft_stats", "draft_commit", "schedule",
                                  "verify_rows", "verify_decide", "residual_stats", "residual_pick",
                                  "assemble", "rnn_step", "rnn_hidden", "draft_loop",
                                  "qk_norm_rope", "cache_append", "cache_read", "cache_attend", "cache_merge",
                                  "add_norm_quant", "linear_layout", "linear_i8", "seen_add", "adjust_logits"};
    return kernel >= 0 && kernel <= DSPARK_KERNEL_ADJUST_LOGITS ? names[kernel] : "?";
}

thread_local char g_last_error[256] = "no error";

// Launch one kernel family through `fn`, counting it and recording the timing events if enabled.
template <typename F>
cudaError_t launch(int kernel, cudaStream_t s, F&& fn)
{
    const bool t = timing(kernel);
    cudaError_t e = cudaSuccess;
    if (t) e = cudaEventRecord(static_cast<cudaEvent_t>(g_timer.events[*g_timer.count].start), s);
    if (e == cudaSuccess) e = fn();
    g_launches.fetch_add(1, std::memory_order_relaxed);
    if (t && e == cudaSuccess) {
        e = cudaEventRecord(static_cast<cudaEvent_t>(g_timer.events[*g_timer.count].stop), s);
        ++*g_timer.count;
    }
    if (e != cudaSuccess)
        snprintf(g_last_error, sizeof g_last_error, "%s: %s (%s)", kernel_name(kernel), cudaGetErrorName(e),
                 cudaGetErrorString(e));
    return e;
}

// Clear a non-sticky error another library left in this thread's runtime state, so that
// the checks after our own launches report only our launches.
void clear_stale_error() { (void)cudaGetLastError(); }

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;


dspark_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

// ------------------------------------------------------------ sample_block

struct SampleLayout {
    size_t x_cur, stats, pick, a_next, yh, state, a_rows, a_lo, zbuf, slots, hdot, total;
};

// the status word sits at offset 0 of every workspace; the resident loop's grid barrier counter
// and abort flag share its 256-byte region
constexpr size_t kGridBarOffset = 64;
constexpr size_t kGridAbortOffset = 128;

dspark_status check_sample(const dspark_sample_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_sample_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->gamma_max < 1 || a->gamma_max > DSPARK_MAX_GAMMA) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->V < 1 || a->V > (1 << 24) || a->r < 1 || a->r > 1024 || a->d < 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((a->conf_token | 1) != 1 || (a->bias_first | 1) != 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->head != DSPARK_HEAD_MARKOV && a->head != DSPARK_HEAD_RNN) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->head == DSPARK_HEAD_RNN && !a->W_rnn) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->path < DSPARK_PATH_AUTO || a->path > DSPARK_PATH_RESIDENT) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->round >= (1ull << 29)) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((long long)a->R * a->gamma_max * a->V >= (1ll << 40)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (!a->U || !a->E || !a->W || !a->h || !a->w_h || !a->w_e || !a->temperature || !a->anchor)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (!a->tokens || !a->conf || !a->surv || !a->draft_lse || !a->draft_logit) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

bool sample_uses_tc(const dspark_sample_args* a)
{
    if (a->path == DSPARK_PATH_CUDA_CORE) return false;
    return tc_supported(a->dtype, a->R, a->V, a->r, a->U, a->E, a->W);
}

// the persistent resident loop, when asked for. AUTO does not take it: measured at R = 128,
// V = 151936 it runs the draft in 1.18 ms against 0.48 ms for the per-step kernels (its transposed
// epilogue and the serial tail between steps cost more than the W traffic it saves)
bool sample_uses_loop(const dspark_sample_args* a)
{
    if (a->path != DSPARK_PATH_RESIDENT) return false;
    return sample_uses_tc(a) && loop_supported(a->dtype, a->head, a->R, a->V, a->r, a->U, a->E, a->W, a->h, a->w_h,
                                               a->w_e);
}

SampleLayout sample_layout(const dspark_sample_args* a)
{
    const int nblk = cdiv(a->V, kNoiseBlock);
    const size_t rows = sample_uses_tc(a) ? tc_stats_rows(a->R) : (size_t)a->R;
    const bool loop = sample_uses_loop(a);
    SampleLayout L;
    size_t o = kStatusBytes;
    L.x_cur = o;
    o = align_up(o + sizeof(int32_t) * a->R, kAlign);
    L.stats = o;   // per block (CUDA-core path), per CTA of the tensor-core kernel, or per CTA of the
                   // loop for two steps (its outputs of step k are written while step k + 1 runs)
    o = align_up(o + sizeof(float2) * rows *
                         (loop ? 2 * loop_ctas(a->R, a->V) : sample_uses_tc(a) ? tc_grid(a->R, nblk) : nblk),
                 kAlign);
    L.pick = o;
    o = align_up(o + sizeof(unsigned long long) * (size_t)a->R * a->gamma_max, kAlign);
    L.a_next = o;   // the tensor-core path keeps kAReplicas copies of the next step's A rows
    o = align_up(o + (sample_uses_tc(a) ? kAReplicas : 1) * (a->dtype == DSPARK_BF16 ? 2 : 4) * (size_t)a->R * a->r,
                 kAlign);
    const bool rnn = a->head == DSPARK_HEAD_RNN;
    L.yh = o;   // RNN head: the h part of the projection, every position
    o = align_up(o + (rnn ? sizeof(float) * (size_t)a->R * a->gamma_max * 3 * a->r : 0), kAlign);
    L.state = o;
    o = align_up(o + (rnn ? sizeof(float) * 2 * (size_t)a->R * a->r : 0), kAlign);
    L.a_rows = o;   // used when the caller does not take the bias operands
    o = align_up(o + (rnn && !a->a_rows ? sizeof(float) * (size_t)a->R * a->gamma_max * a->r : 0), kAlign);
    L.a_lo = o;
    o = align_up(o + (rnn ? 2 * (size_t)a->R * a->r : 0), kAlign);
    L.zbuf = o;   // RNN head on the tensor cores: the step's operand rows, two parities of [R][3r] bf16
    o = align_up(o + (rnn && sample_uses_tc(a) ? 2 * 2 * (size_t)a->R * 3 * a->r : 0), kAlign);
    L.slots = o;   // the loop: per CTA and request, the leading block's logits
    o = align_up(o + (loop ? loop_slot_bytes(a->R, a->V) : 0), kAlign);
    L.hdot = o;    // the loop: w_h . h_k of every position
    o = align_up(o + (loop ? sizeof(float) * (size_t)a->R * a->gamma_max : 0), kAlign);
    L.total = o;
    return L;
}

// ------------------------------------------------------------ verify

struct VerifyLayout {
    size_t row_stats, row_part, lse_t, rej, n_rej, rej_list, res_stats, total;
};

dspark_status check_verify(const dspark_verify_args* a)
{
    // struct_size without target_ready and reserved: 0
    if (!a || (a->struct_size != sizeof(dspark_verify_args) && a->struct_size != offsetof(dspark_verify_args, target_ready)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->struct_size == sizeof(dspark_verify_args) && ((a->target_ready | 1) != 1 || a->reserved != 0))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->gamma_max < 1 || a->gamma_max > DSPARK_MAX_GAMMA) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->V < 1 || a->V > (1 << 24) || a->r < 1 || a->r > 1024) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((a->bias_first | 1) != 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->path < DSPARK_PATH_AUTO || a->path > DSPARK_PATH_TENSOR_CORE) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->round >= (1ull << 29)) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((long long)a->R * (a->gamma_max + 1) * a->V >= (1ll << 40)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (!a->target || !a->U || !a->E || !a->W || !a->anchor || !a->tokens || !a->draft_lse || !a->draft_logit ||
        !a->keep || !a->temperature)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (!a->accepted || !a->next_token || !a->resampled) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

bool verify_uses_tc(const dspark_verify_args* a)
{
    if (a->path == DSPARK_PATH_CUDA_CORE) return false;
    if (a->a_rows) return false;   // fp32 bias operands (RNN head): the CUDA-core residual keeps them exact
    return tc_residual_supported(a->dtype, a->R, a->V, a->r, a->U, a->E, a->W);
}

VerifyLayout verify_layout(const dspark_verify_args* a)
{
    const int nblk = cdiv(a->V, kNoiseBlock);
    const size_t rows = verify_uses_tc(a) ? tc_stats_rows(a->R) : (size_t)a->R;
    VerifyLayout L;
    size_t o = kStatusBytes;
    L.row_stats = o;
    o = align_up(o + sizeof(float2) * (size_t)a->R * (a->gamma_max + 1) * nblk, kAlign);
    L.row_part = o;
    o = align_up(o + sizeof(float2) * (size_t)a->R * (a->gamma_max + 1) * verify_row_partials(nblk), kAlign);
    L.lse_t = o;
    o = align_up(o + sizeof(float) * (size_t)a->R * (a->gamma_max + 1), kAlign);
    L.rej = o;
    o = align_up(o + sizeof(int32_t) * a->R, kAlign);
    L.n_rej = o;
    o = align_up(o + sizeof(int), kAlign);
    L.rej_list = o;
    o = align_up(o + sizeof(int32_t) * a->R, kAlign);
    L.res_stats = o;
    o = align_up(o + sizeof(float) * rows * nblk, kAlign);
    L.total = o;
    return L;
}

// ------------------------------------------------------------ schedule

dspark_status check_schedule(const dspark_schedule_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_schedule_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->gamma_max < 1 || a->gamma_max > DSPARK_MAX_GAMMA) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((long long)a->R * a->gamma_max > DSPARK_MAX_SLOTS) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->mode < DSPARK_SCHED_SYNC || a->mode > DSPARK_SCHED_THRESHOLD) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->mode == DSPARK_SCHED_THRESHOLD && !(a->threshold == a->threshold)) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((long long)a->n_sps < (long long)a->R * (1 + a->gamma_max)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!a->surv || !a->sps || !a->keep || !a->stats) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->mode == DSPARK_SCHED_ASYNC_CAPACITY && !a->surv_capacity) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

// ------------------------------------------------------------ the target layer's attention

dspark_status check_rope(const dspark_qk_norm_rope_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_qk_norm_rope_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq > 1024 || a->Hkv > 1024) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->D < 2 || a->D > 1024 || a->D % 2 || a->rot < 0 || a->rot > a->D || a->rot % 2)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((a->norm | 1) != 1 || (a->interleaved | 1) != 1 || a->reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!(a->eps >= 0.f) || a->eps > FLT_MAX) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->request && a->R < 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T == 0) return DSPARK_OK;   // an empty tensor may have no address
    if (a->ctx_len && !a->request) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!a->q || !a->k || !a->q_out || !a->k_out || !a->position || (a->rot > 0 && !a->freq))
        return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

dspark_status check_cache(const dspark_cache& c)
{
    if (!c.pages || !c.table || !c.ctx_len || c.reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(c.pages) % 16) return DSPARK_ERR_INVALID_ARGUMENT;
    if (c.n_pages < 1 || c.n_pages > INT32_MAX || c.table_width < 1 || c.Hkv < 1 || c.R < 1)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (!dspark_cache_block_bytes(c.page_size, c.D)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (c.R > DSPARK_MAX_SLOTS || c.Hkv > 1024) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if ((long long)c.table_width * c.page_size > INT32_MAX) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    return DSPARK_OK;
}

dspark_status check_append(const dspark_cache_append_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_cache_append_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    const dspark_status st = check_cache(a->cache);
    if (st != DSPARK_OK) return st;
    if (a->T > 0 && (!a->k || !a->v || !a->request || !a->position)) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

dspark_status check_read(const dspark_cache_read_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_cache_read_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    const dspark_status st = check_cache(a->cache);
    if (st != DSPARK_OK) return st;
    if (a->T > 0 && (!a->k_out || !a->v_out || !a->request || !a->position)) return DSPARK_ERR_INVALID_ARGUMENT;
    // 16-byte stores
    if (reinterpret_cast<uintptr_t>(a->k_out) % 16 || reinterpret_cast<uintptr_t>(a->v_out) % 16)
        return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

dspark_status check_attend(const dspark_cache_attend_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_cache_attend_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->Hq < 1 || a->max_q < 1 || a->window < 0 || a->sinks < 0 || a->reserved != 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->path < DSPARK_PATH_AUTO || a->path > DSPARK_PATH_TENSOR_CORE) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!(a->scale > 0.f) || a->scale > FLT_MAX / 2) return DSPARK_ERR_INVALID_ARGUMENT;
    const dspark_status st = check_cache(a->cache);
    if (st != DSPARK_OK) return st;
    if (a->Hq % a->cache.Hkv) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->Hq / a->cache.Hkv > 1024) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->T > 0 && (!a->q || !a->offsets || !a->out)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(a->out) % 16) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

// The status word and, with `align`, the parts of a workspace that kernels read and write in pieces of 16 bytes
dspark_status check_workspace(const void* ws, size_t bytes, size_t need, size_t align)
{
    if (!ws || bytes < need) return DSPARK_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(ws) % align ? DSPARK_ERR_INVALID_ARGUMENT : DSPARK_OK;
}

AttendParams attend_params(const dspark_cache_attend_args* a)
{
    AttendParams p;
    memset(&p, 0, sizeof p);
    p.T = a->T;
    p.Hq = a->Hq;
    p.G = a->Hq / a->cache.Hkv;
    p.dtype = a->dtype;
    p.max_q = a->max_q;
    p.window = a->window;
    p.sinks = a->sinks;
    p.scale = a->scale;
    p.c = a->cache;
    p.page_magic = page_magic(a->cache.page_size);
    p.g_magic = p.G > 1 ? (uint32_t)(((1ull << 32) + p.G - 1) / p.G) : 0u;
    p.q = a->q;
    p.q_ts = a->q_token_stride;
    p.q_hs = a->q_head_stride;
    p.offsets = a->offsets;
    p.out = a->out;
    p.lse = a->lse;
    return p;
}

bool attend_uses_mma(const dspark_cache_attend_args* a, const AttendParams& p)
{
    return a->path != DSPARK_PATH_CUDA_CORE && (attend_tc_supported(p) || attend_mma_supported(p));
}

// ------------------------------------------------------------ the rest of the target's pass

dspark_status check_norm(const dspark_add_norm_quant_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_add_norm_quant_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->N < 1 || (a->norm | 1) != 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!(a->eps >= 0.f) || a->eps > FLT_MAX) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->N > 32768) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->T == 0) return DSPARK_OK;   // an empty tensor may have no address
    if (!a->x || (a->sum && !a->residual) || (!a->codes && !a->y) || !a->codes != !a->scale)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->sum && a->sum == a->y) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->x_stride < 0 || a->residual_stride < 0) return DSPARK_ERR_INVALID_ARGUMENT;
    // rows of an output do not overlap
    if (a->T > 1 && ((a->sum && a->sum_stride < a->N) || (a->y && a->y_stride < a->N) || (a->codes && a->codes_stride < a->N)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

dspark_status check_linear(const dspark_linear_i8_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_linear_i8_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->T < 0 || a->K < 1 || a->N < 1 || a->reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->path < DSPARK_PATH_AUTO || a->path > DSPARK_PATH_TENSOR_CORE) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->out_rows < 0 || (!a->out_row && a->out_rows < a->T)) return DSPARK_ERR_INVALID_ARGUMENT;
    // sums of K products of at most 2^14 stay below 2^31
    if (a->K > 131071 || a->N > (1 << 24)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->T == 0) return DSPARK_OK;
    if (!a->x || !a->x_scale || !a->w || !a->w_scale || !a->out) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->x_stride < 0 || a->w_stride < 0 || (a->out_rows > 1 && a->out_stride < a->N))
        return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

LinearParams linear_params(const dspark_linear_i8_args* a)
{
    LinearParams p;
    memset(&p, 0, sizeof p);
    p.T = a->T;
    p.K = a->K;
    p.N = a->N;
    p.dtype = a->dtype;
    p.out_rows = a->out_rows;
    p.x = a->x;
    p.x_scale = a->x_scale;
    p.w = a->w;
    p.w_scale = a->w_scale;
    p.bias = a->bias;
    p.out_row = a->out_row;
    p.n_rows = a->n_rows;
    p.out = a->out;
    p.x_rs = a->x_stride;
    p.w_rs = a->w_stride;
    p.o_rs = a->out_stride;
    return p;
}

bool linear_uses_tc(const dspark_linear_i8_args* a, const LinearParams& p)
{
    return a->path != DSPARK_PATH_CUDA_CORE && a->T > 0 && linear_tc_supported(p);
}

dspark_status check_seen(const dspark_seen_add_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_seen_add_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->W < 0 || a->V < 1 || (a->prompt | 1) != 1 || a->reserved != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R > DSPARK_MAX_SLOTS || a->V > (1 << 24)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (!a->seen || reinterpret_cast<uintptr_t>(a->seen) % 16 || a->seen_stride % 8 || a->seen_stride < a->V)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->W > 0 && (!a->tokens || a->tokens_stride < 0)) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

dspark_status check_adjust(const dspark_adjust_logits_args* a)
{
    if (!a || a->struct_size != sizeof(dspark_adjust_logits_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->S < 1 || a->V < 1 || a->n_masks < 0 || a->n_bias < 0 || a->reserved != 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->dtype != DSPARK_F32 && a->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R > DSPARK_MAX_SLOTS || a->S > DSPARK_MAX_GAMMA + 1 || a->V > (1 << 24)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (!a->logits || !a->out) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->seen && (reinterpret_cast<uintptr_t>(a->seen) % 16 || a->seen_stride % 8 || a->seen_stride < a->V))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->bias_offsets && a->n_bias > 0 && (!a->bias_token || !a->bias_value)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->mask && a->mask_stride < (a->V + 31) / 32) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->mask_row && !a->mask) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->mask && !a->mask_row && a->n_masks < (long long)a->R * a->S) return DSPARK_ERR_INVALID_ARGUMENT;
    return DSPARK_OK;
}

template <typename T>
T* at(void* ws, size_t off)
{
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace

unsigned long long dspark::wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }

extern "C" {

int32_t dspark_abi_version(void) { return DSPARK_ABI_VERSION; }

const char* dspark_status_string(dspark_status s)
{
    switch (s) {
    case DSPARK_OK: return "ok";
    case DSPARK_ERR_INVALID_ARGUMENT: return "invalid argument";
    case DSPARK_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case DSPARK_ERR_WORKSPACE: return "workspace missing or too small";
    case DSPARK_ERR_CUDA: return "CUDA error";
    case DSPARK_ERR_TIMEOUT: return "bounded device wait ran out";
    case DSPARK_ERR_DEVICE_INPUT: return "out-of-range device input (clamped)";
    case DSPARK_ERR_NONFINITE_INPUT: return "NaN or +inf in a logit or hidden-state input";
    default: return "unknown status";
    }
}

dspark_status dspark_sample_workspace_size(const dspark_sample_args* a, size_t* bytes)
{
    const dspark_status st = check_sample(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = sample_layout(a).total;
    return DSPARK_OK;
}

int32_t dspark_sample_path(const dspark_sample_args* a)
{
    const dspark_status st = check_sample(a);
    if (st != DSPARK_OK) return -st;
    if (a->path == DSPARK_PATH_TENSOR_CORE && !sample_uses_tc(a)) return -DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->path == DSPARK_PATH_RESIDENT && !sample_uses_loop(a)) return -DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (sample_uses_loop(a)) return DSPARK_PATH_RESIDENT;
    return sample_uses_tc(a) ? DSPARK_PATH_TENSOR_CORE : DSPARK_PATH_CUDA_CORE;
}

dspark_status dspark_sample_block(const dspark_sample_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    dspark_status st = check_sample(a);
    if (st != DSPARK_OK) return st;
    if (a->path == DSPARK_PATH_TENSOR_CORE && !sample_uses_tc(a)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (a->path == DSPARK_PATH_RESIDENT && !sample_uses_loop(a)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    const SampleLayout L = sample_layout(a);
    if (!ws || ws_bytes < L.total) return DSPARK_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DraftStep p;
    memset(&p, 0, sizeof p);
    p.R = a->R;
    p.G = a->gamma_max;
    p.V = a->V;
    p.r = a->r;
    p.d = a->d;
    p.nblk = cdiv(a->V, kNoiseBlock);
    p.dtype = a->dtype;
    p.conf_token = a->conf_token;
    p.bias_first = a->bias_first;
    p.gamma = a->gamma;
    p.U = a->U;
    p.E = a->E;
    p.W = a->W;
    p.h = a->h;
    p.w_h = a->w_h;
    p.w_e = a->w_e;
    p.b = a->b;
    p.temperature = a->temperature;
    p.anchor = a->anchor;
    p.seed = a->seed;
    p.round = a->round;
    p.tokens = a->tokens;
    p.conf = a->conf;
    p.surv = a->surv;
    p.draft_lse = a->draft_lse;
    p.draft_logit = a->draft_logit;
    p.sts_temp = a->sts_temp;
    p.wait_ns = wait_limit_ns();
    p.status = at<int>(ws, 0);
    p.x_cur = at<int32_t>(ws, L.x_cur);
    p.stats = at<float2>(ws, L.stats);
    p.n_stats = sample_uses_tc(a) ? tc_grid(a->R, p.nblk) : p.nblk;
    p.pick = at<unsigned long long>(ws, L.pick);
    p.a_next = at<unsigned char>(ws, L.a_next);
    const bool tc = sample_uses_tc(a);
    p.a_replicas = tc && a->head != DSPARK_HEAD_RNN ? kAReplicas : 1;
    p.head = a->head;
    p.W_rnn = a->W_rnn;
    const bool rnn = a->head == DSPARK_HEAD_RNN;
    p.a_rows = rnn ? (a->a_rows ? a->a_rows : at<float>(ws, L.a_rows)) : a->a_rows;
    p.yh = rnn ? at<float>(ws, L.yh) : nullptr;
    p.state = rnn ? at<float>(ws, L.state) : nullptr;
    p.a_lo = rnn && tc ? at<unsigned char>(ws, L.a_lo) : nullptr;
    p.zbuf = rnn && tc ? at<unsigned char>(ws, L.zbuf) : nullptr;
    if (sample_uses_loop(a)) {
        // every step in one persistent launch (after every per-step input event, if any)
        p.n_stats = loop_ctas(a->R, a->V);
        cudaError_t e = cudaSuccess;
        for (int k = 0; a->step_ready && k < a->gamma_max && e == cudaSuccess; ++k)
            if (a->step_ready[k])
                e = cudaStreamWaitEvent(s, static_cast<cudaEvent_t>(const_cast<void*>(a->step_ready[k])), 0);
        if (e == cudaSuccess)
            e = launch(DSPARK_KERNEL_DRAFT_LOOP, s, [&] {
                return launch_draft_loop(p, at<float>(ws, L.slots), at<float>(ws, L.hdot),
                                         at<unsigned int>(ws, kGridBarOffset), at<int>(ws, kGridAbortOffset), s);
            });
        return cuda_status(e);
    }
    cudaError_t e = launch(DSPARK_KERNEL_DRAFT_SETUP, s, [&] { return launch_draft_setup(p, s); });
    if (rnn && e == cudaSuccess) {
        // the h part of the RNN projection, every position: one GEMM before the serial loop
        e = launch(DSPARK_KERNEL_RNN_HIDDEN, s, [&] { return launch_rnn_hidden(p, s); });
        if (e != cudaSuccess)
            snprintf(g_last_error, sizeof g_last_error, "rnn hidden GEMM: %s (%s)", cudaGetErrorName(e),
                     cudaGetErrorString(e));
    }
    // RNN head on the tensor cores: operand-row and W_rnn tensor maps, and the step-0 operand rows
    CUtensorMap zmap, rmap;
    memset(&zmap, 0, sizeof zmap);
    memset(&rmap, 0, sizeof rmap);
    const bool rnn_tc = rnn && e == cudaSuccess && rnn_tc_supported(p) && rnn_tc_maps(p, &zmap, &rmap) == cudaSuccess;
    if (rnn && !rnn_tc) p.zbuf = nullptr;   // the CUDA-core step: the commit writes no operand rows
    if (rnn_tc) e = launch(DSPARK_KERNEL_RNN_STEP, s, [&] { return launch_rnn_z0(p, s); });
    // the commit copies the winning W block with one bulk copy when W admits the block map
    CUtensorMap wmap;
    memset(&wmap, 0, sizeof wmap);
    const bool use_wmap = a->dtype == DSPARK_BF16 && a->r % 16 == 0 && a->r <= 256 &&
                          encode_w_block_map(&wmap, a->W, a->V, a->r) == cudaSuccess;
    for (int k = 0; k < a->gamma_max && e == cudaSuccess; ++k) {
        p.k = k;
        // the caller may still be delivering this step's inputs (U[:, k, :]): wait for its event
        if (a->step_ready && a->step_ready[k]) {
            e = cudaStreamWaitEvent(s, static_cast<cudaEvent_t>(const_cast<void*>(a->step_ready[k])), 0);
            if (e != cudaSuccess) {
                snprintf(g_last_error, sizeof g_last_error, "step_ready[%d]: %s", k, cudaGetErrorName(e));
                break;
            }
        }
        if (rnn)
            e = launch(DSPARK_KERNEL_RNN_STEP, s,
                       [&] { return rnn_tc ? launch_rnn_step_tc(p, zmap, rmap, s) : launch_rnn_step(p, s); });
        if (e == cudaSuccess)
            e = launch(DSPARK_KERNEL_DRAFT_STATS, s,
                       [&] { return tc ? launch_draft_stats_tc(p, s) : launch_draft_stats_simt(p, s); });
        if (e == cudaSuccess)
            e = launch(DSPARK_KERNEL_DRAFT_COMMIT, s, [&] { return launch_draft_commit(p, use_wmap ? &wmap : nullptr, s); });
    }
    return cuda_status(e);
}

dspark_status dspark_schedule_workspace_size(const dspark_schedule_args* a, size_t* bytes)
{
    const dspark_status st = check_schedule(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_schedule(const dspark_schedule_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_schedule(a);
    if (st != DSPARK_OK) return st;
    if (!ws || ws_bytes < kStatusBytes) return DSPARK_ERR_WORKSPACE;
    ScheduleParams p;
    p.R = a->R;
    p.G = a->gamma_max;
    p.mode = a->mode;
    p.n_sps = a->n_sps;
    p.gamma = a->gamma;
    p.surv = a->surv;
    p.surv_capacity = a->surv_capacity;
    p.sps = a->sps;
    p.keep = a->keep;
    p.stats = a->stats;
    p.threshold = a->threshold;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_SCHEDULE, s, [&] { return launch_schedule(p, s); }));
}

dspark_status dspark_assemble_workspace_size(const dspark_assemble_args* a, size_t* bytes)
{
    if (!a || a->struct_size != sizeof(dspark_assemble_args) || !bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_assemble(const dspark_assemble_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    if (!a || a->struct_size != sizeof(dspark_assemble_args)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R < 1 || a->gamma_max < 1 || a->gamma_max > DSPARK_MAX_GAMMA) return DSPARK_ERR_INVALID_ARGUMENT;
    if (a->R > DSPARK_MAX_SLOTS) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    if (!a->keep || !a->anchor || !a->tokens || !a->flat_tokens || !a->flat_request || !a->flat_position ||
        !a->offsets)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (!ws || ws_bytes < kStatusBytes) return DSPARK_ERR_WORKSPACE;
    AssembleParams p;
    p.R = a->R;
    p.G = a->gamma_max;
    p.keep = a->keep;
    p.anchor = a->anchor;
    p.tokens = a->tokens;
    p.flat_tokens = a->flat_tokens;
    p.flat_request = a->flat_request;
    p.flat_position = a->flat_position;
    p.offsets = a->offsets;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_ASSEMBLE, s, [&] { return launch_assemble(p, s); }));
}

dspark_status dspark_verify_workspace_size(const dspark_verify_args* a, size_t* bytes)
{
    const dspark_status st = check_verify(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = verify_layout(a).total;
    return DSPARK_OK;
}

dspark_status dspark_verify(const dspark_verify_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_verify(a);
    if (st != DSPARK_OK) return st;
    if (a->path == DSPARK_PATH_TENSOR_CORE && !tc_supported(a->dtype, a->R, a->V, a->r, a->U, a->E, a->W))
        return DSPARK_ERR_UNSUPPORTED_SHAPE;
    const VerifyLayout L = verify_layout(a);
    if (!ws || ws_bytes < L.total) return DSPARK_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    VerifyParams p;
    memset(&p, 0, sizeof p);
    p.R = a->R;
    p.G = a->gamma_max;
    p.V = a->V;
    p.r = a->r;
    p.nblk = cdiv(a->V, kNoiseBlock);
    p.dtype = a->dtype;
    p.bias_first = a->bias_first;
    p.gamma = a->gamma;
    p.target = a->target;
    p.U = a->U;
    p.E = a->E;
    p.W = a->W;
    p.anchor = a->anchor;
    p.tokens = a->tokens;
    p.draft_lse = a->draft_lse;
    p.a_rows = a->a_rows;
    p.target_ready = a->struct_size == sizeof(dspark_verify_args) ? a->target_ready : 0;
    p.draft_logit = a->draft_logit;
    p.keep = a->keep;
    p.temperature = a->temperature;
    p.seed = a->seed;
    p.round = a->round;
    p.accepted = a->accepted;
    p.next_token = a->next_token;
    p.resampled = a->resampled;
    p.wait_ns = wait_limit_ns();
    p.status = at<int>(ws, 0);
    p.row_stats = at<float2>(ws, L.row_stats);
    p.row_part = at<float2>(ws, L.row_part);
    p.npart = verify_row_partials(p.nblk);
    p.lse_t = at<float>(ws, L.lse_t);
    p.rej = at<int32_t>(ws, L.rej);
    p.n_rej = at<int>(ws, L.n_rej);
    p.rej_list = at<int32_t>(ws, L.rej_list);
    p.res_stats = at<float>(ws, L.res_stats);
    const bool tc = verify_uses_tc(a);
    cudaError_t e = launch(DSPARK_KERNEL_VERIFY_ROWS, s, [&] { return launch_verify_rows(p, s); });
    if (e == cudaSuccess) e = launch(DSPARK_KERNEL_VERIFY_DECIDE, s, [&] { return launch_verify_decide(p, s); });
    if (e == cudaSuccess)
        e = launch(DSPARK_KERNEL_RESIDUAL_STATS, s,
                   [&] { return tc ? launch_residual_stats_tc(p, s) : launch_residual_stats_simt(p, s); });
    if (e == cudaSuccess) e = launch(DSPARK_KERNEL_RESIDUAL_PICK, s, [&] { return launch_residual_pick(p, s); });
    return cuda_status(e);
}

size_t dspark_cache_block_bytes(int32_t page_size, int32_t D)
{
    if (page_size < 16 || page_size > 256 || page_size % 16 || D < 32 || D > 256 || D % 32) return 0;
    return cache_block(page_size, D).bytes;
}

dspark_status dspark_qk_norm_rope_workspace_size(const dspark_qk_norm_rope_args* a, size_t* bytes)
{
    const dspark_status st = check_rope(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_qk_norm_rope(const dspark_qk_norm_rope_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_rope(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    if (a->T == 0) return DSPARK_OK;
    RopeParams p;
    p.T = a->T;
    p.Hq = a->Hq;
    p.Hkv = a->Hkv;
    p.D = a->D;
    p.rot = a->rot;
    p.dtype = a->dtype;
    p.norm = a->norm;
    p.interleaved = a->interleaved;
    p.R = a->R;
    p.eps = a->eps;
    p.q = a->q;
    p.k = a->k;
    p.q_ts = a->q_token_stride;
    p.q_hs = a->q_head_stride;
    p.k_ts = a->k_token_stride;
    p.k_hs = a->k_head_stride;
    p.q_gain = a->q_gain;
    p.k_gain = a->k_gain;
    p.freq = a->freq;
    p.position = a->position;
    p.request = a->request;
    p.ctx_len = a->ctx_len;
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_QK_NORM_ROPE, s, [&] { return launch_qk_norm_rope(p, s); }));
}

dspark_status dspark_cache_append_workspace_size(const dspark_cache_append_args* a, size_t* bytes)
{
    const dspark_status st = check_append(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_cache_append(const dspark_cache_append_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_append(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    if (a->T == 0) return DSPARK_OK;
    CacheRowsParams p;
    memset(&p, 0, sizeof p);
    p.T = a->T;
    p.dtype = a->dtype;
    p.c = a->cache;
    p.k = a->k;
    p.v = a->v;
    p.k_ts = a->k_token_stride;
    p.k_hs = a->k_head_stride;
    p.v_ts = a->v_token_stride;
    p.v_hs = a->v_head_stride;
    p.request = a->request;
    p.position = a->position;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_CACHE_APPEND, s, [&] { return launch_cache_append(p, s); }));
}

dspark_status dspark_cache_read_workspace_size(const dspark_cache_read_args* a, size_t* bytes)
{
    const dspark_status st = check_read(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_cache_read(const dspark_cache_read_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_read(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    if (a->T == 0) return DSPARK_OK;
    CacheRowsParams p;
    memset(&p, 0, sizeof p);
    p.T = a->T;
    p.dtype = a->dtype;
    p.c = a->cache;
    p.request = a->request;
    p.position = a->position;
    p.k_out = a->k_out;
    p.v_out = a->v_out;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_CACHE_READ, s, [&] { return launch_cache_read(p, s); }));
}

dspark_status dspark_cache_attend_workspace_size(const dspark_cache_attend_args* a, size_t* bytes)
{
    const dspark_status st = check_attend(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    const AttendParams p = attend_params(a);
    *bytes = kStatusBytes + (attend_uses_mma(a, p) ? attend_scratch(p, nullptr, nullptr) : 0);
    return DSPARK_OK;
}

dspark_status dspark_cache_attend(const dspark_cache_attend_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_attend(a);
    if (st != DSPARK_OK) return st;
    AttendParams p = attend_params(a);
    if (a->path == DSPARK_PATH_TENSOR_CORE && !attend_uses_mma(a, p)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    const bool mma = attend_uses_mma(a, p);
    const size_t need = kStatusBytes + (mma ? attend_scratch(p, nullptr, nullptr) : 0);
    const dspark_status sw = check_workspace(ws, ws_bytes, need, mma ? 16 : alignof(int));
    if (sw != DSPARK_OK) return sw;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!mma) {
        if (a->T == 0) return DSPARK_OK;
        return cuda_status(launch(DSPARK_KERNEL_CACHE_ATTEND, s, [&] { return launch_cache_attend_simt(p, s); }));
    }
    if (a->T == 0) return DSPARK_OK;
    AttendScratch scratch;
    attend_scratch(p, &scratch, at<char>(ws, kStatusBytes));
    cudaError_t e = launch(DSPARK_KERNEL_CACHE_ATTEND, s, [&] { return launch_cache_attend(p, scratch, s); });
    if (e == cudaSuccess) e = launch(DSPARK_KERNEL_CACHE_MERGE, s, [&] { return launch_cache_merge(p, scratch, s); });
    return cuda_status(e);
}

dspark_status dspark_add_norm_quant_workspace_size(const dspark_add_norm_quant_args* a, size_t* bytes)
{
    const dspark_status st = check_norm(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_add_norm_quant(const dspark_add_norm_quant_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_norm(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    if (a->T == 0) return DSPARK_OK;
    NormParams p;
    p.T = a->T;
    p.N = a->N;
    p.dtype = a->dtype;
    p.norm = a->norm;
    p.eps = a->eps;
    p.x = a->x;
    p.residual = a->residual;
    p.x_rs = a->x_stride;
    p.r_rs = a->residual_stride;
    p.s_rs = a->sum_stride;
    p.y_rs = a->y_stride;
    p.c_rs = a->codes_stride;
    p.gain = a->gain;
    p.n_rows = a->n_rows;
    p.sum = a->sum;
    p.y = a->y;
    p.codes = a->codes;
    p.scale = a->scale;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_ADD_NORM_QUANT, s, [&] { return launch_add_norm_quant(p, s); }));
}

dspark_status dspark_linear_i8_workspace_size(const dspark_linear_i8_args* a, size_t* bytes)
{
    const dspark_status st = check_linear(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    const LinearParams p = linear_params(a);
    *bytes = kStatusBytes + (linear_uses_tc(a, p) ? linear_tc_scratch(p) : 0);
    return DSPARK_OK;
}

dspark_status dspark_linear_i8(const dspark_linear_i8_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_linear(a);
    if (st != DSPARK_OK) return st;
    LinearParams p = linear_params(a);
    const bool tc = linear_uses_tc(a, p);
    if (a->path == DSPARK_PATH_TENSOR_CORE && !tc && a->T > 0) return DSPARK_ERR_UNSUPPORTED_SHAPE;
    const size_t need = kStatusBytes + (tc ? linear_tc_scratch(p) : 0);
    const dspark_status sw = check_workspace(ws, ws_bytes, need, need > kStatusBytes ? 16 : alignof(int));
    if (sw != DSPARK_OK) return sw;
    if (a->T == 0) return DSPARK_OK;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tc) {
        void* scratch = at<char>(ws, kStatusBytes);
        cudaError_t e = launch(DSPARK_KERNEL_LINEAR_LAYOUT, s, [&] { return launch_linear_layout(p, scratch, s); });
        if (e == cudaSuccess) e = launch(DSPARK_KERNEL_LINEAR_I8, s, [&] { return launch_linear_tc(p, scratch, s); });
        return cuda_status(e);
    }
    return cuda_status(launch(DSPARK_KERNEL_LINEAR_I8, s, [&] { return launch_linear_simt(p, s); }));
}

dspark_status dspark_seen_add_workspace_size(const dspark_seen_add_args* a, size_t* bytes)
{
    const dspark_status st = check_seen(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_seen_add(const dspark_seen_add_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_seen(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    SeenParams p;
    p.R = a->R;
    p.W = a->W;
    p.V = a->V;
    p.prompt = a->prompt;
    p.seen_rs = a->seen_stride;
    p.tokens_rs = a->tokens_stride;
    p.seen = a->seen;
    p.tokens = a->tokens;
    p.n = a->n;
    p.extra = a->extra;
    p.fresh = a->fresh;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_SEEN_ADD, s, [&] { return launch_seen_add(p, s); }));
}

dspark_status dspark_adjust_logits_workspace_size(const dspark_adjust_logits_args* a, size_t* bytes)
{
    const dspark_status st = check_adjust(a);
    if (st != DSPARK_OK) return st;
    if (!bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    *bytes = kStatusBytes;
    return DSPARK_OK;
}

dspark_status dspark_adjust_logits(const dspark_adjust_logits_args* a, void* ws, size_t ws_bytes, void* stream)
{
    clear_stale_error();
    const dspark_status st = check_adjust(a);
    if (st != DSPARK_OK) return st;
    const dspark_status sw = check_workspace(ws, ws_bytes, kStatusBytes, alignof(int));
    if (sw != DSPARK_OK) return sw;
    AdjustParams p;
    p.R = a->R;
    p.S = a->S;
    p.V = a->V;
    p.dtype = a->dtype;
    p.n_masks = a->n_masks;
    p.n_bias = a->n_bias;
    p.logits = a->logits;
    p.out = a->out;
    p.seen = a->seen;
    p.seen_rs = a->seen_stride;
    p.repetition = a->repetition;
    p.presence = a->presence;
    p.frequency = a->frequency;
    p.tokens = a->S > 1 ? a->tokens : nullptr;
    p.bias_offsets = a->n_bias > 0 ? a->bias_offsets : nullptr;
    p.bias_token = a->bias_token;
    p.bias_value = a->bias_value;
    p.mask = a->mask;
    p.mask_rs = a->mask_stride;
    p.mask_row = a->mask_row;
    p.keep = a->keep;
    p.status = at<int>(ws, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(DSPARK_KERNEL_ADJUST_LOGITS, s, [&] { return launch_adjust_logits(p, s); }));
}

const char* dspark_last_error(void) { return g_last_error; }

uint64_t dspark_set_wait_limit(uint64_t ns)
{
    return g_wait_ns.exchange(ns == 0 ? kDefaultWaitNs : ns, std::memory_order_relaxed);
}

uint64_t dspark_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

dspark_status dspark_time_kernel(int32_t kernel, dspark_event_pair* events, int32_t capacity, int32_t* count)
{
    if (kernel < 0) {
        g_timer = KernelTimer();
        return DSPARK_OK;
    }
    if (kernel > DSPARK_KERNEL_ADJUST_LOGITS || !events || capacity < 0 || !count) return DSPARK_ERR_INVALID_ARGUMENT;
    g_timer.kernel = kernel;
    g_timer.events = events;
    g_timer.capacity = capacity;
    g_timer.count = count;
    return DSPARK_OK;
}

dspark_status dspark_check(void* ws, void* stream)
{
    if (!ws) return DSPARK_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int h = 0;
    cudaError_t e = cudaMemcpyAsync(&h, ws, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return DSPARK_ERR_CUDA;
    return h;
}

}  // extern "C"
