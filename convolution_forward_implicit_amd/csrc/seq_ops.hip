// Host side of the sequence operators (conv_causal_*, conv_scan_*): argument
// checks, the choice of kernel variants and splits, launches.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "../../include/convfwd.h"
#include "causal_conv.h"
#include "scan_dma.h"
#include "scan_kernels.h"
#include "status.h"

struct conv_causal_plan {
    conv_causal_desc_t desc;
    int64_t esz, ws_bytes, bwd_rows;     // bwd_rows: workgroup rows of partial sums
    char text[256];
};

// A sequence's chunks in `count` segments of `chunks`, `sub` of which make up what one forward workgroup takes.
struct Segments {
    int count, chunks, sub;
};

struct conv_scan_plan {
    conv_scan_desc_t desc;
    int64_t esz;
    int SP, Q, K, NPB;                   // padded states, chunk, chunks, channel blocks
    int64_t units;                       // N * H * NPB
    Segments fwd, dma, bwd;              // forward, forward of whole bf16 vectors, the gradient's state passes
    int slices, heads_per_slice;
    int64_t ws_bytes, bwd_ws_bytes;
    int64_t o_fwd_log;                   // byte offsets in the forward's workspace and in the gradient's
    int64_t o_seg[2], o_log[2], o_bound[2], o_head, o_pb, o_pc;
    char text[320];
};

namespace convfwd {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr double kMaxBytes = 9.0e18;
constexpr double kMaxThreads = 4294967296.0;     // a launch has fewer threads than this

bool one_launch(double workgroups, int threads) { return workgroups * threads < kMaxThreads; }

conv_status_t launched()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? CONV_OK : fail(CONV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

// A tensor as `rows` runs of `width` elements, `ld` apart.
struct Rows {
    const char *name;
    const void *p;
    int64_t rows, width, ld, esz;
};

bool share_memory(const Rows &a, const Rows &b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const int64_t a0 = (int64_t)(uintptr_t)a.p, b0 = (int64_t)(uintptr_t)b.p;
    const int64_t a1 = a0 + ((a.rows - 1) * a.ld + a.width) * a.esz, b1 = b0 + ((b.rows - 1) * b.ld + b.width) * b.esz;
    if (a1 <= b0 || b1 <= a0) return false;
    const int64_t step = a.ld * a.esz;
    if (step != b.ld * b.esz) return true;
    // equal strides: column ranges of one matrix, disjoint iff the runs are, modulo the stride
    int64_t d = (b0 - a0) % step;
    if (d < 0) d += step;
    return d < a.width * a.esz || d + b.width * b.esz > step;
}

// Every output against every input and the outputs before it.
conv_status_t check_overlap(const Rows *out, int nout, const Rows *in, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (share_memory(out[i], in[j])) return fail(CONV_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (share_memory(out[i], out[j]))
                return fail(CONV_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    }
    return CONV_OK;
}

// Alignment of every tensor to its elements, and token strides that hold a row.
conv_status_t check_rows(const Rows *t, int n)
{
    for (int i = 0; i < n; ++i) {
        if (t[i].p && (uintptr_t)t[i].p % t[i].esz)
            return fail(CONV_ERR_INVALID_ARG, "%s is not aligned to its elements", t[i].name);
        if (t[i].ld < t[i].width)
            return fail(CONV_ERR_INVALID_ARG, "%s: %lld elements from token to token, a row has %lld", t[i].name,
                        (long long)t[i].ld, (long long)t[i].width);
        // a chunk of 64 tokens is addressed by 32-bit byte offsets
        if ((double)t[i].ld * t[i].esz * std::max<int64_t>(1, t[i].rows) > kMaxBytes ||
            (t[i].rows > 1 && t[i].ld * t[i].esz >= int64_t(1) << 25))
            return fail(CONV_ERR_UNSUPPORTED, "%s: %lld elements from token to token", t[i].name, (long long)t[i].ld);
    }
    return CONV_OK;
}

bool vector_rows(const Rows &t) { return !t.p || ((uintptr_t)t.p % 16 == 0 && t.ld * t.esz % 16 == 0); }

int64_t or_packed(int64_t ld, int64_t width) { return ld == 0 ? width : ld; }

// What a kernel gets as a tensor's stride.  One row has no next one, and its
// stride may be any: a small one keeps the 32-bit offsets of the rows that a
// tile has none of past the tensor's end (64 rows of 2^27 bytes wrap round).
int64_t stride(const Rows &t) { return t.rows > 1 ? t.ld : std::min<int64_t>(t.ld, 65536); }

conv_status_t check_workspace(const void *ws, int64_t bytes, int64_t need)
{
    if (need == 0) return CONV_OK;
    if (!ws) return fail(CONV_ERR_INVALID_ARG, "workspace is NULL");
    if (bytes < need)
        return fail(CONV_ERR_INVALID_ARG, "workspace has %lld bytes, the plan needs %lld", (long long)bytes, (long long)need);
    if ((uintptr_t)ws % 16) return fail(CONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    return CONV_OK;
}

// ---- causal convolution --------------------------------------------------------
enum ConvKernel { CONV_RUN, CONV_STEP, CONV_BWD };

template <typename T, int F, int V, bool SILU>
void launch_causal(ConvKernel which, const CausalParams &p, int64_t grid, hipStream_t s)
{
    constexpr bool whole = V * sizeof(T) == 16, half = V * sizeof(T) == 8;
    if constexpr (whole || V == 1) {
        if (which == CONV_RUN)
            hipLaunchKernelGGL((causal_conv_kernel<T, F, V, SILU>), dim3((unsigned)grid), dim3(256), 0, s, p);
        else if (which == CONV_STEP)
            hipLaunchKernelGGL((causal_step_kernel<T, F, V, SILU>), dim3((unsigned)grid), dim3(256), 0, s, p);
    }
    if constexpr (half || V == 1) {
        if (which == CONV_BWD)
            hipLaunchKernelGGL((causal_bwd_kernel<T, F, V, SILU>), dim3((unsigned)grid), dim3(256), 0, s, p);
    }
}

template <typename T, int F, int V>
void launch_causal(ConvKernel which, bool silu, const CausalParams &p, int64_t grid, hipStream_t s)
{
    if (silu) launch_causal<T, F, V, true>(which, p, grid, s);
    else launch_causal<T, F, V, false>(which, p, grid, s);
}

template <typename T, int V>
void launch_causal(ConvKernel which, int F, bool silu, const CausalParams &p, int64_t grid, hipStream_t s)
{
    switch (F) {
    case 2: return launch_causal<T, 2, V>(which, silu, p, grid, s);
    case 3: return launch_causal<T, 3, V>(which, silu, p, grid, s);
    case 4: return launch_causal<T, 4, V>(which, silu, p, grid, s);
    case 5: return launch_causal<T, 5, V>(which, silu, p, grid, s);
    case 6: return launch_causal<T, 6, V>(which, silu, p, grid, s);
    case 7: return launch_causal<T, 7, V>(which, silu, p, grid, s);
    default: return launch_causal<T, 8, V>(which, silu, p, grid, s);
    }
}

void launch_causal(ConvKernel which, const conv_causal_desc_t &d, int V, const CausalParams &p, int64_t grid, hipStream_t s)
{
    if (d.dtype == CONV_DT_BF16) {
        if (V == 4) launch_causal<bf16_t, 4>(which, (int)d.F, d.silu, p, grid, s);
        else if (V > 1) launch_causal<bf16_t, 8>(which, (int)d.F, d.silu, p, grid, s);
        else launch_causal<bf16_t, 1>(which, (int)d.F, d.silu, p, grid, s);
    } else {
        if (V == 2) launch_causal<float, 2>(which, (int)d.F, d.silu, p, grid, s);
        else if (V > 1) launch_causal<float, 4>(which, (int)d.F, d.silu, p, grid, s);
        else launch_causal<float, 1>(which, (int)d.F, d.silu, p, grid, s);
    }
}

// channels per access: whole 16-byte vectors where every tensor allows it
int conv_vector(const conv_causal_desc_t &d, int64_t esz, const Rows *t, int n)
{
    bool ok = d.C * esz % 16 == 0;
    for (int i = 0; i < n; ++i) ok = ok && vector_rows(t[i]);
    return ok ? (int)(16 / esz) : 1;
}

int64_t bwd_blocks(const conv_causal_desc_t &d)   // workgroups along a sequence, one at least (dstate)
{
    const int64_t per = kConvBwdRun * kConvRuns;
    return std::max<int64_t>(1, (d.L + per - 1) / per);
}

int64_t channel_blocks(int64_t vectors) { return (vectors + 63) / 64; }   // workgroups across the channels

// ---- scan ------------------------------------------------------------------------
// Where the gradients of A, dt_bias and D go, and the workgroups that add them up.
struct HeadGrads {
    float *da, *dbias, *dd;
    int64_t workgroups;
};

template <typename T, int SP, bool STORE> void launch_states(const ScanParams &p, int64_t grid, hipStream_t s)
{
    if constexpr (sizeof(T) == 2) {
        if (p.vec) {
            hipLaunchKernelGGL((scan_state_dma_kernel<SP, STORE>), dim3((unsigned)grid), dim3(256), 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((scan_state_kernel<T, SP, STORE>), dim3((unsigned)grid), dim3(256), 0, s, p);
}

// The states that the segments leave from zero, in both directions for a gradient.
template <typename T, int SP> void launch_segments(ScanParams p, int64_t units, int ways, hipStream_t s)
{
    if (p.nseg <= p.sub) return;
    p.ahead = units * (p.nseg - p.sub);
    launch_states<T, SP, false>(p, ways * p.ahead, s);
}

template <typename T, int SP> void launch_fwd(const ScanParams &p, int64_t units, hipStream_t s)
{
    launch_segments<T, SP>(p, units, 1, s);
    const dim3 grid((unsigned)(units * (p.nseg / p.sub)));
    if constexpr (sizeof(T) == 2) {
        if (p.vec) {
            hipLaunchKernelGGL((scan_fwd_dma_kernel<SP>), grid, dim3(512), 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((scan_fwd_kernel<T, SP>), grid, dim3(256), 0, s, p);
}

// of scan_reduce_kernel: three sums of each head, and elements of dB and dC where the heads are sliced
int64_t scan_reduce_grid(const conv_scan_plan &pl)
{
    const conv_scan_desc_t &d = pl.desc;
    return 3 * d.H + (pl.slices > 1 ? (d.N * d.L * d.G * pl.SP + 255) / 256 : 0);
}

template <typename T, int SP> void launch_bwd(ScanParams p, int64_t units, HeadGrads g, hipStream_t s)
{
    if (p.N > 0) {
        launch_segments<T, SP>(p, units, 2, s);
        p.ahead = units * p.nseg;
        launch_states<T, SP, true>(p, 2 * p.ahead, s);
        const int64_t grid = (int64_t)p.N * p.K * p.G * p.slices;
        hipLaunchKernelGGL((scan_bwd_kernel<T, SP>), dim3((unsigned)grid), dim3(512), 0, s, p);
    }
    hipLaunchKernelGGL((scan_reduce_kernel<T, SP>), dim3((unsigned)g.workgroups), dim3(256), 0, s, p, g.da, g.dbias,
                       g.dd);       // no sequences: zeros
}

template <typename T> void launch_scan(int SP, const ScanParams &p, int64_t units, const HeadGrads *g, hipStream_t s)
{
    if (SP == 32) return g ? launch_bwd<T, 32>(p, units, *g, s) : launch_fwd<T, 32>(p, units, s);
    if (SP == 64) return g ? launch_bwd<T, 64>(p, units, *g, s) : launch_fwd<T, 64>(p, units, s);
    return g ? launch_bwd<T, 128>(p, units, *g, s) : launch_fwd<T, 128>(p, units, s);
}

// Segments of K chunks so that `units` heads give about `want` workgroups, each
// cut into `fine` times as many for the pass over the states.  A segment's start
// is joined from all before it by the workgroup itself, up to 32; against a launch
// between the two that joins them the gradient of 2 x 2048 x 32 heads went from 160
// to 150 us and 16384 x 64 heads from 255 to 248, 4096 x 32 from 55 to 59.  Finer
// segments pay where a forward workgroup has 16 chunks and more (16384 x 64 heads
// 253 -> 235 us with two; 4096 x 32, 8 chunks: 53 -> 59).
Segments split_segments(int64_t units, int64_t K, int64_t want, int64_t fine)
{
    // time goes by K / n chunks and n joins, a chunk costing about four joins: the
    // least is near n = 2 sqrt(K) (25 chunks of fp32: 27 us with 25 segments, 21 with 10)
    const int64_t most = std::min<int64_t>(32 / fine, (int64_t)std::ceil(2.0 * std::sqrt((double)K)));
    const int64_t n = std::max<int64_t>(1, std::min({K, want / std::max<int64_t>(1, units), most}));
    const int64_t whole = (K + n - 1) / n, sub = n == 1 ? 1 : std::max<int64_t>(1, std::min(fine, whole / 16));
    const int64_t chunks = (whole + sub - 1) / sub, count = (K + chunks * sub - 1) / (chunks * sub) * sub;
    return {(int)count, (int)chunks, (int)sub};
}

// A step's lanes for the states of a channel, and workgroups for the channels of a head.
struct StepShape {
    int lanes, blocks;
};

StepShape step_shape(const conv_scan_desc_t &d)
{
    int lanes = 1;
    while (lanes * 4 < d.S) lanes *= 2;
    const int64_t per = 4 * kStepRows * (64 / lanes);
    return {lanes, (int)((d.P + per - 1) / per)};
}

void scan_params(const conv_scan_plan &pl, ScanParams *p)
{
    const conv_scan_desc_t &d = pl.desc;
    *p = ScanParams{};
    p->N = (int)d.N; p->L = d.L; p->H = (int)d.H; p->P = (int)d.P; p->G = (int)d.G; p->S = (int)d.S;
    p->NPB = pl.NPB; p->K = pl.K; p->softplus = d.softplus;
}

void set_segments(ScanParams *p, const Segments &s)
{
    p->nseg = s.count;
    p->seg = s.chunks;
    p->sub = s.sub;
}

}  // namespace
}  // namespace convfwd

using namespace convfwd;

extern "C" {

conv_status_t conv_causal_create(const conv_causal_desc_t *desc, conv_causal_plan_t **plan)
{
    if (!plan) return fail(CONV_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "descriptor is NULL");
    const conv_causal_desc_t &d = *desc;
    if (d.dtype != CONV_DT_F32 && d.dtype != CONV_DT_BF16) return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", d.dtype);
    if (d.has_bias != 0 && d.has_bias != 1) return fail(CONV_ERR_INVALID_ARG, "has_bias must be 0 or 1");
    if (d.silu != 0 && d.silu != 1) return fail(CONV_ERR_INVALID_ARG, "silu must be 0 or 1");
    if (d.reserved != 0) return fail(CONV_ERR_INVALID_ARG, "reserved must be 0");
    if (d.N < 0 || d.L < 0 || d.C < 1 || d.F < 2)
        return fail(CONV_ERR_INVALID_ARG, "need N >= 0, L >= 0, C >= 1 and F >= 2 (got %lld, %lld, %lld, %lld)",
                    (long long)d.N, (long long)d.L, (long long)d.C, (long long)d.F);
    if (d.F > 8) return fail(CONV_ERR_UNSUPPORTED, "more than 8 taps (F = %lld)", (long long)d.F);
    if (d.N > kMaxDim || d.L > kMaxDim || d.C > kMaxDim) return fail(CONV_ERR_UNSUPPORTED, "N, L or C above 2^30");
    // What neither a prompt nor a step could launch, whole vectors taken where the channels allow them; every call
    // checks its own form.
    const int64_t e = d.dtype == CONV_DT_BF16 ? 2 : 4, vectors = d.C * e % 16 == 0 ? d.C * e / 16 : d.C;
    const int64_t runs = (d.L + kConvRun - 1) / kConvRun;
    const double fwd = (double)d.N * (double)((runs + kConvRuns - 1) / kConvRuns) * (double)channel_blocks(vectors);
    const double step = (double)d.N * (double)vectors / 256;
    const double ws = (double)d.N * (double)bwd_blocks(d) * (double)(d.F + 1) * (double)d.C * 4.0;
    if ((!one_launch(fwd, 256) && !one_launch(step, 256)) || ws >= kMaxBytes)
        return fail(CONV_ERR_UNSUPPORTED, "N x L x C is too large for one launch");
    conv_causal_plan *pl = new (std::nothrow) conv_causal_plan();
    if (!pl) return fail(CONV_ERR_NOMEM, "plan allocation failed");
    pl->desc = d;
    pl->esz = d.dtype == CONV_DT_BF16 ? 2 : 4;
    pl->bwd_rows = d.N * bwd_blocks(d);
    pl->ws_bytes = pl->bwd_rows * (d.F + 1) * d.C * 4;
    snprintf(pl->text, sizeof(pl->text), "causal %s N=%lld L=%lld C=%lld F=%lld%s%s, %d tokens per wave",
             d.dtype == CONV_DT_BF16 ? "bf16" : "f32", (long long)d.N, (long long)d.L, (long long)d.C, (long long)d.F,
             d.has_bias ? " bias" : "", d.silu ? " silu" : "", kConvRun);
    if (getenv("CONVFWD_LOG")) fprintf(stderr, "convfwd: %s\n", pl->text);
    *plan = pl;
    return CONV_OK;
}

static conv_status_t causal_forward(const conv_causal_plan_t *plan, const conv_causal_args_t *a, bool step, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_causal_desc_t &d = plan->desc;
    const int64_t L = step ? 1 : d.L, e = plan->esz, hist = d.F - 1;
    if (!a->w) return fail(CONV_ERR_INVALID_ARG, "w is NULL");
    if ((a->bias != nullptr) != (d.has_bias != 0))
        return fail(CONV_ERR_INVALID_ARG, d.has_bias ? "bias is NULL" : "this plan has no bias");
    if (step && a->lengths) return fail(CONV_ERR_INVALID_ARG, "a step takes no lengths");
    const Rows in[] = {{"x", a->x, d.N * L, d.C, or_packed(a->x_ld, d.C), e},
                       {"w", a->w, 1, d.C * d.F, d.C * d.F, e},
                       {"bias", a->bias, 1, d.C, d.C, e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4},
                       {"state", a->state, d.N * hist, d.C, d.C, e}};
    const Rows out[] = {{"y", a->y, d.N * L, d.C, or_packed(a->y_ld, d.C), e},
                        {"state_out", a->state_out, d.N * hist, d.C, d.C, e}};
    conv_status_t st = check_rows(in, 5);
    if (st == CONV_OK) st = check_rows(out, 2);
    if (st != CONV_OK) return st;
    if (d.N == 0) return CONV_OK;
    if (L > 0 && (!a->x || !a->y)) return fail(CONV_ERR_INVALID_ARG, "x or y is NULL");
    if (step && (!a->state || !a->state_out)) return fail(CONV_ERR_INVALID_ARG, "state or state_out is NULL");
    // a step may move the state on in place: each thread owns its channels
    const bool in_place = step && a->state == a->state_out;
    if ((st = check_overlap(out, 2, in, in_place ? 4 : 5)) != CONV_OK) return st;
    if (L == 0 && !a->state_out) return CONV_OK;
    const Rows vec[] = {in[0], in[1], in[2], in[4], out[0], out[1]};
    const int V = conv_vector(d, e, vec, 6);
    CausalParams p{};
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.state = a->state; p.lengths = a->lengths;
    p.y = a->y; p.state_out = a->state_out;
    p.x_ld = stride(in[0]); p.y_ld = stride(out[0]);
    p.N = (int)d.N; p.C = (int)d.C; p.CV = (int)(d.C / V); p.L = L;
    p.blocks = (L + kConvRun - 1) / kConvRun;
    const int64_t runs = p.blocks + (a->state_out ? 1 : 0);
    const int64_t grid = step ? (d.N * p.CV + 255) / 256 : d.N * ((runs + kConvRuns - 1) / kConvRuns) * channel_blocks(p.CV);
    if (!one_launch((double)grid, 256)) return fail(CONV_ERR_UNSUPPORTED, "N x L x C is too large for one launch");
    (void)hipGetLastError();
    launch_causal(step ? CONV_STEP : CONV_RUN, d, V, p, grid, (hipStream_t)stream);
    return launched();
}

conv_status_t conv_causal_run(const conv_causal_plan_t *plan, const conv_causal_args_t *args, void *stream)
{
    return causal_forward(plan, args, false, stream);
}

conv_status_t conv_causal_step(const conv_causal_plan_t *plan, const conv_causal_args_t *args, void *stream)
{
    return causal_forward(plan, args, true, stream);
}

conv_status_t conv_causal_bwd_workspace_bytes(const conv_causal_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->ws_bytes;
    return CONV_OK;
}

conv_status_t conv_causal_bwd_run(const conv_causal_plan_t *plan, const conv_causal_bwd_args_t *a, void *workspace,
                                  int64_t workspace_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_causal_desc_t &d = plan->desc;
    const int64_t e = plan->esz, hist = d.F - 1;
    if (!a->w || !a->dw) return fail(CONV_ERR_INVALID_ARG, "w or dw is NULL");
    if ((a->bias != nullptr) != (d.has_bias != 0) || (a->dbias != nullptr) != (d.has_bias != 0))
        return fail(CONV_ERR_INVALID_ARG, d.has_bias ? "bias or dbias is NULL" : "this plan has no bias");
    if (a->dstate && !a->state) return fail(CONV_ERR_INVALID_ARG, "dstate without a state");
    const Rows in[] = {{"dy", a->dy, d.N * d.L, d.C, or_packed(a->dy_ld, d.C), e},
                       {"x", a->x, d.N * d.L, d.C, or_packed(a->x_ld, d.C), e},
                       {"w", a->w, 1, d.C * d.F, d.C * d.F, e},
                       {"bias", a->bias, 1, d.C, d.C, e},
                       {"state", a->state, d.N * hist, d.C, d.C, e},
                       {"dstate_out", a->dstate_out, d.N * hist, d.C, d.C, e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4}};
    const Rows out[] = {{"dx", a->dx, d.N * d.L, d.C, or_packed(a->dx_ld, d.C), e},
                        {"dw", a->dw, 1, d.C * d.F, d.C * d.F, e},
                        {"dbias", a->dbias, 1, d.C, d.C, e},
                        {"dstate", a->dstate, d.N * hist, d.C, d.C, e},
                        {"workspace", workspace, 1, plan->ws_bytes, std::max<int64_t>(1, plan->ws_bytes), 1}};
    conv_status_t st = check_rows(in, 7);
    if (st == CONV_OK) st = check_rows(out, 4);
    if (st != CONV_OK) return st;
    if (d.N > 0 && d.L > 0 && (!a->dy || !a->x || !a->dx)) return fail(CONV_ERR_INVALID_ARG, "dy, x or dx is NULL");
    if ((st = check_workspace(workspace, workspace_bytes, plan->ws_bytes)) != CONV_OK) return st;
    if ((st = check_overlap(out, 5, in, 7)) != CONV_OK) return st;
    const Rows vec[] = {in[0], in[1], in[2], in[3], in[4], in[5], out[0], out[3]};
    // A gradient thread holds its run's rows of x and dy: by 8 bytes they leave
    // room for three waves per SIMD, by 16 for one (training case 35 and 54 us).
    const int V = conv_vector(d, e, vec, 8) == 1 ? 1 : (int)(8 / e);
    CausalParams p{};
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.state = a->state; p.lengths = a->lengths;
    p.dy = a->dy; p.dstate_out = a->dstate_out; p.dx = a->dx; p.dstate = a->dstate;
    p.partial = (float *)workspace;
    p.x_ld = stride(in[1]); p.dy_ld = stride(in[0]); p.dx_ld = stride(out[0]);
    p.N = (int)d.N; p.C = (int)d.C; p.CV = (int)(d.C / V); p.L = d.L;
    p.blocks = bwd_blocks(d);
    const int64_t wgs = plan->bwd_rows * channel_blocks(p.CV), sums = (d.F + 1) * channel_blocks(d.C);
    if (!one_launch((double)wgs, 256) || !one_launch((double)sums, 256))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x C is too large for one launch");
    (void)hipGetLastError();
    hipStream_t s = (hipStream_t)stream;
    if (d.N > 0) launch_causal(CONV_BWD, d, V, p, wgs, s);
    const dim3 grid((unsigned)sums);      // no rows: dw and dbias are zeros
    if (d.dtype == CONV_DT_BF16)
        hipLaunchKernelGGL(causal_reduce_kernel<bf16_t>, grid, dim3(256), 0, s, p.partial, (bf16_t *)a->dw,
                           (bf16_t *)a->dbias, plan->bwd_rows, (int)d.C, (int)d.F);
    else
        hipLaunchKernelGGL(causal_reduce_kernel<float>, grid, dim3(256), 0, s, p.partial, (float *)a->dw,
                           (float *)a->dbias, plan->bwd_rows, (int)d.C, (int)d.F);
    return launched();
}

void conv_causal_destroy(conv_causal_plan_t *plan) { delete plan; }

const char *conv_causal_describe(const conv_causal_plan_t *plan) { return plan ? plan->text : ""; }

// ---- scan ------------------------------------------------------------------------
conv_status_t conv_scan_create(const conv_scan_desc_t *desc, conv_scan_plan_t **plan)
{
    if (!plan) return fail(CONV_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "descriptor is NULL");
    const conv_scan_desc_t &d = *desc;
    if (d.dtype != CONV_DT_F32 && d.dtype != CONV_DT_BF16) return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", d.dtype);
    if (d.softplus != 0 && d.softplus != 1) return fail(CONV_ERR_INVALID_ARG, "softplus must be 0 or 1");
    if (d.N < 0 || d.L < 0 || d.H < 1 || d.P < 1 || d.G < 1 || d.S < 1)
        return fail(CONV_ERR_INVALID_ARG, "need N, L >= 0 and H, P, G, S >= 1 (got %lld, %lld, %lld, %lld, %lld, %lld)",
                    (long long)d.N, (long long)d.L, (long long)d.H, (long long)d.P, (long long)d.G, (long long)d.S);
    if (d.H % d.G != 0)
        return fail(CONV_ERR_INVALID_ARG, "H = %lld is not a multiple of G = %lld", (long long)d.H, (long long)d.G);
    if (d.S > 128) return fail(CONV_ERR_UNSUPPORTED, "more than 128 states (S = %lld)", (long long)d.S);
    if (d.P > 65536) return fail(CONV_ERR_UNSUPPORTED, "more than 65536 channels of a head (P = %lld)", (long long)d.P);
    if (d.N > kMaxDim || d.L > kMaxDim || d.H > kMaxDim) return fail(CONV_ERR_UNSUPPORTED, "N, L or H above 2^30");
    conv_scan_plan *pl = new (std::nothrow) conv_scan_plan();
    if (!pl) return fail(CONV_ERR_NOMEM, "plan allocation failed");
    pl->desc = d;
    pl->esz = d.dtype == CONV_DT_BF16 ? 2 : 4;
    pl->SP = d.S <= 32 ? 32 : d.S <= 64 ? 64 : 128;
    pl->Q = d.dtype == CONV_DT_BF16 ? Frag<bf16_t>::Q : Frag<float>::Q;
    pl->K = (int)std::max<int64_t>(1, (d.L + pl->Q - 1) / pl->Q);
    pl->NPB = (int)((d.P + kPB - 1) / kPB);
    const double units = (double)d.N * d.H * pl->NPB, tile = (double)pl->SP * kPB * 4;
    const double rows = (double)d.N * d.L * d.G * pl->SP;
    // What neither a prompt (a workgroup of 64 channels at least) nor a step could launch; every call checks its own.
    if ((!one_launch(units, 256) && !one_launch((double)d.N * d.H * step_shape(d).blocks, 256)) || rows * 4 >= kMaxBytes || units * (pl->K + 1) * tile * 4 >= kMaxBytes) {
        delete pl;
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    }
    pl->units = d.N * d.H * pl->NPB;
    // With fewer heads than compute units the long axis is split, at the price of
    // a first pass over x and B.  One direct-to-LDS workgroup fits a compute unit
    // and two of the others; the first pass's are smaller and finer ones fill
    // the chip.
    const int64_t cus = 256;
    pl->fwd = split_segments(pl->units, pl->K, pl->units >= cus ? 0 : 2 * cus, 1);
    pl->dma = split_segments(pl->units, pl->K, cus, 2);
    pl->bwd = split_segments(pl->units, pl->K, cus, 1);
    const int64_t chunks = d.N * pl->K * d.G, hpg = d.H / d.G;
    // one gradient workgroup fits a compute unit
    const int64_t want = std::max<int64_t>(1, std::min(hpg, cus / std::max<int64_t>(1, chunks)));
    pl->heads_per_slice = (int)((hpg + want - 1) / want);
    pl->slices = (int)((hpg + pl->heads_per_slice - 1) / pl->heads_per_slice);
    const int64_t t = (int64_t)pl->SP * kPB * 4;
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int64_t most = std::max(pl->fwd.count > pl->fwd.sub ? pl->fwd.count : 0, pl->dma.count > pl->dma.sub ? pl->dma.count : 0);
    pl->o_fwd_log = up(pl->units * most * t);
    pl->ws_bytes = pl->o_fwd_log + up(pl->units * most * 4);
    int64_t o = 0;
    for (int k = 0; k < 2; ++k) {
        pl->o_seg[k] = o;
        o += pl->bwd.count > 1 ? up(pl->units * pl->bwd.count * t) : 0;
        pl->o_log[k] = o;
        o += pl->bwd.count > 1 ? up(pl->units * pl->bwd.count * 4) : 0;
        pl->o_bound[k] = o;
        o += up(pl->units * pl->K * t);
    }
    pl->o_head = o;
    o += up(3 * d.N * pl->K * d.H * 4);
    pl->o_pb = o;
    const int64_t part = pl->slices > 1 ? up((int64_t)pl->slices * d.N * d.L * d.G * pl->SP * 4) : 0;
    pl->o_pc = o + part;
    pl->bwd_ws_bytes = o + 2 * part;
    snprintf(pl->text, sizeof(pl->text),
             "scan %s N=%lld L=%lld H=%lld P=%lld G=%lld S=%lld(%d)%s, %d chunks of %d in %d segments "
             "(%d x %d of whole bf16 vectors); gradient: %d segments, %d slices of %d heads",
             d.dtype == CONV_DT_BF16 ? "bf16" : "f32", (long long)d.N, (long long)d.L, (long long)d.H, (long long)d.P,
             (long long)d.G, (long long)d.S, pl->SP, d.softplus ? " softplus" : "", pl->K, pl->Q, pl->fwd.count,
             pl->dma.count / pl->dma.sub, pl->dma.sub, pl->bwd.count, pl->slices, pl->heads_per_slice);
    if (getenv("CONVFWD_LOG")) fprintf(stderr, "convfwd: %s\n", pl->text);
    *plan = pl;
    return CONV_OK;
}

conv_status_t conv_scan_workspace_bytes(const conv_scan_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->ws_bytes;
    return CONV_OK;
}

conv_status_t conv_scan_bwd_workspace_bytes(const conv_scan_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->bwd_ws_bytes;
    return CONV_OK;
}

// 16-byte accesses to heads' channels and groups' states
static bool scan_vector(const conv_scan_plan &pl, const Rows *t, int n)
{
    bool ok = pl.desc.P * pl.esz % 16 == 0 && pl.desc.S * pl.esz % 16 == 0;
    for (int i = 0; i < n; ++i) ok = ok && vector_rows(t[i]);
    return ok;
}

static conv_status_t scan_forward(const conv_scan_plan_t *plan, const conv_scan_args_t *a, bool step, void *ws,
                                  int64_t ws_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_scan_desc_t &d = plan->desc;
    const int64_t L = step ? 1 : d.L, e = plan->esz, rows = d.N * L, need = step ? 0 : plan->ws_bytes;
    if (!a->a) return fail(CONV_ERR_INVALID_ARG, "a is NULL");
    if (step && a->lengths) return fail(CONV_ERR_INVALID_ARG, "a step takes no lengths");
    const int64_t hp = d.H * d.P, gs = d.G * d.S, states = d.N * hp * d.S;
    const Rows in[] = {{"x", a->x, rows, hp, or_packed(a->x_ld, hp), e},
                       {"b", a->b, rows, gs, or_packed(a->b_ld, gs), e},
                       {"c", a->c, rows, gs, or_packed(a->c_ld, gs), e},
                       {"dt", a->dt, rows, d.H, or_packed(a->dt_ld, d.H), e},
                       {"a", a->a, 1, d.H, d.H, 4},
                       {"d", a->d, 1, d.H, d.H, 4},
                       {"dt_bias", a->dt_bias, 1, d.H, d.H, 4},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4},
                       {"state", a->state, 1, states, states, 4}};
    const Rows out[] = {{"y", a->y, rows, hp, or_packed(a->y_ld, hp), e},
                        {"state_out", a->state_out, 1, states, states, 4},
                        {"workspace", ws, 1, need, std::max<int64_t>(1, need), 1}};
    conv_status_t st = check_rows(in, 9);
    if (st == CONV_OK) st = check_rows(out, 2);
    if (st != CONV_OK) return st;
    if (d.N == 0) return CONV_OK;
    if (L > 0 && (!a->x || !a->b || !a->c || !a->dt || !a->y)) return fail(CONV_ERR_INVALID_ARG, "x, b, c, dt or y is NULL");
    if (step && (!a->state || !a->state_out)) return fail(CONV_ERR_INVALID_ARG, "state or state_out is NULL");
    if ((st = check_workspace(ws, ws_bytes, need)) != CONV_OK) return st;
    // a step may update the state in place: each lane owns its part
    const bool in_place = step && a->state == a->state_out;
    if ((st = check_overlap(out, 3, in, in_place ? 8 : 9)) != CONV_OK) return st;
    ScanParams p;
    scan_params(*plan, &p);
    p.L = L;
    p.x = a->x; p.dt = a->dt; p.b = a->b; p.c = a->c; p.a = a->a; p.d = a->d; p.dt_bias = a->dt_bias;
    p.state = a->state; p.lengths = a->lengths; p.y = a->y; p.state_out = a->state_out;
    p.x_ld = stride(in[0]); p.b_ld = stride(in[1]); p.c_ld = stride(in[2]); p.dt_ld = stride(in[3]); p.y_ld = stride(out[0]);
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (step) {
        const StepShape shape = step_shape(d);
        const int lpr = shape.lanes, blocks = shape.blocks;
        const bool vec = d.S % 4 == 0 && ((uintptr_t)a->state | (uintptr_t)a->state_out) % 16 == 0;
        if (!one_launch((double)(d.N * d.H * blocks), 256))
            return fail(CONV_ERR_UNSUPPORTED, "N x H x P is too large for one launch");
        const dim3 grid((unsigned)(d.N * d.H * blocks));
        if (d.dtype == CONV_DT_BF16) {
            if (vec) hipLaunchKernelGGL((scan_step_kernel<bf16_t, true>), grid, dim3(256), 0, s, p, lpr, blocks);
            else hipLaunchKernelGGL((scan_step_kernel<bf16_t, false>), grid, dim3(256), 0, s, p, lpr, blocks);
        } else {
            if (vec) hipLaunchKernelGGL((scan_step_kernel<float, true>), grid, dim3(256), 0, s, p, lpr, blocks);
            else hipLaunchKernelGGL((scan_step_kernel<float, false>), grid, dim3(256), 0, s, p, lpr, blocks);
        }
        return launched();
    }
    if (need > 0) {
        p.seg_state[0] = (float *)ws;
        p.seg_log[0] = (float *)((char *)ws + plan->o_fwd_log);
    }
    const Rows vec[] = {in[0], in[1], in[2], out[0]};
    p.vec = scan_vector(*plan, vec, 4);
    const bool dma = p.vec && d.dtype == CONV_DT_BF16;
    set_segments(&p, dma ? plan->dma : plan->fwd);
    if (!one_launch((double)(plan->units * (p.nseg - p.sub)), 256) ||
        !one_launch((double)(plan->units * (p.nseg / p.sub)), dma ? 512 : 256))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    if (d.dtype == CONV_DT_BF16) launch_scan<bf16_t>(plan->SP, p, plan->units, nullptr, s);
    else launch_scan<float>(plan->SP, p, plan->units, nullptr, s);
    return launched();
}

conv_status_t conv_scan_run(const conv_scan_plan_t *plan, const conv_scan_args_t *args, void *workspace,
                            int64_t workspace_bytes, void *stream)
{
    return scan_forward(plan, args, false, workspace, workspace_bytes, stream);
}

conv_status_t conv_scan_step(const conv_scan_plan_t *plan, const conv_scan_args_t *args, void *stream)
{
    return scan_forward(plan, args, true, nullptr, 0, stream);
}

conv_status_t conv_scan_bwd_run(const conv_scan_plan_t *plan, const conv_scan_bwd_args_t *a, void *workspace,
                                int64_t workspace_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_scan_desc_t &d = plan->desc;
    const int64_t e = plan->esz, rows = d.N * d.L, hp = d.H * d.P, gs = d.G * d.S, states = d.N * hp * d.S;
    if (!a->a || !a->da) return fail(CONV_ERR_INVALID_ARG, "a or da is NULL");
    if ((a->d != nullptr) != (a->dd != nullptr) || (a->dt_bias != nullptr) != (a->ddt_bias != nullptr))
        return fail(CONV_ERR_INVALID_ARG, "dd must be NULL iff d is, and ddt_bias iff dt_bias is");
    const Rows in[] = {{"dy", a->dy, rows, hp, or_packed(a->dy_ld, hp), e},
                       {"x", a->x, rows, hp, or_packed(a->x_ld, hp), e},
                       {"b", a->b, rows, gs, or_packed(a->b_ld, gs), e},
                       {"c", a->c, rows, gs, or_packed(a->c_ld, gs), e},
                       {"dt", a->dt, rows, d.H, or_packed(a->dt_ld, d.H), e},
                       {"a", a->a, 1, d.H, d.H, 4},
                       {"d", a->d, 1, d.H, d.H, 4},
                       {"dt_bias", a->dt_bias, 1, d.H, d.H, 4},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4},
                       {"state", a->state, 1, states, states, 4},
                       {"dstate_out", a->dstate_out, 1, states, states, 4}};
    const Rows out[] = {{"dx", a->dx, rows, hp, or_packed(a->dx_ld, hp), e},
                        {"db", a->db, rows, gs, or_packed(a->db_ld, gs), e},
                        {"dc", a->dc, rows, gs, or_packed(a->dc_ld, gs), e},
                        {"ddt", a->ddt, rows, d.H, or_packed(a->ddt_ld, d.H), e},
                        {"da", a->da, 1, d.H, d.H, 4},
                        {"dd", a->dd, 1, d.H, d.H, 4},
                        {"ddt_bias", a->ddt_bias, 1, d.H, d.H, 4},
                        {"dstate", a->dstate, 1, states, states, 4},
                        {"workspace", workspace, 1, plan->bwd_ws_bytes, std::max<int64_t>(1, plan->bwd_ws_bytes), 1}};
    conv_status_t st = check_rows(in, 11);
    if (st == CONV_OK) st = check_rows(out, 8);
    if (st != CONV_OK) return st;
    if (rows > 0 && (!a->dy || !a->x || !a->b || !a->c || !a->dt || !a->dx || !a->db || !a->dc || !a->ddt))
        return fail(CONV_ERR_INVALID_ARG, "dy, x, b, c, dt, dx, db, dc or ddt is NULL");
    if ((st = check_workspace(workspace, workspace_bytes, plan->bwd_ws_bytes)) != CONV_OK) return st;
    if ((st = check_overlap(out, 9, in, 11)) != CONV_OK) return st;
    ScanParams p;
    scan_params(*plan, &p);
    p.x = a->x; p.dt = a->dt; p.b = a->b; p.c = a->c; p.a = a->a; p.d = a->d; p.dt_bias = a->dt_bias;
    p.state = a->state; p.lengths = a->lengths; p.dy = a->dy; p.dstate_out = a->dstate_out;
    p.dx = a->dx; p.ddt = a->ddt; p.db = a->db; p.dc = a->dc; p.dstate = a->dstate;
    p.dy_ld = stride(in[0]); p.x_ld = stride(in[1]); p.b_ld = stride(in[2]); p.c_ld = stride(in[3]); p.dt_ld = stride(in[4]);
    p.dx_ld = stride(out[0]); p.db_ld = stride(out[1]); p.dc_ld = stride(out[2]); p.ddt_ld = stride(out[3]);
    const Rows vec[] = {in[0], in[1], in[2], in[3], out[0]};
    p.vec = scan_vector(*plan, vec, 5);
    char *ws = (char *)workspace;
    set_segments(&p, plan->bwd);
    const HeadGrads g = {a->da, a->ddt_bias, a->dd, scan_reduce_grid(*plan)};
    if (!one_launch((double)(2 * plan->units * p.nseg), 256) || !one_launch((double)(d.N * plan->K * d.G * plan->slices), 512) ||
        !one_launch((double)g.workgroups, 256))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    for (int k = 0; k < 2; ++k) {
        p.seg_state[k] = (float *)(ws + plan->o_seg[k]);
        p.seg_log[k] = (float *)(ws + plan->o_log[k]);
        p.bound[k] = (float *)(ws + plan->o_bound[k]);
    }
    p.part_head = (float *)(ws + plan->o_head);
    p.part_b = (float *)(ws + plan->o_pb);
    p.part_c = (float *)(ws + plan->o_pc);
    p.slices = plan->slices;
    p.heads_per_slice = plan->heads_per_slice;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d.dtype == CONV_DT_BF16) launch_scan<bf16_t>(plan->SP, p, plan->units, &g, s);
    else launch_scan<float>(plan->SP, p, plan->units, &g, s);
    return launched();
}

void conv_scan_destroy(conv_scan_plan_t *plan) { delete plan; }

const char *conv_scan_describe(const conv_scan_plan_t *plan) { return plan ? plan->text : ""; }

}  // extern "C"
