// Host side of the gated delta rule (conv_delta_*): argument checks, workspace
// layout, launches.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>
#include <type_traits>

#include "../../include/convfwd.h"
#include "delta_chain.h"
#include "seq_host.h"
#include "status.h"

struct conv_delta_plan {
    conv_delta_desc_t desc;
    int64_t esz;
    int SP, K, blocks;                   // padded keys, chunks, blocks of 16 channels of a head
    int slices, heads_per_slice;         // of a group's heads, for what a chunk does without its state
    int64_t ws_bytes, o_heads;
    int PP, grad_slices, grad_heads;     // the gradient's padded channels, and its slices of a group's heads
    int64_t bwd_ws_bytes, o_bwd_heads, o_bound[2], o_rows[2], o_part[2];
    char text[256];
};

namespace convfwd {
namespace {

int64_t up(int64_t v) { return (v + 255) / 256 * 256; }

template <typename T> int64_t keys_of(int SP, bool grad)
{
    return SP == 32 ? keys_bytes<T, 32>(grad) : SP == 64 ? keys_bytes<T, 64>(grad)
         : SP == 128 ? keys_bytes<T, 128>(grad) : keys_bytes<T, 256>(grad);
}
int64_t keys_of(const conv_delta_desc_t &d, int SP, bool grad)
{
    return d.dtype == CONV_DT_BF16 ? keys_of<bf16_t>(SP, grad) : keys_of<float>(SP, grad);
}
int64_t head_of(const conv_delta_desc_t &d, bool grad)
{
    return d.dtype == CONV_DT_BF16 ? head_bytes<bf16_t>(grad) : head_bytes<float>(grad);
}

int64_t state_grid(int64_t units) { return (units + 7) / 8 * 8; }

// A workgroup takes one block of 16 channels, or two where there would be more
// workgroups than compute units, each of which holds one: both blocks go through the
// chunk's barriers and share its loads of K and N.  Above 128 keys there is no room for
// two.  Whole calls of 2048 tokens in us, a block each | two:
//
//   blocks       bf16, 32 keys   64          128         fp32, 32    64          128
//   256            67 |  92       71 |  91    81 | 105    82 | 118    97 | 139   132 | 186
//   264           104 |  92      109 |  94   129 | 107   142 | 123   162 | 141   218 | 189
//   512           115 | 102      126 | 107   148 | 125   154 | 135   182 | 163   256 | 227
//   gradient, 256 234 | 230      260 | 254   319 | 304   284 | 292   335 | 337   423 | 414
//   gradient, 512 512 | 446      577 | 498   682 | 590   585 | 529   690 | 615   849 | 751
//
// (A gradient's 256 blocks are 512 units, both directions.)
bool two_blocks(int SP, double units) { return SP <= kMostPaired && units > 256; }

// Workgroups of a pass over the states of N H heads of `blocks` blocks in so many directions.
double chain_grid(int SP, int directions, int64_t heads, int64_t blocks)
{
    if (two_blocks(SP, (double)directions * heads * blocks)) blocks = (blocks + 1) / 2;
    return (double)directions * state_grid(heads * blocks);
}

template <typename T, int SP, typename F> void paired(DeltaParams &p, int directions, F launch)
{
    if constexpr (SP <= kMostPaired) {
        if (two_blocks(SP, (double)directions * p.N * p.H * p.blocks)) {
            p.blocks = (p.blocks + 1) / 2;
            return launch(std::integral_constant<int, 2>());
        }
    }
    launch(std::integral_constant<int, 1>());
}

template <typename T, int SP> void launch_fwd(DeltaParams p, hipStream_t s)
{
    if (p.K > 0)
        hipLaunchKernelGGL((delta_prepare_kernel<T, SP, false>), dim3((unsigned)((int64_t)p.N * p.K * p.G * p.slices)), dim3(256),
                           0, s, p);
    paired<T, SP>(p, 1, [&](auto cb) {
        hipLaunchKernelGGL((delta_y_kernel<T, SP, decltype(cb)::value>), dim3((unsigned)state_grid((int64_t)p.N * p.H * p.blocks)),
                           dim3(kChainThreads), 0, s, p);
    });
}

// The gradient: what chunks do without their states, both passes over the states,
// the gradients of the chunks and, where a group's heads are sliced, their sums.
template <typename T, int SP> void launch_bwd(DeltaParams p, const conv_delta_plan &pl, hipStream_t s)
{
    const int64_t chunks = (int64_t)p.N * p.K * p.G;
    if (p.K > 0)
        hipLaunchKernelGGL((delta_prepare_kernel<T, SP, true>), dim3((unsigned)(chunks * p.slices)), dim3(256), 0, s, p);
    paired<T, SP>(p, 2, [&](auto cb) {
        hipLaunchKernelGGL((delta_states_kernel<T, SP, decltype(cb)::value>),
                           dim3((unsigned)(2 * state_grid((int64_t)p.N * p.H * p.blocks))), dim3(kChainThreads), 0, s, p);
    });
    if (p.K == 0) return;
    p.slices = pl.grad_slices;
    p.heads_per_slice = pl.grad_heads;
    hipLaunchKernelGGL((delta_grad_kernel<T, SP>), dim3((unsigned)(chunks * p.slices)), dim3(64 * GradShape<T, SP>::NW), 0, s, p);
    if (p.slices > 1) {
        const int64_t grid = ((int64_t)p.N * p.L * p.G * p.S + 255) / 256;
        hipLaunchKernelGGL((delta_reduce_kernel<T>), dim3((unsigned)grid), dim3(256), 0, s, p);
    }
}

template <typename T, int SP> void launch_delta(const DeltaParams &p, const conv_delta_plan &pl, bool grad, hipStream_t s)
{
    if (grad) launch_bwd<T, SP>(p, pl, s);
    else launch_fwd<T, SP>(p, s);
}

template <typename T> void launch_delta(const DeltaParams &p, const conv_delta_plan &pl, bool grad, hipStream_t s)
{
    if (pl.SP == 32) return launch_delta<T, 32>(p, pl, grad, s);
    if (pl.SP == 64) return launch_delta<T, 64>(p, pl, grad, s);
    if (pl.SP == 128) return launch_delta<T, 128>(p, pl, grad, s);
    return launch_delta<T, 256>(p, pl, grad, s);
}

// Slices of a group's `heads` so that `groups` of them give about `want` workgroups.
void slice_heads(int64_t groups, int64_t heads, int64_t want, int *slices, int *per)
{
    const int64_t n = std::max<int64_t>(1, std::min(heads, want / std::max<int64_t>(1, groups)));
    *per = (int)((heads + n - 1) / n);
    *slices = (int)((heads + *per - 1) / *per);
}

// A step's lanes for the keys of a channel, and workgroups for the channels of a head.
struct StepShape {
    int lanes, blocks;
};

StepShape step_shape(const conv_delta_desc_t &d)
{
    int lanes = 1;
    while (lanes * 4 < d.S) lanes *= 2;
    const int64_t per = 4 * kDeltaRows * (64 / lanes);
    return {lanes, (int)((d.P + per - 1) / per)};
}

void delta_params(const conv_delta_plan &pl, DeltaParams *p)
{
    const conv_delta_desc_t &d = pl.desc;
    *p = DeltaParams{};
    p->N = (int)d.N; p->L = d.L; p->H = (int)d.H; p->P = (int)d.P; p->G = (int)d.G; p->S = (int)d.S;
    p->K = pl.K; p->blocks = pl.blocks; p->slices = pl.slices; p->heads_per_slice = pl.heads_per_slice;
    p->scale = (float)d.scale;
}

}  // namespace
}  // namespace convfwd

using namespace convfwd;

extern "C" {

conv_status_t conv_delta_create(const conv_delta_desc_t *desc, conv_delta_plan_t **plan)
{
    if (!plan) return fail(CONV_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "descriptor is NULL");
    const conv_delta_desc_t &d = *desc;
    if (d.dtype != CONV_DT_F32 && d.dtype != CONV_DT_BF16) return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", d.dtype);
    if (d.reserved != 0) return fail(CONV_ERR_INVALID_ARG, "reserved must be 0");
    if (!std::isfinite((float)d.scale)) return fail(CONV_ERR_INVALID_ARG, "scale must be a finite fp32 number");
    if (d.N < 0 || d.L < 0 || d.H < 1 || d.P < 1 || d.G < 1 || d.S < 1)
        return fail(CONV_ERR_INVALID_ARG, "need N, L >= 0 and H, P, G, S >= 1 (got %lld, %lld, %lld, %lld, %lld, %lld)",
                    (long long)d.N, (long long)d.L, (long long)d.H, (long long)d.P, (long long)d.G, (long long)d.S);
    if (d.H % d.G != 0)
        return fail(CONV_ERR_INVALID_ARG, "H = %lld is not a multiple of G = %lld", (long long)d.H, (long long)d.G);
    if (d.S > 256) return fail(CONV_ERR_UNSUPPORTED, "more than 256 keys (S = %lld)", (long long)d.S);
    if (d.P > 65536) return fail(CONV_ERR_UNSUPPORTED, "more than 65536 channels of a head (P = %lld)", (long long)d.P);
    if (d.N > kMaxDim || d.L > kMaxDim || d.H > kMaxDim) return fail(CONV_ERR_UNSUPPORTED, "N, L or H above 2^30");
    conv_delta_plan *pl = new (std::nothrow) conv_delta_plan();
    if (!pl) return fail(CONV_ERR_NOMEM, "plan allocation failed");
    pl->desc = d;
    pl->esz = d.dtype == CONV_DT_BF16 ? 2 : 4;
    pl->SP = d.S <= 32 ? 32 : d.S <= 64 ? 64 : d.S <= 128 ? 128 : 256;
    pl->K = (int)((d.L + kDQ - 1) / kDQ);
    pl->blocks = (int)((d.P + 15) / 16);
    // What neither a prompt nor a step could launch; every call checks its own form.
    const double chunks = (double)d.N * pl->K;
    const double ws = chunks * ((double)d.G * keys_of(d, pl->SP, true) + (double)d.H * head_of(d, true)) +
                      2.0 * (double)d.N * d.H * pl->K * ((d.P + 31.0) * (pl->SP + kDQ) + 2.0 * kApart) * 4.0;
    if ((!one_launch(chain_grid(pl->SP, 1, d.N * d.H, pl->blocks), kChainThreads) &&
         !one_launch((double)d.N * d.H * step_shape(d).blocks, 256)) || ws >= kMaxBytes) {
        delete pl;
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    }
    // two workgroups of the preparation fit a compute unit, one of the gradient's
    const int64_t groups = d.N * pl->K * d.G, hpg = d.H / d.G;
    slice_heads(groups, hpg, 512, &pl->slices, &pl->heads_per_slice);
    slice_heads(groups, hpg, 256, &pl->grad_slices, &pl->grad_heads);
    pl->o_heads = up(d.N * pl->K * d.G * keys_of(d, pl->SP, false));
    pl->ws_bytes = pl->o_heads + up(d.N * pl->K * d.H * head_of(d, false));
    pl->PP = (int)((d.P + 31) / 32 * 32);
    int64_t o = up(groups * keys_of(d, pl->SP, true));
    pl->o_bwd_heads = o;
    o += up(d.N * pl->K * d.H * head_of(d, true));
    const int64_t states = up(d.N * d.H * pl->K * states_floats(pl->PP, pl->SP) * 4), tokens = up(d.N * d.H * pl->K * rows_floats(pl->PP) * 4);
    const int64_t part = hpg > 1 ? up((int64_t)pl->grad_slices * d.N * d.L * d.G * d.S * 4) : 0;
    for (int k = 0; k < 2; ++k) {
        pl->o_bound[k] = o + k * states;
        pl->o_rows[k] = o + 2 * states + k * tokens;
        pl->o_part[k] = o + 2 * states + 2 * tokens + k * part;
    }
    pl->bwd_ws_bytes = o + 2 * (states + tokens + part);
    snprintf(pl->text, sizeof(pl->text),
             "delta %s N=%lld L=%lld H=%lld P=%lld G=%lld S=%lld(%d), %d chunks of %d, %d slices of %d heads; "
             "gradient: %d slices of %d heads",
             d.dtype == CONV_DT_BF16 ? "bf16" : "f32", (long long)d.N, (long long)d.L, (long long)d.H, (long long)d.P,
             (long long)d.G, (long long)d.S, pl->SP, pl->K, kDQ, pl->slices, pl->heads_per_slice,
             pl->grad_slices, pl->grad_heads);
    if (getenv("CONVFWD_LOG")) fprintf(stderr, "convfwd: %s\n", pl->text);
    *plan = pl;
    return CONV_OK;
}

conv_status_t conv_delta_workspace_bytes(const conv_delta_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->ws_bytes;
    return CONV_OK;
}

conv_status_t conv_delta_bwd_workspace_bytes(const conv_delta_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->bwd_ws_bytes;
    return CONV_OK;
}

// 16-byte accesses to the keys
static bool delta_vector(const conv_delta_plan &pl, const Rows *t, int n)
{
    bool ok = pl.desc.S * pl.esz % 16 == 0;
    for (int i = 0; i < n; ++i) ok = ok && vector_rows(t[i]);
    return ok;
}

static conv_status_t delta_forward_call(const conv_delta_plan_t *plan, const conv_delta_args_t *a, bool step, void *ws,
                                        int64_t ws_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_delta_desc_t &d = plan->desc;
    const int64_t L = step ? 1 : d.L, e = plan->esz, rows = d.N * L, need = step ? 0 : plan->ws_bytes;
    if (step && a->lengths) return fail(CONV_ERR_INVALID_ARG, "a step takes no lengths");
    const int64_t hp = d.H * d.P, gs = d.G * d.S, states = d.N * hp * d.S;
    const Rows in[] = {{"q", a->q, rows, gs, or_packed(a->q_ld, gs), e},
                       {"k", a->k, rows, gs, or_packed(a->k_ld, gs), e},
                       {"v", a->v, rows, hp, or_packed(a->v_ld, hp), e},
                       {"g", a->g, rows, d.H, or_packed(a->g_ld, d.H), 4},
                       {"beta", a->beta, rows, d.H, or_packed(a->beta_ld, d.H), e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4},
                       {"state", a->state, 1, states, states, 4}};
    const Rows out[] = {{"y", a->y, rows, hp, or_packed(a->y_ld, hp), e},
                        {"state_out", a->state_out, 1, states, states, 4},
                        {"workspace", ws, 1, need, std::max<int64_t>(1, need), 1}};
    conv_status_t st = check_rows(in, 7);
    if (st == CONV_OK) st = check_rows(out, 2);
    if (st != CONV_OK) return st;
    if (d.N == 0) return CONV_OK;
    if (L > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->y))
        return fail(CONV_ERR_INVALID_ARG, "q, k, v, g, beta or y is NULL");
    if (step && (!a->state || !a->state_out)) return fail(CONV_ERR_INVALID_ARG, "state or state_out is NULL");
    if ((st = check_workspace(ws, ws_bytes, need)) != CONV_OK) return st;
    // a step may update the state in place: each lane owns its part
    const bool in_place = step && a->state == a->state_out;
    if ((st = check_overlap(out, 3, in, in_place ? 6 : 7)) != CONV_OK) return st;
    if (L == 0 && !a->state_out) return CONV_OK;
    DeltaParams p;
    delta_params(*plan, &p);
    p.L = L;
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta; p.state = a->state; p.lengths = a->lengths;
    p.y = a->y; p.state_out = a->state_out;
    p.q_ld = stride(in[0]); p.k_ld = stride(in[1]); p.v_ld = stride(in[2]); p.g_ld = stride(in[3]);
    p.beta_ld = stride(in[4]); p.y_ld = stride(out[0]);
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (step) {
        const StepShape shape = step_shape(d);
        const bool vec = d.S % 4 == 0 && ((uintptr_t)a->state | (uintptr_t)a->state_out) % 16 == 0;
        if (!one_launch((double)(d.N * d.H) * shape.blocks, 256))
            return fail(CONV_ERR_UNSUPPORTED, "N x H x P is too large for one launch");
        const dim3 grid((unsigned)(d.N * d.H * shape.blocks));
        if (d.dtype == CONV_DT_BF16) {
            if (vec) hipLaunchKernelGGL((delta_step_kernel<bf16_t, true>), grid, dim3(256), 0, s, p, shape.lanes, shape.blocks);
            else hipLaunchKernelGGL((delta_step_kernel<bf16_t, false>), grid, dim3(256), 0, s, p, shape.lanes, shape.blocks);
        } else {
            if (vec) hipLaunchKernelGGL((delta_step_kernel<float, true>), grid, dim3(256), 0, s, p, shape.lanes, shape.blocks);
            else hipLaunchKernelGGL((delta_step_kernel<float, false>), grid, dim3(256), 0, s, p, shape.lanes, shape.blocks);
        }
        return launched();
    }
    p.keys = (char *)ws;
    p.heads = (char *)ws + plan->o_heads;
    const Rows vec[] = {in[0], in[1]};
    p.vec = delta_vector(*plan, vec, 2);
    if (!one_launch(chain_grid(plan->SP, 1, d.N * d.H, plan->blocks), kChainThreads) ||
        !one_launch((double)d.N * plan->K * d.G * plan->slices, 256))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    if (d.dtype == CONV_DT_BF16) launch_delta<bf16_t>(p, *plan, false, s);
    else launch_delta<float>(p, *plan, false, s);
    return launched();
}

conv_status_t conv_delta_run(const conv_delta_plan_t *plan, const conv_delta_args_t *args, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    return delta_forward_call(plan, args, false, workspace, workspace_bytes, stream);
}

conv_status_t conv_delta_step(const conv_delta_plan_t *plan, const conv_delta_args_t *args, void *stream)
{
    return delta_forward_call(plan, args, true, nullptr, 0, stream);
}

conv_status_t conv_delta_bwd_run(const conv_delta_plan_t *plan, const conv_delta_bwd_args_t *a, void *workspace,
                                 int64_t workspace_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_delta_desc_t &d = plan->desc;
    const int64_t e = plan->esz, rows = d.N * d.L, hp = d.H * d.P, gs = d.G * d.S, states = d.N * hp * d.S;
    if (a->dstate && !a->state) return fail(CONV_ERR_INVALID_ARG, "dstate without a state");
    const Rows in[] = {{"dy", a->dy, rows, hp, or_packed(a->dy_ld, hp), e},
                       {"q", a->q, rows, gs, or_packed(a->q_ld, gs), e},
                       {"k", a->k, rows, gs, or_packed(a->k_ld, gs), e},
                       {"v", a->v, rows, hp, or_packed(a->v_ld, hp), e},
                       {"g", a->g, rows, d.H, or_packed(a->g_ld, d.H), 4},
                       {"beta", a->beta, rows, d.H, or_packed(a->beta_ld, d.H), e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4},
                       {"state", a->state, 1, states, states, 4},
                       {"dstate_out", a->dstate_out, 1, states, states, 4}};
    const int64_t need = plan->bwd_ws_bytes;
    const Rows out[] = {{"dq", a->dq, rows, gs, or_packed(a->dq_ld, gs), e},
                        {"dk", a->dk, rows, gs, or_packed(a->dk_ld, gs), e},
                        {"dv", a->dv, rows, hp, or_packed(a->dv_ld, hp), e},
                        {"dg", a->dg, rows, d.H, or_packed(a->dg_ld, d.H), 4},
                        {"dbeta", a->dbeta, rows, d.H, or_packed(a->dbeta_ld, d.H), e},
                        {"dstate", a->dstate, 1, states, states, 4},
                        {"workspace", workspace, 1, need, std::max<int64_t>(1, need), 1}};
    conv_status_t st = check_rows(in, 9);
    if (st == CONV_OK) st = check_rows(out, 6);
    if (st != CONV_OK) return st;
    if (d.N == 0) return CONV_OK;
    if (rows > 0 && (!a->dy || !a->q || !a->k || !a->v || !a->g || !a->beta || !a->dq || !a->dk || !a->dv || !a->dg || !a->dbeta))
        return fail(CONV_ERR_INVALID_ARG, "dy, q, k, v, g, beta, dq, dk, dv, dg or dbeta is NULL");
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CONV_OK) return st;
    if ((st = check_overlap(out, 7, in, 9)) != CONV_OK) return st;
    if (rows == 0 && !a->dstate) return CONV_OK;
    DeltaParams p;
    delta_params(*plan, &p);
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta; p.state = a->state; p.lengths = a->lengths;
    p.dy = a->dy; p.dstate_out = a->dstate_out; p.dq = a->dq; p.dk = a->dk; p.dv = a->dv; p.dg = a->dg; p.dbeta = a->dbeta;
    p.dstate = a->dstate;
    p.dy_ld = stride(in[0]); p.q_ld = stride(in[1]); p.k_ld = stride(in[2]); p.v_ld = stride(in[3]); p.g_ld = stride(in[4]);
    p.beta_ld = stride(in[5]);
    p.dq_ld = stride(out[0]); p.dk_ld = stride(out[1]); p.dv_ld = stride(out[2]); p.dg_ld = stride(out[3]);
    p.dbeta_ld = stride(out[4]);
    p.PP = plan->PP;
    p.blocks = plan->PP / 16;
    char *ws = (char *)workspace;
    p.keys = ws;
    p.heads = ws + plan->o_bwd_heads;
    for (int k = 0; k < 2; ++k) {
        p.bound[k] = (float *)(ws + plan->o_bound[k]);
        p.rows[k] = (float *)(ws + plan->o_rows[k]);
        p.part[k] = (float *)(ws + plan->o_part[k]);
    }
    const Rows vec[] = {in[1], in[2]};
    p.vec = delta_vector(*plan, vec, 2);
    // the sums over slices fit any launch: there are some only where N K G is at most 128
    const double groups = (double)d.N * plan->K * d.G;
    if (!one_launch(chain_grid(plan->SP, 2, d.N * d.H, p.blocks), kChainThreads) || !one_launch(groups * plan->slices, 256) ||
        !one_launch(groups * plan->grad_slices, 512))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x H x P is too large for one launch");
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d.dtype == CONV_DT_BF16) launch_delta<bf16_t>(p, *plan, true, s);
    else launch_delta<float>(p, *plan, true, s);
    return launched();
}

void conv_delta_destroy(conv_delta_plan_t *plan) { delete plan; }

const char *conv_delta_describe(const conv_delta_plan_t *plan) { return plan ? plan->text : ""; }

}  // extern "C"
