// Host side of the group norm (conv_gnorm_*): argument checks, the choice of
// vectors and slabs, launches.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "../../include/convfwd.h"
#include "group_norm.h"
#include "seq_host.h"
#include "status.h"

// Slabs of a sample's rows (of the tokens), and rows of each.
struct NormSlabs {
    int64_t count, rows;
};

struct conv_gnorm_plan {
    conv_gnorm_desc_t desc;
    int64_t esz;
    int64_t samples, rows;               // that share statistics: N of L rows, or N L of one
    NormSlabs token_fwd;                 // of each token in registers, forward
    bool by_slabs;                       // the passes over slabs can be launched
    int64_t ws_bytes, bwd_ws_bytes, o_moments, o_sums, o_group, o_pulls;
    char text[256];
};

namespace convfwd {
namespace {

static_assert(NORM_NONE == CONV_NORM_ACT_NONE && NORM_SILU == CONV_NORM_ACT_SILU && NORM_GELU == CONV_NORM_ACT_GELU,
              "the kernels' activations are the descriptor's");

int64_t up(int64_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Channels per access: the widest vector of at most 16 bytes that divides a group and that `ok` allows.
template <typename F> int widest(int64_t C, int64_t esz, F &&ok)
{
    for (int V = (int)(16 / esz); V > 1; V /= 2)
        if (C % V == 0 && ok(V)) return V;
    return 1;
}

// How a workgroup's 256 threads share groups of C channels in vectors of V.
struct Share {
    int lanes, R;                        // of a token's group: lanes, vectors of each
    int groups, blocks;                  // groups of a workgroup, workgroups across all
    int step;                            // rows side by side
};
Share over_rows(const conv_gnorm_desc_t &d, int V)
{
    const int64_t cv = d.C / V, groups = std::max<int64_t>(1, std::min<int64_t>(d.G, 256 / cv));
    return {0, 0, (int)groups, (int)ceil_div(d.G, groups), (int)std::max<int64_t>(1, 256 / (groups * cv))};
}
constexpr int kMostR = 4;
bool in_registers(const conv_gnorm_desc_t &d, int V) { return d.per_token && d.C / V <= 64 * kMostR; }
Share over_tokens(const conv_gnorm_desc_t &d, int V)
{
    const int64_t cv = d.C / V;
    int lanes = 1;
    while (lanes < cv && lanes < 64) lanes *= 2;
    const int64_t slots = 256 / lanes, groups = std::min<int64_t>(d.G, slots);
    const int R = (int)ceil_div(cv, lanes);
    return {lanes, R <= 2 ? R : 4, (int)groups, (int)ceil_div(d.G, groups), (int)(slots / groups)};
}

// `rows` rows of each of `samples` so that there are about `want` workgroups of `unit` rows and more, but not more rows
// than `most`.
NormSlabs split_rows(int64_t samples, int64_t rows, int64_t blocks, int64_t unit, int64_t want, int64_t most)
{
    if (samples == 0 || rows == 0) return {0, 1};
    const int64_t n = std::max<int64_t>(1, want / std::max<int64_t>(1, samples * blocks));
    const int64_t each = std::min(ceil_div(ceil_div(rows, n), unit) * unit, most);
    return {ceil_div(rows, each), each};
}
// The slabs of a call in vectors of V: of its samples' rows, or, of a gradient whose groups are in registers, of its
// tokens; a thread has kNormChain rows of one at most.  Up to that there are two workgroups a compute unit for a pass
// over rows (8 x 3136 x 256 channels, forward and gradient: 17 and 34 us; with one 19 and 37, with four 18 and 40).
NormSlabs row_slabs(const conv_gnorm_desc_t &d, int V)
{
    const Share s = over_rows(d, V);
    return split_rows(d.per_token ? d.N * d.L : d.N, d.per_token ? 1 : d.L, s.blocks, s.step, 512, kNormChain * s.step);
}
NormSlabs token_slabs(const conv_gnorm_desc_t &d, int V)
{
    const Share s = over_tokens(d, V);
    return split_rows(1, d.N * d.L, s.blocks, s.step * (s.R == 1 ? 2 : 1), 512, kNormChain * s.step);
}

template <typename T, int V> void launch_rows(NormParams p, bool grad, int64_t grid, int64_t reduce, hipStream_t s)
{
    const dim3 g((unsigned)grid), b(256);
    const int64_t joins = grid > 0 ? ceil_div(p.samples * p.G, 4) : 0;
    if (grid > 0) {
        hipLaunchKernelGGL((gnorm_stats_kernel<T, V>), g, b, 0, s, p);
        hipLaunchKernelGGL(gnorm_join_kernel, dim3((unsigned)joins), b, 0, s, p);
        if (!grad) hipLaunchKernelGGL((gnorm_apply_kernel<T, V>), g, b, 0, s, p);
        else hipLaunchKernelGGL((gnorm_sums_kernel<T, V>), g, b, 0, s, p);
    }
    if (!grad) return;
    p.reduce_from = ceil_div(joins * 4, kReduceThreads / 64);
    hipLaunchKernelGGL((gnorm_join_sums_kernel<T>), dim3((unsigned)(p.reduce_from + reduce)), dim3(kReduceThreads), 0, s, p);
    if (grid > 0) hipLaunchKernelGGL((gnorm_grad_kernel<T, V>), g, b, 0, s, p);
}

template <typename T, int V, int R>
void launch_tokens(const NormParams &p, bool grad, int64_t grid, int64_t reduce, hipStream_t s)
{
    if (grid > 0) {
        if (grad) hipLaunchKernelGGL((gnorm_token_grad_kernel<T, V, R>), dim3((unsigned)grid), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((gnorm_token_kernel<T, V, R>), dim3((unsigned)grid), dim3(256), 0, s, p);
    }
    if (grad) hipLaunchKernelGGL((gnorm_reduce_kernel<T>), dim3((unsigned)reduce), dim3(kReduceThreads), 0, s, p);
}

template <typename T, int V> void launch_norm(const NormParams &p, int R, bool grad, int64_t grid, int64_t reduce, hipStream_t s)
{
    if (R == 0) launch_rows<T, V>(p, grad, grid, reduce, s);
    else if (R == 1) launch_tokens<T, V, 1>(p, grad, grid, reduce, s);
    else if (R == 2) launch_tokens<T, V, 2>(p, grad, grid, reduce, s);
    else launch_tokens<T, V, 4>(p, grad, grid, reduce, s);
}

// The plan's part of a call and its launch; `vec` are the tensors read and written in vectors.
conv_status_t run_norm(const conv_gnorm_plan &pl, NormParams &p, const Rows *vec, int nvec, bool grad, char *ws, hipStream_t s)
{
    const conv_gnorm_desc_t &d = pl.desc;
    const int V = widest(d.C, pl.esz, [&](int v) {
        bool ok = true;
        for (int i = 0; i < nvec; ++i)
            ok = ok && (!vec[i].p || ((uintptr_t)vec[i].p % (v * pl.esz) == 0 && (vec[i].rows <= 1 || vec[i].ld % v == 0)));
        return ok;
    });
    const bool tokens = in_registers(d, V);
    const Share sh = tokens ? over_tokens(d, V) : over_rows(d, V);
    const NormSlabs sl = !tokens ? row_slabs(d, V) : grad ? token_slabs(d, V) : pl.token_fwd;
    p.samples = pl.samples; p.rows = pl.rows; p.L = d.L; p.tokens = d.N * d.L;
    p.G = (int)d.G; p.C = (int)d.C; p.act = d.act; p.center = d.center; p.eps = (float)d.eps;
    p.slabs = sl.count; p.slab = sl.rows;
    p.blocks = sh.blocks; p.groups = sh.groups; p.lanes = sh.lanes;
    p.stats = (float *)ws;
    p.sums = (float *)(ws + pl.o_sums);
    p.group = (float *)(ws + pl.o_group);
    p.moments = (float *)(ws + pl.o_moments);
    p.pulls = (float *)(ws + pl.o_pulls);
    const double grid = (double)sl.count * sh.blocks * (tokens ? 1.0 : (double)pl.samples);
    const int64_t reduce = grad ? ceil_div(d.G * d.C, 16) : 0;
    // the sums of dw share their launch with those of the samples' groups
    const double joins = grad && !tokens ? (double)pl.samples * d.G / (kReduceThreads / 64) + 1 : 0.0;
    if ((!tokens && !pl.by_slabs) || !one_launch(grid, 256) || !one_launch((double)reduce + joins, kReduceThreads))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x G x C is too large for one launch");
    (void)hipGetLastError();
    if (d.dtype == CONV_DT_BF16) {
        if (V == 8) launch_norm<bf16_t, 8>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
        else if (V == 4) launch_norm<bf16_t, 4>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
        else if (V == 2) launch_norm<bf16_t, 2>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
        else launch_norm<bf16_t, 1>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
    } else {
        if (V == 4) launch_norm<float, 4>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
        else if (V == 2) launch_norm<float, 2>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
        else launch_norm<float, 1>(p, tokens ? sh.R : 0, grad, (int64_t)grid, reduce, s);
    }
    return launched();
}

}  // namespace
}  // namespace convfwd

using namespace convfwd;

extern "C" {

conv_status_t conv_gnorm_create(const conv_gnorm_desc_t *desc, conv_gnorm_plan_t **plan)
{
    if (!plan) return fail(CONV_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "descriptor is NULL");
    const conv_gnorm_desc_t &d = *desc;
    if (d.dtype != CONV_DT_F32 && d.dtype != CONV_DT_BF16) return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", d.dtype);
    if (d.act < CONV_NORM_ACT_NONE || d.act > CONV_NORM_ACT_GELU) return fail(CONV_ERR_INVALID_ARG, "unknown activation %d", d.act);
    for (const int32_t flag : {d.has_bias, d.gated, d.center, d.per_token})
        if (flag != 0 && flag != 1) return fail(CONV_ERR_INVALID_ARG, "has_bias, gated, center and per_token must be 0 or 1");
    if (!(d.eps >= 0) || !std::isfinite((float)d.eps)) return fail(CONV_ERR_INVALID_ARG, "eps must be a finite fp32 number, at least 0");
    if (d.N < 0 || d.L < 0 || d.G < 1 || d.C < 1)
        return fail(CONV_ERR_INVALID_ARG, "need N, L >= 0 and G, C >= 1 (got %lld, %lld, %lld, %lld)", (long long)d.N,
                    (long long)d.L, (long long)d.G, (long long)d.C);
    if (d.N > kMaxDim || d.L > kMaxDim || d.G > kMaxDim || d.C > kMaxDim || (double)d.G * d.C > kMaxDim)
        return fail(CONV_ERR_UNSUPPORTED, "N, L or G x C above 2^30");
    const int64_t esz = d.dtype == CONV_DT_BF16 ? 2 : 4;
    const int V = widest(d.C, esz, [](int) { return true; });
    const int64_t tokens = d.N * d.L;
    if ((double)tokens * d.G * d.C * 8 >= kMaxBytes)
        return fail(CONV_ERR_UNSUPPORTED, "N x L x G x C is too large for one launch");
    conv_gnorm_plan pl{};
    pl.desc = d;
    pl.esz = esz;
    pl.samples = d.per_token ? tokens : d.N;
    pl.rows = d.per_token ? 1 : d.L;
    const Share tok = over_tokens(d, V);
    pl.token_fwd = split_rows(1, tokens, tok.blocks, tok.step * (tok.R == 1 ? 4 : 2), 2048, tokens);
    const NormSlabs slabs = row_slabs(d, V);
    // Tokens whose groups stay in registers need no slabs: their plan is made also where a launch over slabs could not
    // take their number, and a call whose tensors do not allow the vectors for it is refused.
    pl.by_slabs = one_launch((double)pl.samples * slabs.count, 256) && one_launch((double)pl.samples * d.G, 64);
    if (!pl.by_slabs && !in_registers(d, V))
        return fail(CONV_ERR_UNSUPPORTED, "N x L x G x C is too large for one launch");
    // What a call needs goes by the vectors that its tensors allow: a token's group in registers needs the sums of its
    // slabs only.
    int64_t n = 0, sums = 0;
    for (int v = V; v >= 1; v /= 2) {
        if (in_registers(d, v)) sums = std::max(sums, token_slabs(d, v).count);
        else if (pl.by_slabs) n = std::max(n, pl.samples * row_slabs(d, v).count);
    }
    sums = std::max(sums, n);
    const int64_t each = n > 0 ? up(pl.samples * d.G * 8) : 0;      // two numbers of every sample's groups
    pl.o_moments = up(n * d.G * 8);
    pl.ws_bytes = pl.o_moments + each;
    pl.o_sums = pl.ws_bytes;
    pl.o_group = pl.o_sums + up(sums * d.G * d.C * 8);
    pl.o_pulls = pl.o_group + up(n * d.G * 8);
    pl.bwd_ws_bytes = pl.o_pulls + each;
    snprintf(pl.text, sizeof(pl.text), "gnorm %s N=%lld L=%lld G=%lld C=%lld%s%s%s%s, %s, %lld slabs of %lld rows",
             d.dtype == CONV_DT_BF16 ? "bf16" : "f32", (long long)d.N, (long long)d.L, (long long)d.G, (long long)d.C,
             d.has_bias ? " bias" : "", d.act == CONV_NORM_ACT_SILU ? " silu" : d.act == CONV_NORM_ACT_GELU ? " gelu" : "",
             d.gated ? " gated" : "", d.center ? "" : " uncentered", d.per_token ? "each token" : "each sample",
             (long long)(d.per_token ? pl.token_fwd : slabs).count, (long long)(d.per_token ? pl.token_fwd : slabs).rows);
    conv_gnorm_plan *made = new (std::nothrow) conv_gnorm_plan(pl);
    if (!made) return fail(CONV_ERR_NOMEM, "plan allocation failed");
    if (getenv("CONVFWD_LOG")) fprintf(stderr, "convfwd: %s\n", made->text);
    *plan = made;
    return CONV_OK;
}

conv_status_t conv_gnorm_workspace_bytes(const conv_gnorm_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->ws_bytes;
    return CONV_OK;
}

conv_status_t conv_gnorm_bwd_workspace_bytes(const conv_gnorm_plan_t *plan, int64_t *bytes)
{
    if (!plan || !bytes) return fail(CONV_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = plan->bwd_ws_bytes;
    return CONV_OK;
}

conv_status_t conv_gnorm_run(const conv_gnorm_plan_t *plan, const conv_gnorm_args_t *a, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_gnorm_desc_t &d = plan->desc;
    const int64_t e = plan->esz, rows = d.N * d.L, W = d.G * d.C, need = plan->ws_bytes;
    if (!a->w) return fail(CONV_ERR_INVALID_ARG, "w is NULL");
    if ((a->bias != nullptr) != (d.has_bias != 0))
        return fail(CONV_ERR_INVALID_ARG, d.has_bias ? "bias is NULL" : "this plan has no bias");
    if (a->gate && !d.gated) return fail(CONV_ERR_INVALID_ARG, "this plan has no gate");
    const Rows in[] = {{"x", a->x, rows, W, or_packed(a->x_ld, W), e},
                       {"gate", a->gate, rows, W, or_packed(a->gate_ld, W), e},
                       {"w", a->w, 1, W, W, e},
                       {"bias", a->bias, 1, W, W, e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4}};
    const Rows out[] = {{"y", a->y, rows, W, or_packed(a->y_ld, W), e},
                        {"workspace", workspace, 1, need, std::max<int64_t>(1, need), 1}};
    conv_status_t st = check_rows(in, 5);
    if (st == CONV_OK) st = check_rows(out, 1);
    if (st != CONV_OK) return st;
    if (rows == 0) return CONV_OK;
    if (!a->x || !a->y) return fail(CONV_ERR_INVALID_ARG, "x or y is NULL");
    if (d.gated && !a->gate) return fail(CONV_ERR_INVALID_ARG, "gate is NULL");
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CONV_OK) return st;
    if ((st = check_overlap(out, 2, in, 5)) != CONV_OK) return st;
    NormParams p{};
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.gate = a->gate; p.lengths = a->lengths; p.y = a->y;
    p.x_ld = stride(in[0]); p.gate_ld = stride(in[1]); p.y_ld = stride(out[0]);
    const Rows vec[] = {in[0], in[1], in[2], in[3], out[0]};
    return run_norm(*plan, p, vec, 5, false, (char *)workspace, (hipStream_t)stream);
}

conv_status_t conv_gnorm_bwd_run(const conv_gnorm_plan_t *plan, const conv_gnorm_bwd_args_t *a, void *workspace,
                                 int64_t workspace_bytes, void *stream)
{
    if (!plan || !a) return fail(CONV_ERR_INVALID_ARG, "plan or args is NULL");
    const conv_gnorm_desc_t &d = plan->desc;
    const int64_t e = plan->esz, rows = d.N * d.L, W = d.G * d.C, need = plan->bwd_ws_bytes;
    if (!a->w || !a->dw) return fail(CONV_ERR_INVALID_ARG, "w or dw is NULL");
    if ((a->bias != nullptr) != (d.has_bias != 0) || (a->dbias != nullptr) != (d.has_bias != 0))
        return fail(CONV_ERR_INVALID_ARG, d.has_bias ? "bias or dbias is NULL" : "this plan has no bias");
    if ((a->gate || a->dgate) && !d.gated) return fail(CONV_ERR_INVALID_ARG, "this plan has no gate");
    const Rows in[] = {{"dy", a->dy, rows, W, or_packed(a->dy_ld, W), e},
                       {"x", a->x, rows, W, or_packed(a->x_ld, W), e},
                       {"gate", a->gate, rows, W, or_packed(a->gate_ld, W), e},
                       {"w", a->w, 1, W, W, e},
                       {"bias", a->bias, 1, W, W, e},
                       {"lengths", a->lengths, 1, d.N, std::max<int64_t>(1, d.N), 4}};
    const Rows out[] = {{"dx", a->dx, rows, W, or_packed(a->dx_ld, W), e},
                        {"dgate", a->dgate, rows, W, or_packed(a->dgate_ld, W), e},
                        {"dw", a->dw, 1, W, W, e},
                        {"dbias", a->dbias, 1, W, W, e},
                        {"workspace", workspace, 1, need, std::max<int64_t>(1, need), 1}};
    conv_status_t st = check_rows(in, 6);
    if (st == CONV_OK) st = check_rows(out, 4);
    if (st != CONV_OK) return st;
    if (rows > 0 && (!a->dy || !a->x || !a->dx)) return fail(CONV_ERR_INVALID_ARG, "dy, x or dx is NULL");
    if (rows > 0 && d.gated && (!a->gate || !a->dgate)) return fail(CONV_ERR_INVALID_ARG, "gate or dgate is NULL");
    if ((st = check_workspace(workspace, workspace_bytes, need)) != CONV_OK) return st;
    if ((st = check_overlap(out, 5, in, 6)) != CONV_OK) return st;
    NormParams p{};
    p.x = a->x; p.w = a->w; p.bias = a->bias; p.gate = a->gate; p.lengths = a->lengths; p.dy = a->dy;
    p.dx = a->dx; p.dgate = a->dgate; p.dw = a->dw; p.dbias = a->dbias;
    p.dy_ld = stride(in[0]); p.x_ld = stride(in[1]); p.gate_ld = stride(in[2]);
    p.dx_ld = stride(out[0]); p.dgate_ld = stride(out[1]);
    const Rows vec[] = {in[0], in[1], in[2], in[3], in[4], out[0], out[1]};
    return run_norm(*plan, p, vec, 7, true, (char *)workspace, (hipStream_t)stream);
}

void conv_gnorm_destroy(conv_gnorm_plan_t *plan) { delete plan; }

const char *conv_gnorm_describe(const conv_gnorm_plan_t *plan) { return plan ? plan->text : ""; }

}  // extern "C"
