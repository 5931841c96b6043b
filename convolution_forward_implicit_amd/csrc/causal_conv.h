// The short causal depthwise convolution over a sequence, its gradient and its
// single-token step.
//
//   v[n,t,c] = b[c] + sum_{k<F} w[c,k] h[n, t-(F-1)+k, c]
//   y = v (1 / (1 + e^-v)) or v,        h[t] = x[t], and the state's rows for t < 0
//
// The work is 2F flop for two elements moved: every kernel is bound by HBM.
// A wave owns 64 V neighbouring channels (V: 16 bytes, in the gradient 8) of a
// run of tokens, so its accesses are whole lines and its rows' addresses scalar;
// all rows of a run, with the F - 1 before it, are fetched before the first is
// used.  bf16, 4 taps, SiLU: 4096 x 2304 (38 MB) 10.2 us, 3.7 TB/s (13.6 with a
// branch a row, 12.6 with rows in threads, 11.8 without the hint on the stores);
// 32 single tokens 3.2 us, the launch.
#pragma once

#include "seq_common.h"

namespace convfwd {

struct CausalParams {
    const void *x, *w, *bias, *state;
    const int32_t *lengths;
    void *y, *state_out;
    int64_t x_ld, y_ld;       // elements from one token to the next
    int N, C, CV;             // CV: channel vectors of a token
    int64_t L;
    int64_t blocks;           // token runs of a sequence
    // gradient
    const void *dy, *dstate_out;
    void *dx, *dstate;
    float *partial;           // [N * groups of runs][F + 1][C]
    int64_t dy_ld, dx_ld;
};

constexpr int kConvRun = 8;       // tokens of one wave's run, forward
constexpr int kConvBwdRun = 16;   // tokens of one wave's run, gradient
constexpr int kConvRuns = 4;      // runs (waves) of a workgroup

SEQ_DEV int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
SEQ_DEV int64_t scalar(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// The rows t0 .. t0 + M - 1 of h for V channels, as they lie in memory: a token
// of the sequence, a row of the state, or zero.  Every row is fetched, one that
// has none from the nearest that has (and its value dropped): without branches
// the fetches are all under way before the first is used.  n, t0 and len are the
// same in the whole wave.
template <typename T, int F, int V, int M> struct ConvRows {
    typedef typename Pack<T, V>::type vec_t;
    vec_t q[M];
    SEQ_DEV void load(const CausalParams &p, int64_t n, int64_t t0, int64_t len, int c)
    {
        const T *x = (const T *)p.x + n * p.L * p.x_ld;
        const T *old = p.state ? (const T *)p.state + n * (F - 1) * p.C : nullptr;
        vec_t zero;
        __builtin_memset(&zero, 0, sizeof(zero));
        if (len == 0 && (!old || t0 >= 0)) {        // nothing there (L may be 0)
#pragma unroll
            for (int e = 0; e < M; ++e) q[e] = zero;
            return;
        }
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const int64_t t = t0 + e;
            const T *row = x + (t < 0 ? 0 : t < len ? t : len - 1) * p.x_ld;
            if (old && (t < 0 || len == 0)) row = old + (t < 0 ? F - 1 + t : 0) * p.C;
            q[e] = *reinterpret_cast<const vec_t *>(row + c);
        }
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const int64_t t = t0 + e;
            if (!(t < 0 ? old != nullptr : t < len)) q[e] = zero;
        }
    }
    SEQ_DEV float get(int e, int i) const { return pack_get<T, V>(q[e], i); }
};

template <typename T, int F, int V> SEQ_DEV void conv_weights(const CausalParams &p, int c, float (&w)[F][V])
{
    const T *q = (const T *)p.w + (int64_t)c * F;
    float raw[F * V];
    if constexpr (V == 1) {
#pragma unroll
        for (int k = 0; k < F; ++k) raw[k] = (float)q[k];
    } else {
#pragma unroll
        for (int k = 0; k < F; ++k) {
            float part[V];
            load_f32<T, V>(q + k * V, part);
#pragma unroll
            for (int i = 0; i < V; ++i) raw[k * V + i] = part[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < F; ++k) w[k][i] = raw[i * F + k];
}

// One wave: 64 V channels of kConvRun tokens, or (run == blocks) the state that
// the sequence leaves behind.
template <typename T, int F, int V, bool SILU>
__global__ void __launch_bounds__(256) causal_conv_kernel(CausalParams p)
{
    const int64_t runs = p.blocks + (p.state_out ? 1 : 0), groups = (runs + kConvRuns - 1) / kConvRuns;
    const int cb = (p.CV + 63) / 64;
    const int64_t blk = blockIdx.x / cb, n = blk / groups;
    const int64_t run = scalar((blk - n * groups) * kConvRuns + threadIdx.x / 64);
    const int cv = (int)(blockIdx.x - blk * cb) * 64 + (threadIdx.x & 63), c = cv * V;
    if (run >= runs || cv >= p.CV) return;
    const int64_t len = seq_len(p.lengths, n, p.L);
    if (run == p.blocks) {
        ConvRows<T, F, V, F - 1> h;
        h.load(p, n, len - (F - 1), len, c);
#pragma unroll
        for (int j = 0; j < F - 1; ++j)
            *reinterpret_cast<typename Pack<T, V>::type *>((T *)p.state_out + (n * (F - 1) + j) * p.C + c) = h.q[j];
        return;
    }
    const int64_t t0 = run * kConvRun;
    ConvRows<T, F, V, F - 1 + kConvRun> h;
    h.load(p, n, t0 - (F - 1), len, c);
    float w[F][V], b[V];
    conv_weights<T, F, V>(p, c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
    if (p.bias) load_f32<T, V>((const T *)p.bias + c, b);
#pragma unroll
    for (int u = 0; u < kConvRun; ++u) {
        if (t0 + u >= p.L) break;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v = b[i];
#pragma unroll
            for (int k = 0; k < F; ++k) v = fmaf(w[k][i], h.get(u + k, i), v);
            o[i] = t0 + u < len ? (SILU ? v * sigmoid(v) : v) : 0.0f;
        }
        T *row = (T *)p.y + (n * p.L + t0 + u) * p.y_ld;
        stream_f32<T, V>(row + c, o);
    }
}

// One token of every sequence: y from the state and x, and the state moved on
// by one row.  A thread owns its channels of the state, so it may be updated
// in place.
template <typename T, int F, int V, bool SILU>
__global__ void __launch_bounds__(256) causal_step_kernel(CausalParams p)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = id / p.CV;
    if (n >= p.N) return;
    const int c = (int)(id - n * p.CV) * V;
    float h[F][V], w[F][V], o[V];
#pragma unroll
    for (int j = 0; j < F - 1; ++j) load_f32<T, V>((const T *)p.state + (n * (F - 1) + j) * p.C + c, h[j]);
    load_f32<T, V>((const T *)p.x + n * p.x_ld + c, h[F - 1]);
    conv_weights<T, F, V>(p, c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    if (p.bias) load_f32<T, V>((const T *)p.bias + c, o);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < F; ++k) o[i] = fmaf(w[k][i], h[k][i], o[i]);
        if (SILU) o[i] *= sigmoid(o[i]);
    }
    store_f32<T, V>((T *)p.y + n * p.y_ld + c, o);
#pragma unroll
    for (int j = 0; j < F - 1; ++j) store_f32<T, V>((T *)p.state_out + (n * (F - 1) + j) * p.C + c, h[j + 1]);
}

// The gradient: with d = dy act'(v),
//   dh[s] = sum_k w[k] d[s + (F-1) - k],   dw[k] = sum_t d[t] h[t-(F-1)+k],   db = sum_t d[t].
// A wave recomputes v for its run and the F - 1 tokens behind it (d of those
// reaches back into the run), keeps its sums of dw and db in fp32 registers,
// and the workgroup adds its runs in LDS, in a fixed order; causal_reduce_kernel
// adds the workgroups' rows, in a fixed order too.  4 x 2048 x 2304 bf16 (113 MB):
// 34 + 4 us, 3.3 TB/s: about 35 vector instructions an element, the sigmoid's two
// at a quarter of the rate, are 22 us of it, at three waves per SIMD (149 registers
// of fetched rows and sums).  Rows fetched one by one took 80 us where 46 was the
// time; sums that every row enters, tokens behind the sequence as zeros, 41 for 35
// (199 registers, two waves).
template <typename T, int F, int V, bool SILU>
__global__ void __launch_bounds__(256) causal_bwd_kernel(CausalParams p)
{
    __shared__ float part[kConvRuns][64 * V];
    const int cb = (p.CV + 63) / 64;
    const int64_t blk = blockIdx.x / cb;
    const int cvi = threadIdx.x & 63, ri = scalar((int)threadIdx.x / 64);
    const int cv = (int)(blockIdx.x - blk * cb) * 64 + cvi;
    const int64_t n = blk / p.blocks, run = (blk - n * p.blocks) * kConvRuns + ri;
    const bool live = cv < p.CV;
    const int c = cv * V;
    const int64_t len = seq_len(p.lengths, n, p.L), t0 = run * kConvBwdRun;
    float w[F][V], b[V], dw[F][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = b[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < F; ++k) dw[k][i] = w[k][i] = 0.0f;
    }
    if (live && (t0 < p.L || t0 == 0)) {
        typedef typename Pack<T, V>::type vec_t;
        constexpr int M = kConvBwdRun + F - 1;
        ConvRows<T, F, V, M + F - 1> h;
        vec_t dy[M];
        h.load(p, n, t0 - (F - 1), len, c);
        if (len > 0) {
#pragma unroll
            for (int u = 0; u < M; ++u) {
                const T *row = (const T *)p.dy + (n * p.L + (t0 + u < len ? t0 + u : len - 1)) * p.dy_ld;
                dy[u] = *reinterpret_cast<const vec_t *>(row + c);
            }
        }
        conv_weights<T, F, V>(p, c, w);
        if (p.bias) load_f32<T, V>((const T *)p.bias + c, b);
        float d[F][V];             // d[t-(F-1)] .. d[t]
#pragma unroll
        for (int k = 0; k < F; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) d[k][i] = 0.0f;
#pragma unroll
        for (int u = 0; u < M; ++u) {
            const bool in = t0 + u < len;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float g = pack_get<T, V>(dy[u], i);
                if (SILU) {
                    float v = b[i];
#pragma unroll
                    for (int k = 0; k < F; ++k) v = fmaf(w[k][i], h.get(u + k, i), v);
                    const float s = sigmoid(v);
                    g *= s * (1.0f + v * (1.0f - s));
                }
                d[F - 1][i] = in ? g : 0.0f;
            }
            // no term where there is no token: zero times a row of the state or of the
            // last tokens is not zero if that is not finite
            if (u < kConvBwdRun && in) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    db[i] += d[F - 1][i];
#pragma unroll
                    for (int k = 0; k < F; ++k) dw[k][i] = fmaf(d[F - 1][i], h.get(u + k, i), dw[k][i]);
                }
            }
            // dh at s = t - (F-1), once d[s .. s+F-1] is known
            const int64_t s = t0 + u - (F - 1);
            if (u >= F - 1 || (t0 == 0 && p.dstate)) {
                float g[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < F; ++k) g[i] = fmaf(w[k][i], d[F - 1 - k][i], g[i]);
                }
                const int64_t j = s - (len - (F - 1));     // the row of state_out that h[s] became
                if (p.dstate_out && j >= 0 && j < F - 1) {
                    float q[V];
                    load_f32<T, V>((const T *)p.dstate_out + (n * (F - 1) + j) * p.C + c, q);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] += q[i];
                }
                if (s < 0) {
                    store_f32<T, V>((T *)p.dstate + (n * (F - 1) + (F - 1 + s)) * p.C + c, g);
                } else if (s < p.L && u >= F - 1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] = s < len ? g[i] : 0.0f;
                    T *row = (T *)p.dx + (n * p.L + s) * p.dx_ld;
                    stream_f32<T, V>(row + c, g);
                }
            }
#pragma unroll
            for (int k = 0; k < F - 1; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) d[k][i] = d[k + 1][i];
        }
    }
#pragma unroll
    for (int k = 0; k <= F; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) part[ri][cvi * V + i] = k < F ? dw[k < F ? k : 0][i] : db[i];
        __syncthreads();
        for (int e = threadIdx.x; e < 64 * V; e += 256) {
            const int ch = (int)(blockIdx.x - blk * cb) * 64 * V + e;
            if (ch >= p.C) continue;
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < kConvRuns; ++r) sum += part[r][e];
            p.partial[(blk * (F + 1) + k) * p.C + ch] = sum;
        }
    }
}

// dw[c][k] and db[c] from the workgroups' rows: 64 channels x 4 slices of the rows
template <typename T>
__global__ void __launch_bounds__(256) causal_reduce_kernel(const float *partial, T *dw, T *db, int64_t rows, int C,
                                                            int F)
{
    __shared__ float part[4][64];
    const int cb = (C + 63) / 64;
    const int k = blockIdx.x / cb, c = (blockIdx.x - k * cb) * 64 + (threadIdx.x & 63), r = threadIdx.x / 64;
    float s = 0.0f;
    if (c < C) {
        const float *q = partial + (int64_t)k * C + c;
        const int64_t step = (int64_t)(F + 1) * C;
#pragma unroll 8
        for (int64_t i = r; i < rows; i += 4) s += q[i * step];
    }
    part[r][threadIdx.x & 63] = s;
    __syncthreads();
    if (r == 0 && c < C) {
        s = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        if (k < F) dw[(int64_t)c * F + k] = (T)s;
        else if (db) db[c] = (T)s;
    }
}

}  // namespace convfwd
