// Group norm with an activation, channels innermost, and its gradient.
//
//   xhat = (x - mean) / sqrt(var + eps)     mean, var over a group's channels of all a sample's
//                                           pixels, or of each token by itself; without centering
//                                           mean is 0 and var the mean square
//   v = w xhat + b,     y = act(v),   or with a gate z   y = v act(z)
//
// With d = dy act'(v) (gated: dy act(z)), n the values of a group and r = 1 / sqrt(var + eps):
//
//   dx = r (d w - [sum(d w) / n] - xhat sum(d w xhat) / n)     [only where the mean is taken off]
//   dw = sum d xhat,   db = sum d,   dz = dy v act'(z)
//
// A few operations a value, so memory bounds it.
//
// Over pixels (gnorm_stats, _apply, _sums, _grad): a workgroup takes a slab of a
// sample's rows by whole groups; a thread owns V neighbouring channels, whose
// weights it loads once, and steps over the slab's rows.  The first pass leaves each
// slab's mean and sum of squares around it, which gnorm_join makes a group's: a launch
// more, but joined by every workgroup of the next pass they took longer than its rows
// (8 x 3136 x 256 channels in bf16: 14 us where 7.5 are left; in all 6.7 + 4.0 + 7.5, a pass over
// 26 MB at the rate of a large copy 5.2).  The gradient's second pass leaves
// sum d and sum d xhat of every channel of a slab: dw, db and both of a group's sums
// come from these.
//
// Of each token by itself (gnorm_token, gnorm_token_grad): `lanes` lanes hold a group
// in registers, so everything is read once: 4096 x 32 heads of 128 with a gate in bf16,
// 101 MB in 20.4 us, 4.9 TB/s, a large copy's rate.
//
// Numbers.  Squares are summed around a mean that is near theirs, never as mean of
// squares less square of mean: a thread takes the mean of a batch of values it holds
// and joins (count, mean, squares) with what it has, over 64 rows at most; sums over
// threads, slabs and the columns of a wide row are in fp64, always in the same order.
#pragma once

#include "seq_common.h"

namespace convfwd {

enum NormAct { NORM_NONE, NORM_SILU, NORM_GELU };

struct NormParams {
    const void *x, *w, *bias, *gate, *dy;
    const int32_t *lengths;
    void *y, *dx, *dgate, *dw, *dbias;
    int64_t x_ld, gate_ld, y_ld, dy_ld, dx_ld, dgate_ld;
    int64_t samples, rows;          // a sample: the rows that share statistics
    int64_t L, tokens;              // rows of a sequence (lengths' unit), of the call
    int G, C, act, center;
    float eps;
    int64_t slabs, slab;            // of a sample's rows (of the tokens), rows of each
    int blocks, groups;             // across the groups: workgroups, groups of each
    int lanes;
    float *stats;                   // [sample][slab][G][2]: mean, sum of squares around it
    float *sums;                    // [sample][slab][2][G C]: sum d, sum d xhat
    float *group;                   // [sample][slab][G][2]: the same times w, of a group
    float *moments, *pulls;         // [sample][G][2]: mean and r; sum d w / n, sum d w xhat / n
    int64_t reduce_from;            // workgroups from here on add up dw and dbias
};

// ---- activations -----------------------------------------------------------------
// Phi(v), the normal distribution's integral.  For results that are rounded to bf16
// 2^R(|v|) with the fit of the convolutions' epilogue: within 4e-6 of its value down to
// v = -6; of -9e-12 at v = -7 it is 7e-4 off, of -5e-15 at -8 0.8%, of -1e-18 at -9 5%.
template <typename T> SEQ_DEV float normal_cdf(float v)
{
    if constexpr (sizeof(T) == 4) {
        return 0.5f * erfcf(-0.70710678118654752f * v);
    } else {
        const float a = fabsf(v);
        float r = -1.889570263e-06f;
        r = fmaf(r, a, 6.268018558e-05f);
        r = fmaf(r, a, -9.388573895e-04f);
        r = fmaf(r, a, 8.539414817e-03f);
        r = fmaf(r, a, -5.402057739e-02f);
        r = fmaf(r, a, -4.584099095e-01f);
        r = fmaf(r, a, -1.151269077e+00f);
        r = fmaf(r, a, -9.999943512e-01f);
        const float p = exp2_fast(r);
        return v < 0.0f ? p : 1.0f - p;
    }
}
// act(v) and act'(v) of n values
template <typename T, int V> SEQ_DEV void activate(int act, const float (&v)[V], float (&y)[V])
{
    if (act == NORM_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = v[i] * sigmoid(v[i]);
    } else if (act == NORM_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = v[i] * normal_cdf<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = v[i];
    }
}
template <typename T, int V> SEQ_DEV void activate(int act, const float (&v)[V], float (&y)[V], float (&dy)[V])
{
    if (act == NORM_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = sigmoid(v[i]);
            y[i] = v[i] * s;
            dy[i] = fmaf(y[i], 1.0f - s, s);
        }
    } else if (act == NORM_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float c = normal_cdf<T>(v[i]);
            y[i] = v[i] * c;
            dy[i] = fmaf(v[i] * 0.39894228040143268f, exp2_fast(-0.5f * kLog2e * v[i] * v[i]), c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = v[i], dy[i] = 1.0f;
    }
}

// ---- over a sample's rows ----------------------------------------------------------
// rows of sample n that count
SEQ_DEV int64_t norm_rows(const NormParams &p, int64_t n)
{
    if (!p.lengths) return p.rows;
    if (p.rows == p.L) return seq_len(p.lengths, n, p.L);
    const int64_t s = n / p.L;                              // a sample is a token
    return n - s * p.L < seq_len(p.lengths, s, p.L) ? 1 : 0;
}

// What a workgroup takes, and a thread of it: column vectors c, c + 256, .. below
// `wide` of rows r0, r0 + step, ..
struct NormShare {
    int64_t n, slab, row0;      // sample, its slab, first row of the sample's
    int64_t first, live, last;  // of the slab's rows: the first, the end of those that count, of all
    int g0, ng, cv, wide, step, col, r0;
};
template <int V> SEQ_DEV NormShare norm_share(const NormParams &p, uint32_t block)
{
    NormShare s;
    const uint32_t slab = block / (uint32_t)p.blocks, n = slab / (uint32_t)p.slabs;      // fewer than 2^32 workgroups
    s.n = n;
    s.slab = slab - n * (uint32_t)p.slabs;
    s.g0 = (int)(block - slab * (uint32_t)p.blocks) * p.groups;
    s.ng = min(p.groups, p.G - s.g0);
    s.cv = p.C / V;
    s.wide = s.ng * s.cv;
    s.step = s.wide <= 256 ? 256 / s.wide : 1;
    s.r0 = s.wide <= 256 ? (int)threadIdx.x / s.wide : 0;
    s.col = s.wide <= 256 ? (int)threadIdx.x - s.r0 * s.wide : (int)threadIdx.x;
    if (s.r0 >= s.step) s.col = s.wide;
    s.row0 = s.n * p.rows;
    s.first = s.slab * p.slab;
    s.last = s.first + p.slab < p.rows ? s.first + p.slab : p.rows;
    const int64_t rows = norm_rows(p, s.n);
    s.live = s.last < rows ? s.last : rows;
    return s;
}

// (count, mean, squares) of `n` parts that get(i, cnt, mean, m2) names, by LANES lanes:
// in fp64, around the first part's mean, which is near the whole's.
template <int LANES> SEQ_DEV double lanes_sum64(double v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
template <int LANES, typename F> SEQ_DEV void join_parts(int n, F &&get, double &cnt, double &mean, double &m2)
{
    const int l = threadIdx.x & (LANES - 1);
    float c0, mean0, s0;
    get(0, c0, mean0, s0);
    double sum = 0.0, sq = 0.0;
    cnt = 0.0;
#pragma unroll 4
    for (int i = l; i < n; i += LANES) {
        float c, m, s;
        get(i, c, m, s);
        const double d = c > 0.0f ? (double)m - (double)mean0 : 0.0, cd = (double)c * d;
        cnt += (double)c;
        sum += cd;
        sq += c > 0.0f ? fma(cd, d, (double)s) : 0.0;
    }
    cnt = lanes_sum64<LANES>(cnt);
    sum = lanes_sum64<LANES>(sum);
    sq = lanes_sum64<LANES>(sq);
    const double off = cnt > 0.0 ? sum / cnt : 0.0, left = fma(-off, sum, sq);
    mean = (double)mean0 + off;
    m2 = left < 0.0 ? 0.0 : left;       // a NaN stays one
}

// (count, mean, squares) joined with a batch of `b` values of mean bm and squares bs.  d is a mean itself while the
// count is 0: squared it may be infinite, and infinity times 0 no number.
SEQ_DEV void join_batch(float &cnt, float &mean, float &m2, float b, float bm, float bs)
{
    const float all = cnt + b, d = bm - mean, f = all > 0.0f ? b / all : 0.0f;
    mean = fmaf(d, f, mean);
    m2 += fmaf(d * (cnt * f), d, bs);
    cnt = all;
}

constexpr int kNormBatch = 4;       // rows that a thread has under way
// Rows of a slab that a thread may have: it adds their terms up in fp32, and equal terms are rounded the same way every
// time (4096 of 1 + 2^-13 lost 6e-5 of their sum, 16384 equal rows 4e-5 of their squares).  Slabs, and a thread's
// columns of a row wider than a workgroup, are joined in fp64.
constexpr int kNormChain = 64;

// (count, mean, squares) of several columns of a thread, around the first one's mean
struct NormColumns {
    float mean0;
    double cnt = 0.0, sum = 0.0, sq = 0.0;
    SEQ_DEV void add(float c, float mean, float m2)
    {
        if (cnt == 0.0) mean0 = mean;
        const double d = (double)mean - (double)mean0, cd = (double)c * d;
        cnt += (double)c;
        sum += cd;
        sq += fma(cd, d, (double)m2);
    }
    SEQ_DEV void get(float &c, float &mean, float &m2) const
    {
        const double off = sum / cnt, left = fma(-off, sum, sq);
        c = (float)cnt;
        mean = (float)((double)mean0 + off);
        m2 = left < 0.0 ? 0.0f : (float)left;       // a NaN stays one
    }
};
constexpr int kReduceThreads = 1024;    // 16 channels' slabs, by 64 threads each

template <typename T, int V> __global__ void __launch_bounds__(256) gnorm_stats_kernel(NormParams p)
{
    __shared__ float part[3][256];
    const NormShare s = norm_share<V>(p, blockIdx.x);
    const int64_t first = s.first;
    float cnt = 0.0f, mean = 0.0f, m2 = 0.0f;
    NormColumns all;
    for (int col = s.col; col < s.wide; col += 256) {
        const T *x = (const T *)p.x + s.row0 * p.x_ld + (int64_t)s.g0 * p.C + col * V;
        for (int64_t r = first + s.r0; r < s.live; r += kNormBatch * s.step) {
            float v[kNormBatch][V];
#pragma unroll
            for (int b = 0; b < kNormBatch; ++b) {
                const int64_t row = r + b * s.step < s.live ? r + b * s.step : r;       // in place of a row that is none
                load_f32<T, V>(x + row * p.x_ld, v[b]);
            }
            float sum = 0.0f, sq = 0.0f;
            int have = 0;
#pragma unroll
            for (int b = 0; b < kNormBatch; ++b) {
                if (r + b * s.step < s.live) {
                    ++have;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += v[b][i];
                }
            }
            const float n = (float)(have * V), bm = sum / n;
#pragma unroll
            for (int b = 0; b < kNormBatch; ++b) {
                if (r + b * s.step < s.live) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = v[b][i] - bm;
                        sq = fmaf(d, d, sq);
                    }
                }
            }
            join_batch(cnt, mean, m2, n, bm, sq);
        }
        if (s.wide > 256 && cnt > 0.0f) {
            all.add(cnt, mean, m2);
            cnt = mean = m2 = 0.0f;
        }
    }
    if (all.cnt > 0.0) all.get(cnt, mean, m2);
    part[0][threadIdx.x] = cnt;
    part[1][threadIdx.x] = mean;
    part[2][threadIdx.x] = m2;
    __syncthreads();
    // threads that hold parts of group g: all 256 where a row is wider than that
    for (int g = threadIdx.x >> 4; g < s.ng; g += 16) {
        const int cols = s.wide <= 256 ? s.cv : 256, n = s.wide <= 256 ? s.cv * s.step : 256;
        double cnt_g, mean_g, m2_g;
        join_parts<16>(n, [&](int i, float &c, float &m, float &q) {
            const int t = i / cols * s.wide + (s.wide <= 256 ? g * s.cv : 0) + i % cols;
            c = part[0][t], m = part[1][t], q = part[2][t];
        }, cnt_g, mean_g, m2_g);
        if ((threadIdx.x & 15) == 0) {
            float *o = p.stats + ((s.n * p.slabs + s.slab) * p.G + s.g0 + g) * 2;
            o[0] = (float)mean_g;
            o[1] = (float)m2_g;
        }
    }
}

// A group's mean and r from its slabs', or (GRAD) what its gradients are taken off by: a wave each
template <bool GRAD> SEQ_DEV void norm_join(const NormParams &p, uint32_t block)
{
    const uint32_t at = block * (GRAD ? kReduceThreads / 64 : 4) + (threadIdx.x >> 6), sample = at / (uint32_t)p.G;
    const int g = (int)(at - sample * (uint32_t)p.G), lane = threadIdx.x & 63;
    const int64_t n = sample;
    if (n >= p.samples) return;
    const int64_t rows = norm_rows(p, n);
    if constexpr (GRAD) {
        const double count = (double)rows * p.C;
        double a = 0.0, b = 0.0;
#pragma unroll 4
        for (int i = lane; i < (int)p.slabs; i += 64) {
            const float *o = p.group + ((n * p.slabs + i) * p.G + g) * 2;
            a += (double)o[0];
            b += (double)o[1];
        }
        a = lanes_sum64<64>(a);
        b = lanes_sum64<64>(b);
        if (lane == 0) {
            p.pulls[(int64_t)at * 2] = p.center && count > 0.0 ? (float)(a / count) : 0.0f;
            p.pulls[(int64_t)at * 2 + 1] = count > 0.0 ? (float)(b / count) : 0.0f;
        }
    } else {
        double count, m, m2;
        join_parts<64>((int)p.slabs, [&](int i, float &c, float &mm, float &q) {
            const float *o = p.stats + ((n * p.slabs + i) * p.G + g) * 2;
            const int64_t have = rows - i * p.slab;
            c = (float)((have < 0 ? 0 : have < p.slab ? have : p.slab) * p.C);
            mm = o[0], q = o[1];
        }, count, m, m2);
        if (lane == 0) {
            const double var = count > 0.0 ? m2 / count + (p.center ? 0.0 : m * m) : 0.0;
            p.moments[(int64_t)at * 2] = p.center ? (float)m : 0.0f;
            p.moments[(int64_t)at * 2 + 1] = (float)(1.0 / sqrt(var + (double)p.eps));
        }
    }
}
__global__ void __launch_bounds__(256) gnorm_join_kernel(NormParams p) { norm_join<false>(p, blockIdx.x); }

// V weights and biases of a thread's channels
template <typename T, int V> SEQ_DEV void norm_weights(const NormParams &p, int64_t at, float (&w)[V], float (&b)[V])
{
    load_f32<T, V>((const T *)p.w + at, w);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
    if (p.bias) load_f32<T, V>((const T *)p.bias + at, b);
}

template <typename T, int V> SEQ_DEV void norm_out(const NormParams &p, const float (&v)[V], const float (&z)[V], float (&y)[V])
{
    if (p.gate) {
        activate<T, V>(p.act, z, y);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= v[i];
    } else {
        activate<T, V>(p.act, v, y);
    }
}

// Zeros in a slab's rows of a sample none of whose rows count: there is none that a Batch could read instead.
template <typename T, int V> SEQ_DEV void norm_clear(const NormParams &p, const NormShare &s, void *out, int64_t ld)
{
    const float zeros[V] = {};
    for (int col = s.col; col < s.wide; col += 256) {
        T *g = (T *)out + s.row0 * ld + (int64_t)s.g0 * p.C + col * V;
        for (int64_t row = s.first + s.r0; row < s.last; row += s.step) stream_f32<T, V>(g + row * ld, zeros);
    }
}

// Rows row, row + step, .. of a thread's channels, as they are; in place of those that do not count the last that
// does (live > 0): without a branch the loads are all under way at once.
template <typename T, int V> struct Batch {
    typename Pack<T, V>::type q[kNormBatch];
    SEQ_DEV void load(const T *x, int64_t ld, int64_t row, int step, int64_t live)
    {
        const int last = (int)live - 1;
#pragma unroll
        for (int e = 0; e < kNormBatch; ++e) {
            const int r = (int)row + e * step;
            q[e] = *reinterpret_cast<const typename Pack<T, V>::type *>(x + (int64_t)(r < last ? r : last) * ld);
        }
    }
    SEQ_DEV void get(int e, float (&v)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = pack_get<T, V>(q[e], i);
    }
};

template <typename T, int V> __global__ void __launch_bounds__(256) gnorm_apply_kernel(NormParams p)
{
    const NormShare s = norm_share<V>(p, blockIdx.x);
    const int64_t first = s.first + s.r0;
    if (s.live <= 0) return norm_clear<T, V>(p, s, p.y, p.y_ld);
    Batch<T, V> vb, zb;
    for (int col = s.col; col < s.wide; col += 256) {
        const int64_t at = (int64_t)s.g0 * p.C + col * V;
        const float *mo = p.moments + (s.n * p.G + s.g0 + col / s.cv) * 2;
        const float m = mo[0], r = mo[1];
        float w[V], b[V];
        norm_weights<T, V>(p, at, w, b);
        const T *x = (const T *)p.x + s.row0 * p.x_ld + at, *zg = (const T *)p.gate + s.row0 * p.gate_ld + at;
        T *yg = (T *)p.y + s.row0 * p.y_ld + at;
        for (int64_t row = first; row < s.last; row += kNormBatch * s.step) {
            vb.load(x, p.x_ld, row, s.step, s.live);
            if (p.gate) zb.load(zg, p.gate_ld, row, s.step, s.live);
#pragma unroll
            for (int e = 0; e < kNormBatch; ++e) {
                const int64_t at_row = row + e * s.step;
                if (at_row >= s.last) continue;
                float v[V], z[V], y[V];
                vb.get(e, v);
                if (p.gate) zb.get(e, z);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fmaf((v[i] - m) * r, w[i], b[i]);
                norm_out<T, V>(p, v, z, y);
                if (at_row >= s.live)
#pragma unroll
                    for (int i = 0; i < V; ++i) y[i] = 0.0f;
                stream_f32<T, V>(yg + at_row * p.y_ld, y);
            }
        }
    }
}

// d and, where there is a gate, its gradient, of V values; xhat in, act as the plan says
template <typename T, int V>
SEQ_DEV void norm_back(const NormParams &p, const float (&xhat)[V], const float (&w)[V], const float (&b)[V],
                       const float (&z)[V], const float (&dy)[V], float (&d)[V], float (&dz)[V])
{
    float v[V], a[V], da[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fmaf(xhat[i], w[i], b[i]);
    if (p.gate) {
        activate<T, V>(p.act, z, a, da);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = dy[i] * a[i], dz[i] = dy[i] * v[i] * da[i];
    } else {
        activate<T, V>(p.act, v, a, da);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = dy[i] * da[i], dz[i] = 0.0f;
    }
}

template <typename T, int V> __global__ void __launch_bounds__(256) gnorm_sums_kernel(NormParams p)
{
    __shared__ float part[2][256 * V];
    const NormShare s = norm_share<V>(p, blockIdx.x);
    const int64_t first = s.first + s.r0;
    Batch<T, V> vb, zb, db;
    const int64_t W = (int64_t)p.G * p.C;
    float *out = p.sums + (s.n * p.slabs + s.slab) * 2 * W + (int64_t)s.g0 * p.C;
    double whole[2] = {0.0, 0.0};           // of the one group of a wide row
    const int turns = s.wide <= 256 ? 1 : (s.wide + 255) / 256;
    for (int turn = 0; turn < turns; ++turn) {
        const int col = s.col + turn * 256;
        const int64_t at = (int64_t)s.g0 * p.C + col * V;
        float sd[V], sx[V], w[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sd[i] = sx[i] = w[i] = 0.0f;
        if (col < s.wide) {
            const float *mo = p.moments + (s.n * p.G + s.g0 + col / s.cv) * 2;
            const float m = mo[0], r = mo[1];
            norm_weights<T, V>(p, at, w, b);
            const T *x = (const T *)p.x + s.row0 * p.x_ld + at, *zg = (const T *)p.gate + s.row0 * p.gate_ld + at;
            const T *dg = (const T *)p.dy + s.row0 * p.dy_ld + at;
            for (int64_t row = first; row < s.live; row += kNormBatch * s.step) {
                vb.load(x, p.x_ld, row, s.step, s.live);
                db.load(dg, p.dy_ld, row, s.step, s.live);
                if (p.gate) zb.load(zg, p.gate_ld, row, s.step, s.live);
#pragma unroll
                for (int e = 0; e < kNormBatch; ++e) {
                    if (row + e * s.step >= s.live) continue;
                    float v[V], z[V], dy[V], d[V], dz[V];
                    vb.get(e, v);
                    db.get(e, dy);
                    if (p.gate) zb.get(e, z);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = (v[i] - m) * r;
                    norm_back<T, V>(p, v, w, b, z, dy, d, dz);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        sd[i] += d[i];
                        sx[i] = fmaf(d[i], v[i], sx[i]);
                    }
                }
            }
        }
        if (s.wide <= 256) {
#pragma unroll
            for (int i = 0; i < V; ++i) part[0][threadIdx.x * V + i] = sd[i], part[1][threadIdx.x * V + i] = sx[i];
            __syncthreads();
            if ((int)threadIdx.x < s.wide) {
                float a[V], c[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    double u = 0.0, v = 0.0;
                    for (int e = 0; e < s.step; ++e) {
                        u += (double)part[0][(e * s.wide + threadIdx.x) * V + i];
                        v += (double)part[1][(e * s.wide + threadIdx.x) * V + i];
                    }
                    a[i] = (float)u, c[i] = (float)v;
                }
                store_f32<float, V>(out + threadIdx.x * V, a);
                store_f32<float, V>(out + W + threadIdx.x * V, c);
#pragma unroll
                for (int i = 0; i < V; ++i) sd[i] = a[i] * w[i], sx[i] = c[i] * w[i];
            }
            __syncthreads();
            if ((int)threadIdx.x < s.wide)
#pragma unroll
                for (int i = 0; i < V; ++i) part[0][threadIdx.x * V + i] = sd[i], part[1][threadIdx.x * V + i] = sx[i];
            __syncthreads();
        } else if (col < s.wide) {
            store_f32<float, V>(out + col * V, sd);
            store_f32<float, V>(out + W + col * V, sx);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                whole[0] += (double)sd[i] * (double)w[i];
                whole[1] += (double)sx[i] * (double)w[i];
            }
        }
    }
    float *group = p.group + ((s.n * p.slabs + s.slab) * p.G + s.g0) * 2;
    if (s.wide <= 256) {
        for (int g = threadIdx.x >> 4; g < s.ng; g += 16) {
            double a = 0.0, b = 0.0;
            for (int i = threadIdx.x & 15; i < p.C; i += 16) a += (double)part[0][g * p.C + i], b += (double)part[1][g * p.C + i];
            a = lanes_sum64<16>(a);
            b = lanes_sum64<16>(b);
            if ((threadIdx.x & 15) == 0) group[2 * g] = (float)a, group[2 * g + 1] = (float)b;
        }
    } else {                                // one group
        __shared__ double both[2][256];
        both[0][threadIdx.x] = whole[0];
        both[1][threadIdx.x] = whole[1];
        __syncthreads();
        if (threadIdx.x < 16) {
            double a = 0.0, b = 0.0;
            for (int i = threadIdx.x; i < 256; i += 16) a += both[0][i], b += both[1][i];
            a = lanes_sum64<16>(a);
            b = lanes_sum64<16>(b);
            if (threadIdx.x == 0) group[0] = (float)a, group[1] = (float)b;
        }
    }
}

// dw and dbias of 16 channels: the sums of `n` slabs
template <typename T> SEQ_DEV void norm_reduce(const NormParams &p, int64_t block, int64_t n)
{
    constexpr int ROWS = kReduceThreads / 16;
    __shared__ double part[2][ROWS][17];
    const int c = threadIdx.x & 15, l = threadIdx.x >> 4;
    const int64_t W = (int64_t)p.G * p.C, ch = block * 16 + c;
    double d = 0.0, x = 0.0;
    if (ch < W) {
        const float *sums = p.sums + ch;
#pragma unroll 4
        for (int64_t i = l; i < n; i += ROWS) {
            d += (double)sums[i * 2 * W];
            x += (double)sums[(i * 2 + 1) * W];
        }
    }
    part[0][l][c] = d;
    part[1][l][c] = x;
    __syncthreads();
    for (int half = ROWS / 2; half > 0; half >>= 1) {
        if (l < half) {
            part[0][l][c] += part[0][l + half][c];
            part[1][l][c] += part[1][l + half][c];
        }
        __syncthreads();
    }
    if (l == 0 && ch < W) {
        ((T *)p.dw)[ch] = (T)(float)part[1][0][c];
        if (p.dbias) ((T *)p.dbias)[ch] = (T)(float)part[0][0][c];
    }
}

// what the slabs' sums make: of the groups, and dw and dbias
template <typename T> __global__ void __launch_bounds__(kReduceThreads) gnorm_join_sums_kernel(NormParams p)
{
    if (blockIdx.x >= p.reduce_from) norm_reduce<T>(p, blockIdx.x - p.reduce_from, p.samples * p.slabs);
    else norm_join<true>(p, blockIdx.x);
}

template <typename T, int V> __global__ void __launch_bounds__(256) gnorm_grad_kernel(NormParams p)
{
    const NormShare s = norm_share<V>(p, blockIdx.x);
    const int64_t first = s.first + s.r0;
    if (s.live <= 0) {
        norm_clear<T, V>(p, s, p.dx, p.dx_ld);
        if (p.gate) norm_clear<T, V>(p, s, p.dgate, p.dgate_ld);
        return;
    }
    Batch<T, V> vb, zb, db;
    for (int col = s.col; col < s.wide; col += 256) {
        const int64_t at = (int64_t)s.g0 * p.C + col * V, g = s.n * p.G + s.g0 + col / s.cv;
        const float m = p.moments[g * 2], r = p.moments[g * 2 + 1], a1 = p.pulls[g * 2], a2 = p.pulls[g * 2 + 1];
        float w[V], b[V];
        norm_weights<T, V>(p, at, w, b);
        const T *x = (const T *)p.x + s.row0 * p.x_ld + at, *zg = (const T *)p.gate + s.row0 * p.gate_ld + at;
        const T *dg = (const T *)p.dy + s.row0 * p.dy_ld + at;
        T *dx = (T *)p.dx + s.row0 * p.dx_ld + at, *dzg = (T *)p.dgate + s.row0 * p.dgate_ld + at;
        for (int64_t row = first; row < s.last; row += kNormBatch * s.step) {
            vb.load(x, p.x_ld, row, s.step, s.live);
            db.load(dg, p.dy_ld, row, s.step, s.live);
            if (p.gate) zb.load(zg, p.gate_ld, row, s.step, s.live);
#pragma unroll
            for (int e = 0; e < kNormBatch; ++e) {
                const int64_t at_row = row + e * s.step;
                if (at_row >= s.last) continue;
                float v[V], z[V], dy[V], d[V], dz[V];
                vb.get(e, v);
                db.get(e, dy);
                if (p.gate) zb.get(e, z);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = (v[i] - m) * r;
                norm_back<T, V>(p, v, w, b, z, dy, d, dz);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] = r * (fmaf(d[i], w[i], -a1) - v[i] * a2);
                if (at_row >= s.live)
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] = dz[i] = 0.0f;
                stream_f32<T, V>(dx + at_row * p.dx_ld, d);
                if (p.gate) stream_f32<T, V>(dzg + at_row * p.dgate_ld, dz);
            }
        }
    }
}

// ---- of each token by itself ----------------------------------------------------------
// `lanes` lanes share a group of C channels, each with R vectors of V, `lanes` vectors
// apart; a workgroup takes p.slab tokens of p.groups groups.
template <int V> struct TokenShare {
    int64_t row0, last;
    int g, l, slot, rpar, r0, cv;
    bool on;
};
template <int V> SEQ_DEV TokenShare<V> token_share(const NormParams &p)
{
    TokenShare<V> s;
    const int64_t slab = blockIdx.x / p.blocks;
    const int g0 = (int)(blockIdx.x - slab * p.blocks) * p.groups, slots = 256 / p.lanes;
    s.l = (int)threadIdx.x & (p.lanes - 1);
    s.slot = (int)threadIdx.x / p.lanes;
    s.rpar = slots / p.groups;
    s.r0 = s.slot / p.groups;
    s.g = g0 + s.slot - s.r0 * p.groups;
    s.cv = p.C / V;
    s.on = s.r0 < s.rpar && s.g < p.G;
    s.row0 = slab * p.slab;
    s.last = s.row0 + p.slab < p.tokens ? s.row0 + p.slab : p.tokens;
    return s;
}
SEQ_DEV bool token_counts(const NormParams &p, int64_t row)
{
    if (!p.lengths) return true;
    const int64_t n = row / p.L;
    return row - n * p.L < seq_len(p.lengths, n, p.L);
}
SEQ_DEV float lanes_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
// xhat in place of x, from a group's values in R V registers of `lanes` lanes; returns r
template <int V, int R> SEQ_DEV float token_xhat(const NormParams &p, int l, int cv, float (&v)[R][V])
{
    const float inv = 1.0f / (float)p.C;
    float mean = 0.0f, sq = 0.0f;
    if (p.center) {
#pragma unroll
        for (int e = 0; e < R; ++e)
#pragma unroll
            for (int i = 0; i < V; ++i) mean += v[e][i];        // zeros where there is no channel
        mean = lanes_sum(mean, p.lanes) / (float)p.C;
    }
#pragma unroll
    for (int e = 0; e < R; ++e)
        if (l + e * p.lanes < cv)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[e][i] -= mean;
                sq = fmaf(v[e][i], v[e][i], sq);
            }
    const float r = 1.0f / sqrtf(fmaf(lanes_sum(sq, p.lanes), inv, p.eps));
#pragma unroll
    for (int e = 0; e < R; ++e)
#pragma unroll
        for (int i = 0; i < V; ++i) v[e][i] *= r;
    return r;
}

template <typename T, int V, int R> __global__ void __launch_bounds__(256) gnorm_token_kernel(NormParams p)
{
    constexpr int B = R == 1 ? 4 : 2;       // tokens under way
    const TokenShare<V> s = token_share<V>(p);
    const int64_t at = (int64_t)s.g * p.C + s.l * V;
    float w[R][V], b[R][V];
#pragma unroll
    for (int e = 0; e < R; ++e) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[e][i] = b[e][i] = 0.0f;
        if (s.on && s.l + e * p.lanes < s.cv) norm_weights<T, V>(p, at + e * p.lanes * V, w[e], b[e]);
    }
    // all lanes take part in the sums, also those that have no group
    for (int64_t row = s.row0; row < s.last; row += B * s.rpar) {
        float v[B][R][V], z[B][R][V];
        bool live[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int64_t t = row + k * s.rpar + s.r0;
            live[k] = s.on && t < s.last && token_counts(p, t);
#pragma unroll
            for (int e = 0; e < R; ++e) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][e][i] = z[k][e][i] = 0.0f;
                if (live[k] && s.l + e * p.lanes < s.cv) {
                    load_f32<T, V>((const T *)p.x + t * p.x_ld + at + e * p.lanes * V, v[k][e]);
                    if (p.gate) load_f32<T, V>((const T *)p.gate + t * p.gate_ld + at + e * p.lanes * V, z[k][e]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            token_xhat<V, R>(p, s.l, s.cv, v[k]);
            const int64_t t = row + k * s.rpar + s.r0;
            if (!s.on || t >= s.last) continue;
#pragma unroll
            for (int e = 0; e < R; ++e) {
                if (s.l + e * p.lanes >= s.cv) continue;
                float u[V], y[V];
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] = fmaf(v[k][e][i], w[e][i], b[e][i]);
                norm_out<T, V>(p, u, z[k][e], y);
                if (!live[k])
#pragma unroll
                    for (int i = 0; i < V; ++i) y[i] = 0.0f;
                stream_f32<T, V>((T *)p.y + t * p.y_ld + at + e * p.lanes * V, y);
            }
        }
    }
}

template <typename T, int V, int R> __global__ void __launch_bounds__(256) gnorm_token_grad_kernel(NormParams p)
{
    constexpr int B = R == 1 ? 2 : 1;
    __shared__ float part[2][256 * V * R];
    const TokenShare<V> s = token_share<V>(p);
    const int64_t at = (int64_t)s.g * p.C + s.l * V;
    float w[R][V], b[R][V], sd[R][V], sx[R][V];
#pragma unroll
    for (int e = 0; e < R; ++e) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[e][i] = b[e][i] = sd[e][i] = sx[e][i] = 0.0f;
        if (s.on && s.l + e * p.lanes < s.cv) norm_weights<T, V>(p, at + e * p.lanes * V, w[e], b[e]);
    }
    const float inv = 1.0f / (float)p.C;
    for (int64_t row = s.row0; row < s.last; row += B * s.rpar) {
        float v[B][R][V], z[B][R][V], d[B][R][V];
        bool live[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int64_t t = row + k * s.rpar + s.r0;
            live[k] = s.on && t < s.last && token_counts(p, t);
#pragma unroll
            for (int e = 0; e < R; ++e) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][e][i] = z[k][e][i] = d[k][e][i] = 0.0f;
                if (live[k] && s.l + e * p.lanes < s.cv) {
                    const int64_t o = at + e * p.lanes * V;
                    load_f32<T, V>((const T *)p.x + t * p.x_ld + o, v[k][e]);
                    load_f32<T, V>((const T *)p.dy + t * p.dy_ld + o, d[k][e]);
                    if (p.gate) load_f32<T, V>((const T *)p.gate + t * p.gate_ld + o, z[k][e]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int64_t t = row + k * s.rpar + s.r0;
            const float r = token_xhat<V, R>(p, s.l, s.cv, v[k]);
            float dz[R][V], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int e = 0; e < R; ++e) {
                float dd[V];
                norm_back<T, V>(p, v[k][e], w[e], b[e], z[k][e], d[k][e], dd, dz[e]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (live[k]) {
                        sd[e][i] += dd[i];
                        sx[e][i] = fmaf(dd[i], v[k][e][i], sx[e][i]);
                    }
                    d[k][e][i] = dd[i] * w[e][i];
                    s1 += d[k][e][i];
                    s2 = fmaf(d[k][e][i], v[k][e][i], s2);
                }
            }
            s1 = p.center ? lanes_sum(s1, p.lanes) * inv : 0.0f;
            s2 = lanes_sum(s2, p.lanes) * inv;
            if (!s.on || t >= s.last) continue;
#pragma unroll
            for (int e = 0; e < R; ++e) {
                if (s.l + e * p.lanes >= s.cv) continue;
                const int64_t o = at + e * p.lanes * V;
                float dx[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dx[i] = live[k] ? r * (d[k][e][i] - s1 - v[k][e][i] * s2) : 0.0f;
                    dz[e][i] = live[k] ? dz[e][i] : 0.0f;
                }
                stream_f32<T, V>((T *)p.dx + t * p.dx_ld + o, dx);
                if (p.gate) stream_f32<T, V>((T *)p.dgate + t * p.dgate_ld + o, dz[e]);
            }
        }
    }
    // the slab's sums: the slots of a group, in order
#pragma unroll
    for (int e = 0; e < R; ++e)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            part[0][(e * V + i) * 256 + threadIdx.x] = sd[e][i];
            part[1][(e * V + i) * 256 + threadIdx.x] = sx[e][i];
        }
    __syncthreads();
    if (!s.on || s.r0 > 0) return;
    const int64_t W = (int64_t)p.G * p.C, slab = blockIdx.x / p.blocks;
    float *out = p.sums + slab * 2 * W + at;
#pragma unroll
    for (int e = 0; e < R; ++e) {
        if (s.l + e * p.lanes >= s.cv) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            double a = 0.0, c = 0.0;
            for (int k = 0; k < s.rpar; ++k) {
                const int th = (int)threadIdx.x + k * p.groups * p.lanes;
                a += (double)part[0][(e * V + i) * 256 + th];
                c += (double)part[1][(e * V + i) * 256 + th];
            }
            out[e * p.lanes * V + i] = (float)a;
            out[W + e * p.lanes * V + i] = (float)c;
        }
    }
}

template <typename T> __global__ void __launch_bounds__(kReduceThreads) gnorm_reduce_kernel(NormParams p)
{
    norm_reduce<T>(p, blockIdx.x, p.slabs);
}

}  // namespace convfwd
